"""A cache without pages (a server's before its first allocation) is no error of
the arguments: its pools have no address, so theirs do not coincide."""
from __future__ import annotations

from test_kv_host import ALIAS, AT, VALID, append, attend, cache, evict


def empty(prefix="", **kw):
    return cache(prefix, pages=0, k=0, v=0, **kw)


def test_calls_on_a_cache_without_pages():
    for e4m3 in (0, 1):
        assert append(empty(e4m3=e4m3)) in VALID
        assert append(empty(e4m3=e4m3), starts=AT["starts"], tokens=100) in VALID
        assert attend(empty(e4m3=e4m3)) in VALID
        assert evict(empty(e4m3=e4m3), empty("t", e4m3=e4m3)) in VALID


def test_keys_and_values_in_one_place_are_refused_where_there_are_some():
    assert append(cache(v=AT["k"])) == ALIAS
