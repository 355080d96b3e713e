"""The pages' refusals and the functions that guard their addresses, on a machine without a GPU."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from gemm_epilogue_02_gb300.build import ARCH, nvcc
from page_helpers import Pool, choose, page_bounds, page_score, power

OK, INVALID, ALIGN, UNSUPPORTED, ALIAS = 0, 1, 2, 3, 4
VALID = (OK, UNSUPPORTED, INVALID)     # no GPU here; on one these addresses are no device memory
MB = 1 << 20
AT = {n: (i + 1) * 64 * MB for i, n in enumerate(
    ["k", "v", "ks", "vs", "bounds", "bscale", "table", "lengths", "starts", "Q", "to", "ton", "uses", "touses", "parents", "in_use",
     "ws", "tokens", "O", "aws"])}


def cache(**kw):
    c = tg.KvCache()
    d = dict(k=AT["k"], v=AT["v"], pages=32, page_size=16, heads=4, dim=64, e4m3=0, page_stride=16 * 4 * 64, slot_stride=4 * 64,
             head_stride=64, k_scale=0, v_scale=0, scale_page_stride=16 * 4, scale_slot_stride=4, scale_head_stride=1)
    if kw.get("e4m3"):
        d.update(k_scale=AT["ks"], v_scale=AT["vs"])
    d.update(kw)
    for n, x in d.items():
        setattr(c, n, (x or None) if n in ("k", "v", "k_scale", "v_scale") else x)
    return c


def bounds(**kw):
    c = tg.KvPageBounds()
    d = dict(bounds=AT["bounds"], scale=AT["bscale"])
    d.update(kw)
    c.bounds, c.scale = d["bounds"] or None, d["scale"] or None
    return c


def call(fn, fmt, fields, kw):
    unknown = set(kw) - set(fields)
    assert not unknown, unknown
    fields.update(kw)
    keep = list(fields.values())
    return fn(fmt.pack(*[ctypes.addressof(f) if isinstance(f, ctypes.Structure) else f for f in keep]))


SEQ = dict(table=AT["table"], lengths=AT["lengths"], width=8, stride=8, batch=8)


def kv_bounds(c=None, b=None, **kw):
    return call(tg.tgemm_kv_bounds, tg.KV_BOUNDS_ARGS, dict(cache=c or cache(), bounds=b or bounds(), **SEQ, starts=AT["starts"], dtype=1), kw)


def kv_select(c=None, b=None, **kw):
    return call(tg.tgemm_kv_select, tg.KV_SELECT_ARGS, dict(
        cache=c or cache(), bounds=b or bounds(), **SEQ, Q=AT["Q"], heads=16, qb=1024, qh=64, to=AT["to"], ton=AT["ton"], tob=16, toh=4,
        keep=4, first=1, recent=1, dtype=1), kw)


def kv_grow(c=None, **kw):
    return call(tg.tgemm_kv_grow, tg.KV_GROW_ARGS, dict(cache=c or cache(), uses=AT["uses"], **SEQ, tokens=AT["tokens"]), kw)


def kv_free(c=None, **kw):
    return call(tg.tgemm_kv_free, tg.KV_FREE_ARGS, dict(cache=c or cache(), uses=AT["uses"], **SEQ), kw)


def kv_fork(c=None, **kw):
    return call(tg.tgemm_kv_fork, tg.KV_FORK_ARGS, dict(
        cache=c or cache(), uses=AT["uses"], **SEQ, parents=AT["parents"], to=AT["to"], ton=AT["ton"], tow=8, tos=8, children=5), kw)


def kv_compact(c=None, **kw):
    return call(tg.tgemm_kv_compact, tg.KV_COMPACT_ARGS, dict(
        cache=c or cache(), bounds=bounds(), uses=AT["uses"], **SEQ, to=AT["to"], tow=8, tos=8, touses=AT["touses"], in_use=AT["in_use"],
        ws=AT["ws"], wsb=MB), kw)


def lists(c=None, head_stride=8, **kw):
    d = dict(cache=c or cache(), **SEQ, w=0, ww=0, wb=0, wh=0, Q=AT["Q"], O=AT["O"], heads=16, qb=1024, qh=64, ob=1024, oh=64,
             window=0, scale=0.125, cap=0.0, ws=AT["aws"], wsb=60 * MB, dtype=0)
    return call(lambda a: tg.tgemm_attention_decode_lists(a, head_stride), tg.ATTENTION_DECODE_ARGS, d, kw)


CALLS = [kv_bounds, kv_select, kv_grow, kv_free, kv_fork, kv_compact, lists]


def test_valid_calls():
    for f in CALLS:
        assert f() in VALID, f.__name__
        assert f(cache(e4m3=1)) in VALID, f.__name__
    assert kv_bounds(starts=0) in VALID and kv_grow(tokens=0) in VALID
    assert kv_compact(to=AT["table"], touses=AT["uses"]) in VALID              # in place
    assert kv_compact(bounds=0) in VALID
    assert lists(head_stride=0) in VALID
    for f, kw in ((kv_bounds, dict(batch=0)), (kv_select, dict(batch=0)), (kv_grow, dict(batch=0)), (kv_free, dict(batch=0)),
                  (kv_fork, dict(children=0))):
        assert f(**kw) == OK, f.__name__
    assert kv_fork(to=AT["table"] + 8 * 8 * 4, ton=AT["lengths"] + 32) in VALID        # other rows of the parents' arrays


@pytest.mark.parametrize("f", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", [
    (dict(k=0), INVALID), (dict(pages=-1), INVALID), (dict(dim=60), INVALID), (dict(page_size=0), INVALID), (dict(e4m3=2), INVALID),
    (dict(v=AT["v"] + 2), ALIGN),
])
def test_bad_caches(f, kw, code):
    assert f(cache(**kw)) == code


@pytest.mark.parametrize("f", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(batch=65536), INVALID), (dict(width=-1), INVALID), (dict(stride=7), INVALID),
    (dict(width=2 ** 27, stride=2 ** 27), INVALID), (dict(table=0), INVALID), (dict(lengths=0), INVALID), (dict(table=AT["table"] + 2), ALIGN),
    (dict(lengths=AT["lengths"] + 1), ALIGN),
])
def test_bad_sequences(f, kw, code):
    assert f(**kw) == code


@pytest.mark.parametrize("f", [kv_bounds, kv_grow, kv_free, kv_fork, kv_compact], ids=lambda f: f.__name__)
def test_lists_that_cannot_be_counted(f):
    """2^31 pages and more in 1024 lists."""
    c = cache(page_size=1, page_stride=256)
    assert f(c, width=2 ** 22, stride=2 ** 22, batch=512) == INVALID


@pytest.mark.parametrize("f", [kv_grow, kv_free, kv_fork, kv_compact], ids=lambda f: f.__name__)
@pytest.mark.parametrize("c", [
    dict(page_size=1, page_stride=64, heads=1, slot_stride=64, pages=2 ** 30 + 1),
    dict(page_size=2 ** 20, heads=2048, slot_stride=2048 * 64, page_stride=2 ** 37),
])
def test_pools_that_cannot_be_counted(f, c):
    kw = dict(bounds=0) if f is kv_compact else {}
    assert f(cache(**c), width=0, **kw) == INVALID


@pytest.mark.parametrize("f", [kv_bounds, kv_select], ids=lambda f: f.__name__)
@pytest.mark.parametrize("b,code", [
    (dict(bounds=0), INVALID), (dict(scale=0), INVALID), (dict(bounds=AT["bounds"] + 8), ALIGN), (dict(scale=AT["bscale"] + 2), ALIGN),
])
def test_bad_bounds(f, b, code):
    assert f(b=bounds(**b)) == code
    assert kv_compact(bounds=bounds(**b)) == code
    assert f(cache(dim=72, head_stride=72, slot_stride=288, page_stride=4608)) == INVALID


@pytest.mark.parametrize("f,kw,code", [
    (kv_bounds, dict(dtype=2), INVALID), (kv_bounds, dict(starts=AT["starts"] + 2), ALIGN), (kv_bounds, dict(b=bounds(bounds=AT["k"])), ALIAS),
    (kv_bounds, dict(b=bounds(scale=AT["bounds"])), ALIAS),
    (kv_select, dict(dtype=2), INVALID), (kv_select, dict(heads=15), INVALID), (kv_select, dict(heads=4 * 65), INVALID),
    (kv_select, dict(keep=0), INVALID), (kv_select, dict(recent=0), INVALID), (kv_select, dict(first=-1), INVALID),
    (kv_select, dict(first=4), INVALID), (kv_select, dict(recent=4), INVALID), (kv_select, dict(Q=0), INVALID),
    (kv_select, dict(Q=AT["Q"] + 2), ALIGN), (kv_select, dict(qh=60), ALIGN), (kv_select, dict(toh=3), INVALID), (kv_select, dict(tob=3), INVALID),
    (kv_select, dict(to=0), INVALID), (kv_select, dict(ton=0), INVALID), (kv_select, dict(to=AT["table"]), ALIAS),
    (kv_select, dict(ton=AT["lengths"] + 16), ALIAS), (kv_select, dict(to=AT["ton"] - 8), ALIAS), (kv_select, dict(to=AT["k"]), ALIAS),
    (kv_select, dict(to=AT["Q"]), ALIAS), (kv_select, dict(ton=AT["bounds"]), ALIAS),
    (kv_select, dict(c=cache(page_size=1, page_stride=256), width=2 ** 17 + 1, stride=2 ** 18), INVALID),
    (kv_grow, dict(uses=0), INVALID), (kv_grow, dict(uses=AT["uses"] + 2), ALIGN), (kv_grow, dict(uses=AT["table"]), ALIAS),
    (kv_grow, dict(uses=AT["k"]), ALIAS), (kv_grow, dict(lengths=AT["table"] + 64), ALIAS), (kv_grow, dict(tokens=AT["tokens"] + 1), ALIGN),
    (kv_free, dict(uses=0), INVALID), (kv_free, dict(uses=AT["lengths"]), ALIAS),
    (kv_fork, dict(uses=0), INVALID), (kv_fork, dict(parents=0), INVALID), (kv_fork, dict(parents=AT["parents"] + 2), ALIGN),
    (kv_fork, dict(to=0), INVALID), (kv_fork, dict(ton=0), INVALID), (kv_fork, dict(tos=7), INVALID), (kv_fork, dict(children=-1), INVALID),
    (kv_fork, dict(ton=AT["uses"] + 8), ALIAS), (kv_fork, dict(c=cache(v=AT["k"])), ALIAS),
    (kv_compact, dict(uses=0), INVALID), (kv_compact, dict(touses=0), INVALID), (kv_compact, dict(in_use=0), INVALID),
    (kv_compact, dict(ws=0), INVALID), (kv_compact, dict(wsb=100), INVALID), (kv_compact, dict(ws=AT["ws"] + 4), ALIGN),
    (kv_compact, dict(to=0), INVALID), (kv_compact, dict(tow=7), INVALID), (kv_compact, dict(tos=6), INVALID),
    (kv_compact, dict(to=AT["table"] + 4), ALIAS), (kv_compact, dict(touses=AT["uses"] + 4), ALIAS), (kv_compact, dict(in_use=AT["uses"]), ALIAS),
    (kv_compact, dict(ws=AT["uses"]), ALIAS), (kv_compact, dict(touses=AT["bounds"]), ALIAS), (kv_compact, dict(to=AT["lengths"]), ALIAS),
    (kv_compact, dict(c=cache(v=AT["k"])), ALIAS),
    (lists, dict(cap=-1.0), INVALID),
], ids=lambda x: x.__name__ if callable(x) else str(x)[:40])
def test_refusals(f, kw, code):
    assert f(**kw) == code


@pytest.mark.parametrize("stride", [7, -8, 2 ** 41])
def test_strides_of_the_heads_lists(stride):
    assert lists(head_stride=stride) == INVALID


def test_no_structures():
    lib = tg.load()
    for name in ("tgemm_kv_bounds", "tgemm_kv_select", "tgemm_kv_grow", "tgemm_kv_fork", "tgemm_kv_free", "tgemm_kv_compact"):
        assert getattr(lib, name)(None, None) == INVALID
    assert lib.tgemm_attention_decode_lists(None, 8, None) == INVALID
    assert kv_bounds(cache=0) == INVALID and kv_bounds(bounds=0) == INVALID and kv_select(bounds=0) == INVALID
    for pages in (0, 1, 10 ** 6):
        assert tg.tgemm_kv_compact_workspace(pages) >= 12 * pages
    with pytest.raises(tg.TgemmError):
        tg.tgemm_kv_compact_workspace(-1)


@pytest.mark.parametrize("f,kw", [
    (kv_fork, dict(parents=AT["uses"] + 64)), (kv_fork, dict(parents=AT["to"])), (kv_fork, dict(parents=AT["ton"] + 16)),
    (kv_fork, dict(parents=AT["v"])), (kv_fork, dict(uses=AT["table"] + 128)), (kv_fork, dict(uses=AT["lengths"] - 124)),
    (kv_fork, dict(to=AT["lengths"] - 8)), (kv_fork, dict(ton=AT["table"] + 252)), (kv_fork, dict(table=AT["k"] + 256)),
    (kv_fork, dict(lengths=AT["v"])), (kv_fork, dict(c=cache(e4m3=1), parents=AT["ks"])),
    (kv_grow, dict(tokens=AT["uses"] + 124)), (kv_grow, dict(tokens=AT["lengths"])), (kv_grow, dict(tokens=AT["table"] + 60)),
], ids=lambda x: x.__name__ if callable(x) else "-".join(x))
def test_what_is_read_is_not_written(f, kw):
    """Parents, their lists and lengths, and the numbers of new tokens, against what the call writes."""
    assert f(**kw) == ALIAS


@pytest.mark.parametrize("f,kw", [
    (kv_bounds, dict(table=AT["bounds"] + 64)), (kv_bounds, dict(lengths=AT["bscale"] + 8)), (kv_bounds, dict(starts=AT["bscale"])),
    (kv_bounds, dict(starts=AT["bounds"] - 32)), (kv_bounds, dict(table=AT["bscale"] + 508)),
    (kv_compact, dict(bounds=bounds(bounds=AT["k"]))), (kv_compact, dict(bounds=bounds(scale=AT["v"] + 256))),
    (kv_compact, dict(bounds=bounds(scale=AT["bounds"] + 4))), (kv_compact, dict(c=cache(e4m3=1), bounds=bounds(scale=AT["ks"]))),
], ids=lambda x: x.__name__ if callable(x) else "-".join(x))
def test_bounds_lie_apart(f, kw):
    """Bounds against the lists that say which are written, and against the rows that move."""
    assert f(**kw) == ALIAS


@pytest.mark.parametrize("tob,toh,code", [(8, 4, ALIAS), (15, 4, ALIAS), (4, 32, VALID), (4, 31, ALIAS), (12, 8, ALIAS), (9, 4, ALIAS), (32, 4, VALID)])
def test_lists_that_are_written_lie_apart(tob, toh, code):
    """Lists of 4 of 4 heads and 8 sequences."""
    got = kv_select(tob=tob, toh=toh)
    assert got == code if code == ALIAS else got in code and got == kv_select()


# ---------------------------------------------------------------- the functions as compiled for the host
@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("page") / "libpagehost.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "page_host_check.cu")
    subprocess.run([nvcc(), *ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", lib, src], check=True,
                   capture_output=True)
    h = ctypes.CDLL(lib)
    h.check_scale.argtypes, h.check_scale.restype = [ctypes.c_float], ctypes.c_float
    h.check_completed.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    return h


def test_powers(host):
    """The least power of two with top <= 127 s."""
    tops = [0.0, 1e-45, 2.0 ** -126, 127 * 2.0 ** -100, 1.0, 126.99999, 127.0, 127.00001, 128.0, 3.4028234663852886e38]
    tops += [float(np.float32(127 * 2.0 ** e * f)) for e in range(-110, 121, 7) for f in (1 - 2.0 ** -23, 1.0, 1 + 2.0 ** -22)]
    for top in tops:
        top = float(np.float32(top))
        s = host.check_scale(top)
        assert s == power(top) and top <= 127 * s and (s == 2.0 ** -100 or top > 127 * s / 2)


def test_completed_pages(host):
    at = ctypes.c_int()
    for page in (1, 7, 16):
        for n in (0, 1, 15, 16, 17, 100, 2 ** 30):
            for fresh in (0, 1, 16, n, n + 1, -3, 2 ** 31, -2 ** 31):
                to = host.check_completed(n, fresh, page, ctypes.byref(at))
                assert to == n // page and 0 <= at.value <= to
                if 0 <= fresh <= n:
                    assert at.value == (n - fresh) // page


def test_spans(host):
    out = (ctypes.c_int * 5)()
    for page in (1, 16, 24):
        for n in (0, 1, 16, 100, 5000, 2 ** 30):
            for keep, first, recent in ((1, 0, 1), (4, 1, 1), (10, 3, 7), (2 ** 30, 0, 5)):
                host.check_span(n, page, keep, first, recent, out)
                count = -(-n // page)
                assert out[0] == count and out[1] == min(count, keep)
                if count <= keep:
                    assert out[2] == count and out[3] == out[4] == 0
                else:
                    assert out[2] == first and out[3] == count - first - recent >= out[4] == keep - first - recent >= 0


def test_fork_lengths(host):
    lengths, bad = (ctypes.c_int * 4)(5, 0, 48, -2), ctypes.c_int()
    for parent, width, to_width, want, wrong in ((0, 4, 4, 5, 0), (1, 4, 4, 0, 0), (2, 4, 4, 48, 0), (2, 4, 2, 0, 1), (2, 2, 4, 32, 1),
                                                 (3, 4, 4, 0, 1), (4, 4, 4, 0, 1), (-1, 4, 4, 0, 0), (-2, 4, 4, 0, 1)):
        assert host.check_fork(lengths, 4, parent, width, 16, to_width, ctypes.byref(bad)) == want and bad.value == wrong
    assert [host.check_pages(n, 16) for n in (0, 1, 16, 17, 2 ** 31 - 1)] == [0, 1, 1, 2, 2 ** 27]


# ---------------------------------------------------------------- the helpers' definitions
def test_bounds_hold():
    """No key leaves its bounds, and no product with the query in whole numbers the score."""
    g = np.random.default_rng(0)
    for _ in range(50):
        keys = g.normal(size=(9, 16)) * 10.0 ** g.integers(-3, 4)
        lo, hi, s = page_bounds(keys)
        assert (s * lo <= keys).all() and (keys <= s * hi).all() and np.abs(lo).max() <= 127 and np.abs(hi).max() <= 127
        q = g.normal(size=(2, 16))
        t = [power(np.abs(x).max()) for x in q]
        whole = [np.rint(x / u) * u for x, u in zip(q, t)]
        assert page_score(q, lo, hi, s) >= max((keys @ w).max() for w in whole) - 1e-9


def test_choice_and_pool_helpers():
    assert choose([0, 5, 5, 1, 9, 2], 4, 1, 1) == [0, 1, 4, 5] and choose([1, 2], 5, 0, 1) == [0, 1]
    p = Pool([0, 1, 0, 0], 4, 8)
    table, lengths = [[1] + [-1] * 7, [-1] * 8], [3, 0]
    p.grow(table, lengths, [6, 20])
    assert lengths == [9, 0] and table[0][:3] == [1, 0, 2] and p.error and p.uses == [1, 1, 1, 0]


# ---------------------------------------------------------------- the Python calls
def pools(**kw):
    return tg.PagedCache(*(torch.zeros(6, 16, 2, 64, dtype=torch.float16) for _ in range(2)))


def page_bounds_of(pages=6, heads=2, dim=64):
    return tg.PageBounds(torch.zeros(pages, heads, 2, dim, dtype=torch.int8), torch.zeros(pages, heads))


I32 = torch.int32


def vec(n):
    return torch.zeros(n, dtype=I32)


@pytest.mark.parametrize("args", [
    (torch.zeros(6, 2, 2, 64), torch.zeros(6, 2)), (torch.zeros(6, 2, 64, dtype=torch.int8), torch.zeros(6, 2)),
    (torch.zeros(6, 2, 3, 64, dtype=torch.int8), torch.zeros(6, 2)), (torch.zeros(6, 2, 2, 64, dtype=torch.int8), torch.zeros(6, 3)),
    (torch.zeros(6, 2, 2, 64, dtype=torch.int8), torch.zeros(6, 2, dtype=torch.float64)),
    (torch.zeros(6, 2, 2, 128, dtype=torch.int8)[..., ::2], torch.zeros(6, 2)), (torch.zeros(6, 2, 2, 64, dtype=torch.int8), torch.zeros(2, 6).T),
])
def test_bounds_tensors(args):
    with pytest.raises(ValueError):
        tg.PageBounds(*args)


@pytest.mark.parametrize("fn,args", [
    (tg.kv_bounds, lambda c: (c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3))),           # right, but for its device
    (tg.kv_bounds, lambda c: (c, page_bounds_of(5), torch.zeros(3, 4, dtype=I32), vec(3))),
    (tg.kv_bounds, lambda c: (c, page_bounds_of(), torch.zeros(3, 4), vec(3))),
    (tg.kv_bounds, lambda c: (c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(2))),
    (tg.kv_bounds, lambda c: (c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), vec(3))),
    (tg.kv_select, lambda c: (torch.zeros(3, 4, 64).half(), c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 2, 2, dtype=I32), vec(3))),
    (tg.kv_select, lambda c: (torch.zeros(3, 3, 64).half(), c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 2, 2, dtype=I32), vec(3))),
    (tg.kv_select, lambda c: (torch.zeros(3, 4, 64).bfloat16(), c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 2, 2, dtype=I32), vec(3))),
    (tg.kv_select, lambda c: (torch.zeros(3, 4, 64).half(), c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 3, 2, dtype=I32), vec(3))),
    (tg.kv_select, lambda c: (torch.zeros(3, 4, 64).half(), c, page_bounds_of(), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 2, 2), vec(3))),
    (tg.attention_decode, lambda c: (torch.zeros(3, 4, 64).half(), c, torch.zeros(3, 3, 4, dtype=I32), vec(3), torch.zeros(3, 4, 64).half())),
    (tg.attention_decode, lambda c: (torch.zeros(3, 4, 64).half(), c, torch.zeros(3, 2, 4), vec(3), torch.zeros(3, 4, 64).half())),
    (tg.kv_grow, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3))),
    (tg.kv_grow, lambda c: (c, vec(5), torch.zeros(3, 4, dtype=I32), vec(3))),
    (tg.kv_grow, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), vec(2))),
    (tg.kv_fork, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), vec(2), torch.zeros(2, 4, dtype=I32), vec(2))),
    (tg.kv_fork, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), vec(3), torch.zeros(2, 4, dtype=I32), vec(2))),
    (tg.kv_free, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3))),
    (tg.kv_free, lambda c: (c, vec(6).float(), torch.zeros(3, 4, dtype=I32), vec(3))),
    (tg.kv_compact, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 4, dtype=I32), vec(6), vec(1))),
    (tg.kv_compact, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 3, dtype=I32), vec(6), vec(1))),
    (tg.kv_compact, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(2, 4, dtype=I32), vec(6), vec(1))),
    (tg.kv_compact, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 4, dtype=I32), vec(6), vec(2))),
    (tg.kv_compact, lambda c: (c, vec(6), torch.zeros(3, 4, dtype=I32), vec(3), torch.zeros(3, 4, dtype=I32), vec(6), vec(1), page_bounds_of(7))),
])
def test_python_refusals(fn, args):
    """None of these reaches the library."""
    with pytest.raises(ValueError):
        fn(*args(pools()))
