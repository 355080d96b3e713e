"""The paged cache's refusals and the functions that guard its addresses, on a
machine without a GPU: argument checks of the C ABI and of the Python calls,
page, length and start checks as compiled for the host, and the helpers'
definitions against brute force."""
from __future__ import annotations

import ctypes
import math
import subprocess

import numpy as np
import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from gemm_epilogue_02_gb300.build import ARCH, nvcc
from kv_helpers import E4M3, attend64, evict_reference, make_table

OK, INVALID, ALIGN, UNSUPPORTED, ALIAS = 0, 1, 2, 3, 4
# Fake, aligned, disjoint addresses: validation reads addresses only.
MB = 1 << 20
AT = {n: (i + 1) * 64 * MB for i, n in enumerate(
    ["k", "v", "ks", "vs", "tk", "tv", "tks", "tvs", "K", "V", "Q", "O", "table", "to_table", "lengths", "starts", "weights",
     "kept", "to_lengths", "to_weights", "workspace"])}
VALID = (OK, UNSUPPORTED, INVALID)     # no GPU here; on one these addresses are no device memory


def cache(prefix="", **kw):
    c = tg.KvCache()
    d = dict(k=AT[prefix + "k"], v=AT[prefix + "v"], pages=32, page_size=16, heads=4, dim=64, e4m3=0,
             page_stride=16 * 4 * 64, slot_stride=4 * 64, head_stride=64, k_scale=0, v_scale=0,
             scale_page_stride=16 * 4, scale_slot_stride=4, scale_head_stride=1)
    if kw.get("e4m3"):
        d.update(k_scale=AT[prefix + "ks"], v_scale=AT[prefix + "vs"])
    d.update(kw)
    for n, x in d.items():
        setattr(c, n, (x or None) if n in ("k", "v", "k_scale", "v_scale") else x)
    return c


BAD_CACHES = [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=2 ** 31), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=(1 << 20) + 1), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID),
    (dict(dim=60), INVALID), (dict(dim=264), INVALID), (dict(e4m3=2), INVALID), (dict(e4m3=1, k_scale=0), INVALID),
    (dict(e4m3=1, dim=72), INVALID), (dict(head_stride=56), INVALID), (dict(slot_stride=-256), INVALID),
    (dict(page_stride=2 ** 62), INVALID), (dict(k=AT["k"] + 8), ALIGN), (dict(v=AT["v"] + 2), ALIGN),
    (dict(slot_stride=260), ALIGN), (dict(e4m3=1, k_scale=AT["ks"] + 2), ALIGN), (dict(e4m3=1, scale_slot_stride=0), INVALID),
]


def call(fn, fmt, fields, **kw):
    """fn on the packed fields, a dict in the structure's order; cache structures by address."""
    unknown = set(kw) - set(fields)
    assert not unknown, unknown
    fields.update(kw)
    keep = [f for f in fields.values() if isinstance(f, tg.KvCache)]
    return fn(fmt.pack(*[ctypes.addressof(f) if isinstance(f, tg.KvCache) else f for f in fields.values()]), 0), keep


def append(c=None, **kw):
    return call(tg.tgemm_kv_append, tg.KV_APPEND_ARGS, dict(
        cache=c or cache(), table=AT["table"], lengths=AT["lengths"], width=8, stride=8, batch=8, w=0, ww=0, wb=0, wh=0,
        K=AT["K"], V=AT["V"], starts=0, tokens=8, ts=256, hs=64, dtype=0), **kw)[0]


def attend(c=None, **kw):
    return call(tg.tgemm_attention_decode, tg.ATTENTION_DECODE_ARGS, dict(
        cache=c or cache(), table=AT["table"], lengths=AT["lengths"], width=8, stride=8, batch=8, w=0, ww=0, wb=0, wh=0,
        Q=AT["Q"], O=AT["O"], heads=16, qb=1024, qh=64, ob=1024, oh=64, window=0, scale=0.125, cap=0.0, ws=AT["workspace"],
        wsb=60 * MB, dtype=0), **kw)[0]


def evict(c=None, to=None, **kw):
    return call(tg.tgemm_kv_evict, tg.KV_EVICT_ARGS, dict(
        cache=c or cache(), table=AT["table"], lengths=AT["lengths"], width=8, stride=8, batch=8, w=AT["weights"], ww=128,
        wb=512, wh=128, to=to or cache("t"), to_table=AT["to_table"], unused=0, tw=4, tstride=4, to_batch=8,
        tow=AT["to_weights"], toww=64, towb=256, towh=64, kept=AT["kept"], tl=AT["to_lengths"], keep=64, recent=8), **kw)[0]


def test_valid_calls():
    for e4m3 in (0, 1):
        assert append(cache(e4m3=e4m3)) in VALID and attend(cache(e4m3=e4m3)) in VALID
        assert evict(cache(e4m3=e4m3), cache("t", e4m3=e4m3)) in VALID
    assert append(starts=AT["starts"], tokens=100) in VALID
    assert attend(w=AT["weights"], ww=128, wb=512, wh=128) in VALID
    assert append(batch=0, tokens=0, K=0, V=0, table=0, lengths=0) == OK
    assert attend(batch=0, Q=0, O=0, table=0, lengths=0) == OK
    assert evict(batch=0, to_batch=0, table=0, lengths=0, to_table=0, w=0, kept=0, tl=0, tow=0) == OK


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(kw, code):
    assert append(cache(**kw)) == code
    assert attend(cache(**kw)) == code
    assert evict(cache(**kw)) == code
    assert evict(to=cache("t", **{n: x + AT["tk"] - AT["k"] if n in ("k", "v", "k_scale") and x else x
                                  for n, x in kw.items()})) == code


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=7), INVALID), (dict(dtype=2), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=70000, tokens=70000), INVALID), (dict(width=-1), INVALID), (dict(stride=7), INVALID),
    (dict(table=0), INVALID), (dict(lengths=0), INVALID), (dict(ts=-256), INVALID), (dict(K=AT["K"] + 2), ALIGN),
    (dict(ts=260), ALIGN), (dict(hs=65), ALIGN), (dict(lengths=AT["lengths"] + 1), ALIGN), (dict(K=AT["v"] + 512), ALIAS),
    (dict(V=AT["k"]), ALIAS), (dict(w=AT["weights"], ww=128, wb=512, wh=100), INVALID), (dict(w=AT["weights"] + 2, ww=8, wb=512, wh=128), ALIGN),
])
def test_append_refusals(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(heads=6), INVALID), (dict(heads=0), INVALID), (dict(dtype=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=math.inf), INVALID),
    (dict(window=-1), INVALID), (dict(ws=0), INVALID), (dict(wsb=16), INVALID), (dict(ws=AT["workspace"] + 8), ALIGN),
    (dict(Q=AT["Q"] + 2), ALIGN), (dict(qb=1028), ALIGN), (dict(oh=68), ALIGN), (dict(oh=56), INVALID), (dict(O=AT["Q"] + 1024), ALIAS),
    (dict(O=AT["k"]), ALIAS), (dict(ws=AT["v"]), ALIAS), (dict(lengths=0), INVALID), (dict(stride=4), INVALID),
    (dict(batch=65535, width=1 << 20, stride=1 << 20), INVALID), (dict(width=(1 << 26) + 1, stride=1 << 27), INVALID),
])
def test_attention_decode_refusals(kw, code):
    assert attend(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), INVALID), (dict(recent=-1), INVALID), (dict(to_batch=7), INVALID), (dict(w=0), INVALID), (dict(kept=0), INVALID), (dict(tl=0), INVALID),
    (dict(tow=0), INVALID), (dict(toww=63), INVALID), (dict(kept=AT["kept"] + 2), ALIGN), (dict(tl=AT["lengths"] + 8), ALIAS),
    (dict(tow=AT["weights"] + 128), ALIAS), (dict(kept=AT["to_weights"]), ALIAS), (dict(to_table=0), INVALID), (dict(wh=100), INVALID),
])
def test_evict_refusals(kw, code):
    assert evict(**kw) == code


def test_evict_refuses_caches_that_do_not_match():
    assert evict(to=cache("t", dim=128, page_stride=16 * 4 * 128, slot_stride=512, head_stride=128)) == INVALID
    assert evict(to=cache("t", heads=2)) == INVALID
    assert evict(to=cache("t", e4m3=1)) == INVALID


def test_null_arguments():
    for fn in (tg.load().tgemm_kv_append, tg.load().tgemm_attention_decode, tg.load().tgemm_kv_evict):
        assert fn(None, None) == INVALID
    assert attend(cache=0) == INVALID and append(cache=0) == INVALID and evict(cache=0) == INVALID and evict(to=None, **{"to_table": 0}) == INVALID


def test_workspace_sizes():
    small = tg.tgemm_attention_decode_workspace(1, 8, 8, 64, 100, False)
    assert small > 0 and tg.tgemm_attention_decode_workspace(64, 32, 8, 128, 32768, False) >= small
    with_w = tg.tgemm_attention_decode_workspace(4, 32, 8, 128, 5000, True)
    assert with_w >= tg.tgemm_attention_decode_workspace(4, 32, 8, 128, 5000, False)
    for bad in ((-1, 8, 8, 64, 1), (1, 7, 2, 64, 1), (1, 8, 0, 64, 1), (1, 8, 8, 0, 1), (1, 8, 8, 512, 1), (1, 8, 8, 64, -1)):
        with pytest.raises(tg.TgemmError):
            tg.tgemm_attention_decode_workspace(*bad, False)


# ---------------------------------------------------------------- the Python calls
def py_cache(dtype=torch.float16, heads=2, dim=64, **kw):
    k, v = (torch.zeros(3, 4, heads, dim).to(dtype) for _ in range(2))
    if dtype == E4M3:
        kw = dict(k_scale=torch.ones(3, 4, heads), v_scale=torch.ones(3, 4, heads), **kw)
    return tg.PagedCache(k, v, **kw)


def test_paged_cache_refusals():
    k = torch.zeros(3, 4, 2, 64, dtype=torch.float16)
    s = torch.ones(3, 4, 2)
    for args in ((k[0], k[0]), (k, k[:, :2]), (k, k.bfloat16()), (k.float(), k.float()), (k.to(E4M3), k.to(E4M3)), (k, k, s, s),
                 (k.to(E4M3), k.to(E4M3), s, s.double()), (k.to(E4M3), k.to(E4M3), s[:2], s), (k[..., ::2], k[..., ::2]),
                 (k, torch.zeros(3, 2, 4, 64, dtype=torch.float16).transpose(1, 2))):
        with pytest.raises(ValueError):
            tg.PagedCache(*args)
    c = tg.PagedCache(*(torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16).transpose(1, 2) for _ in range(2)))
    assert (c.pages, c.page_size, c.heads, c.dim) == (3, 4, 2, 64)
    assert (c._struct.slot_stride, c._struct.head_stride) == (64, 256)


def test_python_refusals():
    c, e = py_cache(), py_cache(E4M3)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    w = torch.zeros(2, 2, 12)
    for bad in (dict(K=x[:1], V=x[:1]), dict(K=x.float(), V=x.float()), dict(K=x.bfloat16(), V=x.bfloat16()), dict(V=x[:, :1]),
                dict(table=t.long()), dict(lengths=n[:1]), dict(starts=n), dict(weights=w[:1]), dict(weights=w.double()),
                dict(table=t.t()), dict()):      # the last: all in order, but not on a GPU
        a = dict(K=x, V=x, table=t, lengths=n, starts=None, weights=None)
        a.update(bad)
        with pytest.raises(ValueError):
            tg.kv_append(c, a["K"], a["V"], a["table"], a["lengths"], starts=a["starts"], weights=a["weights"])
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (dict(Q=x[:, :1]), dict(Q=x[..., :32]), dict(Q=x.bfloat16()), dict(lengths=n[:1]), dict(weights=w[..., ::2]), dict()):
        a = dict(Q=x, O=x.clone(), lengths=n, weights=None)
        a.update(bad)
        with pytest.raises(ValueError):
            tg.attention_decode(a["Q"], c, t, a["lengths"], a["O"], weights=a["weights"], workspace=ws)
    kept = torch.zeros(2, 2, 5, dtype=torch.int32)
    for bad in (dict(to=e), dict(kept=kept.long()), dict(kept=kept[:1]), dict(tw=w[..., :4]), dict(tl=n[:1]), dict()):
        a = dict(to=py_cache(), kept=kept, tl=n.clone(), tw=w.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            tg.kv_evict(c, t, n, w, a["to"], t, a["kept"], a["tl"], a["tw"])


# ---------------------------------------------------------------- guards, as compiled for the host
@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("kv") / "libkvhost.so")
    src = __file__.replace("test_kv_host.py", "kv_host_check.cu")
    subprocess.run([nvcc(), *ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o",
                    lib, src], check=True, capture_output=True)
    h = ctypes.CDLL(lib)
    h.check_row.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p]
    h.check_sequence.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong]
    h.check_tiles.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p]
    for f in (h.check_first, h.check_owner):
        f.argtypes = [ctypes.c_longlong] * 3
    h.check_pad.argtypes = [ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int]
    h.check_first.restype = ctypes.c_longlong
    h.check_key.argtypes, h.check_key.restype = [ctypes.c_uint], ctypes.c_uint
    return h


def test_lengths_are_cut_to_the_page_list(host):
    out = ctypes.c_int()
    for length, width, page, want, bad in ((0, 4, 16, 0, 0), (64, 4, 16, 64, 0), (65, 4, 16, 64, 1), (-1, 4, 16, 0, 1),
                                           (-2 ** 31, 4, 16, 0, 1), (2 ** 31 - 1, 4, 16, 64, 1), (1, 0, 16, 0, 1),
                                           (2 ** 31 - 1, 2047, 1 << 20, 2047 << 20, 1)):
        assert host.check_length(length, width, page, ctypes.byref(out)) == bad and out.value == want


def test_rows_of_positions_and_bad_pages(host):
    page, slot = ctypes.c_int(), ctypes.c_int()
    for size in (1, 2, 3, 16, 20, 1000):
        lst = np.random.default_rng(size).permutation(50).astype(np.int32)
        for pos in range(0, 50 * size, max(1, size // 3)):
            ok = host.check_row(lst.ctypes.data, pos, size, 50, ctypes.byref(page), ctypes.byref(slot))
            assert ok == 1 and page.value == lst[pos // size] and slot.value == pos % size
    for bad in (-1, 50, 51, 2 ** 31 - 1, -2 ** 31):
        lst = np.array([bad, 3], np.int32)
        assert host.check_row(lst.ctypes.data, 5, 16, 50, ctypes.byref(page), ctypes.byref(slot)) == 0
        assert host.check_row(lst.ctypes.data, 16, 16, 50, ctypes.byref(page), ctypes.byref(slot)) == 1


def test_tokens_find_their_sequence(host):
    for new in ([3], [0, 2, 0, 0, 5, 1, 0], [1] * 20, [0], [0, 0, 4]):
        for first in (0, 3):
            starts = np.cumsum([first] + new).astype(np.int32)
            want = [-1] * first + [b for b, c in enumerate(new) for _ in range(c)] + [-1, -1]
            got = [host.check_sequence(starts.ctypes.data, len(new), t) for t in range(len(want))]
            assert got == want


def test_keys_order_weights_as_numbers(host):
    vals = [-math.inf, -3.5, -1e-42, 0.0, 1e-42, 0.25, 0.5, 7.0, 1e30, math.inf]
    key = lambda x: host.check_key(int(np.float32(x).view(np.uint32)))
    keys = [key(v) for v in vals]
    assert keys == sorted(keys) and len(set(keys)) == len(keys)
    assert key(-0.0) == key(0.0)
    assert key(math.nan) < keys[0] and host.check_key(0xFFC00000) < keys[0]


def runs(host, lengths, window, tile, heads, places):
    """The runs of attention_decode, [(first, end)], each item's [first, end) tiles in them, the CTAs that share a
    run and the heads that a run goes through."""
    lo = ctypes.c_int()
    out = (ctypes.c_int * 3)()
    host.check_limits(out)
    lengths_of = [host.check_length_of(k) for k in range(out[2])]
    lanes = heads if places >= 8 * heads else 1
    through, most = heads // lanes, places // lanes
    counts = [host.check_tiles(n, window, tile, 1, ctypes.byref(lo)) for n in lengths]
    pad = 0
    if len(lengths) <= 32 and len(lengths) * through <= most:
        units = (ctypes.c_longlong * out[2])(*[sum(-(-c // u) for c in counts) * through for u in lengths_of])
        pad = host.check_pad(units, sum(counts) * through, most)
    if pad > 1:
        counts = [host.check_tiles(n, window, tile, pad, ctypes.byref(lo)) for n in lengths]
    total = sum(counts) * through
    ctas = total // pad if pad else min(most, total)
    items, at = [], 0
    for c in counts:
        for _ in range(through):
            items.append((at, at + c))
            at += c
    return [(host.check_first(c, ctas, total), host.check_first(c + 1, ctas, total)) for c in range(ctas)], items, total, lanes


@pytest.mark.parametrize("seed", range(60))
def test_runs_cover_every_tile_once_and_parts_have_slots_of_their_own(host, seed):
    rng = np.random.default_rng(seed)
    places = int(rng.choice([1, 2, 7, 152, 304, 320]))
    batch = int(rng.choice([1, 2, 5, 40, 300]))
    most = int(rng.choice([1, 64, 300, 5000, 200000]))
    lengths = rng.integers(0, most + 1, batch).tolist()
    window = int(rng.choice([0, 0, 1, 100]))
    tile = int(rng.choice([64, 96, 192]))
    cta_runs, items, total, lanes = runs(host, lengths, window, tile, int(rng.choice([1, 2, 3, 8, 24, 64])), places)
    assert len(cta_runs) * lanes <= places
    assert cta_runs[0][0] == 0 and cta_runs[-1][1] == total
    assert all(a < b for a, b in cta_runs) and all(x[1] == y[0] for x, y in zip(cta_runs, cta_runs[1:]))
    limits = (ctypes.c_int * 3)()
    host.check_limits(limits)
    slots, counters, tops = set(), set(), set()
    for first, end in items:
        c0, c1 = (host.check_owner(t, len(cta_runs), total) for t in (first, end - 1))
        assert cta_runs[c0][0] <= first < cta_runs[c0][1] and cta_runs[c1][0] < end <= cta_runs[c1][1]
        if c0 == c1:
            continue
        for lane in range(lanes):
            parts = [host.check_slot(c, c0, lane, lanes) for c in range(c0, c1 + 1)]
            assert not slots & set(parts) and len(set(parts)) == len(parts)
            assert max(parts) < 2 * limits[0]
            slots |= set(parts)
            groups = -(-len(parts) // limits[1])
            assert groups <= limits[1]
            heads = set(parts[::limits[1]])
            assert not counters & heads
            counters |= heads
            assert parts[0] not in tops
            tops.add(parts[0])


@pytest.mark.parametrize("lengths,heads", [([77, 300, 0, 2000], 2), ([4096], 8), ([2000] * 4, 8), ([100, 300] * 8, 8), ([30], 100)])
def test_few_tiles_make_runs_that_end_with_their_item(host, lengths, heads):
    cta_runs, items, _, _ = runs(host, lengths, 0, 96, heads, 304)
    assert all(any(a <= r[0] and r[1] <= b for a, b in items) for r in cta_runs)
    assert {a for a, _ in items} <= {r[0] for r in cta_runs}


def test_many_tiles_make_equal_runs(host):
    for lengths in ([100000, 3, 70000], [1000] * 60):
        cta_runs, _, total, lanes = runs(host, lengths, 0, 96, 8, 304)
        sizes = [b - a for a, b in cta_runs]
        assert len(cta_runs) == 304 // lanes and max(sizes) - min(sizes) <= 1


def test_owners_of_tiles_outside_stay_inside(host):
    """What inconsistent lengths could ask for must not lead out of the runs."""
    for t in (-5, -1, 100, 10 ** 12):
        assert 0 <= host.check_owner(t, 7, 100) < 7


def test_tiles_of_lengths_and_windows(host):
    lo = ctypes.c_int()
    for n, window, tile, pad, want, want_lo in ((0, 0, 64, 1, 1, 0), (0, 5, 64, 4, 4, 0), (1, 0, 64, 1, 1, 0), (64, 0, 64, 1, 1, 0),
                                                (65, 0, 64, 1, 2, 0), (65, 0, 64, 4, 4, 0), (65, 64, 64, 1, 1, 1),
                                                (1000, 130, 64, 1, 3, 870), (1 << 30, 0, 64, 4, 1 << 24, 0)):
        assert host.check_tiles(n, window, tile, pad, ctypes.byref(lo)) == want and lo.value == want_lo


# ---------------------------------------------------------------- the tests' own definitions
def test_attend64_against_brute_force():
    g = torch.Generator().manual_seed(0)
    q, k, v = torch.randn(4, 8, generator=g), torch.randn(5, 2, 8, generator=g).double(), torch.randn(5, 2, 8, generator=g).double()
    o, p, mag, reach, top = attend64(q, k, v, 0.3, cap=2.0)
    for h in range(4):
        s = [2.0 * math.tanh(0.3 * sum(float(q[h, d]) * float(k[j, h // 2, d]) for d in range(8)) / 2.0) for j in range(5)]
        z = sum(math.exp(x) for x in s)
        for d in range(8):
            assert abs(float(o[h, d]) - sum(math.exp(s[j]) / z * float(v[j, h // 2, d]) for j in range(5))) < 1e-12
        assert abs(float(p[h].sum()) - 1) < 1e-12


def test_evict_reference_small():
    w = np.array([1, 5, 5, 0, 2, 9], np.float32)
    assert evict_reference(w, 6, 3, 0) == [1, 2, 5]
    assert evict_reference(w, 6, 3, 1) == [1, 2, 5]
    assert evict_reference(w, 6, 3, 2) == [1, 4, 5]
    assert evict_reference(w, 6, 2, 5) == [4, 5]
    assert evict_reference(w, 2, 4, 1) == [0, 1]
    assert evict_reference(np.array([np.nan, -np.inf, 1], np.float32), 3, 2, 0) == [1, 2]


def test_make_table_names_every_page_once():
    t, pages = make_table([0, 5, 33], 16, 2, 0)
    used = [p for p in t.flatten().tolist() if p != 0x7FFFFFFF]
    assert len(used) == 4 == len(set(used)) and max(used) < pages
