"""Refusals of the head norms with the position rotation, on a machine without a GPU."""
from __future__ import annotations

import ctypes
from decimal import Decimal, getcontext

import pytest
import torch

import gemm_epilogue_02_gb300 as tg

OK, INVALID, ALIGN, UNSUPPORTED, ALIAS = 0, 1, 2, 3, 4
VALID = (OK, UNSUPPORTED, INVALID)     # no GPU here; on one these addresses are no device memory
MB = 1 << 20
AT = {n: (i + 1) * 256 * MB for i, n in enumerate(["q", "k", "qo", "ko", "qw", "kw", "pos", "gq", "gk", "gqw", "gkw", "ws"])}
TOKENS, HQ, HK, DIM = 100, 8, 2, 64


class Rotation:
    def __init__(self, pairs=32, axes=None, interleaved=0, turns=True):
        self.t = (ctypes.c_uint64 * 256)(*range(1, 257))
        self.a = (ctypes.c_int32 * 256)(*(axes or [0] * 256)[:256]) if axes else None
        c = tg.RotaryStruct()
        c.turns, c.axes = ctypes.addressof(self.t) if turns else None, ctypes.addressof(self.a) if axes else None
        c.pairs, c.interleaved = pairs, interleaved
        self.c = c

    @property
    def at(self):
        return ctypes.addressof(self.c)


def fields(**kw):
    d = {}
    for name, heads in (("q", HQ), ("k", HK), ("qo", HQ), ("ko", HK)):
        d.update({name: AT[name], name + "_t": heads * DIM, name + "_h": DIM})
    d.update(qw=AT["qw"], kw=AT["kw"], pos=AT["pos"], axis_stride=TOKENS, axes=1, tokens=TOKENS, hq=HQ, hk=HK, dim=DIM, shift=0,
             rotary=None, f32=0, norm=1, eps=1e-6, dtype=1)
    unknown = set(kw) - set(d)
    assert not unknown, unknown
    d.update(kw)
    return d


def forward(rotation=None, **kw):
    rotation = rotation or Rotation()
    d = fields(**kw)
    if d["rotary"] is None:
        d["rotary"] = rotation.at
    return tg.tgemm_qk_norm_rope(tg.QK_NORM_ROPE_ARGS.pack(*d.values()))


def backward(rotation=None, **kw):
    rotation = rotation or Rotation()
    more = dict(gq=AT["gq"], gq_t=HQ * DIM, gq_h=DIM, gk=AT["gk"], gk_t=HK * DIM, gk_h=DIM, gqw=AT["gqw"], gkw=AT["gkw"], ws=AT["ws"],
                wsb=64 * MB)
    for n in list(kw):
        if n in more:
            more[n] = kw.pop(n)
    d = fields(**kw)
    if d["rotary"] is None:
        d["rotary"] = rotation.at
    return tg.tgemm_qk_norm_rope_backward(tg.QK_NORM_ROPE_BACKWARD_ARGS.pack(*d.values(), *more.values()))


def test_valid_calls():
    assert forward() in VALID and backward() in VALID
    assert forward(tokens=0) == OK and backward(tokens=0, gqw=0, gkw=0) == OK
    assert forward(hq=0, hk=0) == OK
    assert forward(hk=0, k=0, ko=0) in VALID                      # queries alone
    none = dict(hk=0, k=0, k_t=0, k_h=0, ko=0, ko_t=0, ko_h=0)
    assert forward(**none) == forward() and backward(**none, gk=0, gk_t=0, gk_h=0) == backward()
    assert forward(Rotation(4), dim=8, q_t=64, q_h=8) in VALID
    # in place, and side by side with other rows of a projection's output
    assert forward(qo=AT["q"], ko=AT["k"]) in VALID
    row = (HQ + 2 * HK) * DIM
    side = dict(q_t=row, k=AT["q"] + 2 * HQ * DIM, k_t=row)
    assert forward(**side) in VALID
    assert forward(**side, qo=AT["q"], qo_t=row, ko=AT["q"] + 2 * HQ * DIM, ko_t=row) in VALID
    assert forward(**side, ko=AT["q"] + 2 * (HQ + HK) * DIM, ko_t=row) in VALID          # where the values were
    assert backward(qo=AT["gq"], ko=AT["gk"]) in VALID and backward(qo=AT["q"], ko=AT["k"]) in VALID
    assert backward(gqw=0, gkw=0, ws=0, wsb=0) in VALID
    assert backward(norm=0, qw=0, kw=0, gqw=0, gkw=0, q=0, k=0) in VALID       # a rotation alone does not read q and k
    assert forward(rotary=0, pos=0, axes=0, axis_stride=0) in VALID           # a norm alone
    assert forward(Rotation(axes=[0, 1] * 16), axes=2, axis_stride=0) in VALID         # axes that share positions


COMMON = [
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 31), INVALID), (dict(hq=-1), INVALID), (dict(hq=65536), INVALID),
    (dict(dim=60), INVALID), (dict(dim=264, q_t=8 * 264, q_h=264), INVALID), (dict(dim=0), INVALID), (dict(dtype=2), INVALID),
    (dict(norm=2), INVALID), (dict(f32=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(norm=0), INVALID), (dict(shift=2 ** 31), INVALID), (dict(axes=0), INVALID), (dict(axes=33), INVALID),
    (dict(pos=0), INVALID), (dict(pos=AT["pos"] + 2), ALIGN), (dict(qw=AT["qw"] + 1), ALIGN), (dict(f32=1, kw=AT["kw"] + 2), ALIGN),
    (dict(axes=2, axis_stride=2 ** 41), INVALID), (dict(axis_stride=-1), INVALID), (dict(qo=0), INVALID),
    (dict(qo=AT["qo"] + 8), ALIGN), (dict(qo_t=HQ * DIM + 4), ALIGN), (dict(qo_h=DIM - 8), INVALID), (dict(ko_h=-DIM), INVALID),
    (dict(qo=AT["q"] + 64), ALIAS), (dict(qo=AT["k"]), ALIAS), (dict(ko=AT["qo"]), ALIAS), (dict(qo=AT["pos"] - 1024), ALIAS),
    (dict(qo=AT["qw"]), ALIAS), (dict(qo=AT["q"], qo_t=HQ * DIM + 64), ALIAS), (dict(q_t=2 ** 62), INVALID),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(q=0), INVALID), (dict(k=AT["k"] + 2), ALIGN)])
def test_forward_refusals(kw, code):
    assert forward(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(q=0), INVALID), (dict(gq=0), INVALID), (dict(gk=AT["gk"] + 8), ALIGN), (dict(ws=0), INVALID), (dict(wsb=1024), INVALID),
    (dict(ws=AT["ws"] + 8), ALIGN), (dict(gqw=AT["gqw"] + 2), ALIGN), (dict(norm=0, qw=0, kw=0), INVALID),
    (dict(qo=AT["gq"] + 16), ALIAS), (dict(qo=AT["gk"]), ALIAS), (dict(gqw=AT["gkw"]), ALIAS), (dict(gqw=AT["ws"]), ALIAS),
    (dict(gqw=AT["qw"]), ALIAS), (dict(qo=AT["ws"]), ALIAS), (dict(gkw=AT["q"]), ALIAS), (dict(ws=AT["gq"]), ALIAS),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("rotation,code", [
    (Rotation(33), INVALID), (Rotation(-1), INVALID), (Rotation(30), INVALID), (Rotation(16, interleaved=2), INVALID),
    (Rotation(32, turns=False), INVALID), (Rotation(32, axes=[1] * 32), INVALID), (Rotation(32, axes=[-1] * 32), INVALID),
])
def test_rotation_refusals(rotation, code):
    assert forward(rotation) == code and backward(rotation) == code


def test_no_structure_and_no_work():
    assert tg.load().tgemm_qk_norm_rope(None, None) == INVALID and tg.load().tgemm_qk_norm_rope_backward(None, None) == INVALID
    assert forward(rotary=0, norm=0, qw=0, kw=0) == INVALID
    with pytest.raises(tg.TgemmError):
        tg.tgemm_qk_norm_rope_backward_workspace(12)
    assert tg.tgemm_qk_norm_rope_backward_workspace(128) > 0


def test_frequencies_become_turns():
    """f / (2 pi) * 2^64 modulo 2^64, to one unit."""
    getcontext().prec = 90
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    f = [10000.0 ** (-i / 64) for i in range(64)] + [0.0, -1.5, 7.0, 1e-300, 1.8e19, -12345678.9, 2.0 ** -60, 3e-19]
    for x, t in zip(f, tg.Rotary(f)._turns):
        want = int((Decimal(x) / (2 * pi) * Decimal(2) ** 64).to_integral_value(rounding="ROUND_FLOOR")) % 2 ** 64
        assert min((t - want) % 2 ** 64, (want - t) % 2 ** 64) <= 1


@pytest.mark.parametrize("f,kw", [
    ([1.0] * 6, {}), ([1.0, float("nan"), 1.0, 1.0], {}), ([1.0, float("inf")], dict(interleaved=True)), ([1.0] * 4, dict(axes=[0, 1])),
    ([1.0] * 4, dict(axes=[0, 0, 0, 32])), ([1.0] * 4, dict(axes=[0, 0, 0, -1])), ([2.0 ** 64] * 4, {}),
])
def test_rotary_refusals(f, kw):
    with pytest.raises(ValueError):
        tg.Rotary(f, **kw)


def tensors(**kw):
    d = dict(Q=torch.zeros(5, 4, 64, dtype=torch.float16), K=torch.zeros(5, 2, 64, dtype=torch.float16),
             positions=torch.zeros(1, 5, dtype=torch.int32), rotary=tg.Rotary([1.0] * 32), Q_out=torch.zeros(5, 4, 64, dtype=torch.float16),
             K_out=torch.zeros(5, 2, 64, dtype=torch.float16), q_weight=torch.ones(64), k_weight=torch.ones(64))
    d.update(kw)
    return d


H = torch.float16


@pytest.mark.parametrize("kw", [
    dict(), dict(Q=torch.zeros(5, 4, 64)), dict(Q=torch.zeros(5, 256, dtype=H)), dict(K=torch.zeros(4, 2, 64, dtype=H)),
    dict(K=torch.zeros(5, 2, 32, dtype=H)), dict(K=torch.zeros(5, 2, 64, dtype=torch.bfloat16)), dict(K=None), dict(K_out=None),
    dict(Q_out=torch.zeros(5, 3, 64, dtype=H)), dict(Q_out=torch.zeros(5, 64, 4, dtype=H).transpose(1, 2)),
    dict(Q=torch.zeros(5, 64, 4, dtype=H).transpose(1, 2)), dict(positions=None), dict(positions=torch.zeros(1, 5)),
    dict(positions=torch.zeros(1, 4, dtype=torch.int32)), dict(rotary=tg.Rotary([1.0] * 32, axes=[1] * 32)),
    dict(rotary=tg.Rotary([1.0] * 36)), dict(q_weight=torch.ones(63)), dict(q_weight=torch.ones(64, dtype=torch.float64)),
    dict(q_weight=torch.ones(64, dtype=H)), dict(q_weight=torch.ones(128)[::2]), dict(eps=None),
    dict(eps=None, rotary=None, q_weight=None, k_weight=None),
])
def test_python_refusals(kw):
    """The first is right but for its device: none of these reaches the library."""
    d = tensors(**kw)
    with pytest.raises(ValueError):
        tg.qk_norm_rope(**d)
    grads = {"Q_out_grad": d["Q_out"], "K_out_grad": d["K_out"], "Q_grad": d["Q_out"], "K_grad": d["K_out"]}
    with pytest.raises(ValueError):
        tg.qk_norm_rope_backward(**grads, **{n: x for n, x in d.items() if not n.endswith("_out")})


@pytest.mark.parametrize("kw", [dict(q_weight_grad=torch.zeros(63)), dict(k_weight_grad=torch.zeros(64, dtype=H)),
                                dict(q_weight_grad=torch.zeros(64), eps=None, q_weight=None, k_weight=None)])
def test_python_gradient_refusals(kw):
    d = tensors(**{n: x for n, x in kw.items() if not n.endswith("_grad")})
    with pytest.raises(ValueError):
        tg.qk_norm_rope_backward(d["Q_out"], d["K_out"], d["Q"], d["K"], d["positions"], d["rotary"], d["Q_out"], d["K_out"],
                                 q_weight=d["q_weight"], k_weight=d["k_weight"], **{n: x for n, x in kw.items() if not n.endswith("weight")})


@pytest.mark.parametrize("eps,code", [(1e39, INVALID), (float("inf"), INVALID), (3.4e38, VALID), (1e-60, VALID), (0.0, VALID)])
def test_range_of_eps(eps, code):
    for call in (forward, backward):
        assert call(eps=eps) == code if code == INVALID else call(eps=eps) in code and call(eps=eps) == call()


@pytest.mark.parametrize("tokens,heads,t,h,code", [
    (100, 8, 512, 64, VALID), (100, 8, 504, 64, ALIAS), (100, 8, 64, 6400, VALID), (100, 8, 64, 6392, ALIAS), (100, 8, 64, 64, ALIAS),
    (2, 2, 64, 64, ALIAS), (1, 8, 64, 64, VALID), (100, 1, 64, 64, VALID), (100, 2, 192, 128, VALID), (100, 8, 128, 192, ALIAS),
    (3, 2, 128, 192, VALID), (100, 2, 128, 200, ALIAS),
])
def test_rows_that_are_written_lie_apart(tokens, heads, t, h, code):
    """Steps of t elements from token to token and h from head to head, rows of 64."""
    kw = dict(tokens=tokens, hq=heads, q_t=heads * DIM, qo_t=t, qo_h=h)
    offsets = sorted(i * t + j * h for i in range(tokens) for j in range(heads))
    assert any(b - a < DIM for a, b in zip(offsets, offsets[1:])) == (code == ALIAS)
    for call, more in ((forward, {}), (backward, dict(gq_t=heads * DIM))):
        got = call(**kw, **more)
        assert got == code if code == ALIAS else got in code and got == call()
