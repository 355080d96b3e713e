"""Head norms with the position rotation, and their gradient, against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from rope_helpers import TDT, angles64, backward64, close, forward64

pytestmark = pytest.mark.gpu


def frequencies(pairs, base=10000.0):
    return [base ** (-i / max(1, pairs)) for i in range(pairs)]


def case(tokens, q_heads, k_heads, dim, dtype, axes=1, far=1000, seed=0, fused=True, gain=1.0):
    """Queries and keys as slices of one projection (or apart), and positions."""
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = (torch.randn(tokens, q_heads + 2 * k_heads, dim, generator=g) * gain).to(TDT[dtype]).cuda()
        q, k = x[:, :q_heads], x[:, q_heads:q_heads + k_heads]
    else:
        q, k = ((torch.randn(tokens, h, dim, generator=g) * gain).to(TDT[dtype]).cuda() for h in (q_heads, k_heads))
    positions = torch.randint(0, far + 1, (axes, tokens), generator=g).to(torch.int32).cuda()
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).to(TDT[dtype]).cuda() for _ in range(2)]
    return q, k, positions, w


SHAPES = [
    # tokens, q_heads, k_heads, dim, pairs, interleaved, axes
    (1, 8, 8, 64, 32, False, 1), (1, 1, 1, 128, 64, False, 1), (7, 3, 1, 128, 64, True, 1), (33, 5, 2, 80, 40, False, 2),
    (19, 6, 3, 80, 20, False, 1), (40, 4, 4, 96, 24, True, 1), (65, 24, 8, 112, 28, False, 3), (17, 2, 2, 256, 128, False, 1),
    (9, 3, 2, 256, 64, True, 3), (5, 2, 1, 8, 4, False, 1), (5, 2, 1, 8, 3, True, 1), (300, 32, 8, 128, 64, False, 3),
    (13, 9, 5, 72, 36, False, 1), (21, 7, 3, 200, 16, False, 1), (11, 40, 1, 248, 124, False, 2), (600, 1, 1, 64, 0, False, 1),
    (3, 1, 0, 128, 64, False, 1),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(cuda_lib, shape, dtype):
    tokens, q_heads, k_heads, dim, pairs, interleaved, n_axes = shape
    q, k, positions, w = case(tokens, q_heads, k_heads, dim, dtype, n_axes, far=70000, seed=tokens)
    if k_heads == 0:
        k = None
    f, axes = frequencies(pairs), [i * n_axes // max(1, pairs) for i in range(pairs)]
    rotary = tg.Rotary(f, axes=axes, interleaved=interleaved)
    angle = angles64(positions, f, axes)
    qo = torch.full((tokens + 2, q_heads + 1, dim + 8), 77.0, dtype=q.dtype, device="cuda")   # what lies around stays
    q_out, k_out = qo[1:-1, :q_heads, :dim], None if k is None else torch.empty(k.shape, dtype=k.dtype, device="cuda")
    tg.qk_norm_rope(q, k, positions, rotary, q_out, k_out, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    close(q_out, *forward64(q, w[0], 1e-6, angle, interleaved), dtype)
    if k is not None:
        close(k_out, *forward64(k, w[1], 1e-6, angle, interleaved), dtype)
    qo[1:-1, :q_heads, :dim] = 77.0
    assert (qo == 77.0).all()

    g = torch.Generator().manual_seed(1)
    dq, dk = (None if t is None else torch.randn(t.shape, generator=g).to(t.dtype).cuda() for t in (q, k))
    dqi, dki = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    dw = [torch.full((dim,), float("nan"), device="cuda") for _ in range(2)]
    tg.qk_norm_rope_backward(dq, dk, q, k, positions, rotary, dqi, dki, q_weight=w[0], k_weight=w[1], q_weight_grad=dw[0],
                             k_weight_grad=dw[1])
    torch.cuda.synchronize()
    for x, wi, dy, dx, dwi in ((q, w[0], dq, dqi, dw[0]), (k, w[1], dk, dki, dw[1])):
        if x is None:
            assert (dwi == 0).all()          # no rows
            continue
        want, bound, want_w, bound_w = backward64(x, wi, dy, 1e-6, angle, interleaved)
        close(dx, want, bound, dtype)
        assert ((dwi.double().cpu() - want_w).abs() <= bound_w).all()
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gradient_against_differences(cuda_lib, dtype):
    """Central differences of the definition in 64 bits along random directions."""
    tokens, heads, dim, pairs, eps = 5, 3, 64, 16, 1e-3
    q, k, positions, w = case(tokens, heads, heads, dim, dtype, seed=3)
    f = frequencies(pairs)
    angle = angles64(positions, f, [0] * pairs)
    rotary = tg.Rotary(f)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(tokens, heads, dim, generator=g).to(TDT[dtype])
    dx, dw = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(dim, device="cuda")
    tg.qk_norm_rope_backward(dy.cuda(), None, q, None, positions, rotary, dx, None, q_weight=w[0], q_weight_grad=dw, eps=eps)
    want, bound, _, bound_w = backward64(q, w[0], dy, eps, angle, False)
    u = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    for i in range(6):
        d, dd = torch.randn(q.shape, generator=g, dtype=torch.float64), torch.randn(dim, generator=g, dtype=torch.float64)
        h = 1e-4

        def loss(t):
            return (dy.double() * forward64(q.double().cpu() + t * d, w[0].double().cpu() + t * dd, eps, angle, False)[0]).sum()

        slope = (loss(h) - loss(-h)) / (2 * h)
        got = (dx.double().cpu() * d).sum() + (dw.double().cpu() * dd).sum()
        # the third derivative of x / |x| is of order 1 / |x|^3 here: h^2 times it, well below 1e-4 of the slope's size
        room = ((u * want.abs() + bound) * d.abs()).sum() + (bound_w * dd.abs()).sum() + 1e-4 * (dy.double().abs().sum() * h + 1)
        assert abs(got - slope) <= room


@pytest.mark.parametrize("far", [2 ** 31 - 1, -2 ** 31, 10 ** 6])
def test_far_positions(cuda_lib, far):
    """Angles keep 2^-31 of a turn at any position; what 64 bits lose of far * f themselves is allowed for."""
    tokens, heads, dim = 64, 2, 128
    q, k, _, _ = case(tokens, heads, heads, dim, "fp16", seed=9)
    step = -1 if far > 0 else 1
    positions = (far + step * torch.arange(tokens)).to(torch.int32).view(1, -1).cuda()
    f = frequencies(64)
    q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    tg.qk_norm_rope(q, k, positions, tg.Rotary(f), q_out, k_out, eps=None)
    angle = angles64(positions, f, [0] * 64)
    want, bound = forward64(q, None, None, angle, False)
    close(q_out, want, bound + abs(far) * 2.0 ** -52 * q.double().cpu().abs().amax(), "fp16")


@pytest.mark.parametrize("shift", [-1, 5])
def test_shift_and_lengths(cuda_lib, shift):
    q, k, positions, w = case(12, 4, 2, 64, "bf16", seed=2)
    f = frequencies(32)
    out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
    tg.qk_norm_rope(q, k, positions[0], tg.Rotary(f), *out, q_weight=w[0], k_weight=w[1], shift=shift)     # [tokens]
    angle = angles64(positions, f, [0] * 32, shift)
    close(out[0], *forward64(q, w[0], 1e-6, angle, False), "bf16")


def test_axes_that_share_positions(cuda_lib):
    q, k, positions, w = case(9, 4, 2, 64, "fp16", seed=20)
    f = frequencies(32)
    one, three = ([torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)] for _ in range(2))
    tg.qk_norm_rope(q, k, positions, tg.Rotary(f), *one, q_weight=w[0], k_weight=w[1])
    tg.qk_norm_rope(q, k, positions.expand(3, -1), tg.Rotary(f, axes=[i % 3 for i in range(32)]), *three, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert torch.equal(one[0], three[0]) and torch.equal(one[1], three[1])


@pytest.mark.parametrize("mode", ["norm_only", "rotation_only", "f32_weights", "no_weights"])
def test_parts_of_it(cuda_lib, mode):
    tokens, dim, pairs = 50, 96, 48
    q, k, positions, w = case(tokens, 5, 2, dim, "bf16", seed=4, fused=False)
    f = frequencies(pairs)
    rotary = None if mode == "norm_only" else tg.Rotary(f)
    eps = None if mode == "rotation_only" else 1e-5
    if mode == "f32_weights":
        w = [torch.randn(dim, device="cuda") for _ in range(2)]
    elif mode != "norm_only":
        w = [None, None]
    out = [torch.empty_like(t) for t in (q, k)]
    tg.qk_norm_rope(q, k, None if rotary is None else positions, rotary, *out, q_weight=w[0], k_weight=w[1], eps=eps)
    angle = angles64(positions, f, [0] * pairs) if rotary else torch.zeros(tokens, 1, 0, dtype=torch.float64)
    dy = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q, k)]
    dx = [torch.empty_like(t) for t in (q, k)]
    tg.qk_norm_rope_backward(*dy, q, k, None if rotary is None else positions, rotary, *dx, q_weight=w[0], k_weight=w[1], eps=eps)
    for i, x in enumerate((q, k)):
        close(out[i], *forward64(x, w[i], eps, angle, False), "bf16")
        want, bound, _, _ = backward64(x, w[i], dy[i], eps, angle, False)
        close(dx[i], want, bound, "bf16")


def test_in_place(cuda_lib):
    """Inside the projection's output, and gradients over what they come from: the same as apart."""
    q, k, positions, w = case(77, 6, 3, 128, "bf16", seed=6)
    rotary = tg.Rotary(frequencies(64))
    apart = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
    tg.qk_norm_rope(q, k, positions, rotary, *apart, q_weight=w[0], k_weight=w[1])
    v_before = q._base[:, 9:].clone()
    q0, k0 = q.clone(), k.clone()
    tg.qk_norm_rope(q, k, positions, rotary, q, k, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert torch.equal(q, apart[0]) and torch.equal(k, apart[1]) and torch.equal(q._base[:, 9:], v_before)
    dy = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q0, k0)]
    dx = [torch.empty_like(t) for t in (q0, k0)]
    dw = [torch.empty(128, device="cuda") for _ in range(4)]
    ws = tg.qk_norm_rope_backward_workspace(q0, k0)
    args = dict(q_weight=w[0], k_weight=w[1], workspace=ws)
    tg.qk_norm_rope_backward(*dy, q0, k0, positions, rotary, *dx, q_weight_grad=dw[0], k_weight_grad=dw[1], **args)
    over = [t.clone() for t in dy]
    tg.qk_norm_rope_backward(*over, q0, k0, positions, rotary, *over, q_weight_grad=dw[2], k_weight_grad=dw[3], **args)
    inputs = [q0.clone(), k0.clone()]
    tg.qk_norm_rope_backward(*dy, *inputs, positions, rotary, *inputs, **args)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(over[i], dx[i]) and torch.equal(inputs[i], dx[i]) and torch.equal(dw[i], dw[2 + i])


@pytest.mark.parametrize("scale", [0.0, 1e-4, 200.0])
def test_sizes_of_values(cuda_lib, scale):
    """Rows of zeros, small and large ones."""
    q, k, positions, w = case(10, 3, 2, 64, "fp16", seed=8, gain=scale)
    f = frequencies(32)
    out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
    tg.qk_norm_rope(q, k, positions, tg.Rotary(f), *out, q_weight=w[0], k_weight=w[1])
    angle = angles64(positions, f, [0] * 32)
    close(out[0], *forward64(q, w[0], 1e-6, angle, False), "fp16")
    close(out[1], *forward64(k, w[1], 1e-6, angle, False), "fp16")


def test_not_finite_values_stay_in_their_row(cuda_lib):
    q, k, positions, w = case(9, 4, 2, 128, "bf16", seed=11, fused=False)
    rotary = tg.Rotary(frequencies(64))
    clean = [torch.empty_like(t) for t in (q, k)]
    tg.qk_norm_rope(q, k, positions, rotary, *clean, q_weight=w[0], k_weight=w[1])
    q[3, 1, 5], k[7, 0, 100] = float("nan"), float("inf")
    out = [torch.empty_like(t) for t in (q, k)]
    tg.qk_norm_rope(q, k, positions, rotary, *out, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert out[0][3, 1].isnan().all() and out[1][7, 0, [36, 100]].isnan().all()
    clean[0][3, 1], out[0][3, 1] = 0, 0
    clean[1][7, 0], out[1][7, 0] = 0, 0
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1], clean[1])


def test_no_tokens(cuda_lib):
    q, k = (torch.empty(0, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2))
    positions = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    rotary = tg.Rotary(frequencies(32))
    tg.qk_norm_rope(q, k, positions, rotary, q, k)
    w = torch.ones(64, device="cuda")
    dw = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    tg.qk_norm_rope_backward(q, k, q, k, positions, rotary, q, k, q_weight=w, k_weight=w, q_weight_grad=dw[0], k_weight_grad=dw[1])
    torch.cuda.synchronize()
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


def test_the_same_bits_again(cuda_lib):
    q, k, positions, w = case(700, 8, 2, 128, "bf16", seed=12)
    rotary = tg.Rotary(frequencies(64))
    dy = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q, k)]
    results = []
    ws = None
    for again in (False, True, True, False):
        ws = ws if again else tg.qk_norm_rope_backward_workspace(q, k)     # left fit for the next call
        dx = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
        dw = [torch.empty(128, device="cuda") for _ in range(2)]
        tg.qk_norm_rope_backward(*dy, q, k, positions, rotary, *dx, q_weight=w[0], k_weight=w[1], q_weight_grad=dw[0],
                                 k_weight_grad=dw[1], workspace=ws)
        results.append(dx + dw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))


def test_graph_and_side_stream(cuda_lib):
    """Captured once, replayed for the positions and rows found at each replay; on another stream than the current one;
    eager calls between replays use their own workspace."""
    q, k, positions, w = case(40, 4, 2, 64, "fp16", seed=13)
    rotary = tg.Rotary(frequencies(32))
    dy = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q, k)]

    def everything(stream=None, ws=None):
        out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)] * 1
        dx = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
        dw = [torch.empty(64, device="cuda") for _ in range(2)]
        tg.qk_norm_rope(q, k, positions, rotary, *out, q_weight=w[0], k_weight=w[1], stream=stream)
        tg.qk_norm_rope_backward(*dy, q, k, positions, rotary, *dx, q_weight=w[0], k_weight=w[1], q_weight_grad=dw[0],
                                 k_weight_grad=dw[1], workspace=ws, stream=stream)
        return out + dx + dw

    ws = tg.qk_norm_rope_backward_workspace(q, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = everything(ws=ws)
    side = torch.cuda.Stream()
    for i in range(3):
        positions.random_(0, 5000)
        q.normal_()
        graph.replay()
        plain = everything()
        torch.cuda.synchronize()
        aside = everything(stream=side)
        side.synchronize()
        for a, b, c in zip(captured, plain, aside):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_debug_build_finds_nothing(cuda_lib):
    from gemm_epilogue_02_gb300 import _binding
    dbg = tg.load_debug()
    assert dbg.tgemm_debug_last_check() == 0
    release = _binding._lib
    results = []
    for lib in (release, dbg):
        _binding._lib = lib
        try:
            row = []
            for shape in SHAPES[:10]:
                tokens, q_heads, k_heads, dim, pairs, interleaved, n_axes = shape
                q, k, positions, w = case(tokens, q_heads, k_heads, dim, "bf16", n_axes, seed=tokens)
                f, axes = frequencies(pairs), [i * n_axes // max(1, pairs) for i in range(pairs)]
                rotary = tg.Rotary(f, axes=axes, interleaved=interleaved)
                out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
                dw = [torch.empty(dim, device="cuda") for _ in range(2)]
                tg.qk_norm_rope(q, k, positions, rotary, *out, q_weight=w[0], k_weight=w[1])
                row += [t.clone() for t in out]
                tg.qk_norm_rope_backward(*out, q, k, positions, rotary, *out, q_weight=w[0], k_weight=w[1], q_weight_grad=dw[0],
                                         k_weight_grad=dw[1])
                row += out + dw
            torch.cuda.synchronize()
            results.append(row)
        finally:
            _binding._lib = release
    assert dbg.tgemm_last_device_status() == 0 and dbg.tgemm_debug_last_check() == 0
    assert all(torch.equal(a, b) for a, b in zip(*results))


def odd_values(x, at, seed=0):
    """x with infinities, NaN and zeros of both signs in some of the elements `at` of its rows."""
    g = torch.Generator().manual_seed(seed)
    y = x.clone()
    for value in (float("inf"), float("-inf"), float("nan"), 0.0, -0.0):
        where = torch.zeros(x.shape, dtype=torch.bool)
        where[..., at] = torch.rand(x[..., at].shape, generator=g) < 0.1
        y[where.to(x.device)] = value
    return y


def same_bits(a, b):
    """Equal, signs of zeros included; NaN to NaN."""
    return bool(((a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())).all())


PARTS = [(128, 32, False), (128, 24, True), (96, 20, False), (8, 3, True), (256, 64, False), (72, 8, False), (64, 0, False), (112, 49, True)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,pairs,interleaved", PARTS)
def test_elements_past_the_pairs_stay(cuda_lib, dim, pairs, interleaved, dtype):
    """Infinities, NaN and the signs of zeros past the pairs stay where they are and touch nothing else, in both directions;
    so do those of the pairs."""
    q, k, positions, _ = case(23, 5, 2, dim, dtype, seed=30, far=900)
    f = frequencies(pairs)
    rotary, angle = tg.Rotary(f, interleaved=interleaved), angles64(positions, f, [0] * pairs)
    past = list(range(2 * pairs, dim))
    for where in (past, list(range(2 * pairs))):
        x = [odd_values(t, where, seed=31) for t in (q, k)] if where else [q.clone(), k.clone()]
        out, back = ([torch.empty_like(t) for t in x] for _ in range(2))
        tg.qk_norm_rope(*x, positions, rotary, *out, eps=None)
        tg.qk_norm_rope_backward(*x, x[0], x[1], positions, rotary, *back, eps=None)
        torch.cuda.synchronize()
        for t, y, z in zip(x, out, back):
            assert same_bits(y[..., past], t[..., past]) and same_bits(z[..., past], t[..., past])
            if where is past:
                clean = t.double().cpu()
                clean[..., past] = 0
                for got, a in ((y, angle), (z, -angle)):
                    want, bound = forward64(clean, None, None, a, interleaved)
                    close(got[..., :2 * pairs], want[..., :2 * pairs], bound[..., :2 * pairs], dtype)


@pytest.mark.parametrize("pairs,interleaved", [(32, False), (24, True), (0, False)])
def test_infinity_past_the_pairs_with_the_norm(cuda_lib, pairs, interleaved):
    """A row with an infinity has r = 0: the infinity becomes NaN, every other element 0."""
    q, k, positions, w = case(6, 4, 2, 128, "bf16", seed=32, fused=False)
    q[2, 1, 77], k[5, 0, 120] = float("inf"), float("-inf")
    out = [torch.empty_like(t) for t in (q, k)]
    rotary = tg.Rotary(frequencies(pairs), interleaved=interleaved) if pairs else None
    tg.qk_norm_rope(q, k, positions, rotary, *out, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    for row, at in ((out[0][2, 1], 77), (out[1][5, 0], 120)):
        assert row[at].isnan()
        row[at] = 0
        assert (row == 0).all()
    assert out[0].isfinite().all() and out[1].isfinite().all()


@pytest.mark.parametrize("q_heads,k_heads,dim,pairs,interleaved", [
    (6, 3, 128, 64, False), (4, 1, 64, 32, False), (1, 1, 96, 48, True), (3, 5, 72, 36, False), (7, 2, 256, 128, False), (1, 0, 32, 16, False),
])
def test_gradient_without_eps(cuda_lib, q_heads, k_heads, dim, pairs, interleaved):
    """eps = 0, heads that do not fill the rows a warp has at a time: the weights' gradients are those of the rows there are."""
    q, k, positions, w = case(37, q_heads, max(1, k_heads), dim, "bf16", seed=33)
    if k_heads == 0:
        k = None
    f = frequencies(pairs)
    rotary, angle = tg.Rotary(f, interleaved=interleaved), angles64(positions, f, [0] * pairs)
    g = torch.Generator().manual_seed(34)
    dq, dk = (None if t is None else torch.randn(t.shape, generator=g).to(t.dtype).cuda() for t in (q, k))
    dqi, dki = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    dw = [torch.empty(dim, device="cuda") for _ in range(2)]
    tg.qk_norm_rope_backward(dq, dk, q, k, positions, rotary, dqi, dki, q_weight=w[0], k_weight=w[1], q_weight_grad=dw[0],
                             k_weight_grad=dw[1], eps=0.0)
    torch.cuda.synchronize()
    for x, wi, dy, dx, dwi in ((q, w[0], dq, dqi, dw[0]), (k, w[1], dk, dki, dw[1])):
        if x is None:
            assert (dwi == 0).all()
            continue
        want, bound, want_w, bound_w = backward64(x, wi, dy, 0.0, angle, interleaved)
        close(dx, want, bound, "bf16")
        assert ((dwi.double().cpu() - want_w).abs() <= bound_w).all()


def test_smallest_eps(cuda_lib):
    """An eps below fp32's numbers is not 0: a row of zeros stays one, and so does its gradient's part in the weights'."""
    q, _, positions, w = case(9, 3, 1, 64, "bf16", seed=35, fused=False)
    q[4, 1] = 0
    f = frequencies(32)
    rotary, angle = tg.Rotary(f), angles64(positions, f, [0] * 32)
    out, dw = torch.empty_like(q), torch.empty(64, device="cuda")
    tg.qk_norm_rope(q, None, positions, rotary, out, None, q_weight=w[0], eps=1e-60)
    dy, dx = torch.randn(q.shape, device="cuda").bfloat16(), torch.empty_like(q)
    dy[4, 1] = 0
    tg.qk_norm_rope_backward(dy, None, q, None, positions, rotary, dx, None, q_weight=w[0], q_weight_grad=dw, eps=1e-60)
    torch.cuda.synchronize()
    close(out, *forward64(q, w[0], 1e-60, angle, False), "bf16")
    want, bound, want_w, bound_w = backward64(q, w[0], dy, 1e-60, angle, False)
    close(dx, want, bound, "bf16")
    assert ((dw.double().cpu() - want_w).abs() <= bound_w).all()
