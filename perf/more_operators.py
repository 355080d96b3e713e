"""Cases of the operators around the paged key-value cache: norms of queries and keys with the position rotation (rotate,
rotate_back), sparse attention over pages that a cheap score selects (bounds, sparse), and the pages themselves (fork,
compact).

The cache is two pools, keys and values, [pages, page_size, kv_heads, dim], in 16 bits or in e4m3 with one fp32 scale per row;
a sequence's pages are listed in its row of a page table, and uses[page] counts the sequences that hold it.

    rotate       y = R(x * r * w) of each query and key head, r = 1 / sqrt(mean x^2 + eps), R the rotation of the first `rot`
                 elements: pair i, elements (i, i + rot / 2) or (2 i, 2 i + 1), by the angle positions[axis_i] * frequency_i.
    rotate_back  its gradients: those of x and of the two weight vectors.
    bounds       of each page that the newest tokens complete, and each key head: top = the largest |k|, scale = the least
                 power of two (2^-100 at least) with top <= 127 scale, lo = floor(least k_d / scale), hi = ceil(largest k_d / scale).
    sparse       a page's score is the largest over the group's heads of S = scale_page scale_q sum_d max(q_d lo_d, q_d hi_d), q_d
                 the query in whole numbers (nearest, even) of a power of two scale_q found as above. Of a sequence's pages
                 `keep` stay: the first `first`, the last `recent`, and of the others those of largest score (ties to the
                 lowest position). Attention of the query over these pages' positions follows.
    fork         one step of a search: the children of the step before are freed, each child takes over its parent's positions
                 (full pages are shared, the rows of a last, partly filled one are copied to a page of its own) and grows by
                 one token. New pages are the lowest free ones, in the order of the children.
    compact      the pages in use move below their number: those above it, in order, to the free ones below, in order.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # One request's newest token in a small model: the smallest call, all latency.
        dict(name="rotate_one_token", op="rotate", tokens=1, q_heads=16, k_heads=4, dim=64, rot=64, axes=1, interleaved=False,
             dtype="fp16", far=5000),
        # A long prompt of text and pictures: positions in time, height and width.
        dict(name="rotate_prompt_axes", op="rotate", tokens=24571, q_heads=32, k_heads=8, dim=128, rot=128, axes=3,
             interleaved=False, dtype="bf16", far=1000000),
        # A short training sequence with odd sizes: half of each head rotated, pairs side by side.
        dict(name="rotate_back_uneven", op="rotate_back", tokens=333, q_heads=6, k_heads=3, dim=96, rot=48, axes=1,
             interleaved=True, dtype="fp16", far=400),
        # An ordinary training batch.
        dict(name="rotate_back_batch", op="rotate_back", tokens=16384, q_heads=32, k_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, dtype="bf16", far=8192),
        # A serving batch's step: one token each, some of which complete a page.
        dict(name="bounds_step", op="bounds", batch=128, new=1, most=1, context=4000, kv_heads=8, dim=128, page=16,
             dtype="bf16", cache="16"),
        # Prompts of uneven length, a cache in 8 bits, an odd page size.
        dict(name="bounds_prompts_e4m3", op="bounds", batch=13, new=1, most=30000, context=0, kv_heads=8, dim=128, page=24,
             dtype="bf16", cache="e4m3"),
        # One request with a document.
        dict(name="sparse_one", op="sparse", batch=1, least=20011, most=20011, kv_heads=8, group=4, dim=128, page=16,
             dtype="fp16", cache="16", keep=64, first=1, recent=4),
        # A full serving batch of ragged long contexts, the largest.
        dict(name="sparse_batch", op="sparse", batch=32, least=1, most=65536, kv_heads=8, group=8, dim=128, page=32,
             dtype="bf16", cache="16", keep=128, first=1, recent=8),
        # A small search over two prompts.
        dict(name="fork_beams", op="fork", batch=2, least=500, most=1000, children=8, kv_heads=8, dim=64, page=16,
             dtype="fp16", cache="16", spare=1.2),
        # Many samples of each of several long prompts.
        dict(name="fork_samples", op="fork", batch=16, least=1, most=16384, children=128, kv_heads=8, dim=128, page=64,
             dtype="bf16", cache="16", spare=1.5),
        # A small pool with holes where requests have ended.
        dict(name="compact_small", op="compact", batch=5, least=1, most=400, kv_heads=4, dim=64, page=16, dtype="fp16",
             cache="16", spare=1.6, shared=2),
        # A large pool after a busy hour.
        dict(name="compact_large", op="compact", batch=48, least=100, most=9000, kv_heads=8, dim=128, page=64, dtype="bf16",
             cache="16", spare=1.8, shared=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_back", "bounds", "sparse", "sparse", "fork", "compact"])
    case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), dim=rng.choice([64, 64, 80, 96, 112, 128, 128, 256]))
    if op in ("rotate", "rotate_back"):
        case.update(q_heads=rng.choice([1, 3, 8, 16, 24, 32, 40, 64]), k_heads=rng.choice([1, 2, 3, 4, 8, 8, 16]),
                    axes=rng.choice([1, 1, 1, 2, 3]), interleaved=rng.random() < 0.3, far=_log(rng, 10, 1000000))
        case["rot"] = case["dim"] if rng.random() < 0.7 else case["dim"] // 2
        most = (20000 if op == "rotate" else 14000) * 40 * 128 // ((case["q_heads"] + case["k_heads"]) * case["dim"])
        case["tokens"] = _log(rng, 1, min(most, 100000))
        return case
    case.update(cache=rng.choice(["16", "16", "e4m3"]), kv_heads=rng.choice([1, 2, 3, 4, 8, 8, 16]),
                page=rng.choice([8, 16, 16, 20, 24, 32, 64, 128]))
    rows = 8 * 128 / (case["kv_heads"] * case["dim"])              # positions of a row of the listed cases' size
    if op == "bounds":
        batch = _log(rng, 1, 200)
        if rng.random() < 0.4:
            case.update(batch=batch, new=1, most=1, context=_log(rng, 1, max(2, min(8000, int(200000 * rows) // batch))))
        else:
            case.update(batch=batch, new=0, most=_log(rng, 1, max(2, min(40000, int(200000 * rows) // batch))),
                        context=_log(rng, 1, 200))
    elif op == "sparse":
        batch = _log(rng, 1, 64)
        group = min(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 24]), 128 // case["kv_heads"])
        most = _log(rng, rng.choice([1, 500]), max(2, min(131072, int(800000 * rows) // batch)))
        keep = _log(rng, 2, max(3, min(2 + most // case["page"], int(80000 * rows) // batch // case["page"] // max(1, group // 8))))
        case.update(batch=batch, least=rng.choice([0, 1, max(1, most // 2), most]), most=most, keep=keep, group=group,
                    first=rng.choice([0, 0, 1]), recent=rng.choice([1, 1, max(1, keep // 8), keep - 1]))
    else:
        batch = _log(rng, 1, 64)
        most = _log(rng, 1, max(2, min(16384, int(200000 * rows) // batch)))
        case.update(batch=batch, least=rng.choice([0, 1, max(1, most // 2), most]), most=most, spare=rng.choice([1.1, 1.5, 1.9]))
        if op == "fork":
            case.update(children=_log(rng, 1, 160))
        else:
            case.update(shared=rng.choice([0, 1, batch]))
    return case


# ---------------------------------------------------------------- inputs
def _ints(gen, least, most, n):
    """n whole numbers in least..most, the first of them the largest."""
    out = torch.randint(least, most + 1, (n,), generator=gen).tolist()
    out[0] = most
    return out


def _lengths(case):
    """(lengths, new tokens or parents) of each sequence, on the host. They belong to the case; a seed changes what the rows
    hold and where they lie."""
    gen = torch.Generator().manual_seed(case["batch"] * 7919 + case["most"])
    if case["op"] == "bounds":
        new = _ints(gen, case["new"], case["most"], case["batch"])
        context = _ints(gen, case["context"] // 2, case["context"], case["batch"])
        return [c + n for c, n in zip(context, new)], new
    lengths = _ints(gen, case["least"], case["most"], case["batch"])
    if case["op"] == "fork":
        return lengths, _ints(gen, 0, case["batch"] - 1, case["children"])
    return lengths, None


def _frequencies(case):
    """Radians that each pair turns by per position, and the axis whose position counts."""
    half = case["rot"] // 2
    return [10000.0 ** (-i / half) for i in range(half)], [i * case["axes"] // half for i in range(half)]


def _table(counts, page, spare, seed):
    """A page table [batch, most pages + 1] (-1 past a sequence's own) over shuffled pages, and the pool's number of pages."""
    need = [(n + page - 1) // page for n in counts]
    pages = int(sum(need) * spare) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed), dtype=torch.int64).to(torch.int32)
    table = torch.full((len(counts), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _split(x):
    """The e4m3 elements and the scale of each row of x [..., dim]."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (x / scale.unsqueeze(-1)).to(E4M3), scale


def _pools(case, pages, gen):
    """k, v, k_scale, v_scale (the scales None for a 16-bit cache): normal values, a few channels of the keys larger."""
    out, shape = [], (case["page"], case["kv_heads"], case["dim"])
    step = max(1, 2 ** 27 // math.prod(shape))
    for which in range(2):
        parts, scales = [], []
        for at in range(0, pages, step):
            x = torch.randn((min(step, pages - at),) + shape, device="cuda", dtype=DT[case["dtype"]], generator=gen)
            x[..., :2] *= 3 - 2 * which
            if case["cache"] == "e4m3":
                e, s = _split(x)
                parts.append(e.view(torch.uint8))
                scales.append(s)
            else:
                parts.append(x)
        out.append((torch.cat(parts).view(E4M3), torch.cat(scales)) if scales else (torch.cat(parts), None))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _prepare_rotate(case, gen):
    tokens, heads, dim, dt = case["tokens"], case["q_heads"] + case["k_heads"], case["dim"], DT[case["dtype"]]
    # One projection's output: queries, keys and values of a token side by side.
    x = torch.randn((tokens, heads + case["k_heads"], dim), device="cuda", generator=gen).mul_(1.5).to(dt)
    at = torch.randint(0, case["far"], (1,), device="cuda", generator=gen)
    time = torch.arange(tokens, device="cuda") + at
    places = torch.randint(0, 256, (2, tokens), device="cuda", generator=gen)         # rows and columns of pictures
    positions = torch.cat([time.unsqueeze(0), places])[:case["axes"]].to(torch.int32).contiguous()
    frequencies, axes = _frequencies(case)
    state = dict(case=case, q=x[:, :case["q_heads"]], k=x[:, case["q_heads"]:heads], positions=positions, frequencies=frequencies,
                 axes=axes, rates=torch.tensor(frequencies, dtype=torch.float64, device="cuda"),
                 axis=torch.tensor(axes, device="cuda"))
    for name, n in (("q", case["q_heads"]), ("k", case["k_heads"])):
        state[name + "_weight"] = (1 + 0.2 * torch.randn(dim, device="cuda", generator=gen)).to(dt)
        state[name + "_out"] = torch.empty((tokens, n, dim), device="cuda", dtype=dt)
        if case["op"] == "rotate_back":
            state[name + "_grad"] = torch.randn((tokens, n, dim), device="cuda", generator=gen).to(dt)
            state[name + "_weight_grad"] = torch.empty(dim, device="cuda")
    if own:
        import gemm_epilogue_02_gb300 as tg
        state["rotary"] = tg.Rotary(frequencies, axes=axes, interleaved=case["interleaved"])
        if case["op"] == "rotate_back":
            state["workspace"] = tg.qk_norm_rope_backward_workspace(state["q"], state["k"])
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("rotate", "rotate_back"):
        return _prepare_rotate(case, gen)
    lengths, more = _lengths(case)
    batch, heads, dim, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    table, pages = _table(lengths, page, case.get("spare", 1.0), seed + 1)
    if case["op"] == "fork":
        pages += 2 * case["children"]
    if case["op"] == "compact":
        # Some sequences are children of others: the same full pages, a last page of their own (or the parent's, if it is full).
        width = table.shape[1]
        for b in range(case["shared"]):
            full = lengths[b] // page
            row = torch.full((1, width), -1, dtype=torch.int32)
            row[0, :full] = table[b, :full]
            table = torch.cat([table, row])
            lengths = lengths + [full * page]
    k, v, ks, vs = _pools(case, pages, gen)
    uses = torch.zeros(pages, dtype=torch.int32)
    for b, n in enumerate(lengths):
        uses[table[b, :(n + page - 1) // page].long()] += 1
    state = dict(case=case, k=k, v=v, k_scale=ks, v_scale=vs, table=table.cuda(), uses=uses.cuda(),
                 lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    if case["op"] in ("bounds", "sparse"):
        # What earlier steps have left.
        state.update(bounds=torch.randint(-127, 128, (pages, heads, 2, dim), device="cuda", generator=gen, dtype=torch.int8),
                     bounds_scale=torch.ones((pages, heads), device="cuda"))
    if case["op"] == "bounds":
        starts = torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(more).cumsum(0)])
        state["starts"] = None if case["new"] == case["most"] == 1 else starts.to(torch.int32).cuda()
    elif case["op"] == "sparse":
        step = max(1, 2 ** 27 // (page * heads * dim))
        for at in range(0, pages, step):
            part = slice(at, at + step)
            lo_hi, scale = _page_bounds(_values(k[part], ks[part] if ks is not None else None))
            state["bounds"][part], state["bounds_scale"][part] = lo_hi, scale
        q = torch.randn((batch, heads * case["group"], dim), device="cuda", generator=gen) * 2
        state.update(q=q.to(DT[case["dtype"]]), scale=dim ** -0.5, out=torch.zeros_like(q, dtype=DT[case["dtype"]]),
                     to_table=torch.full((batch, heads, case["keep"]), -1, dtype=torch.int32, device="cuda"),
                     to_lengths=torch.zeros(batch, dtype=torch.int32, device="cuda"))
    elif case["op"] == "fork":
        state.update(parents=torch.tensor(more, dtype=torch.int32, device="cuda"),
                     to_table=torch.full((case["children"], table.shape[1]), -1, dtype=torch.int32, device="cuda"),
                     to_lengths=torch.zeros(case["children"], dtype=torch.int32, device="cuda"))
    else:
        state.update(to_table=torch.full(table.shape, -1, dtype=torch.int32, device="cuda"), to_uses=torch.zeros_like(state["uses"]),
                     in_use=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if own:
        import gemm_epilogue_02_gb300 as tg
        state["cache"] = tg.PagedCache(k, v, ks, vs)
        if case["op"] in ("bounds", "sparse"):
            state["page_bounds"] = tg.PageBounds(state["bounds"], state["bounds_scale"])
        if case["op"] == "sparse":
            state["workspace"] = tg.attention_decode_workspace(state["q"], state["cache"], state["to_table"])
        if case["op"] == "compact":
            state["workspace"] = tg.kv_compact_workspace(state["cache"])
    return state


# ---------------------------------------------------------------- plain forms
def _angles(s):
    """cos and sin of every token's angles, [tokens, 1, rot / 2], from 64 bits: far positions need them."""
    a = s["positions"].double()[s["axis"]].T * s["rates"]
    return torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)


def _turn(s, x, cos, sin):
    """The first rot elements of x's rows turned; sin negated turns them back."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    head = x[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["case"]["interleaved"] else (head[..., :half], head[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], -1).flatten(-2) if s["case"]["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _rotated(s, x, w, cos, sin):
    x = x.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(s, y, cos, sin)


def _run_rotate(s):
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.qk_norm_rope(s["q"], s["k"], s["positions"], s["rotary"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=EPS)
    else:
        cos, sin = _angles(s)
        s["q_out"].copy_(_rotated(s, s["q"], s["q_weight"], cos, sin))
        s["k_out"].copy_(_rotated(s, s["k"], s["k_weight"], cos, sin))
    return [s["q_out"], s["k_out"]]


def _back(s, x, w, dy, cos, sin):
    x, g = x.float(), _turn(s, dy.float(), cos, -sin)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit, gw = x * r, g * w.float()
    return r * (gw - unit * (gw * unit).mean(-1, keepdim=True)), (g * unit).sum((0, 1))


def _run_rotate_back(s):
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.qk_norm_rope_backward(s["q_grad"], s["k_grad"], s["q"], s["k"], s["positions"], s["rotary"], s["q_out"], s["k_out"],
                                 q_weight=s["q_weight"], k_weight=s["k_weight"], q_weight_grad=s["q_weight_grad"],
                                 k_weight_grad=s["k_weight_grad"], eps=EPS, workspace=s["workspace"])
    else:
        cos, sin = _angles(s)
        dx, dw = _back(s, s["q"], s["q_weight"], s["q_grad"], cos, sin)
        s["q_out"].copy_(dx), s["q_weight_grad"].copy_(dw)
        dx, dw = _back(s, s["k"], s["k_weight"], s["k_grad"], cos, sin)
        s["k_out"].copy_(dx), s["k_weight_grad"].copy_(dw)
    return [s["q_out"], s["k_out"], s["q_weight_grad"], s["k_weight_grad"]]


def _bytes(x):
    """e4m3 tensors have few operations of their own: they are moved as bytes."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _values(x, scale):
    return x.float() if scale is None else x.float() * scale.unsqueeze(-1)


def _power(top):
    """The least power of two s >= 2^-100 with top <= 127 s."""
    m, e = torch.frexp(top)
    e = torch.where(m * 128 > 127, e - 6, e - 7).clamp(min=-100)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, torch.full_like(e, -100)))


def _page_bounds(x):
    """(bounds int8 [n, heads, 2, dim], scale [n, heads]) of pages of keys x [n, page, heads, dim] in 32 bits."""
    lo, hi = x.amin(1), x.amax(1)
    scale = _power(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    s = scale.unsqueeze(-1)
    return torch.stack([torch.floor(lo / s), torch.ceil(hi / s)], 2).to(torch.int8), scale


def _run_bounds(s):
    case = s["case"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_bounds(s["cache"], s["page_bounds"], s["table"], s["lengths"], starts=s["starts"])
    else:
        new = 1 if s["starts"] is None else s["starts"][1:] - s["starts"][:-1]
        lo, hi = (s["lengths"] - new) // case["page"], s["lengths"] // case["page"]
        i = torch.arange(s["table"].shape[1], device="cuda")
        pages = s["table"][(i >= lo.unsqueeze(1)) & (i < hi.unsqueeze(1))].long()
        if pages.numel():
            keys = _values(_bytes(s["k"])[pages].view(s["k"].dtype), s["k_scale"][pages] if s["k_scale"] is not None else None)
            s["bounds"][pages], s["bounds_scale"][pages] = _page_bounds(keys)
    return [s["bounds"], s["bounds_scale"]]


def _run_sparse(s):
    case = s["case"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_select(s["q"], s["cache"], s["page_bounds"], s["table"], s["lengths"], s["to_table"], s["to_lengths"],
                     first=case["first"], recent=case["recent"])
        tg.attention_decode(s["q"], s["cache"], s["to_table"], s["to_lengths"], s["out"], scale=s["scale"],
                            workspace=s["workspace"])
        return [s["to_table"], s["to_lengths"], s["out"]]
    batch, heads, group, dim, page, keep = (case[n] for n in ("batch", "kv_heads", "group", "dim", "page", "keep"))
    n = s["lengths"].long()
    count = (n + page - 1) // page                                                   # pages of each sequence
    i = torch.arange(s["table"].shape[1], device="cuda")
    there = i < count.unsqueeze(1)                                                   # [batch, width]
    pages = torch.where(there, s["table"].long(), 0)
    q = s["q"].float().view(batch, heads, group, dim)
    scale_q = _power(q.abs().amax(-1))                                               # [batch, heads, group]
    whole = torch.round(q / scale_q.unsqueeze(-1))
    bounds = s["bounds"][pages].float().permute(0, 2, 3, 4, 1)                       # [batch, heads, 2, dim, width]
    # Whole numbers below 2^24: 32 bits hold their sums.
    score = torch.matmul(whole.clamp(max=0), bounds[:, :, 0]) + torch.matmul(whole.clamp(min=0), bounds[:, :, 1])
    score = (score * s["bounds_scale"][pages].permute(0, 2, 1).unsqueeze(2) * scale_q.unsqueeze(-1)).amax(2)
    always = (i < case["first"]) | (i >= (count - case["recent"]).unsqueeze(1))
    score = score.masked_fill(always.unsqueeze(1), math.inf).masked_fill(~there.unsqueeze(1), -math.inf)
    kept = min(keep, s["table"].shape[1])
    best = torch.sort(torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :kept], dim=-1)[0]
    chosen = torch.gather(pages.unsqueeze(1).expand(-1, heads, -1), 2, best)         # pages of no sequence come last
    have = count.clamp(max=keep)
    s["to_table"].fill_(-1)
    s["to_table"][..., :kept] = torch.where(torch.arange(kept, device="cuda") < have.view(-1, 1, 1), chosen, -1).to(torch.int32)
    length = torch.where(count > 0, (have - 1) * page + n - (count - 1) * page, 0)
    s["to_lengths"].copy_(length)
    head = torch.arange(heads, device="cuda").view(1, -1, 1)

    def rows(name):
        """The chosen pages' rows, [batch, heads, kept * page, dim], in 32 bits."""
        x = _bytes(s[name]).transpose(1, 2)[chosen, head].view(s[name].dtype)
        return _values(x, s[name + "_scale"].transpose(1, 2)[chosen, head] if s[name + "_scale"] is not None else None).flatten(2, 3)

    in_list = torch.arange(kept * page, device="cuda") < length.view(-1, 1)
    t = torch.matmul(q, rows("k").transpose(-1, -2)) * s["scale"]
    t = t.masked_fill(~in_list.view(batch, 1, 1, -1), -math.inf)
    p = torch.exp(t - t.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(torch.matmul(p, rows("v")).view(s["out"].shape))
    return [s["to_table"], s["to_lengths"], s["out"]]


def _cache_parts(s):
    return [s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None]


def _run_fork(s):
    page = s["case"]["page"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_free(s["cache"], s["uses"], s["to_table"], s["to_lengths"])
        tg.kv_fork(s["cache"], s["uses"], s["table"], s["lengths"], s["parents"], s["to_table"], s["to_lengths"])
        tg.kv_grow(s["cache"], s["uses"], s["to_table"], s["to_lengths"])
        return _cache_parts(s) + [s["uses"], s["to_table"], s["to_lengths"]]
    i = torch.arange(s["to_table"].shape[1], device="cuda")

    def count(mask, by):
        """Adds `by` to the uses of the children's pages under the mask."""
        held = s["to_table"][mask].long()
        s["uses"].index_add_(0, held, torch.full_like(held, by, dtype=torch.int32))

    count(i < ((s["to_lengths"].long() + page - 1) // page).unsqueeze(1), -1)
    # Fork.
    parent = s["parents"].long()
    n = s["lengths"].long()[parent]
    full, rest = n // page, n % page
    s["to_table"].copy_(torch.where(i < full.unsqueeze(1), s["table"][parent], s["to_table"]))
    count(i < full.unsqueeze(1), 1)
    free = (s["uses"] == 0).nonzero()[:, 0]
    part = (rest > 0).nonzero()[:, 0]
    fresh = free[:part.numel()]
    s["to_table"][part, full[part]] = fresh.to(torch.int32)
    s["uses"][fresh] = 1
    source = s["table"].long()[parent[part], full[part]]
    filled = torch.arange(page, device="cuda") < rest[part].unsqueeze(1)
    for x in _cache_parts(s):
        x = _bytes(x)
        kept = filled.view(filled.shape + (1,) * (x.dim() - 2))
        x[fresh] = torch.where(kept, x[source], x[fresh])
    # Grow by one token.
    part = (n % page == 0).nonzero()[:, 0]
    fresh = (s["uses"] == 0).nonzero()[:part.numel(), 0]
    s["to_table"][part, full[part]] = fresh.to(torch.int32)
    s["uses"][fresh] = 1
    s["to_lengths"].copy_(n + 1)
    return _cache_parts(s) + [s["uses"], s["to_table"], s["to_lengths"]]


def _run_compact(s):
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_compact(s["cache"], s["uses"], s["table"], s["lengths"], s["to_table"], s["to_uses"], s["in_use"],
                      workspace=s["workspace"])
    else:
        page, pages = s["case"]["page"], s["uses"].shape[0]
        used = s["uses"] > 0
        total = used.sum()
        number = torch.arange(pages, device="cuda")
        source = (used & (number >= total)).nonzero()[:, 0]
        target = (~used & (number < total)).nonzero()[:, 0]
        to = number.clone()
        to[source] = target
        for x in _cache_parts(s):
            _bytes(x)[target] = _bytes(x)[source]
        s["to_uses"].copy_(s["uses"])
        s["to_uses"][target] = s["uses"][source]
        s["to_uses"][source] = 0
        s["in_use"].copy_(total)
        held = torch.arange(s["table"].shape[1], device="cuda") < ((s["lengths"].long() + page - 1) // page).unsqueeze(1)
        s["to_table"].copy_(torch.where(held, to[torch.where(held, s["table"].long(), 0)], s["to_table"].long()))
    return _cache_parts(s) + [s["to_table"], s["to_uses"], s["in_use"]]


RUN = {"rotate": _run_rotate, "rotate_back": _run_rotate_back, "bounds": _run_bounds, "sparse": _run_sparse, "fork": _run_fork,
       "compact": _run_compact}


def run(state):
    return RUN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    dim = case["dim"]
    if case["op"] in ("rotate", "rotate_back"):
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * dim
        back = case["op"] == "rotate_back"
        return {"bytes": n * (6 if back else 4) + 4 * case["axes"] * case["tokens"] + dim * (12 if back else 4),
                "flops": n * (16 if back else 8)}
    heads, page = case["kv_heads"], case["page"]
    size = 1 if case["cache"] == "e4m3" else 2
    row = dim * size + (4 if size == 1 else 0)                                        # a row of k, or of v
    lengths, more = _lengths(case)
    if case["op"] == "bounds":
        done = sum(n // page - (n - m) // page for n, m in zip(lengths, more))
        return {"bytes": done * heads * (page * row + 2 * dim + 4) + 4 * len(lengths), "flops": done * heads * page * dim * 2}
    if case["op"] == "sparse":
        all_pages = sum((n + page - 1) // page for n in lengths)
        kept = sum(n if n <= case["keep"] * page else (case["keep"] - 1) * page + (n - 1) % page + 1 for n in lengths)
        lists = sum(min((n + page - 1) // page, case["keep"]) for n in lengths)
        scored = sum((n + page - 1) // page for n in lengths if n > case["keep"] * page)
        q = case["batch"] * heads * case["group"] * dim * 4
        return {"bytes": scored * heads * (2 * dim + 4) + kept * heads * 2 * row + 4 * all_pages + lists * heads * 4 + q,
                "flops": heads * case["group"] * dim * 4 * (scored + kept)}
    if case["op"] == "fork":
        rest = sum(lengths[p] % page for p in more)
        entries = sum((lengths[p] + page) // page for p in more)                      # a child's list, grown by one token
        return {"bytes": rest * heads * 4 * row + entries * 24, "flops": entries}
    used = sum((n + page - 1) // page for n in lengths)
    pages = int(used * case["spare"]) + 3
    # The pages in use lie anywhere: used (1 - used / pages) of them above their number.
    moved = used * (pages - used) // pages
    return {"bytes": moved * page * heads * 4 * row + used * 8 + pages * 8, "flops": pages}


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_rotate(case, seed):
    s = prepare(case, seed)
    dim, rot, half = case["dim"], case["rot"], case["rot"] // 2
    first = [2 * i if case["interleaved"] else i for i in range(half)]
    second = [2 * i + 1 if case["interleaved"] else i + half for i in range(half)]
    # Every token's rotation as complex numbers of length one.
    angle = torch.stack([s["positions"][a].double() * f for f, a in zip(s["frequencies"], s["axes"])], 1).unsqueeze(1)
    z = torch.polar(torch.ones_like(angle), angle)
    grads, weight_grads = [], []
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"].double()
        norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        root = torch.sqrt(norm ** 2 / dim + EPS)
        if case["op"] == "rotate":
            y = x / root * w
            turned = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = turned.real, turned.imag
            grads.append(y)
            continue
        g = s[name + "_grad"].double()
        turned = torch.complex(g[..., first], g[..., second]) * z.conj()
        g[..., first], g[..., second] = turned.real, turned.imag
        weight_grads.append(torch.einsum("thd,thd->d", g, x / root))
        h = g * w
        grads.append(h / root - x * (h * x).sum(-1, keepdim=True) / (dim * root ** 3))
    return grads + weight_grads


def _exact_power(top):
    """The least power of two s >= 2^-100 with top <= 127 s, of numbers in 64 bits on the host."""
    out = []
    for t in top.flatten().tolist():
        e = -100
        if t > 127 * 2.0 ** e:
            e = max(-100, math.ceil(math.log2(t / 127)) - 2)
            while t > 127 * 2.0 ** e:
                e += 1
        out.append(2.0 ** e)
    return torch.tensor(out, dtype=torch.float64).view(top.shape)


def _exact_rows(s, name, page, h):
    """The rows of one head on a page, [page_size, dim], as the values they stand for; those of e4m3 are fp32 numbers."""
    x = s[name][page, :, h]
    if s[name + "_scale"] is None:
        return x.double()
    return (x.float().double() * s[name + "_scale"][page, :, h].double().unsqueeze(-1)).float().double()


def _exact_bounds(case, seed):
    s = prepare(case, seed)
    lengths, new = _lengths(case)
    table, bounds, scale = s["table"].cpu(), s["bounds"].cpu(), s["bounds_scale"].double().cpu()
    done = [int(table[b, i]) for b, (n, m) in enumerate(zip(lengths, new))
            for i in range((n - m) // case["page"], n // case["page"])]
    if len(done) > 20000:
        return None
    for p in done:
        rows = torch.stack([_exact_rows(s, "k", p, h) for h in range(case["kv_heads"])])
        least, most = rows.min(1).values.cpu(), rows.max(1).values.cpu()
        scale[p] = _exact_power(torch.maximum(-least, most).max(-1).values)
        bounds[p, :, 0] = torch.floor(least / scale[p].unsqueeze(1)).to(torch.int8)
        bounds[p, :, 1] = torch.ceil(most / scale[p].unsqueeze(1)).to(torch.int8)
    return [bounds, scale]


def _exact_sparse(case, seed):
    s = prepare(case, seed)
    lengths, _ = _lengths(case)
    page, group, keep = case["page"], case["group"], case["keep"]
    if case["batch"] * case["kv_heads"] > 600:
        return None
    to_table = torch.full(s["to_table"].shape, -1, dtype=torch.int32)
    to_lengths = torch.zeros(case["batch"], dtype=torch.int32)
    out = torch.zeros(s["out"].shape, dtype=torch.float64)
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        count = -(-n // page)
        pages = s["table"][b, :count].long()
        k = min(count, keep)
        to_lengths[b] = n - (count - k) * page
        for h in range(case["kv_heads"]):
            q = s["q"][b, h * group:(h + 1) * group].double()
            chosen = torch.arange(count)
            if count > keep:
                unit = _exact_power(q.abs().max(1).values.cpu()).to(q.device).unsqueeze(1)
                steps = torch.round(q / unit)
                lo, hi = s["bounds"][pages, h, 0].double(), s["bounds"][pages, h, 1].double()
                reach = torch.zeros(group, count, dtype=torch.float64, device="cuda")
                for j in range(group):
                    reach[j] = torch.maximum(steps[j] * lo, steps[j] * hi).sum(1)
                best = (reach * unit * s["bounds_scale"][pages, h].double()).max(0).values.cpu()
                fixed = list(range(case["first"])) + list(range(count - case["recent"], count))
                middle = torch.argsort(-best[case["first"]:count - case["recent"]], stable=True) + case["first"]
                chosen = torch.tensor(sorted(fixed + middle[:keep - len(fixed)].tolist()))
            ids = pages[chosen.cuda()]
            to_table[b, h, :k] = ids.to(torch.int32).cpu()
            rows = []
            for name in ("k", "v"):
                x = _bytes(s[name])[ids, :, h].view(s[name].dtype).float().double()
                if s[name + "_scale"] is not None:
                    x = x * s[name + "_scale"][ids, :, h].double().unsqueeze(-1)
                rows.append(x.reshape(-1, case["dim"])[:int(to_lengths[b])])
            p = torch.softmax(rows[0] @ q.T * s["scale"], 0)
            out[b, h * group:(h + 1) * group] = (p.T @ rows[1]).cpu()
    return [to_table, to_lengths, out]


def _as_numbers(s):
    return [x.float().double() if x.dtype == E4M3 else x.double() for x in _cache_parts(s)]


def _exact_fork(case, seed):
    s = prepare(case, seed)
    lengths, parents = _lengths(case)
    page, pools = case["page"], _as_numbers(s)
    table, to_table, uses = s["table"].tolist(), s["to_table"].tolist(), s["uses"].tolist()

    def fresh():
        p = uses.index(0)
        uses[p] = 1
        return p

    for c, b in enumerate(parents):
        for i in range(lengths[b] // page):
            to_table[c][i] = table[b][i]
            uses[table[b][i]] += 1
    for c, b in enumerate(parents):
        i, rest = divmod(lengths[b], page)
        if rest:
            to_table[c][i] = fresh()
            for x in pools:
                x[to_table[c][i], :rest] = x[table[b][i], :rest]
    for c, b in enumerate(parents):
        if lengths[b] % page == 0:
            to_table[c][lengths[b] // page] = fresh()
    return pools + [torch.tensor(uses, dtype=torch.int32), torch.tensor(to_table, dtype=torch.int32),
                    torch.tensor([lengths[b] + 1 for b in parents], dtype=torch.int32)]


def _exact_compact(case, seed):
    s = prepare(case, seed)
    page, pools, uses = case["page"], _as_numbers(s), s["uses"].tolist()
    total = sum(u > 0 for u in uses)
    to = dict(zip([p for p in range(total, len(uses)) if uses[p] > 0], [p for p in range(total) if uses[p] == 0]))
    for p, t in to.items():
        uses[t], uses[p] = uses[p], 0
        for x in pools:
            x[t] = x[p]
    to_table, lengths = s["to_table"].tolist(), s["lengths"].tolist()
    for b, row in enumerate(s["table"].tolist()):
        for i in range(-(-lengths[b] // page)):
            to_table[b][i] = to.get(row[i], row[i])
    return pools + [torch.tensor(to_table, dtype=torch.int32), torch.tensor(uses, dtype=torch.int32),
                    torch.tensor([total], dtype=torch.int32)]


def exact(case, seed):
    """The outputs from the definitions: pages, heads and lists one by one, real numbers in 64 bits."""
    return {"rotate": _exact_rotate, "rotate_back": _exact_rotate, "bounds": _exact_bounds, "sparse": _exact_sparse,
            "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, seed)
