"""Cases of the paged key-value cache's operators: writing new tokens (append), attention of one new token per sequence
(attend) and eviction by accumulated attention weight (evict).

The cache is two pools, keys and values, of shape [pages, page_size, kv_heads, dim], in 16 bits or in e4m3 with one fp32
scale per row (pools of scales [pages, page_size, kv_heads]); a sequence's pages are listed in its row of a page table.

    append   sequence b brings n_b tokens (starts[b] .. starts[b + 1] of the token axis); lengths[b] counts them already, so
             its token i goes to position lengths[b] - n_b + i.  e4m3: scale = max |x| / 448 of the row (1 for a row of
             zeros), element = x / scale rounded to nearest even.  The row's accumulated weight starts at zero.
    attend   o = sum_j softmax_j(s) v_j over positions max(0, n - window) <= j < n (window 0: all), s_j = scale q . k_j,
             passed through cap * tanh(s / cap) when cap > 0; heads share keys in groups; n = 0 gives zeros.  With weights,
             weights[b, g, j] grows by the sum of group g's softmax weights on j.
    evict    of n positions k = min(n, keep) stay: the last min(recent, k), and of those before them the ones of largest
             weight, ties to the lowest position.  They are copied in order to other pages.
"""
import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # One request's newest token in a small model: the smallest call, all latency.
        dict(name="append_one_token", op="append", batch=1, new=1, most=1, context=77, kv_heads=8, dim=64, page=16,
             dtype="fp16", cache="16"),
        # A serving batch's newest tokens, beside the contexts they extend.
        dict(name="append_batch_256", op="append", batch=256, new=1, most=1, context=500, kv_heads=8, dim=128, page=16,
             dtype="bf16", cache="16"),
        # Prompts of uneven length written in one call, quantised on the way in; an odd page size.
        dict(name="append_prompts_e4m3", op="append", batch=11, new=1, most=8191, context=0, kv_heads=8, dim=128, page=24,
             dtype="bf16", cache="e4m3"),
        # The first steps of one chat: a context of a few dozen tokens, one key head for each query head.
        dict(name="attend_one_short", op="attend", batch=1, least=77, most=77, kv_heads=8, group=1, dim=64, page=16,
             dtype="fp16", cache="16", cap=0.0, window=0, weights=False),
        # An ordinary serving batch of ragged contexts, grouped heads.
        dict(name="attend_batch_ragged", op="attend", batch=32, least=1, most=4096, kv_heads=8, group=4, dim=128, page=16,
             dtype="bf16", cache="16", cap=0.0, window=0, weights=False),
        # One long document: few rows, so the work has to be split over its length.
        dict(name="attend_one_long", op="attend", batch=1, least=262143, most=262143, kv_heads=8, group=8, dim=128, page=64,
             dtype="bf16", cache="16", cap=0.0, window=0, weights=False),
        # All query heads on one key head, a head dimension that is no power of two, capped scores, a window.
        dict(name="attend_window_capped", op="attend", batch=7, least=1000, most=30000, kv_heads=1, group=24, dim=96, page=24,
             dtype="fp16", cache="16", cap=30.0, window=8192, weights=False),
        # A cache held in 8 bits, with the weights that eviction goes by.
        dict(name="attend_e4m3_weights", op="attend", batch=16, least=500, most=16384, kv_heads=8, group=8, dim=128, page=32,
             dtype="bf16", cache="e4m3", cap=0.0, window=0, weights=True),
        # The largest: a full batch of long contexts.
        dict(name="attend_full_batch", op="attend", batch=48, least=1, most=32768, kv_heads=8, group=4, dim=128, page=64,
             dtype="bf16", cache="16", cap=0.0, window=0, weights=False),
        # A short cache trimmed by a fifth.
        dict(name="evict_one_short", op="evict", batch=1, least=333, most=333, kv_heads=8, dim=64, page=16, dtype="fp16",
             cache="16", keep=256, recent=32, coarse=False),
        # A batch brought back to a budget; some sequences are still below it.
        dict(name="evict_batch", op="evict", batch=16, least=1000, most=8192, kv_heads=8, dim=128, page=32, dtype="bf16",
             cache="16", keep=2048, recent=256, coarse=False),
        # Long 8-bit caches; weights with many equal values.
        dict(name="evict_long_e4m3", op="evict", batch=2, least=100000, most=131072, kv_heads=8, dim=128, page=64,
             dtype="bf16", cache="e4m3", keep=16384, recent=1000, coarse=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), cache=rng.choice(["16", "16", "e4m3"]),
                dim=rng.choice([64, 64, 80, 96, 112, 128, 128, 256]), kv_heads=rng.choice([1, 2, 3, 4, 8, 8, 16]),
                page=rng.choice([1, 8, 16, 16, 20, 24, 32, 64, 128]))
    if op == "append":
        rows = 40000 * 8 * 128 // (case["kv_heads"] * case["dim"])       # cache positions of the largest drawn case
        batch = _log(rng, 1, 300)
        if rng.random() < 0.5:
            case.update(batch=batch, new=1, most=1, context=_log(rng, 1, max(2, min(2000, rows // batch))))
        else:
            case.update(batch=batch, new=0, most=_log(rng, 1, max(2, min(20000, rows // batch))), context=_log(rng, 1, 200))
    elif op == "attend":
        rows = 700000 * 8 * 128 // (case["kv_heads"] * case["dim"])
        batch = _log(rng, 1, 128)
        most = _log(rng, 1, max(2, min(262144, rows // batch)))
        case.update(batch=batch, least=rng.choice([0, 1, max(1, most // 2), most]), most=most,
                    group=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 24]),
                    cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, 0, _log(rng, 1, 2 * most)]),
                    weights=rng.random() < 0.3)
        case["group"] = min(case["group"], 128 // case["kv_heads"])
    else:
        rows = 150000 * 8 * 128 // (case["kv_heads"] * case["dim"])
        batch = _log(rng, 1, 64)
        most = _log(rng, 2, max(4, min(131072, rows // batch)))
        keep = _log(rng, 1, most)
        case.update(batch=batch, least=rng.choice([0, 1, max(1, most // 2), most]), most=most, keep=keep,
                    recent=rng.choice([0, 1, keep // 8, keep // 2, keep]), coarse=rng.random() < 0.5)
    return case


def _ints(gen, least, most, n):
    """n whole numbers in least..most, the first of them the largest."""
    out = torch.randint(least, most + 1, (n,), generator=gen).tolist()
    out[0] = most
    return out


def _lengths(case):
    """(lengths, new tokens) of each sequence, on the host.  They belong to the case; a seed changes what the rows hold and
    where they lie."""
    gen = torch.Generator().manual_seed(case["batch"] * 7919 + case["most"])
    if case["op"] == "append":
        new = _ints(gen, case["new"], case["most"], case["batch"])
        context = _ints(gen, case["context"] // 2, case["context"], case["batch"])
        return [c + n for c, n in zip(context, new)], new
    return _ints(gen, case["least"], case["most"], case["batch"]), None


def _table(counts, page, extra, seed):
    """A page table [batch, most pages] (-1 past a sequence's own) over shuffled pages, and the pool's number of pages."""
    need = [(n + page - 1) // page for n in counts]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed), dtype=torch.int64).to(torch.int32)
    table = torch.full((len(counts), max(1, max(need))), -1, dtype=torch.int32)
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


def _pool(case, pages, gen, shape=None):
    """Random rows of a pool: normal values, with a few channels larger than the others."""
    shape = (pages, case["page"], case["kv_heads"], case["dim"]) if shape is None else shape
    x = torch.randn(shape, device="cuda", dtype=DT[case["dtype"]], generator=gen)
    x[..., :2] *= 3
    return x


def _pools(case, pages, gen):
    """k, v, k_scale, v_scale (the scales None for a 16-bit cache)."""
    out = []
    for _ in range(2):
        if case["cache"] == "e4m3":
            step = max(1, 2 ** 27 // (case["page"] * case["kv_heads"] * case["dim"]))
            parts = [_split(_pool(case, min(step, pages - at), gen)) for at in range(0, pages, step)]
            out.append((torch.cat([p[0].view(torch.uint8) for p in parts]).view(E4M3), torch.cat([p[1] for p in parts])))
        else:
            out.append((_pool(case, pages, gen), None))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lengths, new = _lengths(case)
    table, pages = _table(lengths, case["page"], 3, seed + 1)
    k, v, ks, vs = _pools(case, pages, gen)
    state = dict(case=case, lengths_host=lengths, new_host=new, k=k, v=v, k_scale=ks, v_scale=vs,
                 table=table.cuda(), lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    batch, heads, dim = case["batch"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        shape = (starts[-1], heads, dim)
        state.update(k_new=_pool(case, 0, gen, shape), v_new=_pool(case, 0, gen, shape),
                     starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                     weights=torch.ones(batch, heads, max(lengths), device="cuda"))
    elif case["op"] == "attend":
        q = torch.randn((batch, heads * case["group"], dim), device="cuda", generator=gen) * 2
        state.update(q=q.to(DT[case["dtype"]]), scale=dim ** -0.5,
                     out=torch.zeros((batch, heads * case["group"], dim), device="cuda", dtype=DT[case["dtype"]]),
                     weights=torch.rand((batch, heads, max(1, max(lengths))), device="cuda", generator=gen)
                     if case["weights"] else None)
    else:
        kept = [min(n, case["keep"]) for n in lengths]
        to_table, to_pages = _table(kept, case["page"], 0, seed + 2)
        # Accumulated weights: a heavy tail, and nothing yet on some positions.
        w = torch.rand((batch, heads, max(lengths)), device="cuda", generator=gen) ** 8 * 40
        if case["coarse"]:
            w = (w * 16).floor() / 16
        w = torch.where(torch.rand(w.shape, device="cuda", generator=gen) < 0.05, torch.zeros_like(w), w)
        state.update(weights=w, to_table=to_table.cuda(), to_k=torch.zeros((to_pages,) + k.shape[1:], device="cuda").to(k.dtype),
                     to_v=torch.zeros((to_pages,) + k.shape[1:], device="cuda").to(k.dtype),
                     to_k_scale=torch.zeros((to_pages,) + k.shape[1:3], device="cuda") if ks is not None else None,
                     to_v_scale=torch.zeros((to_pages,) + k.shape[1:3], device="cuda") if ks is not None else None,
                     kept=torch.full((batch, heads, case["keep"]), -1, dtype=torch.int32, device="cuda"),
                     to_lengths=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                     to_weights=torch.zeros((batch, heads, case["keep"]), device="cuda"))
    if own:
        import gemm_epilogue_02_gb300 as tg
        state["cache"] = tg.PagedCache(k, v, ks, vs)
        if case["op"] == "attend":
            state["workspace"] = tg.attention_decode_workspace(state["q"], state["cache"], state["table"],
                                                               weights=case["weights"])
        if case["op"] == "evict":
            state["to_cache"] = tg.PagedCache(state["to_k"], state["to_v"], state["to_k_scale"], state["to_v_scale"])
    return state


def _rows(state, b, positions, table="table"):
    """Flat row numbers (page * page_size + slot) of sequence b's positions."""
    page = state["case"]["page"]
    return state[table][b].long()[positions // page] * page + positions % page


def _flat(pool):
    return pool.view((-1,) + pool.shape[2:])


def _bytes(x):
    """e4m3 tensors have few operations of their own: they are moved as bytes."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _values(pool, scale, rows):
    x = _flat(_bytes(pool))[rows]
    if scale is None:
        return x.float()
    return x.view(E4M3).float() * _flat(scale)[rows].unsqueeze(-1)


def _run_append(s):
    case = s["case"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_append(s["cache"], s["k_new"], s["v_new"], s["table"], s["lengths"],
                     starts=None if case["new"] == case["most"] == 1 else s["starts"], weights=s["weights"])
    else:
        tokens = torch.arange(s["k_new"].shape[0], device="cuda")
        seq = torch.searchsorted(s["starts"][1:].long(), tokens, right=True)
        pos = s["lengths"].long()[seq] - s["starts"].long()[seq + 1] + tokens
        rows = s["table"].long()[seq, pos // case["page"]] * case["page"] + pos % case["page"]
        for new, pool, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
            if scale is None:
                _flat(pool)[rows] = new
            else:
                x, sc = _split(new)
                _flat(pool.view(torch.uint8))[rows] = x.view(torch.uint8)
                _flat(scale)[rows] = sc
        s["weights"][seq, :, pos] = 0.0
    return [x for x in (s["k"], s["v"], s["k_scale"], s["v_scale"], s["weights"]) if x is not None]


def _run_attend(s):
    case = s["case"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.attention_decode(s["q"], s["cache"], s["table"], s["lengths"], s["out"], scale=s["scale"], cap=case["cap"],
                            window=case["window"], weights=s["weights"], workspace=s["workspace"])
    else:
        heads, group = case["kv_heads"], case["group"]
        s["out"].zero_()
        for b, n in enumerate(s["lengths_host"]):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == lo:
                continue
            rows = _rows(s, b, torch.arange(lo, n, device="cuda"))
            k, v = _values(s["k"], s["k_scale"], rows), _values(s["v"], s["v_scale"], rows)
            q = s["q"][b].float().view(heads, group, -1)
            score = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]
            if case["cap"]:
                score = case["cap"] * torch.tanh(score / case["cap"])
            p = torch.exp(score - score.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            s["out"][b] = torch.matmul(p, v.permute(1, 0, 2)).view(heads * group, -1).to(s["out"].dtype)
            if s["weights"] is not None:
                s["weights"][b, :, lo:n] += p.sum(1)
    return [x for x in (s["out"], s["weights"]) if x is not None]


def _run_evict(s):
    case = s["case"]
    if own:
        import gemm_epilogue_02_gb300 as tg
        tg.kv_evict(s["cache"], s["table"], s["lengths"], s["weights"], s["to_cache"], s["to_table"], s["kept"],
                    s["to_lengths"], s["to_weights"], recent=case["recent"])
    else:
        s["kept"].fill_(-1)
        s["to_weights"].zero_()
        for b, n in enumerate(s["lengths_host"]):
            k = min(n, case["keep"])
            r = min(case["recent"], k)
            w = s["weights"][b, :, :n]
            best = torch.sort(w[:, :n - r], dim=-1, descending=True, stable=True)[1][:, :k - r]
            last = torch.arange(n - r, n, device="cuda").expand(w.shape[0], r)
            kept = torch.cat([torch.sort(best, dim=-1)[0], last], -1)                       # [heads, k], ascending
            s["kept"][b, :, :k] = kept.to(torch.int32)
            s["to_weights"][b, :, :k] = torch.gather(w, 1, kept)
            head = torch.arange(w.shape[0], device="cuda").unsqueeze(1)
            rows = _rows(s, b, kept)
            to = _rows(s, b, torch.arange(k, device="cuda"), "to_table").expand_as(rows)
            for name in ("k", "v", "k_scale", "v_scale"):
                if s[name] is not None:
                    _flat(_bytes(s["to_" + name]))[to, head] = _flat(_bytes(s[name]))[rows, head]
        s["to_lengths"].copy_(s["lengths"].clamp(max=case["keep"]))
    return [x for x in (s["kept"], s["to_lengths"], s["to_weights"], s["to_k"], s["to_v"], s["to_k_scale"],
                        s["to_v_scale"]) if x is not None]


def run(state):
    return {"append": _run_append, "attend": _run_attend, "evict": _run_evict}[state["case"]["op"]](state)


def work(case):
    heads, dim = case["kv_heads"], case["dim"]
    row = 2 * dim * (1 if case["cache"] == "e4m3" else 2) + (8 if case["cache"] == "e4m3" else 0)   # a row of k and of v
    lengths, new = _lengths(case)
    if case["op"] == "append":
        return {"bytes": sum(new) * heads * (4 * dim + row + 4), "flops": sum(new) * heads * dim * 2}
    if case["op"] == "attend":
        used = sum(min(n, case["window"] or n) for n in lengths)
        qo = case["batch"] * heads * case["group"] * dim * 4
        return {"bytes": used * heads * (row + (8 if case["weights"] else 0)) + qo,
                "flops": used * heads * case["group"] * dim * 4}
    kept = sum(min(n, case["keep"]) for n in lengths)
    return {"bytes": heads * (4 * sum(lengths) + kept * (2 * row + 12)), "flops": sum(lengths) * heads}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    page, heads = case["page"], case["kv_heads"]
    table = s["table"].cpu()

    def row_of(b, j, tab=table):
        return tab[b, j // page].long() * page + j % page

    def rows64(pool, scale, idx, h):
        x = pool.view(-1, heads, case["dim"])[:, h].contiguous().view(torch.uint8 if pool.dtype == E4M3 else pool.dtype)[idx]
        x = (x.view(E4M3) if pool.dtype == E4M3 else x).double()
        return x if scale is None else x * scale.view(-1, heads)[idx, h].double().unsqueeze(1)

    if case["op"] == "append":
        weights = s["weights"].double()
        for b in range(case["batch"]):
            weights[b, :, s["lengths_host"][b] - s["new_host"][b]:s["lengths_host"][b]] = 0.0
        out = []
        flat = torch.cat([row_of(b, torch.arange(s["lengths_host"][b] - s["new_host"][b], s["lengths_host"][b]))
                          for b in range(case["batch"])]).cuda()
        scales = []
        for name in ("k", "v"):
            pool = s[name].double() if s[name].dtype != E4M3 else s[name].float().double()
            x = s[name + "_new"].double()
            if s[name + "_scale"] is None:
                pool.view(-1, heads, case["dim"])[flat] = x
            else:
                # The quotient's rounding to 8 bits goes by the scale as it is stored, in 32 bits.
                top = x.abs().max(-1).values
                scale = torch.where(top == 0, torch.ones_like(top), top / 448).float()
                pool.view(-1, heads, case["dim"])[flat] = (x / scale.double().unsqueeze(-1)).to(E4M3).double()
                whole = s[name + "_scale"].double()
                whole.view(-1, heads)[flat] = scale.double()
                scales.append(whole)
            out.append(pool)
        return out + scales + [weights]

    if case["op"] == "attend":
        group = case["group"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        weights = s["weights"].double() if s["weights"] is not None else None
        for b, n in enumerate(s["lengths_host"]):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == lo:
                continue
            idx = row_of(b, torch.arange(lo, n)).cuda()
            k = s["k"].view(-1, heads, case["dim"]).view(torch.uint8 if s["k_scale"] is not None else s["k"].dtype)[idx]
            v = s["v"].view(-1, heads, case["dim"]).view(torch.uint8 if s["k_scale"] is not None else s["v"].dtype)[idx]
            for h in range(heads):
                if s["k_scale"] is not None:
                    kh = k[:, h].contiguous().view(E4M3).double() * s["k_scale"].view(-1, heads)[idx, h].double()[:, None]
                    vh = v[:, h].contiguous().view(E4M3).double() * s["v_scale"].view(-1, heads)[idx, h].double()[:, None]
                else:
                    kh, vh = k[:, h].double(), v[:, h].double()
                q = s["q"][b, h * group:(h + 1) * group].double()
                t = kh @ q.T * s["scale"]
                if case["cap"] > 0:
                    t = torch.tanh(t / case["cap"]) * case["cap"]
                p = torch.softmax(t, 0)
                out[b, h * group:(h + 1) * group] = p.T @ vh
                if weights is not None:
                    weights[b, h, lo:n] += p.sum(1)
        return [x for x in (out, weights) if x is not None]

    kept_out = torch.full(s["kept"].shape, -1, dtype=torch.int32)
    w_out = torch.zeros(s["to_weights"].shape, dtype=torch.float64)
    to = {n: s["to_" + n].float().double() for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}
    weights = s["weights"].cpu().double()
    to_table = s["to_table"].cpu()
    for b, n in enumerate(s["lengths_host"]):
        k = min(n, case["keep"])
        r = min(case["recent"], k)
        target = row_of(b, torch.arange(k), to_table).cuda()
        for h in range(heads):
            w = weights[b, h, :n]
            chosen = torch.argsort(-w[:n - r], stable=True)[:k - r]
            mark = torch.zeros(n, dtype=torch.bool)
            mark[chosen] = True
            mark[n - r:] = True
            kept = mark.nonzero()[:, 0]
            kept_out[b, h, :k] = kept.to(torch.int32)
            w_out[b, h, :k] = w[kept]
            source = row_of(b, kept).cuda()
            for name in ("k", "v"):
                to[name].view(-1, heads, case["dim"])[target, h] = rows64(s[name], None, source, h)
                if s[name + "_scale"] is not None:
                    to[name + "_scale"].view(-1, heads)[target, h] = s[name + "_scale"].view(-1, heads)[source, h].double()
    sizes = torch.tensor([min(n, case["keep"]) for n in s["lengths_host"]], dtype=torch.int32)
    return [kept_out, sizes, w_out] + [to[n] for n in ("k", "v", "k_scale", "v_scale") if n in to]
