"""Cases, plain forms and exact results of the paged 4-bit key-value cache's operators.

One layer's cache is a pool of pages, [num_pages][num_heads][page_size] slots of head_dim 4-bit codes with an fp16
minimum and an fp16 scale for each group of 64 or 128 of them, and a table that names each sequence's pages in order.
A cache that tracks its slots holds for each of them two numbers more: the attention weight that it has been given so
far (fp32) and the number of the token in it (int32).

  attend  softmax attention of new tokens' query rows over the slots that they see; a tracked cache's weights grow by
          the probabilities: out = sum_t p_t v_t, p = softmax_t(q . k_t), weights_t += sum over rows and heads of p_t
  append  the new tokens' k and v rows into their slots, in the 4-bit form
  evict   per sequence and head, down to `budget` slots: those of the last `recent` tokens, then those of the largest
          weight, ties to the lowest slot; kept slots at or above the budget fill the holes below it in order

The caches' codes come back as the bytes that hold them and are compared byte for byte: the format fixes every
rounding on the way to a code, so there is no room between two right results.
"""
import math

import torch

own = False

POOLS = ("k_codes", "k_mins", "k_scales", "v_codes", "v_mins", "v_scales")


def listed():
    return [
        # one decode step of the OPT-125M block: 4 sequences, a few dozen tokens each; latency is all there is
        dict(name="attend, opt-125m block", op="attend", seqs=4, heads=12, kv_heads=12, head_dim=64, group=64, page=64,
             lo=33, hi=40, rows=1, track=False),
        # the decode step of the OPT-6.7B block of 512 sequences past a prompt of 512 tokens
        dict(name="attend, opt-6.7b block", op="attend", seqs=512, heads=32, kv_heads=32, head_dim=128, group=64,
             page=64, lo=513, hi=544, rows=1, track=False),
        # one sequence with a long context: the work has to be split over its length
        dict(name="attend, one long sequence", op="attend", seqs=1, heads=32, kv_heads=32, head_dim=128, group=64,
             page=64, lo=100003, hi=100003, rows=1, track=False),
        # a serving batch of very different lengths, 8 query heads to a key-value head, small pages
        dict(name="attend, ragged shared heads", op="attend", seqs=24, heads=64, kv_heads=8, head_dim=128, group=128,
             page=16, lo=1, hi=16384, rows=1, track=False),
        # a few draft tokens verified at once, wide heads, a page size that is no power of two
        dict(name="attend, draft rows", op="attend", seqs=8, heads=32, kv_heads=4, head_dim=256, group=64, page=48,
             lo=700, hi=9000, rows=5, track=False),
        # decode with the attention weights gathered for eviction, the OPT-6.7B layer at its budget
        dict(name="attend tracked, opt-6.7b", op="attend", seqs=64, heads=32, kv_heads=32, head_dim=128, group=64,
             page=64, lo=1500, hi=2112, rows=1, track=True),
        # the same for few long ragged sequences and shared heads
        dict(name="attend tracked, shared heads", op="attend", seqs=3, heads=32, kv_heads=8, head_dim=128, group=64,
             page=128, lo=5, hi=40000, rows=1, track=True),
        # one decode step's k and v of the OPT-6.7B block of 512 sequences
        dict(name="append, decode rows", op="append", seqs=512, kv_heads=32, head_dim=128, group=64, page=64, lo=513,
             hi=544, rows=1, track=False),
        # prompts of different lengths, padded to 512 tokens, into a tracked cache of the OPT-30B layer
        dict(name="append, padded prompts", op="append", seqs=32, kv_heads=56, head_dim=128, group=64, page=64, lo=1,
             hi=512, rows=512, track=True),
        # a handful of slots of a small block
        dict(name="evict, opt-125m block", op="evict", seqs=4, kv_heads=12, head_dim=64, group=64, page=16, lo=33,
             hi=48, budget=32, recent=8),
        # generation at a budget of 2048 tokens: back to it whenever a page more has filled
        dict(name="evict, steady", op="evict", seqs=64, kv_heads=32, head_dim=128, group=64, page=64, lo=2049, hi=2112,
             budget=2048, recent=256),
        # long prompts cut down at once
        dict(name="evict, prompts", op="evict", seqs=4, kv_heads=32, head_dim=128, group=64, page=64, lo=700, hi=16384,
             budget=1024, recent=512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    most = 512 * 544 * 32 * 128  # values of K in the largest listed case
    op = rng.choice(("attend", "attend", "attend", "append", "evict"))
    d = rng.choice((64, 128, 128, 256))
    case = dict(op=op, head_dim=d, group=rng.choice((64, 128)) if d > 64 else 64, page=rng.choice((16, 32, 48, 64, 80, 128, 256)))
    kv = rng.choice((1, 2, 3, 4, 5, 8, 12, 16, 32, 40, 56))
    case["kv_heads"] = kv
    if op == "attend":
        ratio = rng.choice((1, 1, 1, 2, 3, 4, 5, 8, 12))
        rows = rng.choice((1, 1, 1, 2, 3, 7))
        hi = _log(rng, 1, 100003)
        room = most // (kv * d * ratio * rows) // hi
        while room < 1:
            hi //= 2
            room = most // (kv * d * ratio * rows) // hi
        case |= dict(heads=kv * ratio, rows=rows, track=rng.random() < 0.4, seqs=_log(rng, 1, min(512, room)))
        hi = max(hi, rows)
        case |= dict(lo=rng.choice((rows, hi, max(rows, hi // 2))), hi=hi)
    elif op == "append":
        rows = rng.choice((1, 1, _log(rng, 2, 600)))
        case |= dict(rows=rows, track=rng.random() < 0.5, seqs=_log(rng, 1, max(1, min(512, most // (8 * rows * kv * d)))))
        hi = rows if rows > 1 else _log(rng, 1, 700)
        case |= dict(lo=rng.choice((1, hi)), hi=hi)
    else:
        budget = _log(rng, 16, 4096)
        hi = budget + rng.choice((1, case["page"], _log(rng, 1, 12000)))
        case |= dict(budget=budget, recent=rng.choice((0, 1, budget // 8, budget // 2)), lo=rng.choice((hi, budget + 1, max(1, budget // 2))), hi=hi)
        case |= dict(seqs=_log(rng, 1, max(1, min(64, most // (3 * hi * kv * d)))))
    return case


# ------------------------------------------------------------------ inputs ------------


def _quantise(x, group):
    """x [..., D] fp16 -> (codes uint8 [..., D/2], mins fp16 [..., D/group], scales fp16): groups along the last dim."""
    g = x.float().unflatten(-1, (-1, group))
    low = g.amin(-1, keepdim=True) + 0.0
    scale = ((g.amax(-1, keepdim=True) - low) / torch.full_like(low, 15.0)).half()
    step = scale.float()
    inverse = torch.where(step > 0, torch.ones_like(step) / step, torch.zeros_like(step))
    c = ((g - low) * inverse).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), low.squeeze(-1).half(), torch.where(step > 0, scale, torch.zeros_like(scale)).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=gen)
    S, H, D, G, ps = case["seqs"], case["kv_heads"], case["head_dim"], case["group"], case["page"]
    op, rows = case["op"], case.get("rows", 1)
    lengths = torch.randint(case["lo"], case["hi"] + 1, (S,), **dev)
    lengths[0] = case["hi"]
    slots = torch.full_like(lengths, case["hi"] + (1 if op == "append" else 0)) if op == "append" else lengths
    # every sequence's pages in a shuffled order out of a pool with a few more; -1 where it has none
    width = -(-(case["hi"] + 1) // ps)
    need = (slots + ps - 1) // ps
    have = torch.arange(width, device="cuda") < need[:, None]
    pages = S * width + 3
    table = torch.where(have, torch.randperm(pages, **dev)[: S * width].view(S, width), -1).to(torch.int32)
    st = dict(case=dict(case), table=table, max_len=case["hi"] + (op == "append"))

    def rowsof(n, *shape):  # fp16 normal values in pieces
        return torch.cat([torch.randn((min(n - i, 1 << 14), *shape), **dev).half() for i in range(0, n, 1 << 14)])

    if op != "append":
        # keys whose channels differ in size, and whose sizes make a softmax with a few large terms among many small ones
        channel = torch.exp(0.5 * torch.randn(H, 1, D, **dev))
        parts = []
        per = max(1, (1 << 28) // (H * ps * D))
        for p in range(0, pages, per):
            n = min(per, pages - p)
            parts.append(_quantise((torch.randn((n, H, ps, D), **dev) * channel).half(), G) + _quantise(torch.randn((n, H, ps, D), **dev).half(), G))
        for i, name in enumerate(POOLS):
            st[name] = torch.cat([q[i] for q in parts]) if len(parts) > 1 else parts[0][i]
        del parts
    else:
        for name in POOLS:
            st[name] = torch.zeros((pages, H, ps, D // 2 if "codes" in name else D // G), dtype=torch.uint8 if "codes" in name else torch.float16, device="cuda")
    if op == "evict" or case.get("track"):
        w = torch.exp(2.0 * torch.randn((pages, H, ps), **dev) - 8.0)  # a few steps' worth, a few slots with most of it
        st["weights"] = torch.where(torch.rand((pages, H, ps), **dev) < 0.02, torch.zeros_like(w), w)  # some were never seen
        st["tokens"] = torch.zeros((pages, H, ps), dtype=torch.int32, device="cuda")
    if op == "attend":
        st["q"] = rowsof(S * rows, case["heads"] * D) * (1.5 * D**-0.5)
        st["positions"] = (lengths - rows).to(torch.int32)  # the slot of each sequence's first new row
        st["out"] = torch.empty_like(st["q"])
    elif op == "append":
        qkv = rowsof(S * rows, 3 * H * D)  # k and v are thirds of the projection's rows
        st["k"], st["v"] = qkv[:, H * D : 2 * H * D], qkv[:, 2 * H * D :]
        if rows > 1:
            st["counts"] = lengths.to(torch.int32)
            st["positions"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        else:
            st["counts"] = None
            st["positions"] = (lengths - 1).to(torch.int32)
        st["first"] = (st["positions"] + torch.randint(0, 1000, (S,), **dev)).to(torch.int32) if case["track"] else None
    else:
        # slots below the budget hold tokens of any age, those above it the latest ones in order
        budget, hi = case["budget"], case["hi"]
        old = min(budget, hi)
        seen = torch.argsort(torch.rand((S, H, old + old // 2), **dev), -1)[:, :, :old]
        age = torch.arange(width * ps - old, device="cuda") + old + old // 2
        tokens = torch.cat([seen, age.expand(S, H, -1)], -1).to(torch.int32)
        at = table.clamp(min=0).long()
        cut = tokens.view(S, H, width, ps).permute(0, 2, 1, 3)
        st["tokens"][at[have]] = cut[have]
        st["lengths"] = lengths.to(torch.int32)
        st["next"] = torch.where(lengths > old, lengths + old // 2, old + old // 2).to(torch.int32)
        st["new_lengths"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        st["weights_out"], st["tokens_out"] = torch.zeros_like(st["weights"]), torch.zeros_like(st["tokens"])
    if own:
        import bit_compressed_decode_b200 as fg

        st["cache"] = fg.PagedKVCache(pages, H, D, ps, table, group=G, arrays=[st[n] for n in POOLS], weights=st.get("weights"), tokens=st.get("tokens"))
        if op == "attend":
            st["workspace"] = torch.empty(fg.fg_paged_attention_workspace_bytes(st["cache"], case["heads"], S * rows, rows, st["max_len"], case["track"]), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ the operators -----


def run(st):
    if own:
        return _framework(st)
    return {"attend": _attend, "append": _append, "evict": _evict}[st["case"]["op"]](st)


def _framework(st):
    import bit_compressed_decode_b200 as fg

    case, cache = st["case"], st["cache"]
    if case["op"] == "attend":
        fg.fg_paged_attention(cache, st["q"], st["positions"], rows_per_seq=case["rows"], max_len=st["max_len"], accumulate=case["track"], out=st["out"], workspace=st["workspace"])
    elif case["op"] == "append":
        fg.fg_paged_kv_append(cache, st["k"], st["v"], st["positions"], rows_per_seq=case["rows"], row_counts=st["counts"], first_tokens=st["first"])
    else:
        fg.fg_paged_kv_evict(cache, st["lengths"], st["next"], case["budget"], case["recent"], new_lengths=st["new_lengths"], weights_out=st["weights_out"], tokens_out=st["tokens_out"])
    return _results(st)


def _results(st):
    case = st["case"]
    if case["op"] == "attend":
        return dict(out=st["out"], **(dict(weights=st["weights"]) if case["track"] else {}))
    got = {n: st[n] for n in POOLS}
    if case["op"] == "append":
        return got | (dict(weights=st["weights"], tokens=st["tokens"]) if case["track"] else {})
    return got | dict(weights=st["weights_out"], tokens=st["tokens_out"], lengths=st["new_lengths"])


def _values(codes, mins, scales):
    """fp32 [..., D] of codes [..., D/2] and mins, scales [..., D/group]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (mins.shape[-1], -1))
    return (c * scales.float()[..., None] + mins.float()[..., None]).flatten(-2)


def _attend(st):
    case, at = st["case"], st["table"].clamp(min=0).long()
    S, H, D, rows = case["seqs"], case["kv_heads"], case["head_dim"], case["rows"]
    R = case["heads"] // H

    def dense(pool):  # [S, H, slots, ...]
        return st[pool][at].transpose(1, 2).flatten(2, 3)

    q = st["q"].float().view(S, rows, H, R, D).permute(0, 2, 1, 3, 4).reshape(S, H, rows * R, D)
    scores = q @ _values(dense("k_codes"), dense("k_mins"), dense("k_scales")).transpose(-1, -2)
    last = st["positions"][:, None] + torch.arange(rows, device="cuda")  # [S, rows]: the last slot that a row sees
    seen = torch.arange(scores.shape[-1], device="cuda") <= last[:, :, None]
    seen = seen.repeat_interleave(R, 1)[:, None]
    scores = torch.where(seen, scores, -math.inf)
    p = torch.where(seen, torch.exp(scores - scores.amax(-1, keepdim=True)), 0.0)
    p = p / p.sum(-1, keepdim=True)
    out = p @ _values(dense("v_codes"), dense("v_mins"), dense("v_scales"))
    st["out"].copy_(out.view(S, H, rows, R, D).permute(0, 2, 1, 3, 4).reshape(S * rows, -1))
    if case["track"]:
        add = p.sum(2).unflatten(-1, (at.shape[1], -1)).transpose(1, 2)
        st["weights"].index_put_((at,), add, accumulate=True)
    return _results(st)


def _append(st):
    case, n = st["case"], st["k"].shape[0]
    rows, ps, H = case["rows"], case["page"], case["kv_heads"]
    r = torch.arange(n, device="cuda")
    s = r // rows
    if st["counts"] is not None:
        r = torch.where(r % rows < st["counts"][s], r, s * rows)  # a row behind the prompt's end: its first row once more
    slot = st["positions"][s].long() + r % rows
    at = (st["table"][s, slot // ps].long()[:, None], torch.arange(H, device="cuda")[None], (slot % ps)[:, None])
    for a in "kv":
        x = st[a][r].view(n, H, case["head_dim"])
        for name, value in zip(("codes", "mins", "scales"), _quantise(x, case["group"])):
            st["%s_%s" % (a, name)][at] = value
    if case["track"]:
        st["weights"][at] = torch.zeros((n, H), device="cuda")
        st["tokens"][at] = (st["first"][s] + r % rows).to(torch.int32)[:, None].expand(n, H)
    return _results(st)


def _evict(st):
    case, at = st["case"], st["table"].clamp(min=0).long()
    S, H, ps, budget = case["seqs"], case["kv_heads"], case["page"], case["budget"]
    n = st["lengths"].long()[:, None, None]
    w, t = (st[x][at].transpose(1, 2).flatten(2, 3) for x in ("weights", "tokens"))
    slot = torch.arange(w.shape[-1], device="cuda")
    inside = slot < n
    rank = torch.where(t >= st["next"][:, None, None] - case["recent"], math.inf, w)
    order = torch.where(inside, rank, -1.0).sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, True) & inside
    low = slot[:budget]
    moved = keep & (slot >= budget)
    movers = torch.where(moved, slot, slot.numel()).sort(-1).values[..., : low.numel()]
    hole = ~keep[..., : low.numel()]
    src = torch.where(hole, movers.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), low)
    fine = low < n.clamp(max=budget)
    src, dst = torch.where(fine, src, src[..., :1]), torch.where(fine, low, 0)  # behind the last slot: the first once more
    head = torch.arange(H, device="cuda")[None, :, None]
    seq = torch.arange(S, device="cuda")[:, None, None]
    source = (at[seq, src // ps], head, src % ps)
    target = (at[seq, dst // ps], head, dst % ps)
    for name in POOLS:
        st[name][target] = st[name][source]
    st["weights_out"][target] = st["weights"][source]
    st["tokens_out"][target] = st["tokens"][source]
    st["new_lengths"].copy_(st["lengths"].clamp(max=budget))
    return _results(st)


# ------------------------------------------------------------------ what they cost ----


def work(case):
    S, H, D, groups = case["seqs"], case["kv_heads"], case["head_dim"], case["head_dim"] // case["group"]
    slot = D + 8 * groups  # bytes of a slot: K and V codes, four fp16 numbers a group
    lengths = case["hi"] + (S - 1) * (case["lo"] + case["hi"]) / 2  # of all sequences together, on average
    if case["op"] == "attend":
        rows, heads = case["rows"], case["heads"]
        return dict(bytes=lengths * H * (slot + 8 * case["track"]) + 4 * S * rows * heads * D, flops=4 * lengths * rows * heads * D)
    if case["op"] == "append":
        n = lengths if case["rows"] > 1 else S
        return dict(bytes=n * H * (4 * D + slot + 8 * case["track"]), flops=8 * n * H * D)
    # evict: weights and tokens of every slot read and those of the kept written; the moved slots read and written
    n, budget = lengths / S, case["budget"]
    over = max(0.0, n - budget)
    recent = min(case["recent"], budget, n)
    moved = min(over, recent) + max(0.0, over - recent) * (budget - recent) / max(1.0, n - recent)
    return dict(bytes=S * H * (8 * n + 8 * min(n, budget) + 2 * slot * moved), flops=S * H * n)


# ------------------------------------------------------------------ in 64 bits --------


def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["op"]](case, st)


def _slots(st, pool, s, n, dtype):
    """Sequence s's first n slots of a pool, [H, n, ...], page by page as the table names them."""
    ps = st["case"]["page"]
    pages = [int(p) for p in st["table"][s, : -(-n // ps)]]
    return torch.cat([st[pool][p] for p in pages], 1)[:, :n].to(dtype)


def _exact_attend(case, st):
    S, H, D, G, rows = case["seqs"], case["kv_heads"], case["head_dim"], case["group"], case["rows"]
    R, ps, f64 = case["heads"] // H, case["page"], torch.float64
    out = torch.zeros((S, rows, H, R, D), dtype=f64, device="cuda")
    weights = st["weights"].to(f64) if case["track"] else None
    q = st["q"].to(f64).view(S, rows, H, R, D)
    for s in range(S):
        n = int(st["positions"][s]) + rows
        side = {}
        for a in "kv":
            c = _slots(st, a + "_codes", s, n, torch.int32)
            x = torch.empty((H, n, D), dtype=f64, device="cuda")
            x[..., 0::2], x[..., 1::2] = c % 16, c // 16
            for g in range(D // G):
                x[..., g * G : (g + 1) * G] *= _slots(st, a + "_scales", s, n, f64)[..., g : g + 1]
                x[..., g * G : (g + 1) * G] += _slots(st, a + "_mins", s, n, f64)[..., g : g + 1]
            side[a] = x
        for r in range(rows):
            m = n - rows + r + 1
            p = torch.softmax(torch.einsum("hrd,htd->hrt", q[s, r], side["k"][:, :m]), -1)
            out[s, r] = torch.einsum("hrt,htd->hrd", p, side["v"][:, :m])
            if case["track"]:
                share = p.sum(1)
                for i in range(0, m, ps):
                    weights[int(st["table"][s, i // ps]), :, : min(ps, m - i)] += share[:, i : i + ps]
    return dict(out=out.view(S * rows, -1), **(dict(weights=weights) if case["track"] else {}))


def _exact_append(case, st):
    S, H, D, G, rows, ps = case["seqs"], case["kv_heads"], case["head_dim"], case["group"], case["rows"], case["page"]
    got = {n: None if "codes" in n else st[n].double() for n in POOLS}
    if case["track"]:
        got |= dict(weights=st["weights"].double(), tokens=None)
    for s in range(S):
        n = rows if st["counts"] is None else int(st["counts"][s])
        at = int(st["positions"][s]) + torch.arange(n, device="cuda")
        page, off = st["table"][s].long()[at // ps], at % ps
        for a in "kv":
            g = st[a][s * rows : s * rows + n].double().view(n, H, D // G, G)
            got[a + "_mins"][page, :, off] = g.min(-1).values
            got[a + "_scales"][page, :, off] = (g.max(-1).values - g.min(-1).values) / 15
        if case["track"]:
            got["weights"][page, :, off] = 0.0
    return got


def _exact_evict(case, st):
    S, H, ps, budget = case["seqs"], case["kv_heads"], case["page"], case["budget"]
    names = [n for n in POOLS if "codes" not in n]
    got = {n: st[n].cpu().double() for n in names}
    got["weights"], got["tokens"] = st["weights_out"].cpu().double(), st["tokens_out"].cpu()
    table, old = st["table"].cpu().tolist(), {n: got[n].clone() for n in names}
    w_all, t_all = st["weights"].cpu(), st["tokens"].cpu()
    for s in range(S):
        n = int(st["lengths"][s])
        page = torch.tensor([table[s][i // ps] for i in range(n)])
        off = torch.arange(n) % ps
        since = int(st["next"][s]) - case["recent"]
        for h in range(H):
            w, t = w_all[page, h, off].tolist(), t_all[page, h, off].tolist()
            order = sorted(range(n), key=lambda i: (t[i] < since, 0.0 if t[i] >= since else -w[i], i))
            keep = set(order[:budget])
            src = list(range(min(n, budget)))
            above = iter(sorted(i for i in keep if i >= budget))
            src = torch.tensor([i if i in keep else next(above) for i in src])
            dst = torch.arange(len(src))
            for name in names:
                got[name][page[dst], h, off[dst]] = old[name][page[src], h, off[src]]
            got["weights"][page[dst], h, off[dst]] = w_all[page[src], h, off[src]].double()
            got["tokens"][page[dst], h, off[dst]] = t_all[page[src], h, off[src]]
    return {n: None for n in POOLS if "codes" in n} | got | dict(lengths=st["lengths"].cpu().clamp(max=budget))
