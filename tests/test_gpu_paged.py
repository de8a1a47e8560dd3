"""The paged 4-bit KV cache against plain implementations in 64 bits: append (bit for bit), attention with and without
the accumulation of its weights, eviction (exact), and a run of them together.

Attention's tolerance, per output value.  The kernel holds scores, softmax and sums in fp32.  Its output is rounded to
fp16: 2^-11 of it.  The weight w = p * scale that multiplies a group's codes enters the tensor core as two fp16 numbers,
2^-22 of it (2^-25 absolute where the second is subnormal), against codes of at most 15.  The codes are fp16 subnormals
c * 2^-20, and a product with one is aligned by the exponent -14: what is kept of the 16 products of an MMA is a multiple
of 2^-24 * 2 w_max 2^-14, that is 2^-17 w_max in units of a code, so that an MMA drops less than 16 * 2^-17 w_max, and all
of them less than 2^-13 sum p scale.  With q.k = sum_g (min_g sum q + scale_g sum q c), each of the <= D + 2 D/G fp32
additions and products of a score is off by 2^-24 of magnitudes below A = sum |q| (|min| + 15 scale) in each direction,
twice that on a tensor core that truncates; exp2 adds 2^-21 and each of the n/128 + 8 chained additions and rescalings
of the sums 2^-23.  So
  |out - ref| <= 2^-11 |ref| + (2^-13 + 15 * 2^-22) sum p scale + 2 delta sum p (|min| + 15 scale) + n 2^-25 * 15 * 4 / l
  delta = 2 (D + 2 D/G) 2^-23 max A + 2^-21 + (n/128 + 8) 2^-23,  l = sum exp(s - max s)
(4: the running reference of the exponent may lie 2 binary orders below the maximum).  A slot's weight grows by sums of
p: delta of the growth, and 2^-23 per addition (one for each row and head) of the total."""
import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si

pytestmark = pytest.mark.gpu

fg = None


@pytest.fixture(autouse=True)
def _bind_library(fg_lib):
    global fg
    fg = fg_lib


RANGE = 4


def flagged(code=RANGE):
    with pytest.raises(fg.FgError) as e:
        fg.fg_sync_status()
    assert e.value.code == code


def make_cache(rng, lengths, H, D, G, ps, track=False, extra=3, spread=1.0, poison=True):
    """A cache of random groups: lengths[s] slots of each sequence hold data, every other slot of every page holds NaN,
    infinite or huge numbers, and table entries past a sequence's pages hold numbers that are no pages."""
    S = len(lengths)
    width = max(1, max(-(-n // ps) for n in lengths)) + 1
    pages = sum(-(-n // ps) for n in lengths) + extra
    order = rng.permutation(pages)
    table = np.full((S, width), -7, np.int32)
    table[:, 1::2] = 2**31 - 1
    used, at = np.zeros((pages, ps), bool), 0
    for s, n in enumerate(lengths):
        for i in range(-(-n // ps)):
            table[s, i] = order[at]
            used[order[at], : min(ps, n - i * ps)] = True
            at += 1
    NG = D // G
    arrays = []
    for _ in range(2):
        arrays.append(rng.integers(0, 256, (pages, H, ps, D // 2), dtype=np.uint8))
        arrays.append((rng.normal(-2.4, 0.4, (pages, H, ps, NG)) * spread).astype(np.float16))
        arrays.append((np.abs(rng.normal(0.31, 0.05, (pages, H, ps, NG))) * spread).astype(np.float16))
    if poison:
        free = ~np.broadcast_to(used[:, None, :, None], (pages, H, ps, NG))
        bad = np.array([np.nan, np.inf, -np.inf, 65504, -65504], np.float16)
        for i in (1, 2, 4, 5):
            arrays[i] = np.where(free, bad[rng.integers(0, 5, free.shape)], arrays[i])
    dev = [torch.from_numpy(a).cuda() for a in arrays]
    c = fg.PagedKVCache(pages, H, D, ps, torch.from_numpy(table).cuda(), group=G, arrays=dev, track=track)
    if track:
        w = np.exp(rng.normal(-7, 2, (pages, H, ps))).astype(np.float32)
        c.weights.copy_(torch.from_numpy(w))
        c.tokens.copy_(torch.from_numpy(rng.integers(0, 1 << 20, (pages, H, ps), dtype=np.int32)))
    return c


def dense(cache, pool, s, n):
    """Sequence s's first n slots of a pool as numpy [H, n, ...]."""
    ps = cache.page_size
    t = cache.page_table[s].cpu().numpy()
    a = pool.cpu().numpy()
    if n == 0:
        return a[:0].reshape((a.shape[1], 0) + a.shape[3:])
    return np.concatenate([a[t[i]] for i in range(-(-n // ps))], 1)[:, :n]


def values(cache, s, n, side):
    """(values, magnitudes |min| + 15 scale, scales, each [H, n, D] float64) of k or v."""
    c = dense(cache, getattr(cache, side + "_codes"), s, n)
    mn = np.repeat(dense(cache, getattr(cache, side + "_mins"), s, n).astype(np.float64), cache.group, -1)
    sc = np.repeat(dense(cache, getattr(cache, side + "_scales"), s, n).astype(np.float64), cache.group, -1)
    codes = np.stack((c & 15, c >> 4), -1).reshape(c.shape[:-1] + (-1,)).astype(np.float64)
    return mn + codes * sc, np.abs(mn) + 15 * sc, sc


def ref_attention(cache, q, positions, rows_per_seq, counts=None):
    """(out, tolerance, {(s): (growth of weights [H, n], its tolerance)}) in float64."""
    q = q.cpu().numpy().astype(np.float64)
    rows, D, H = q.shape[0], cache.head_dim, cache.num_heads
    R = q.shape[1] // D // H
    q = q.reshape(rows, H, R, D)
    out, tol, grown = np.zeros_like(q), np.zeros_like(q), {}
    NG = D // cache.group
    for s in range(rows // rows_per_seq):
        count = rows_per_seq if counts is None else counts[s]
        if positions[s] < 0 or count == 0:
            continue
        n = positions[s] + count
        k, ka, _ = values(cache, s, n, "k")
        v, va, vs = values(cache, s, n, "v")
        add, add_tol = np.zeros((H, n)), np.zeros((H, n))
        for i in range(count):
            r, m = s * rows_per_seq + i, positions[s] + i + 1
            sc = np.einsum("hrd,htd->hrt", q[r], k[:, :m])
            e = np.exp(sc - sc.max(-1, keepdims=True))
            l = e.sum(-1, keepdims=True)
            p = e / l
            A = np.einsum("hrd,htd->hrt", np.abs(q[r]), ka[:, :m]).max(-1, keepdims=True)
            delta = 2 * (D + 2 * NG) * 2.0**-23 * A + 2.0**-21 + (m / 128 + 8) * 2.0**-23
            o = np.einsum("hrt,htd->hrd", p, v[:, :m])
            out[r] = o
            tol[r] = (2.0**-11 * np.abs(o) + (2.0**-13 + 15 * 2.0**-22) * np.einsum("hrt,htd->hrd", p, vs[:, :m])
                      + 2 * delta * np.einsum("hrt,htd->hrd", p, va[:, :m]) + m * 2.0**-25 * 60 / l)
            add[:, :m] += p.sum(1)
            add_tol[:, :m] += (2 * delta * p).sum(1)
        grown[s] = (add, add_tol)
    return out.reshape(rows, -1), tol.reshape(rows, -1), grown


def check_attention(cache, q, positions, rows_per_seq=1, counts=None, max_len=None, accumulate=False, workspace=None):
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    before = cache.weights.clone() if accumulate else None
    out = fg.fg_paged_attention(cache, q, pos, rows_per_seq=rows_per_seq, row_counts=cnt, max_len=max_len,
                                accumulate=accumulate, workspace=workspace)
    fg.fg_sync_status()
    ref, tol, grown = ref_attention(cache, q, positions, rows_per_seq, counts)
    err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), (err.max(), (err / np.maximum(tol, 1e-30)).max())
    if accumulate:
        want, slack = before.cpu().numpy().astype(np.float64), np.zeros(before.shape)
        per = rows_per_seq * (q.shape[1] // cache.head_dim // cache.num_heads)
        t = cache.page_table.cpu().numpy()
        for s, (add, add_tol) in grown.items():
            for i in range(0, add.shape[1], cache.page_size):
                a, b = add[:, i:i + cache.page_size], add_tol[:, i:i + cache.page_size]
                at = (t[s, i // cache.page_size], slice(None), slice(0, a.shape[1]))
                want[at] += a
                slack[at] += b + (per + 2) * 2.0**-23 * want[at]
        got = cache.weights.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - want) <= slack), (np.abs(got - want) / np.maximum(slack, 1e-30)).max()
    return out


def queries(rng, rows, heads, D, size=1.5):
    return torch.from_numpy((rng.normal(0, size * D**-0.5, (rows, heads * D))).astype(np.float16)).cuda()


# ------------------------------------------------------------------ append ------------


@pytest.mark.parametrize("D,G,ps", [(64, 64, 16), (128, 64, 48), (128, 128, 64), (256, 64, 16), (256, 128, 80)])
@pytest.mark.parametrize("rows,counts,positions", [
    (1, None, [0, 15, 16, -1, 70]), (5, None, [0, 14, -1, 60, 31]), (40, [40, 0, 1, 17, 33], [0, 3, 47, 48, -1])])
def test_append_bits(D, G, ps, rows, counts, positions):
    rng = np.random.default_rng(D + ps + rows)
    S, H = len(positions), 3
    cap = 128
    c = make_cache(rng, [cap] * S, H, D, G, ps, track=True)
    before = [a.clone() for a in c.arrays() + [c.weights, c.tokens]]
    qkv = si.normal_f16(3, 5, (S * rows, 3 * H * D), 1.0)
    qkv[0, H * D:H * D + G] = 0.5                                       # a constant group: scale 0
    dev = torch.from_numpy(qkv).cuda()
    k, v = dev[:, H * D:2 * H * D], dev[:, 2 * H * D:]
    if counts is not None:                                              # the padding may hold anything
        for s in range(S):
            dev[s * rows + counts[s]:(s + 1) * rows] = float("nan")
    first = torch.arange(100, 100 + S, dtype=torch.int32, device="cuda") * 1000
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    fg.fg_paged_kv_append(c, k, v, i32(positions), rows_per_seq=rows, row_counts=i32(counts), first_tokens=first)
    fg.fg_sync_status()
    want = [a.cpu().numpy() for a in before]
    t = c.page_table.cpu().numpy()
    for s in range(S):
        for i in range(rows if counts is None else counts[s]):
            if positions[s] < 0:
                continue
            p = positions[s] + i
            at = (t[s, p // ps], slice(None), p % ps)
            for side, x in ((0, k), (3, v)):
                r = oracle.quantize(x[s * rows + i].cpu().numpy().reshape(H, D), group=G)
                want[side][at], want[side + 1][at], want[side + 2][at] = r.codes, r.mins, r.scales
            want[6][at], want[7][at] = 0.0, 100000 + s * 1000 + i
    for a, w in zip(c.arrays() + [c.weights, c.tokens], want):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), w.view(np.uint8))


def test_append_equals_the_contiguous_cache():
    S, H, D, L, P = 3, 4, 128, 128, 21
    a, b = fg.KVCache(S, H, D, L), fg.KVCache(S, H, D, L)
    k = torch.from_numpy(si.normal_f16(1, 22, (S * P, H * D), 1.0)).cuda()
    v = torch.from_numpy(si.normal_f16(1, 23, (S * P, H * D), 1.0)).cuda()
    pos = torch.tensor([0, 40, 107], dtype=torch.int32, device="cuda")
    fg.fg_kv_append(a, k, v, pos, rows_per_seq=P)
    c = fg.PagedKVCache.from_cache(b, track=True)
    fg.fg_paged_kv_append(c, k, v, pos, rows_per_seq=P)
    fg.fg_sync_status()
    for x, y in zip(a.arrays(), b.arrays()):
        assert torch.equal(x, y)
    assert c.tokens[1, 2, 40:61].tolist() == list(range(40, 61))        # without first_tokens: the slots' own numbers


def test_append_flags_bad_slots_and_leaves_the_rest():
    rng = np.random.default_rng(1)
    H, D, ps = 2, 128, 16
    c = make_cache(rng, [48] * 6, H, D, 64, ps, track=True)
    c.page_table[1, 0] = c.num_pages                                    # a page that is none
    c.page_table[2, 0] = -1
    before = [a.clone() for a in c.arrays() + [c.weights, c.tokens]]
    k = torch.from_numpy(si.normal_f16(2, 22, (12, H * D), 1.0)).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # past the table's pages; two bad pages; below -1; a count above rows_per_seq; a count below 0
    fg.fg_paged_kv_append(c, k, k, i32([c.max_pages * ps, 3, 15, -2, 0, 0]), rows_per_seq=2, row_counts=i32([2, 2, 1, 2, 3, -1]))
    flagged()
    for a, b in zip(c.arrays() + [c.weights, c.tokens], before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    fg.fg_paged_kv_append(c, k, k, i32([2**31 - 1, -1, -1, -1, -1, 4]), rows_per_seq=2)   # no overflow past int32
    flagged()
    r = oracle.quantize(k[11].cpu().numpy().reshape(H, D))
    page = int(c.page_table[5, 0])
    assert np.array_equal(c.v_codes[page, :, 5].cpu().numpy(), r.codes)
    fg.fg_sync_status()                                                 # and the flag is gone


# ------------------------------------------------------------------ attention ---------

SHAPES = [  # D, G, page, kv heads, ratio
    (64, 64, 16, 2, 1), (64, 64, 64, 3, 4), (128, 64, 48, 2, 1), (128, 64, 16, 1, 8), (128, 128, 64, 2, 3),
    (256, 64, 80, 1, 5), (256, 128, 32, 2, 1), (128, 64, 128, 4, 9), (256, 64, 16, 1, 17), (64, 64, 32, 1, 2),
]


@pytest.mark.parametrize("accumulate", [False, True], ids=["plain", "tracked"])
@pytest.mark.parametrize("D,G,ps,H,R", SHAPES)
def test_attention_one_new_token(D, G, ps, H, R, accumulate):
    rng = np.random.default_rng(D * 7 + ps + R)
    lengths = [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 300, 511]
    c = make_cache(rng, lengths, H, D, G, ps, track=accumulate)
    q = queries(rng, len(lengths), H * R, D)
    check_attention(c, q, [n - 1 for n in lengths], accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True], ids=["plain", "tracked"])
@pytest.mark.parametrize("D,G,ps,H,R", SHAPES)
def test_attention_rows_counts_and_inactive_sequences(D, G, ps, H, R, accumulate):
    rng = np.random.default_rng(D + ps * 5 + R)
    rows = 6
    counts = [6, 0, 1, 5, 6, 3]
    positions = [0, 9, 200, 31, -1, 16 * 9 - 2]
    c = make_cache(rng, [max(0, p) + n if p >= 0 else 0 for p, n in zip(positions, counts)], H, D, G, ps, track=accumulate)
    q = queries(rng, len(counts) * rows, H * R, D)
    for s, n in enumerate(counts):                                      # the padding's queries may hold anything
        q[s * rows + n:(s + 1) * rows] = float("nan")
    q.view(len(counts), rows, -1)[4] = float("inf")
    zeros = torch.zeros_like(q)
    qz = torch.where(torch.isfinite(q), q, zeros)
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = fg.fg_paged_attention(c, q, pos, rows_per_seq=rows, row_counts=cnt)
    fg.fg_sync_status()
    for s, n in enumerate(counts):
        dead = out.view(len(counts), rows, -1)[s, (n if positions[s] >= 0 else 0):]
        assert torch.count_nonzero(dead) == 0 and torch.isfinite(dead).all()
    assert torch.equal(out, check_attention(c, qz, positions, rows, counts, accumulate=accumulate))


@pytest.mark.parametrize("accumulate", [False, True], ids=["plain", "tracked"])
@pytest.mark.parametrize("D,G,ps,H,R,lengths", [
    (128, 64, 64, 2, 1, [20011]), (128, 128, 16, 1, 8, [9000, 1, 4097]), (64, 64, 48, 1, 1, [30000, 12]),
    (256, 64, 128, 1, 4, [5000, 2049])])
def test_attention_split_over_long_sequences(D, G, ps, H, R, lengths, accumulate):
    rng = np.random.default_rng(D + R)
    c = make_cache(rng, lengths, H, D, G, ps, track=accumulate)
    q = queries(rng, len(lengths), H * R, D, 3.0)
    out = check_attention(c, q, [n - 1 for n in lengths], max_len=max(lengths), accumulate=accumulate)
    if not accumulate:                                                  # less scratch, or none: split less
        need = fg.fg_paged_attention_workspace_bytes(c, H * R, len(lengths), 1, max(lengths))
        for nbytes in (need // 3, 0):
            check_attention(c, q, [n - 1 for n in lengths], max_len=max(lengths),
                            workspace=torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
    else:
        need = fg.fg_paged_attention_workspace_bytes(c, H * R, len(lengths), 1, max(lengths), True)
        if need:
            with pytest.raises(fg.FgError, match="WORKSPACE"):
                fg.fg_paged_attention(c, q, torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device="cuda"),
                                      max_len=max(lengths), accumulate=True,
                                      workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert out.shape == q.shape


@pytest.mark.parametrize("accumulate", [False, True], ids=["plain", "tracked"])
@pytest.mark.parametrize("D,G,R,rows", [(128, 64, 8, 6), (64, 64, 5, 7), (256, 128, 1, 9), (128, 128, 1, 1)])
def test_attention_partitioned_tiles_and_counts(D, G, R, rows, accumulate):
    """Long enough to be shared by all warps: tiles without a live column, cut and whole items, inactive sequences."""
    rng = np.random.default_rng(D + R)
    counts = [rows, 0, 1, max(1, rows - 2), rows, rows, 1]
    positions = [0, 9, 3001, 31, -1, 2500, 700]
    c = make_cache(rng, [max(0, p) + n if p >= 0 else 0 for p, n in zip(positions, counts)], 2, D, G, 48, track=accumulate)
    assert c.max_pages * 48 > 2048
    out = check_attention(c, queries(rng, len(counts) * rows, 2 * R, D), positions, rows, counts, accumulate=accumulate)
    for s, n in enumerate(counts):
        assert torch.count_nonzero(out.view(len(counts), rows, -1)[s, (n if positions[s] >= 0 else 0):]) == 0


@pytest.mark.parametrize("rows,R", [(33, 1), (20, 5)])
def test_attention_prompt_rows(rows, R):
    rng = np.random.default_rng(rows)
    H, D = 2, 128
    positions = [0, 100]
    c = make_cache(rng, [p + rows for p in positions], H, D, 64, 32, track=True)
    check_attention(c, queries(rng, 2 * rows, H * R, D), positions, rows, accumulate=True)


@pytest.mark.parametrize("size,spread", [(40.0, 1.0), (1.5, 2000.0), (0.0, 1.0), (300.0, 30.0)])
def test_attention_extreme_scores_and_scales(size, spread):
    """One-hot softmaxes, scales near fp16's largest, equal scores."""
    rng = np.random.default_rng(int(size))
    H, D, lengths = 2, 128, [1, 77, 700]
    c = make_cache(rng, lengths, H, D, 64, 64, track=True, spread=spread)
    check_attention(c, queries(rng, 3, 2 * H, D, size if spread == 1.0 else size / spread), [n - 1 for n in lengths],
                    accumulate=True)


def test_attention_rising_scores():
    """Scores that grow along the sequence: the running maximum moves all the way."""
    rng = np.random.default_rng(5)
    H, D, n = 1, 64, 900
    c = make_cache(rng, [n], H, D, 64, 64, track=True)
    t = c.page_table[0].cpu().tolist()
    for i in range(n):
        c.k_mins[t[i // 64], :, i % 64] = i * 0.02 - 2.4
    check_attention(c, torch.full((1, D), 0.05, dtype=torch.float16, device="cuda"), [n - 1], accumulate=True)


def test_attention_strides_and_untouched_rows():
    rng = np.random.default_rng(8)
    H, R, D, lengths = 2, 2, 128, [70, 5, 200]
    c = make_cache(rng, lengths, H, D, 64, 16)
    q = queries(rng, 5, H * R, D)
    wide = torch.full((5, 3 * H * R * D + 8), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 8:8 + H * R * D] = q
    big = torch.full((6, H * R * D + 64), 7.0, dtype=torch.float16, device="cuda")
    pos = torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device="cuda")
    fg.fg_paged_attention(c, wide[:3, 8:8 + H * R * D], pos, out=big[:3, :H * R * D])
    fg.fg_sync_status()
    assert torch.equal(big[:3, :H * R * D], check_attention(c, q[:3].contiguous(), [n - 1 for n in lengths]))
    assert (big[3:] == 7.0).all() and (big[:, H * R * D:] == 7.0).all()


def test_attention_flags_bad_sequences_only():
    rng = np.random.default_rng(9)
    H, D, ps = 2, 128, 16
    lengths = [40, 40, 40, 40, 40, 40, 40]
    c = make_cache(rng, lengths, H, D, 64, ps, track=True)
    c.page_table[0, 1] = c.num_pages
    c.page_table[1, 2] = -1
    before = c.weights.clone()
    q = queries(rng, 7, H, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # bad pages, past max_len, below -1, bad counts, and one good sequence
    out = fg.fg_paged_attention(c, q, i32([39, 39, 40, -2, 39, 39, 39]), row_counts=i32([1, 1, 1, 1, 2, -1, 1]), max_len=40,
                                accumulate=True)
    flagged()
    assert torch.count_nonzero(out[:6]) == 0
    got = c.weights.clone()
    mine = c.page_table[6, :3].long()
    assert torch.count_nonzero(got[mine] - before[mine]) > 0
    got[mine] = before[mine]
    assert torch.equal(got, before)
    c.weights.copy_(before)
    good = fg.fg_paged_attention(c, q, i32([-1] * 6 + [39]), accumulate=True)
    fg.fg_sync_status()
    assert torch.equal(good, out)


def test_attention_equals_the_contiguous_caches():
    """Over one cache, the paged call and the contiguous one agree to the sum of their roundings."""
    S, H, D, L = 4, 4, 128, 320
    cache = fg.KVCache(S, H, D, L)
    k = torch.from_numpy(si.normal_f16(1, 22, (S * L, H * D), 1.0)).cuda()
    v = torch.from_numpy(si.normal_f16(1, 23, (S * L, H * D), 1.0)).cuda()
    fg.fg_kv_append(cache, k, v, torch.zeros(S, dtype=torch.int32, device="cuda"), rows_per_seq=L)
    q = torch.from_numpy(si.normal_f16(1, 24, (S, H * D), D**-0.5)).cuda()
    pos = [3, 100, 319, 256]
    c = fg.PagedKVCache.from_cache(cache)
    out = check_attention(c, q, pos)
    old = fg.fg_attention_decode(cache, q, torch.tensor(pos, dtype=torch.int32, device="cuda"))
    # the contiguous kernel's bound is 2e-3 of the largest output (tests of the individual kernels)
    assert (out.float() - old.float()).abs().max() <= 4e-3 * old.float().abs().max()


def test_attention_is_deterministic():
    rng = np.random.default_rng(3)
    c = make_cache(rng, [5000, 3, 777], 2, 128, 64, 64, track=True)
    q = queries(rng, 3, 8, 128)
    pos = torch.tensor([4999, 2, 776], dtype=torch.int32, device="cuda")
    w0, got = c.weights.clone(), []
    for _ in range(5):
        c.weights.copy_(w0)
        got.append((fg.fg_paged_attention(c, q, pos, accumulate=True).clone(), c.weights.clone()))
    for o, w in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(w, got[0][1])


# ------------------------------------------------------------------ one slot with most of the weight --------------
#
# A query row with a single one in it reads one dim of the keys, whose minima and steps are multiples of 2^-6: scores are
# exact, and what is left of the tolerance above is the weights' own.  With T the span of a row's scores (nats):
#   p       the product with log2 e and its subtraction from the running maximum, 2^-23 T each, exp2 2^-22 and the same
#           for rescalings: (T + 8) 2^-22 of it
#   sums    a warp that has all slots adds two a block of 32 to a lane's sums: (n / 16 + 16) 2^-24 of their terms, and the
#           same for the sum that divides
#   w       two fp16 numbers, 2^-22 of w, of w times a power of two under which the run's largest scale lies in [2^12,
#           2^13]: where the second is subnormal 2^-25 absolute of that, 2^-37 max scale, against codes of 15
#   MMA     16 products aligned to the largest: 2^-13 sum p scale, as above
#   output  2^-11 of it, 2^-25 where it is subnormal
# With N = sum p (|min| + 15 scale) and l = sum exp(s - max s):
#   |out - ref| <= 2^-11 |ref| + 2^-25 + (2^-13 + 15 * 2^-22) sum p scale + 15 * 2^-37 n max scale / l
#                  + 2 ((T + 8) 2^-22 + (n / 16 + 16) 2^-24) N


def sink_cache(rng, n, H, D, G, ps, vscale, span, track=False, sink=0, step=2.0**-3):
    """A sequence of n slots whose dim scores are -span + step code for all slots but `sink`, whose own is 0 with V a tenth of
    the others' size.  V's scales lie around vscale, its minima at -7.5 scales."""
    c = make_cache(rng, [n], H, D, G, ps, track=track)
    t = c.page_table[0].cpu().numpy()
    page, off = t[np.arange(n) // ps], np.arange(n) % ps
    NG = D // G
    km, ks = np.full((n, H, NG), -span, np.float16), np.full((n, H, NG), step, np.float16)
    km[sink], ks[sink] = 0, 0
    vs = (vscale * np.exp(0.2 * rng.normal(size=(n, H, NG)))).astype(np.float16)
    vs[sink] = np.float16(vscale * 0.1)
    vm = (-7.5 * vs.astype(np.float64)).astype(np.float16)
    at = (torch.from_numpy(page).long().cuda(), slice(None), torch.from_numpy(off).cuda())
    for pool, x in ((c.k_mins, km), (c.k_scales, ks), (c.v_mins, vm), (c.v_scales, vs)):
        pool[at] = torch.from_numpy(x).cuda()
    return c


def unit_queries(rows, heads, D, size=1.0):
    """Row r's head h: `size` at one dim, another for every row and head; zeros else."""
    q = np.zeros((rows, heads, D), np.float16)
    for r in range(rows):
        for h in range(heads):
            q[r, h, (7 * r + 13 * h + 3) % D] = size
    return torch.from_numpy(q.reshape(rows, -1)).cuda()


def sharp_attention(cache, q, n, rows):
    """(out, tolerance, growth, its tolerance) of the rows of a sequence with n slots in all, by the formulas above."""
    q = q.cpu().numpy().astype(np.float64)
    D, H = cache.head_dim, cache.num_heads
    q = q.reshape(rows, H, -1, D)
    k, _, _ = values(cache, 0, n, "k")
    v, va, vs = values(cache, 0, n, "v")
    out, tol = np.zeros_like(q), np.zeros_like(q)
    add, add_tol = np.zeros((H, n)), np.zeros((H, n))
    for r in range(rows):
        m = n - rows + r + 1
        sc = np.einsum("hrd,htd->hrt", q[r], k[:, :m])
        span = float((sc.max(-1) - sc.min(-1)).max())
        e = np.exp(sc - sc.max(-1, keepdims=True))
        l = e.sum(-1, keepdims=True)
        p = e / l
        mean = lambda x: np.einsum("hrt,htd->hrd", p, x[:, :m])
        rel = (span + 8) * 2.0**-22 + (n / 16 + 16) * 2.0**-24
        o = mean(v)
        out[r] = o
        tol[r] = (2.0**-11 * np.abs(o) + 2.0**-25 + (2.0**-13 + 15 * 2.0**-22) * mean(vs)
                  + 15 * 2.0**-37 * m * vs[:, :m].max() / l + 2 * rel * mean(va))
        add[:, :m] += p.sum(1)
        add_tol[:, :m] += 2 * rel * p.sum(1)
    return out.reshape(rows, -1), tol.reshape(rows, -1), add, add_tol


def check_sharp(cache, q, n, rows=1, seqs=1, workspace=None, max_len=None, share=None):
    """`seqs` sequences over the same pages (only read); share: the least part of the outputs' spread that the tolerance is."""
    ref, tol, _, _ = sharp_attention(cache, q, n, rows)
    if share is not None:
        assert tol.max() <= share * np.abs(ref).max(), (tol.max(), np.abs(ref).max())
    c = cache
    if seqs > 1:
        c = fg.PagedKVCache(cache.num_pages, cache.num_heads, cache.head_dim, cache.page_size,
                            cache.page_table.repeat(seqs, 1).contiguous(), group=cache.group, arrays=cache.arrays())
    pos = torch.full((seqs,), n - rows, dtype=torch.int32, device="cuda")
    out = fg.fg_paged_attention(c, q.repeat(seqs, 1).contiguous(), pos, rows_per_seq=rows, max_len=max_len, workspace=workspace)
    fg.fg_sync_status()
    err = np.abs(out.view(seqs, rows, -1).cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), ((err / tol).max(), err.max(), np.abs(ref).max())


SINKS = [  # D, G, page, kv heads, ratio, rows: one column, one tile, two tiles, four groups, several rows
    (128, 64, 64, 2, 1, 1), (64, 64, 16, 2, 1, 1), (256, 128, 32, 1, 1, 1), (128, 128, 64, 1, 8, 1), (64, 64, 48, 1, 16, 1),
    (256, 64, 16, 1, 4, 1), (128, 64, 32, 1, 3, 3)]


def tail_span(n, mass=0.02, top=15 / 8):
    """Nats below the sink at which n slots of -span + code / 8 hold about `mass` of the weight, a multiple of 1/8."""
    return round(8 * np.log(n * np.expm1(top) / top / mass)) / 8


@pytest.mark.parametrize("vscale", [0.03, 0.001])
@pytest.mark.parametrize("way", ["short", "whole", "parts", "many"])
@pytest.mark.parametrize("D,G,ps,H,R,rows", SINKS)
def test_attention_sink_and_small_values(D, G, ps, H, R, rows, way, vscale):
    """One slot with 98 % of the weight and the rest on thousands, V small: the rest's share of the output stands.  In one
    run of a warp or CTA (short, whole, many: more items than warps), and in parts."""
    rng = np.random.default_rng(D + R + len(way))
    n = 1000 if way == "short" else 16384
    c = sink_cache(rng, n, H, D, G, ps, vscale, tail_span(n))
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    check_sharp(c, unit_queries(rows, H * R, D), n, rows, seqs=2600 // H if way == "many" else 1,
                workspace=none if way == "whole" else None, max_len=n, share=0.01)


@pytest.mark.parametrize("sink", [0, 777, 15000, 16383])
@pytest.mark.parametrize("R", [1, 4])
def test_attention_sink_anywhere(R, sink):
    n = 16384
    c = sink_cache(np.random.default_rng(sink), n, 1, 128, 64, 64, 0.002, tail_span(n), sink=sink)
    check_sharp(c, unit_queries(1, R, 128), n, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), share=0.01)


@pytest.mark.parametrize("R", [1, 5])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 64), (256, 128)])
@pytest.mark.parametrize("span,n", [(0.0, 700), (300.0, 700), (300.0, 5000), (1.0, 1)])
def test_attention_exact_scores(D, G, R, span, n):
    """Equal and one-hot softmaxes of exact scores: the outputs to their own rounding and the sums'."""
    rng = np.random.default_rng(n + R)
    c = sink_cache(rng, n, 2, D, G, 32, 0.3, span, step=0.0)
    check_sharp(c, unit_queries(1, 2 * R, D), n, share=0.01 if span else None)


@pytest.mark.parametrize("R", [1, 4])
@pytest.mark.parametrize("per_slot", [2.0**-6, 2.0**-5])
def test_attention_largest_scales_and_rising_scores(R, per_slot):
    """V from -65504 to 65504 (scales of 8733) under scores that rise by a binade or two from block to block: the running
    maximum lags, and p is up to 4."""
    rng = np.random.default_rng(R)
    n, D = 700, 128
    c = sink_cache(rng, n, 2, D, 64, 64, 1.0, 0.0, step=0.0)
    t = c.page_table[0].cpu().tolist()
    for i in range(n):
        c.k_mins[t[i // 64], :, i % 64] = i * per_slot
        c.v_mins[t[i // 64], :, i % 64] = -65504.0
        c.v_scales[t[i // 64], :, i % 64] = 8733.0
    q = unit_queries(1, 2 * R, D)
    _, tol, _, _ = sharp_attention(c, q, n, 1)
    assert tol.max() < 0.001 * 2 * 65504
    check_sharp(c, q, n)


@pytest.mark.parametrize("R", [1, 4, 12])
def test_attention_scales_of_all_sizes(R):
    """V's scales from 2^-24 to 8733 along the sequence, growing and shrinking, some 0: the tolerance is the largest's."""
    rng = np.random.default_rng(R)
    n, D = 3000, 128
    c = sink_cache(rng, n, 1, D, 64, 64, 1.0, 0.0, step=2.0**-4)
    t = c.page_table[0].cpu().tolist()
    for i in range(n):
        e = -24 + 37 * i / 2000 if i < 2000 else 13 - 37 * (i - 2000) / 1000
        x = 0.0 if i % 17 == 0 else 2.0**e
        c.v_scales[t[i // 64], :, i % 64] = x
        c.v_mins[t[i // 64], :, i % 64] = -7.5 * x
    for m in (30, 200, 1000, n):                                        # where only the small ones are seen, and all
        check_sharp(c, unit_queries(1, R, D), m)


@pytest.mark.parametrize("R", [1, 4])
@pytest.mark.parametrize("n", [1000, 16384])
def test_tracked_sink(R, n):
    """The same with the weights gathered: the output and each slot's growth."""
    D = 128
    c = sink_cache(np.random.default_rng(n), n, 2, D, 64, 64, 0.01, tail_span(n), track=True)
    c.weights.zero_()
    q = unit_queries(1, 2 * R, D)
    ref, tol, add, add_tol = sharp_attention(c, q, n, 1)
    out = fg.fg_paged_attention(c, q, torch.tensor([n - 1], dtype=torch.int32, device="cuda"), accumulate=True, max_len=n)
    fg.fg_sync_status()
    assert np.all(np.abs(out.cpu().numpy().astype(np.float64) - ref) <= tol)
    got = dense(c, c.weights, 0, n).astype(np.float64)
    assert np.all(np.abs(got - add) <= add_tol + R * 2.0**-23 * add)


# ------------------------------------------------------------------ eviction ----------


def ref_evict(cache, lengths, nxt, budget, recent):
    """Per sequence and head, the slot that each kept place is filled from."""
    src = {}
    for s, n in enumerate(lengths):
        if n <= budget:
            continue
        w, t = dense(cache, cache.weights, s, n), dense(cache, cache.tokens, s, n)
        for h in range(cache.num_heads):
            rank = lambda i: (0, 0.0, i) if t[h, i] >= nxt[s] - recent else (2, 0.0, i) if np.isnan(w[h, i]) else (1, -float(w[h, i]), i)
            keep = set(sorted(range(n), key=rank)[:budget])
            above = iter(sorted(i for i in keep if i >= budget))
            src[s, h] = [i if i in keep else next(above) for i in range(budget)]
    return src


def check_evict(cache, lengths, nxt, budget, recent, in_place=True, max_len=None, same_lengths=False):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pools = cache.arrays() + [cache.weights, cache.tokens]
    src = ref_evict(cache, lengths, nxt, budget, recent)
    want = [a.cpu().numpy().copy() for a in pools]
    t, ps = cache.page_table.cpu().numpy(), cache.page_size
    old = [w.copy() for w in want]
    wout = tout = None
    if not in_place:
        wout, tout = torch.full_like(cache.weights, -1.0), torch.full_like(cache.tokens, -1)
        want += [wout.cpu().numpy(), tout.cpu().numpy()]
    for s, n in enumerate(lengths):
        for h in range(cache.num_heads):
            m = np.array(src.get((s, h), range(max(0, n))), np.int64)
            i = np.arange(len(m))
            to, fr = (t[s, i // ps], h, i % ps), (t[s, m // ps], h, m % ps)
            for x in range(6 if not in_place else 8):
                want[x][to] = old[x][fr]
            if not in_place:
                want[8][to], want[9][to] = old[6][fr], old[7][fr]
    ln = i32(lengths)
    new = fg.fg_paged_kv_evict(cache, ln, i32(nxt), budget, recent, weights_out=wout, tokens_out=tout, max_len=max_len,
                               new_lengths=ln if same_lengths else None)
    fg.fg_sync_status()
    assert new.tolist() == [min(n, budget) for n in lengths]
    for a, w in zip(pools + ([] if in_place else [wout, tout]), want):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), w.view(np.uint8))


def tokens_in_order(cache, lengths):
    t, ps = cache.page_table.cpu(), cache.page_size
    for s, n in enumerate(lengths):
        for i in range(0, max(0, n), ps):
            cache.tokens[t[s, i // ps], :, :min(ps, n - i)] = torch.arange(i, min(n, i + ps), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "apart"])
@pytest.mark.parametrize("D,G,ps,H,budget,recent", [
    (64, 64, 16, 3, 32, 8), (128, 64, 48, 2, 100, 0), (128, 128, 64, 1, 64, 64), (256, 64, 16, 2, 257, 100),
    (256, 128, 80, 1, 1, 0), (128, 64, 64, 2, 512, 1), (64, 64, 32, 1, 16, 16)])
def test_evict_exact(D, G, ps, H, budget, recent, in_place):
    rng = np.random.default_rng(budget + ps)
    lengths = [0, 1, budget - 1, budget, budget + 1, budget + 2, budget + ps, 2 * budget + 3, 3 * budget + 700, -1]
    c = make_cache(rng, [max(0, n) for n in lengths], H, D, G, ps, track=True)
    tokens_in_order(c, lengths)
    check_evict(c, lengths, lengths, budget, recent, in_place)


@pytest.mark.parametrize("what", ["ties", "zeros", "nan", "inf", "negative", "protected_in_holes", "all_protected", "sorted", "reversed"])
def test_evict_ranks(what):
    rng = np.random.default_rng(len(what))
    H, budget, lengths = 2, 96, [97, 400, 1000]
    c = make_cache(rng, lengths, H, 128, 64, 32, track=True)
    tokens_in_order(c, lengths)
    nxt = list(lengths)
    if what == "ties":
        c.weights.copy_(torch.from_numpy(rng.integers(0, 3, c.weights.shape)))
    elif what == "zeros":
        c.weights.copy_(torch.from_numpy(np.where(rng.random(c.weights.shape) < 0.5, 0.0, -0.0)))
    elif what == "nan":
        c.weights[torch.rand(c.weights.shape, device="cuda") < 0.95] = float("nan")
    elif what == "inf":
        c.weights[torch.rand(c.weights.shape, device="cuda") < 0.5] = float("inf")
    elif what == "negative":
        c.weights.neg_()
    elif what == "protected_in_holes":                                  # tokens of any age in any slot
        c.tokens.copy_(torch.from_numpy(rng.permutation(c.tokens.numel()).reshape(c.tokens.shape).astype(np.int32) % 2000))
        nxt = [2000] * 3
    elif what == "all_protected":                                       # more protected slots than the budget
        c.tokens.fill_(2**31 - 1)
        nxt = [2**31 - 1] * 3
    else:
        t, ps = c.page_table.cpu(), c.page_size
        for s, n in enumerate(lengths):
            for i in range(n):
                c.weights[t[s, i // ps], :, i % ps] = i if what == "sorted" else n - i
    check_evict(c, lengths, nxt, budget, 24)


@pytest.mark.parametrize("weights", ["ties", "apart"])
@pytest.mark.parametrize("n,budget", [(20000, 1024), (9000, 8000), (40000, 39999), (5000, 16), (70001, 30000)])
def test_evict_long(n, budget, weights):
    rng = np.random.default_rng(n)
    c = make_cache(rng, [n, 100], 1, 64, 64, 64, track=True)
    tokens_in_order(c, [n, 100])
    if weights == "ties":
        c.weights.copy_(torch.round(c.weights * 2000))
    check_evict(c, [n, 100], [n, 100], budget, min(budget, 128), max_len=n)


@pytest.mark.parametrize("n,budget", [(140001, 70000), (131072, 65536)])
def test_evict_more_than_65535_moves(n, budget):
    """Holes and movers past 16 bits, all of a word's slots among them."""
    c = make_cache(np.random.default_rng(n), [n], 1, 64, 64, 64, track=True)
    tokens_in_order(c, [n])
    c.weights.copy_(torch.where(c.tokens >= budget, 1.0 + c.weights, 0.0))
    check_evict(c, [n], [n], budget, 0, max_len=n)


def test_evict_writes_lengths_in_place():
    rng = np.random.default_rng(4)
    lengths = [300, 20, 64, -1, 0]
    c = make_cache(rng, [300, 20, 64, 0, 0], 2, 64, 64, 16, track=True)
    tokens_in_order(c, lengths)
    check_evict(c, lengths, lengths, 48, 4, same_lengths=True)


def test_evict_flags_bad_sequences_only():
    rng = np.random.default_rng(6)
    lengths = [100, 100, 100, 100, 100]
    c = make_cache(rng, lengths, 2, 64, 64, 16, track=True)
    tokens_in_order(c, lengths)
    c.page_table[0, 6] = -3
    c.page_table[1, 0] = c.num_pages
    before = [a.clone() for a in c.arrays() + [c.weights, c.tokens]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    new = fg.fg_paged_kv_evict(c, i32([100, 100, c.max_pages * 16 + 1, -2, 16]), i32(lengths), 50, 10)
    flagged()
    assert new.tolist() == [100, 100, c.max_pages * 16 + 1, -2, 16]
    new = fg.fg_paged_kv_evict(c, i32([-1, -1, 100, -1, -1]), i32(lengths), 100, 10, max_len=99)
    flagged()
    assert new.tolist() == [-1, -1, 100, -1, -1]
    for a, b in zip(c.arrays() + [c.weights, c.tokens], before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def evict_known(c, lengths, budget, gone, new_lengths=None):
    """Evicts from a one-head cache whose weights are 1 but at the slots gone[s] (all below the budget), which are as many as
    a sequence has above it, and checks what filled them; pages are the table's in order."""
    ps = c.page_size
    c.weights.fill_(1.0)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    at, fill = [], []
    for s, n in enumerate(lengths):
        if n <= budget:
            continue
        hole, mover = torch.tensor(sorted(gone[s]), device="cuda"), torch.arange(budget, n, device="cuda")
        assert len(hole) == n - budget
        t = c.page_table[s].long()
        at.append((t[hole // ps], 0, hole % ps))
        c.weights[at[-1]] = 0.0
        src = (t[mover // ps], 0, mover % ps)
        fill.append([a[src].clone() for a in c.arrays() + [c.weights, c.tokens]])
    sums = [a.view(-1)[::4097].clone() for a in c.arrays()]             # what stays, by sample
    new = fg.fg_paged_kv_evict(c, ln, ln, budget, 0, new_lengths=ln if new_lengths == "same" else None)
    fg.fg_sync_status()
    assert new.tolist() == [min(n, budget) for n in lengths]
    for x, want in zip(at, fill):
        for a, w in zip(c.arrays() + [c.weights, c.tokens], want):
            assert torch.equal(a[x], w)
    changed = sum(len(g) for g in gone)
    for a, b in zip(c.arrays(), sums):
        assert torch.count_nonzero(a.view(-1)[::4097] != b) <= changed


@pytest.mark.parametrize("lengths", ["same", "apart"])
@pytest.mark.parametrize("page_bits,pages,sizes,budget", [
    (25, 1, [3000, 100, 2600], 2500),                                   # a page of max_len slots, as a contiguous cache has
    (24, 2, [2**24 + 500, 2**24 - 700], 2**24 - 100)])                  # and lengths that end in a second one
def test_evict_largest_pages(page_bits, pages, sizes, budget, lengths):
    ps, S, D = 1 << page_bits, len(sizes), 64
    if torch.cuda.mem_get_info()[0] < 3 * S * pages * ps * 80:
        pytest.skip("not enough device memory")
    rng = np.random.default_rng(page_bits)
    order = torch.from_numpy(rng.permutation(S * pages).reshape(S, pages).astype(np.int32)).cuda()
    c = fg.PagedKVCache(S * pages, 1, D, ps, order, track=True)
    gen = torch.Generator("cuda").manual_seed(3)
    for a in c.arrays():
        a.copy_(torch.randint(0, 256, a.shape, dtype=torch.uint8, device="cuda", generator=gen))
    c.tokens.copy_(torch.randint(0, 1 << 30, c.tokens.shape, dtype=torch.int32, device="cuda", generator=gen))
    c.tokens.clamp_(max=budget - 1)                                     # (none counts as recent)
    gone = [rng.choice(budget, max(0, n - budget), replace=False).tolist() for n in sizes]
    evict_known(c, sizes, budget, gone, lengths)


def test_evict_more_moves_than_32_bits_of_vectors():
    """2^27 slots of 256 values move: 2^31 vectors of codes.  k and v share their pools (both get the same moves)."""
    n, D, ps = 1 << 28, 256, 1 << 20
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough device memory")
    pages = n // ps
    codes = torch.empty((pages, 1, ps, D // 2), dtype=torch.uint8, device="cuda")
    nums = torch.empty((pages, 1, ps, D // 128), dtype=torch.float16, device="cuda")
    tokens = torch.arange(n, dtype=torch.int32, device="cuda").view(pages, 1, ps)
    gen = torch.Generator("cuda").manual_seed(1)
    for p in range(pages):
        codes[p] = torch.randint(0, 256, codes[p].shape, dtype=torch.uint8, device="cuda", generator=gen)
        nums[p] = torch.randn(nums[p].shape, dtype=torch.float16, device="cuda", generator=gen)
    table = torch.from_numpy(np.random.default_rng(1).permutation(pages).reshape(1, -1).astype(np.int32)).cuda()
    low, high = table[0, :pages // 2].long(), table[0, pages // 2:].long()
    weights = torch.ones((pages, 1, ps), dtype=torch.float32, device="cuda")
    weights[low] = 0.0
    c = fg.PagedKVCache(pages, 1, D, ps, table, group=128, arrays=[codes, nums, nums] * 2, weights=weights, tokens=tokens)
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    new = fg.fg_paged_kv_evict(c, i32(n), i32(2**30), n // 2, 0)
    fg.fg_sync_status()
    assert new.tolist() == [n // 2]
    for a, b in zip(low.tolist(), high.tolist()):
        for pool in (codes, nums, weights, tokens):
            assert torch.equal(pool[a], pool[b])


def test_evict_workspace():
    """More slots than a CTA's shared memory holds: scratch is asked for, and refused without."""
    c = make_cache(np.random.default_rng(2), [100, 100], 1, 64, 64, 64, track=True)
    assert fg.fg_paged_kv_evict_workspace_bytes(c, 64) == 0
    wide = fg.PagedKVCache(c.num_pages, 1, 64, 64, torch.zeros((2, 4000), dtype=torch.int32, device="cuda"),
                           arrays=c.arrays(), weights=c.weights, tokens=c.tokens)
    n = torch.tensor([100, -1], dtype=torch.int32, device="cuda")
    assert fg.fg_paged_kv_evict_workspace_bytes(wide, 64) > 0
    with pytest.raises(fg.FgError, match="WORKSPACE"):
        fg.fg_paged_kv_evict(wide, n, n, 64, 0, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert fg.fg_paged_kv_evict_workspace_bytes(wide, 64, max_len=1000) == 0


# ------------------------------------------------------------------ together ----------


def test_pools_past_32_bits():
    """Pages whose bytes lie past 2^32 of their pool: the same bits as a small pool's."""
    rng = np.random.default_rng(77)
    H, D, ps, lengths = 2, 256, 256, [700, 3000]
    small = make_cache(rng, lengths, H, D, 64, ps, track=True)
    pages = (2**32 + 2**24) // (H * ps * (D // 2))                      # of codes alone
    if torch.cuda.mem_get_info()[0] < 3 * pages * H * ps * (D + 72):
        pytest.skip("not enough device memory")
    shift = pages - small.num_pages
    big = [torch.empty((pages,) + a.shape[1:], dtype=a.dtype, device="cuda") for a in small.arrays() + [small.weights, small.tokens]]
    for x, y in zip(big, small.arrays() + [small.weights, small.tokens]):
        x[shift:] = y
    t = small.page_table
    table = torch.where((t >= 0) & (t < small.num_pages), t + shift, t)
    c = fg.PagedKVCache(pages, H, D, ps, table, arrays=big[:6], weights=big[6], tokens=big[7])
    q = queries(rng, 2, 3 * H, D)
    kv = queries(rng, 2, H, D, 16.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = []
    for k in (small, c):
        o = fg.fg_paged_attention(k, q, i32([n - 1 for n in lengths]), accumulate=True)
        fg.fg_paged_kv_append(k, kv, kv, i32([n - 1 for n in lengths]))
        new = fg.fg_paged_kv_evict(k, i32(lengths), i32(lengths), 512, 100)
        fg.fg_sync_status()
        got.append((o, new, [a[-small.num_pages:].clone() for a in k.arrays() + [k.weights, k.tokens]]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for x, y in zip(got[0][2], got[1][2]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("R,rows,limit", [(1, 1, 300), (1, 1, 6000), (3, 2, 300), (3, 2, 6000)])
def test_first_call_captured_and_many_sequences(R, rows, limit):
    """Many ragged sequences, most of them short or out, captured at once; the plan's bound far above the lengths."""
    rng = np.random.default_rng(limit + R)
    lengths = [int(x) for x in rng.integers(0, 60, 150)] + [290]
    pos = [n - rows if n >= rows else -1 for n in lengths]
    c = make_cache(rng, lengths, 1, 64, 64, 16, track=True)
    q = queries(rng, len(lengths) * rows, R, 64)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    w0 = c.weights.clone()
    ws = torch.empty(fg.fg_paged_attention_workspace_bytes(c, R, len(lengths) * rows, rows, limit, True), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fg.fg_paged_attention(c, q, p, rows_per_seq=rows, max_len=limit, accumulate=True, out=out, workspace=ws)
    g.replay()
    fg.fg_sync_status()
    w1 = c.weights.clone()
    c.weights.copy_(w0)
    assert torch.equal(out, check_attention(c, q, pos, rows, max_len=limit, accumulate=True))
    assert torch.equal(c.weights, w1)


def step(c, qkv, H, R, D, pos, first, out, ws, stream=None):
    hq = H * R * D
    fg.fg_paged_kv_append(c, qkv[:, hq:hq + H * D], qkv[:, hq + H * D:], pos, first_tokens=first, stream=stream)
    fg.fg_paged_attention(c, qkv[:, :hq], pos, accumulate=True, out=out, workspace=ws, stream=stream)


def test_generation_at_a_budget():
    """Prompts into pages, then decode steps; whenever a sequence has filled a page beyond the budget its heads evict
    back to it and it goes on.  Every step's attention and weights are checked over the cache as it stands, every
    eviction against its rule, and no kept token's codes ever change."""
    rng = np.random.default_rng(12)
    S, H, R, D, G, ps, budget, recent = 3, 2, 2, 128, 64, 16, 64, 24
    width = budget // ps + 2
    table = torch.from_numpy(rng.permutation(S * width + 2)[:S * width].reshape(S, width).astype(np.int32)).cuda()
    c = fg.PagedKVCache(S * width + 2, H, D, ps, table, group=G, track=True)
    prompts, P = [70, 9, 80], 80
    data = {}                                                           # token -> (k, v) rows of a sequence
    rows = lambda n: (torch.from_numpy(rng.normal(0, 1, (n, H * D)).astype(np.float16)).cuda() for _ in range(2))
    k, v = rows(S * P)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    fg.fg_paged_kv_append(c, k, v, i32([0] * S), rows_per_seq=P, row_counts=i32(prompts))
    for s in range(S):
        for i in range(prompts[s]):
            data[s, i] = (k[s * P + i], v[s * P + i])
    lengths, seen = list(prompts), list(prompts)
    evictions = 0
    for it in range(40):
        if max(lengths) >= budget + ps:
            check_evict(c, lengths, seen, budget, recent, max_len=width * ps)
            lengths = [min(n, budget) for n in lengths]
            evictions += 1
        k, v = rows(S)
        fg.fg_paged_kv_append(c, k, v, i32(lengths), first_tokens=i32(seen))
        for s in range(S):
            data[s, seen[s]] = (k[s], v[s])
        lengths, seen = [n + 1 for n in lengths], [n + 1 for n in seen]
        check_attention(c, queries(rng, S, H * R, D), [n - 1 for n in lengths], max_len=width * ps, accumulate=True)
    assert evictions >= 2
    for s in range(S):
        tok = dense(c, c.tokens, s, lengths[s])
        codes = dense(c, c.v_codes, s, lengths[s])
        for h in range(H):
            assert len(set(tok[h])) == lengths[s] and set(range(seen[s] - recent, seen[s])) <= set(tok[h])
            for i in range(lengths[s]):
                r = oracle.quantize(data[s, int(tok[h, i])][1].cpu().numpy().reshape(H, D), group=G)
                assert np.array_equal(codes[h, i], r.codes[h])


def test_prefilled_contiguous_cache_goes_on_in_paged_calls():
    h, H, F, S, P = 256, 4, 512, 3, 20
    D = h // H
    cfg = fg.LayerConfig(h, H, F)
    lw = fg.LayerWeights.from_fp16(cfg, si.layer_weights_f16(0, h, F, std=0.05, bias_std=0.05, ln_random=True))
    cache = fg.KVCache(S, H, D, 64)
    x = torch.from_numpy(si.hidden_block(0, si.STREAM["prompt"], S, P, h)).cuda()
    fg.fg_layer_prefill(cfg, lw, cache, x, torch.zeros(S, dtype=torch.int32, device="cuda"))
    c = fg.PagedKVCache.from_cache(cache, track=True)
    rng = np.random.default_rng(2)
    check_attention(c, queries(rng, S, H, D), [P - 1] * S, accumulate=True)
    tokens_in_order(c, [P] * S)
    check_evict(c, [P] * S, [P] * S, 16, 4)


def test_prefilled_slots_carry_their_own_numbers():
    """A prefilled cache that goes on as a tracked one: its prompt's last tokens are the recent ones."""
    S, H, D, L, P, budget, recent = 2, 3, 64, 64, 40, 24, 16
    cache = fg.KVCache(S, H, D, L)
    k = torch.from_numpy(si.normal_f16(1, 22, (S * P, H * D), 1.0)).cuda()
    v = torch.from_numpy(si.normal_f16(1, 23, (S * P, H * D), 1.0)).cuda()
    fg.fg_kv_append(cache, k, v, torch.zeros(S, dtype=torch.int32, device="cuda"), rows_per_seq=P)
    c = fg.PagedKVCache.from_cache(cache, track=True)
    c.weights[:, :, :recent] = 1.0                                      # the oldest have all the weight
    check_evict(c, [P] * S, [P] * S, budget, recent)
    kept = c.tokens[:, :, :budget].cpu().numpy()
    want = list(range(budget - recent)) + list(range(P - recent, P))
    assert all(sorted(kept[s, h]) == want for s in range(S) for h in range(H))
    given = torch.full_like(c.tokens, 7)                                # the caller's own pool stays as it is
    assert fg.PagedKVCache.from_cache(cache, tokens=given, track=True).tokens is given and (given == 7).all()
    assert fg.PagedKVCache.from_cache(cache).tokens is None


def test_decode_layer_over_pages():
    """A decode layer put together from the public calls over shuffled pages, against fg_layer_decode over the contiguous
    cache: the same bits in the cache, the layer's output within 1e-2 of its change (what the layer's own tests allow)."""
    h, H, F, S, P, ps, L = 256, 4, 512, 3, 20, 16, 64
    D, qs = h // H, (h // H)**-0.5
    cfg = fg.LayerConfig(h, H, F)
    lw = fg.LayerWeights.from_fp16(cfg, si.layer_weights_f16(0, h, F, std=0.05, bias_std=0.05, ln_random=True))
    flat = fg.KVCache(S, H, D, L)
    x = torch.from_numpy(si.hidden_block(0, si.STREAM["prompt"], S, P, h)).cuda()
    fg.fg_layer_prefill(cfg, lw, flat, x, torch.zeros(S, dtype=torch.int32, device="cuda"))
    table = torch.from_numpy(np.random.default_rng(1).permutation(S * (L // ps)).reshape(S, -1).astype(np.int32)).cuda()
    paged = fg.PagedKVCache(S * (L // ps), H, D, ps, table, track=True)
    at = table.long()
    pages = lambda a: a.view(S, H, L // ps, ps, -1).transpose(1, 2)
    for a, b in zip(flat.arrays(), paged.arrays()):
        b[at] = pages(a)
    m, v = lw.matrix, lw.vector
    for step in range(3):
        x = torch.from_numpy(si.decode_inputs(0, step, S, h)).cuda()
        pos = torch.full((S,), P + step, dtype=torch.int32, device="cuda")
        want = fg.fg_layer_decode(cfg, lw, flat, x, pos)
        a = fg.fg_layernorm(x, v("ln1_g"), v("ln1_b"))
        qkv = fg.fg_linear_w4a16(a, m("wqkv"), bias=v("bqkv"), qscale_cols=h, qscale=qs)
        fg.fg_paged_kv_append(paged, qkv[:, h:2 * h], qkv[:, 2 * h:], pos)
        o = fg.fg_paged_attention(paged, qkv[:, :h], pos, max_len=L, accumulate=True)
        h1 = fg.fg_linear_w4a16(o, m("wo"), bias=v("bo"), residual=x)
        f = fg.fg_linear_w4a16(fg.fg_layernorm(h1, v("ln2_g"), v("ln2_b")), m("w1"), bias=v("b1"), relu=True)
        y = fg.fg_linear_w4a16(f, m("w2"), bias=v("b2"), residual=h1)
        fg.fg_sync_status()
        for p, q in zip(flat.arrays(), paged.arrays()):
            assert torch.equal(pages(p)[:, :2], q[at][:, :2])
        change = (want.double() - x.double()).abs().max()
        assert (y.double() - want.double()).abs().max() <= 1e-2 * change
    # a head's three rows of probabilities: sums of 1
    total = paged.weights[at].sum((1, 3)).double()
    assert (total - 3.0).abs().max() <= 3 * 64 * 2.0**-23


def test_side_stream_and_graph_replay():
    """One step captured once and replayed, two graphs that share a workspace, and calls on a stream of their own."""
    rng = np.random.default_rng(21)
    S, H, R, D, ps, L0 = 3, 2, 4, 128, 64, 3000
    mk = lambda: make_cache(np.random.default_rng(5), [L0 + 8] * S, H, D, 64, ps, track=True)
    a, b = mk(), mk()
    xs = [queries(rng, S, H * R + 2 * H, D, 3.0) for _ in range(4)]
    need = fg.fg_paged_attention_workspace_bytes(a, H * R, S, 1, None, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out_a = torch.empty((S, H * R * D), dtype=torch.float16, device="cuda")
    pos_a = torch.full((S,), L0, dtype=torch.int32, device="cuda")
    x = torch.empty_like(xs[0])
    side = torch.cuda.Stream()
    x.copy_(xs[0])
    torch.cuda.synchronize()
    want = []
    for i, q in enumerate(xs):                                          # eager, on a side stream
        pos = torch.full((S,), L0 + i, dtype=torch.int32, device="cuda")
        out = torch.empty_like(out_a)
        torch.cuda.synchronize()
        step(b, q, H, R, D, pos, None, out, None, stream=side)
        side.synchronize()
        want.append((out, b.weights.clone()))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(a, x, H, R, D, pos_a, None, out_a, ws)
        graphs.append(g)
    ws.fill_(0xFF)                                                      # nothing in the workspace is relied on
    for i, q in enumerate(xs):
        x.copy_(q)
        pos_a.fill_(L0 + i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out_a, want[i][0]) and torch.equal(a.weights, want[i][1])
    fg.fg_sync_status()


def test_two_calls_at_once():
    """Two caches on two streams, a workspace each: the bits of the calls one after the other."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    lengths = [[6000, 50, 1200], [3000, 3001, 2]]
    caches, alone = ([make_cache(np.random.default_rng(i), n, 2, 128, 64, 32, track=True) for i, n in enumerate(lengths)]
                     for _ in range(2))
    qs = [queries(np.random.default_rng(9 + i), 3, 4, 128) for i in range(2)]
    pos = [torch.tensor([x - 1 for x in n], dtype=torch.int32, device="cuda") for n in lengths]
    ln = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in lengths]
    want = []
    for c, q, p, n in zip(alone, qs, pos, ln):
        want.append([fg.fg_paged_attention(c, q, p, accumulate=True) for _ in range(4)] + [fg.fg_paged_kv_evict(c, n, n, 100, 10)])
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(fg.fg_paged_attention(caches[i], qs[i], pos[i], accumulate=True, stream=streams[i]))
    for i in range(2):
        got[i].append(fg.fg_paged_kv_evict(caches[i], ln[i], ln[i], 100, 10, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))
        for x, y in zip(caches[i].arrays() + [caches[i].weights, caches[i].tokens], alone[i].arrays() + [alone[i].weights, alone[i].tokens]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    fg.fg_sync_status()


def test_evict_in_a_graph():
    rng = np.random.default_rng(31)
    lengths = [400, 90, 399]
    mk = lambda: make_cache(np.random.default_rng(7), lengths, 2, 64, 64, 16, track=True)
    a, b = mk(), mk()
    for c in (a, b):
        tokens_in_order(c, lengths)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    new = torch.empty_like(ln)
    need = fg.fg_paged_kv_evict_workspace_bytes(a, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fg.fg_paged_kv_evict(a, ln, ln, 128, 32, new_lengths=new, workspace=ws)
    ws.fill_(0xFF)
    g.replay()
    fg.fg_paged_kv_evict(b, ln, ln, 128, 32)
    fg.fg_sync_status()
    assert new.tolist() == [128, 90, 128]
    for x, y in zip(a.arrays() + [a.weights, a.tokens], b.arrays() + [b.weights, b.tokens]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    new2 = torch.empty_like(ln)
    fg.fg_paged_kv_evict(a, new, ln, 128, 32, new_lengths=new2)         # within the budget: nothing moves
    fg.fg_sync_status()
    for x, y in zip(a.arrays(), b.arrays()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_group_zero_is_the_default():
    table = torch.tensor([[0]], dtype=torch.int32, device="cuda")
    a, b = (fg.PagedKVCache(1, 2, 128, 16, table, group=g) for g in (0, 64))
    assert a.group == 64 and [x.shape for x in a.arrays()] == [x.shape for x in b.arrays()]
    x = torch.from_numpy(si.normal_f16(1, 22, (1, 256), 1.0)).cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c in (a, b):
        fg.fg_paged_kv_append(c, x, x, zero)
    fg.fg_sync_status()
    assert all(torch.equal(p, q) for p, q in zip(a.arrays(), b.arrays()))


def test_single_rows_of_any_stride():
    """One row has no next one: k and v, q and out may come from tensors of different and of odd widths."""
    H, R, D = 2, 2, 128
    a, b = (make_cache(np.random.default_rng(3), [40], H, D, 64, 16) for _ in range(2))
    pos = torch.tensor([39], dtype=torch.int32, device="cuda")
    q, x = queries(np.random.default_rng(4), 1, H * R, D), queries(np.random.default_rng(5), 1, H * D, 1)
    odd = lambda t, n: torch.cat([t, torch.zeros((1, n), dtype=t.dtype, device="cuda")], 1).repeat(2, 1)[:1, :t.shape[1]]
    fg.fg_paged_kv_append(a, x, x, pos)
    fg.fg_paged_kv_append(b, odd(x, 3), odd(x, 8), pos)
    want = fg.fg_paged_attention(a, q, pos)
    got = fg.fg_paged_attention(b, odd(q, 5), pos, out=odd(torch.zeros_like(q), 1))
    fg.fg_sync_status()
    assert all(torch.equal(m.view(torch.uint8), n.view(torch.uint8)) for m, n in zip(a.arrays(), b.arrays()))
    assert torch.equal(want, got)


def test_binding_refuses_what_it_can_see():
    rng = np.random.default_rng(1)
    c = make_cache(rng, [40, 40], 2, 128, 64, 16, track=True)
    q = queries(rng, 2, 2, 128)
    pos = torch.tensor([39, 39], dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :200]), dict(q=q.cpu()), dict(q=q[:, ::2]), dict(positions=pos.long()),
                dict(positions=pos[:1]), dict(positions=pos.cpu()), dict(out=q[:1]), dict(out=q[:, :128]),
                dict(row_counts=pos.float()), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fg.fg_paged_attention(**(dict(cache=c, q=q, positions=pos) | bad))
    with pytest.raises(fg.FgError, match="SHAPE"):
        fg.fg_paged_attention(c, q[:, :128], pos)                       # one query head for two key-value heads
    with pytest.raises(ValueError):
        fg.fg_paged_kv_append(c, q, q[:1], pos)
    with pytest.raises(ValueError):
        fg.fg_paged_kv_evict(c, pos, pos, 16, 4, weights_out=c.weights[:1])
    with pytest.raises(ValueError):
        fg.PagedKVCache(4, 2, 128, 16, c.page_table, arrays=c.arrays()[:5] + [c.v_scales[:1]])
    with pytest.raises(fg.FgError, match="SHAPE"):
        fg.PagedKVCache(4, 2, 128, 40, c.page_table)
    plain = fg.PagedKVCache(c.num_pages, 2, 128, 16, c.page_table, arrays=c.arrays())
    with pytest.raises(fg.FgError, match="INVALID"):
        fg.fg_paged_attention(plain, q, pos, accumulate=True)
    with pytest.raises(fg.FgError, match="INVALID"):
        fg.fg_paged_kv_evict(plain, pos, pos, 16, 4)
    none = fg.fg_paged_attention(c, q[:0], pos)                         # no rows: nothing to do
    assert none.shape == (0, 256)
    fg.fg_sync_status()
