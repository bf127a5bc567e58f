"""The key/value-cache operators on the GPU against their definitions in 64 bits
(cache_parity.py, which also derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

from cache_parity import Cache, kept_ref, mask_words, random_tree, tree_ref, weights_ref, within
from parity import guarded_empty, guards_intact

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF, F32 = torch.bfloat16, torch.float32


def status_ok():
    from exact_io_aware_57_b200 import attn

    torch.cuda.synchronize()
    assert attn.attn_device_status() == 0


def run_tree(cache, Hq, T, shape, dtype, row_lens=None, seed=0, scale=None, see=None, sigma=1.0):
    """Inputs, the call and its check against the definition; returns the outputs."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, Hkv, d = cache.B, cache.Hkv, cache.d
    q = (sigma * torch.randn(B, T, Hq, d, generator=g)).to(dtype)
    kn, vn = torch.randn(B, T, Hkv, d, generator=g).to(dtype), torch.randn(B, T, Hkv, d, generator=g).to(dtype)
    lens = [T] * B if row_lens is None else list(row_lens)
    for b, r in enumerate(lens):  # padding rows hold anything
        q[b, r:], kn[b, r:], vn[b, r:] = math.nan, math.nan, math.nan
    mask = None
    if shape == "none":
        see = None
    elif shape == "chain":
        see = [np.tril(np.ones((T, T), dtype=bool))] * B
    else:
        if see is None:
            see = [random_tree(T, rng) for _ in range(B)]
        mask = mask_words(np.stack(see) if shape == "tree" else see[0]).cuda()
        if shape == "shared":
            see = [see[0]] * B
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    k, v, cl, table = cache.gpu()
    ob, o = guarded_empty((B, T, Hq, d), dtype)
    lb, lse = guarded_empty((B, Hq, T), F32)
    attn.attn_fwd_tree(q.cuda(), k, v, cl, k_new=None if see is None else kn.cuda(),
                       v_new=None if see is None else vn.cuda(), block_table=table, tree_mask=mask,
                       row_lens=None if row_lens is None else torch.tensor(lens, dtype=torch.int32).cuda(),
                       scale=scale, out=o, lse=lse)
    status_ok()
    assert guards_intact(ob) and guards_intact(lb)
    o_r, l_r, tol_o, tol_l = tree_ref(q, cache.rows_k, cache.rows_v, kn, vn, see, lens, sc)
    within(lse, l_r, tol_l, "lse")
    within(o, o_r, tol_o, "o")
    return o, lse


TREE = [
    # lens, Hq, Hkv, d, page, T, shape, row_lens, dtype
    ([1000], 8, 2, 128, 16, 1, "chain", None, BF),
    ([300, 0, 1, 127, 128, 129], 8, 8, 128, 64, 1, "chain", None, BF),
    ([640, 77, 3000], 32, 4, 128, 16, 13, "tree", [13, 1, 7], BF),
    ([500, 260], 16, 2, 64, 32, 61, "tree", [60, 61], BF),
    ([257, 130], 6, 2, 128, 128, 100, "shared", None, BF),      # group of 3, rows over several tiles
    ([200], 4, 1, 64, 256, 150, "tree", None, BF),              # two tiles of new keys, three mask words
    ([90, 1], 2, 2, 128, 8, 130, "chain", [130, 129], BF),
    ([77, 33], 4, 4, 64, 0, 2, "none", None, BF),               # contiguous, odd capacity
    ([0, 5], 4, 2, 128, 0, 3, "none", [3, 0], BF),              # nothing to see at all
    ([400], 160, 1, 128, 24, 1, "chain", None, BF),             # a group of more than 128 heads
    ([2500], 5, 1, 64, 40, 5, "tree", None, BF),
    ([129, 64, 1], 8, 4, 128, 16, 6, "tree", [6, 2, 0], F32),
    ([700], 4, 4, 64, 0, 1, "chain", None, F32),
    ([60, 0], 6, 2, 128, 8, 70, "tree", None, F32),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,T,shape,row_lens,dtype", TREE)
def test_tree(lens, Hq, Hkv, d, page, T, shape, row_lens, dtype):
    run_tree(Cache(lens, Hkv, d, page, dtype), Hq, T, shape, dtype, row_lens)


@pytest.mark.parametrize("T,shape,d,page", [(1, "chain", 128, 16), (7, "tree", 64, 8), (40, "tree", 128, 0),
                                            (50, "chain", 64, 32), (64, "tree", 128, 128)])
def test_tree_at_every_place_of_a_tile(T, shape, d, page):
    """New keys behind 1 .. 128 slots of a tile: sharing it or in a tile of their own."""
    lens = [1, 7, 8, 9, 31, 33, 63, 64, 65, 77, 88, 95, 119, 120, 121, 127, 128]
    rng = np.random.default_rng(T)
    run_tree(Cache([n + 128 * int(k) for n, k in zip(lens, rng.integers(0, 3, len(lens)))], 1, d, page, BF), 2, T, shape,
             BF, [int(x) for x in rng.integers(0, T + 1, len(lens))])


@pytest.mark.parametrize("T,Hq,d", [(61, 8, 128), (130, 8, 64), (33, 16, 128), (200, 6, 64)])
@pytest.mark.parametrize("longest", [300, 2500])
def test_tree_row_tiles_side_by_side(T, Hq, d, longest):
    """Sequences that fill no, one, an odd or an even number of row tiles, so that runs
    begin and end at every place of a unit."""
    rng = np.random.default_rng(T + longest)
    lens = [int(x) for x in rng.integers(0, longest, 17)]
    run_tree(Cache(lens, 2, d, 32, BF), Hq, T, "tree", BF, [int(rng.choice([0, 1, T // 4, T // 2 + 1, T])) for _ in lens])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_rows_without_any_key(dtype):
    """A mask that leaves a row empty, over an empty and over a used cache."""
    see = [np.eye(5, dtype=bool) for _ in range(2)]
    see[0][2] = False
    see[1][3] = False
    o, lse = run_tree(Cache([0, 9], 2, 64, 8, dtype), 4, 5, "tree", dtype, see=see)
    assert torch.all(o[0, 2] == 0) and torch.all(lse[0, :, 2] == -math.inf)
    assert torch.all(torch.isfinite(lse[1, :, 3]))


@pytest.mark.parametrize("scale,sigma", [(0.5, 2.0), (-0.2, 1.0), (0.0, 1.0)])
def test_tree_scales(scale, sigma):
    run_tree(Cache([333, 1200], 2, 128, 64, BF), 8, 9, "tree", BF, scale=scale, sigma=sigma)


@pytest.mark.parametrize("T,Hq", [(1, 4), (3, 8), (40, 8)])
def test_tree_scores_that_rise_and_fall(T, Hq):
    """Scores hundreds apart, larger from tile to tile in one sequence and smaller in the
    other: references are raised on the way, and first ones stay the largest."""
    cache = Cache([900, 900], 2, 128, 16, BF)
    for b, ramp in enumerate((torch.linspace(0, 60, 900), torch.linspace(60, 0, 900))):
        cache.rows_k[b] = (cache.rows_k[b].float() * ramp[:, None, None]).to(BF)
        for i in range(900):
            cache.k[cache.at(b, i)] = cache.rows_k[b][i]
    run_tree(cache, Hq, T, "chain", BF)


def test_tree_infinite_stale_rows():
    run_tree(Cache([100, 250], 2, 128, 32, BF, stale=math.inf), 8, 4, "chain", BF)


@pytest.mark.parametrize("B,Hkv", [(70, 3), (1, 1), (2, 40)])
def test_tree_many_and_few_units(B, Hkv):
    """Sequences of very different lengths shared out over the SMs."""
    rng = np.random.default_rng(B)
    run_tree(Cache([int(x) for x in rng.integers(0, 900, B)], Hkv, 64, 16, BF), 2 * Hkv, 3, "tree", BF)


@pytest.mark.parametrize("T,Hq", [(1, 2), (5, 16)])
def test_tree_more_sequences_than_threads(T, Hq):
    rng = np.random.default_rng(9)
    run_tree(Cache([int(x) for x in rng.integers(0, 40, 700)], 1, 64, 8, BF), Hq, T, "chain", BF,
             [int(x) for x in rng.integers(0, T + 1, 700)])


def test_tree_long_context():
    run_tree(Cache([40000], 1, 128, 256, BF), 4, 2, "chain", BF)


def test_tree_equals_attention_over_dense_keys():
    """One chunk of a prompt over its cached beginning equals the causal forward's rows."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(3)
    n, T = 300, 40
    q, k, v = (torch.randn(1, n, h, 128, generator=g).bfloat16().cuda() for h in (8, 2, 2))
    o, lse = attn.attn_fwd(q, k, v, causal=True)
    lens = torch.tensor([n - T], dtype=torch.int32).cuda()
    o2, lse2 = attn.attn_fwd_tree(q[:, -T:].contiguous(), k, v, lens, k_new=k[:, -T:].contiguous(),
                                  v_new=v[:, -T:].contiguous())
    status_ok()
    assert float((o[:, -T:].float() - o2.float()).abs().max()) <= 2 * 2.0 ** -8 * float(v.float().abs().max())
    assert float((lse[:, :, -T:] - lse2).abs().max()) <= 1e-4


WEIGHTS = [
    # lens, Hq, Hkv, d, page, T, accepted (None: all rows), extra cap, in place, dtype
    ([700], 8, 2, 128, 16, 1, None, 0, True, BF),
    ([300, 1, 128, 129], 4, 4, 64, 64, 1, None, 70, False, BF),
    ([500, 300], 32, 4, 128, 32, 61, [5, 1], 3, False, BF),
    ([200, 200], 6, 2, 128, 0, 200, None, 0, False, BF),       # prompts of their own keys
    ([400], 4, 1, 64, 0, 400, None, 9, True, BF),
    ([65, 0, 3], 4, 2, 128, 24, 9, [9, 0, 3], 20, False, BF),
    ([4], 160, 1, 128, 0, 4, None, 0, False, BF),
    ([3, 40], 4, 2, 64, 8, 8, [8, 8], 1, False, BF),           # more rows than slots: the first see nothing
    ([5 + i % 31 for i in range(700)], 2, 1, 64, 8, 1, None, 2, False, BF),   # more sequences than threads
    ([1500], 24, 2, 128, 0, 1500, None, 0, False, BF),         # 12 heads: row tiles of 120 rows
    ([300], 2, 1, 128, 0, 300, None, 0, False, F32),
    ([129, 64], 8, 4, 64, 16, 6, [6, 2], 5, True, F32),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,T,accepted,extra,inplace,dtype", WEIGHTS)
def test_weights(lens, Hq, Hkv, d, page, T, accepted, extra, inplace, dtype):
    from exact_io_aware_57_b200 import attn

    g, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)
    cache, B = Cache(lens, Hkv, d, page, dtype), len(lens)
    q = torch.randn(B, T, Hq, d, generator=g).to(dtype)
    counts = [T] * B if accepted is None else accepted
    rows = [list(range(T)) if accepted is None else sorted(rng.choice(T, c, replace=False).tolist()) for c in counts]
    scale = 1.0 / math.sqrt(d)
    lse = torch.full((B, Hq, T), math.nan)
    for b in range(B):
        for i, t in enumerate(rows[b]):
            last = lens[b] - counts[b] + i
            for h in range(Hq):
                kh = cache.rows_k[b][:max(last + 1, 0), h // (Hq // Hkv)].double()
                lse[b, h, t] = float(torch.logsumexp(kh @ q[b, t, h].double() * scale, 0)) if last >= 0 else -math.inf
    cap = max(lens) + extra
    w = torch.rand(B, Hkv, cap, generator=g)
    k, _, cl, table = cache.gpu()
    ob, out = guarded_empty((B, Hkv, cap), F32)
    wd = w.cuda()
    if inplace:
        out.copy_(wd)
        wd = out
    lists = {}
    if accepted is not None:  # entries behind the count name nothing
        width = max(max(counts), 1)
        lists = dict(rows=torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32).cuda(),
                     row_lens=torch.tensor(counts, dtype=torch.int32).cuda())
    got = attn.attn_cache_weights(q.cuda(), lse.cuda(), k, cl, wd, block_table=table, out=out, **lists)
    status_ok()
    assert got is out and guards_intact(ob)
    ref, tol = weights_ref(q, lse, cache.rows_k, w, rows, counts, scale)
    within(out, ref, tol, "weights")


@pytest.mark.parametrize("d,Hkv,group", [(64, 2, 4), (128, 1, 8), (64, 4, 5)])
@pytest.mark.parametrize("lens,counts", [
    # chunks at the ends of sequences: units of many and of one or two steps in one run
    ([8701, 3695, 4337, 328, 1187, 4313, 6386, 2628, 4324], [1376, 318, 562, 58, 764, 516, 432, 672, 1270]),
    ([700, 0, 129, 1300, 64, 700, 257], [700, 0, 129, 65, 64, 1, 130]),
    ([2049], [2049]),
])
def test_weights_of_chunks(lens, counts, d, Hkv, group):
    """Several row tiles per head, units shared by CTAs and warpgroups; the reference in
    64 bits on the GPU, its bound that of weights_ref."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(9)
    B, n, scale = len(lens), max(counts), 1.0 / math.sqrt(d)
    cache = Cache(lens, Hkv, d, 128, BF)
    k, _, cl, table = cache.gpu()
    q = torch.randn(B, n, Hkv * group, d, generator=g).to(BF).cuda()
    ref = torch.rand(B, Hkv, max(lens), generator=g).double().cuda()
    tol = 2.0 ** -22 * ref
    w, lse = ref.float(), torch.full((B, Hkv * group, n), -math.inf, device="cuda")
    ref = w.double()
    for b, (m, c) in enumerate(zip(lens, counts)):
        rows = cache.rows_k[b].double().cuda()
        hide = torch.arange(m, device="cuda")[None, :] > (m - c + torch.arange(c, device="cuda"))[:, None]
        for h in range(Hkv * group if c else 0):
            kh, qh = rows[:, h // group], q[b, :c, h].double()
            s = (qh @ kh.T * scale).masked_fill(hide, -math.inf)
            lse[b, h, :c] = torch.logsumexp(s, 1).float()
            p = torch.exp(s - lse[b, h, :c].double()[:, None])
            e = (d + 2) * 2.0 ** -24 * scale * (qh.abs() @ kh.abs().T) + 1e-5
            ref[b, h // group, :m] += p.sum(0)
            tol[b, h // group, :m] += (p * (e + 2.0 ** -22)).sum(0)
    for _ in range(3):  # the order in which warpgroups finish varies
        out = attn.attn_cache_weights(q, lse, k, cl, w, block_table=table, out=torch.empty_like(w),
                                      row_lens=torch.tensor(counts, dtype=torch.int32).cuda())
        status_ok()
        within(out, ref.cpu(), tol.cpu(), "weights")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_of_a_prompt_sum_to_its_rows(dtype):
    """From zeros (weights None): every row hands out one unit per head."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(8)
    n, Hq, Hkv = 513, 8, 2
    q, k, v = (torch.randn(2, n, h, 128, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    _, lse = attn.attn_fwd(q, k, v, causal=True)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    w = attn.attn_cache_weights(q, lse, k, lens, None)
    status_ok()
    assert w.shape == (2, Hkv, n)
    # each of n * group unit sums is off by at most 1e-4 relative (see cache_parity)
    assert float((w.double().sum(-1) / (n * Hq // Hkv) - 1).abs().max()) <= 1e-4


APPEND = [
    # lens, Hkv, d, page, T, accepted, dtype
    ([0, 5, 16, 31], 2, 64, 16, 1, None, BF),
    ([100, 7], 3, 128, 32, 61, [5, 1], BF),
    ([3, 0], 1, 128, 0, 300, None, F32),
    ([60], 8, 64, 8, 9, [0], F32),
]


@pytest.mark.parametrize("lens,Hkv,d,page,T,accepted,dtype", APPEND)
def test_append(lens, Hkv, d, page, T, accepted, dtype):
    from exact_io_aware_57_b200 import attn

    g, rng = torch.Generator().manual_seed(2), np.random.default_rng(2)
    B = len(lens)
    counts = [T] * B if accepted is None else accepted
    rows = [list(range(T)) if accepted is None else sorted(rng.choice(T, c, replace=False).tolist()) for c in counts]
    cache = Cache(lens, Hkv, d, page, dtype, room=T, stale=7.0)
    kn, vn = torch.randn(B, T, Hkv, d, generator=g).to(dtype), torch.randn(B, T, Hkv, d, generator=g).to(dtype)
    k, v, cl, table = cache.gpu()
    lists = {}
    if accepted is not None:
        width = max(max(counts), 1) + 1
        lists = dict(rows=torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32).cuda(),
                     row_lens=torch.tensor(counts, dtype=torch.int32).cuda())
    new = attn.attn_cache_append(kn.cuda(), vn.cuda(), k, v, cl, block_table=table, **lists)
    status_ok()
    for b in range(B):
        for i, t in enumerate(rows[b]):
            cache.k[cache.at(b, lens[b] + i)] = kn[b, t]
            cache.v[cache.at(b, lens[b] + i)] = vn[b, t]
    assert torch.equal(k.cpu(), cache.k) and torch.equal(v.cpu(), cache.v)
    assert new.tolist() == [n + c for n, c in zip(lens, counts)] and cl.tolist() == lens


EVICT = [
    # lens, Hkv, d, page, page_out, keep, recent, dtype
    ([1000, 37, 0, 100, 101], 2, 64, 16, 32, 100, 10, BF),
    ([5000], 3, 128, 0, 64, 1025, 0, BF),
    ([300, 70], 1, 128, 64, 0, 64, 64, F32),     # only the recent ones stay
    ([33, 34], 8, 64, 8, 8, 33, 1, F32),
    ([20000], 1, 64, 256, 256, 1, 0, BF),
]
# long ones: a share of the weights for each CTA, and shares beyond shared memory
EVICT_LONG = [([70000], 2, 64, 0, 0, 30000, 5, BF), ([120000], 1, 64, 128, 256, 50000, 0, BF)]


@pytest.mark.parametrize("lens,Hkv,d,page,page_out,keep,recent,dtype,values",
                         [(*c, v) for c in EVICT for v in ("random", "ties", "equal", "special")] +
                         [(*c, v) for c in EVICT_LONG for v in ("random", "ties")])
def test_evict(lens, Hkv, d, page, page_out, keep, recent, dtype, values):
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(4)
    B, cap = len(lens), max(lens) + 3
    cache = Cache(lens, Hkv, d, page, dtype, stale=7.0)
    dst = Cache([min(n, keep) for n in lens], Hkv, d, page_out, dtype, stale=9.0, seed=1)
    dst.k.fill_(9.0)
    dst.v.fill_(9.0)
    w = torch.rand(B, Hkv, cap, generator=g)
    if values == "ties":
        w = (w * 8).floor() / 8
    elif values == "equal":
        w.fill_(0.25)
    elif values == "special":
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-40, -1e-40, 3e38])
        w = odd[torch.randint(0, len(odd), w.shape, generator=g)]
    k, v, cl, table = cache.gpu()
    ko, vo, _, tout = dst.gpu()
    wb, w_out = guarded_empty((B, Hkv, cap), F32)
    w_out, kept, new = attn.attn_cache_evict(k, v, w.cuda(), cl, keep, ko, vo, recent=recent, block_table=table,
                                             out_table=tout, weights_out=w_out)
    status_ok()
    assert guards_intact(wb) and new.tolist() == [min(n, keep) for n in lens]
    kept, w_out = kept.cpu(), w_out.cpu()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            idx = kept_ref(w[b, h], n, keep, recent)
            assert kept[b, h].tolist() == idx + [-1] * (keep - len(idx))
            want = torch.zeros(cap)
            want[:len(idx)] = w[b, h, idx]
            assert torch.equal(w_out[b, h].nan_to_num(123.0), want.nan_to_num(123.0))
            for i, j in enumerate(idx):
                p, r = dst.at(b, i)
                dst.k[p, r, h], dst.v[p, r, h] = cache.rows_k[b][j, h], cache.rows_v[b][j, h]
    assert torch.equal(ko.cpu(), dst.k) and torch.equal(vo.cpu(), dst.v)


def test_a_run_together():
    """Prompt -> cache -> weights -> eviction -> verified trees, each step on the last one's
    results, on a stream of its own, against the same run in 64 bits."""
    from exact_io_aware_57_b200 import attn

    g, rng = torch.Generator().manual_seed(11), np.random.default_rng(11)
    B, Hq, Hkv, d, n, keep, recent, T = 2, 8, 2, 128, 333, 96, 16, 9
    scale = 1.0 / math.sqrt(d)
    q, k, v = (torch.randn(B, n, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    pool = Cache([0, 0], Hkv, d, 16, BF, room=keep + 3 * T)
    lens = torch.full((B,), n, dtype=torch.int32).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
        kc, vc, _, table = pool.gpu()
        _, lse = attn.attn_fwd(qd, kd, vd, causal=True)
        w = attn.attn_cache_weights(qd, lse, kd, lens, None)
        w, kept, lens = attn.attn_cache_evict(kd, vd, w, lens, keep, kc, vc, recent=recent, out_table=table)
        steps, kept = [], kept.cpu()
        for _ in range(3):
            qn, kn, vn = (torch.randn(B, T, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
            see = [random_tree(T, rng) for _ in range(B)]
            path = [np.flatnonzero(see[b][T - 1]).tolist() for b in range(B)]
            rows = torch.tensor([p + [-1] * (T - len(p)) for p in path], dtype=torch.int32).cuda()
            cnt = torch.tensor([len(p) for p in path], dtype=torch.int32).cuda()
            o, lse = attn.attn_fwd_tree(qn.cuda(), kc, vc, lens, k_new=kn.cuda(), v_new=vn.cuda(), block_table=table,
                                        tree_mask=mask_words(np.stack(see)).cuda())
            lens = attn.attn_cache_append(kn.cuda(), vn.cuda(), kc, vc, lens, block_table=table, rows=rows,
                                          row_lens=cnt)
            w = attn.attn_cache_weights(qn.cuda(), lse, kc, lens, w, block_table=table, rows=rows, row_lens=cnt)
            steps.append((qn, kn, vn, see, path, o, lse))
    st.synchronize()
    assert attn.attn_device_status() == 0
    # the prompt's weights in 64 bits choose the same slots, up to near ties at the border
    full = torch.zeros(B, Hkv, n, dtype=torch.float64)
    hide = ~torch.tril(torch.ones(n, n, dtype=torch.bool))
    for b in range(B):
        for h in range(Hq):
            s = (q[b, :, h].double() @ k[b, :, h // 4].double().T * scale).masked_fill(hide, -math.inf)
            full[b, h // 4] += torch.softmax(s, 1).sum(0)
    keys, vals, want = [], [], torch.zeros(B, Hkv, w.shape[2], dtype=torch.float64)
    for b in range(B):
        for h in range(Hkv):
            old = full[b, h, :n - recent]
            stay = kept[b, h][:keep - recent].long()
            assert kept[b, h][keep - recent:].tolist() == list(range(n - recent, n))
            gone = torch.ones(n - recent, dtype=torch.bool)
            gone[stay] = False
            assert float(old[stay].min()) >= float(old[gone].max()) * (1 - 2e-4)
            want[b, h, :keep] = full[b, h, kept[b, h].long()]
        keys.append(torch.stack([k[b, kept[b, h].long(), h] for h in range(Hkv)], 1))
        vals.append(torch.stack([v[b, kept[b, h].long(), h] for h in range(Hkv)], 1))
    tol = 2e-4 * want
    for qn, kn, vn, see, path, o, lse in steps:
        o_r, l_r, tol_o, tol_l = tree_ref(qn, keys, vals, kn, vn, see, [T] * B, scale)
        within(o, o_r, tol_o, "o")
        within(lse, l_r, tol_l, "lse")
        for b in range(B):
            keys[b], vals[b] = torch.cat([keys[b], kn[b, path[b]]]), torch.cat([vals[b], vn[b, path[b]]])
        want, t = weights_ref(qn, l_r, keys, want, path, [len(p) for p in path], scale)
        tol = tol + t + 2e-4 * (want + 0)
    within(w, want, tol, "weights")
    assert lens.tolist() == [x.shape[0] for x in keys]


def test_step_captured_into_a_graph():
    """A captured decode step replays as the cache grows: lengths are read on the device."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 128, 16, 5
    cache = Cache([15, 130, 0], Hkv, d, page, BF, room=steps)
    k, v, lens, table = cache.gpu()
    q, kn, vn = (torch.zeros(B, 1, h, d, dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv))
    w = torch.zeros(B, Hkv, 160, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
    ws = torch.empty(attn.attn_fwd_tree_workspace_size(B, Hq, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    ww = torch.empty(attn.attn_cache_weights_workspace_size(B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    new = torch.empty_like(lens)

    def step():
        attn.attn_fwd_tree(q, k, v, lens, k_new=kn, v_new=vn, block_table=table, out=o, lse=lse, workspace=ws)
        attn.attn_cache_append(kn, vn, k, v, lens, block_table=table, new_lens=new)
        lens.copy_(new)
        attn.attn_cache_weights(q, lse, k, lens, w, block_table=table, workspace=ww)

    graph = torch.cuda.CUDAGraph()
    keep = lens.clone()
    with torch.cuda.graph(graph):
        step()
    assert torch.equal(lens, keep)  # nothing ran yet
    want = torch.zeros(B, Hkv, 160, dtype=torch.float64)
    tol = torch.zeros_like(want)
    keys, vals = list(cache.rows_k), list(cache.rows_v)
    for _ in range(steps):
        qn, k1, v1 = (torch.randn(B, 1, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        q.copy_(qn), kn.copy_(k1), vn.copy_(v1)
        graph.replay()
        status_ok()
        o_r, l_r, tol_o, tol_l = tree_ref(qn, keys, vals, k1, v1, [np.ones((1, 1), dtype=bool)] * B, [1] * B,
                                          1 / math.sqrt(d))
        within(o, o_r, tol_o, "o")
        within(lse, l_r, tol_l, "lse")
        keys = [torch.cat([a, k1[b]]) for b, a in enumerate(keys)]
        vals = [torch.cat([a, v1[b]]) for b, a in enumerate(vals)]
        want, t = weights_ref(qn, lse.cpu(), keys, want, [[0]] * B, [1] * B, 1 / math.sqrt(d))
        tol = tol + t
        within(w, want, tol, "weights")
    assert lens.tolist() == [a.shape[0] for a in keys]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_that_are_not_acceptable(dtype):
    """Bad lengths and counts are reported and leave the other sequences alone."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(1)
    cache = Cache([40, 40, 40], 2, 64, 16, dtype, room=8, stale=5.0)
    k, v, _, table = cache.gpu()
    q, kn, vn = (torch.randn(3, 2, h, 64, generator=g).to(dtype) for h in (4, 2, 2))
    qd, knd, vnd = q.cuda(), kn.cuda(), vn.cuda()
    o_r, l_r, tol_o, tol_l = tree_ref(q, cache.rows_k, cache.rows_v, kn, vn, [np.tril(np.ones((2, 2), dtype=bool))] * 3,
                                      [2, 2, 2], 0.125)
    for bad_lens, bad_rows in (([40, -1, 40], [2, 2, 2]), ([40, 10 ** 6, 40], [2, 2, 2]), ([40, 40, 40], [2, 3, 2]),
                               ([40, 40, 40], [2, -1, 2])):
        lens = torch.tensor(bad_lens, dtype=torch.int32).cuda()
        rl = torch.tensor(bad_rows, dtype=torch.int32).cuda()
        o, lse = attn.attn_fwd_tree(qd, k, v, lens, k_new=knd, v_new=vnd, block_table=table, row_lens=rl)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
        assert torch.all(o[1] == 0) and torch.all(lse[1] == -math.inf)
        for b in (0, 2):
            within(o[b], o_r[b], tol_o[b], "o")
            within(lse[b], l_r[b], tol_l[b], "lse")
        w = torch.full((3, 2, 64), 0.5, device="cuda")
        attn.attn_cache_weights(qd, lse, k, lens, w, block_table=table, row_lens=rl)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
        assert torch.all(w[1] == 0.5) and torch.all(w[0, :, :38] > 0.5)
        k2, v2 = k.clone(), v.clone()
        new = attn.attn_cache_append(knd, vnd, k2, v2, lens, block_table=table, row_lens=rl)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
        assert new.tolist() == [42, bad_lens[1], 42]
        for s in range(40, 48):
            assert torch.equal(k2[cache.at(1, s)], k[cache.at(1, s)])
        assert torch.equal(k2[cache.at(0, 41)].cpu(), kn[0, 1])
    # rows that do not exist, and a page outside the pool
    rows = torch.tensor([[0, 1], [0, 2], [1, 0]], dtype=torch.int32).cuda()
    lens = torch.tensor([40, 40, 40], dtype=torch.int32).cuda()
    k2, v2 = k.clone(), v.clone()
    attn.attn_cache_append(knd, vnd, k2, v2, lens, block_table=table, rows=rows)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
    assert torch.equal(k2[cache.at(2, 40)].cpu(), kn[2, 1])
    w = torch.zeros(3, 2, 64, device="cuda")
    attn.attn_cache_weights(qd, torch.zeros(3, 4, 2, device="cuda"), k, lens, w, block_table=table, rows=rows)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
    for page in (-1, 10 ** 6):
        t2 = table.clone()
        t2[1, 1] = page
        o, lse = attn.attn_fwd_tree(qd, k, v, lens, k_new=knd, v_new=vnd, block_table=t2)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
        for b in (0, 2):
            within(o[b], o_r[b], tol_o[b], "o")
        attn.attn_cache_weights(qd, lse, k, lens, w, block_table=t2)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_INVALID


def test_evict_that_does_not_fit():
    from exact_io_aware_57_b200 import attn

    cache = Cache([50, 20], 2, 64, 8, BF, stale=7.0)
    k, v, lens, table = cache.gpu()
    ko = torch.full((4, 8, 2, 64), 9.0, dtype=BF, device="cuda")
    vo = ko.clone()
    tout = torch.tensor([[0, 1, 2], [2, 3, 1]], dtype=torch.int32).cuda()[:, :3].contiguous()
    w = torch.rand(2, 2, 50).cuda()
    w_out, kept, new = attn.attn_cache_evict(k, v, w, lens, 30, ko, vo, block_table=table, out_table=tout)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
    assert new.tolist() == [50, 20] and torch.all(kept[0] == -1)
    assert kept[1, 0].tolist() == list(range(20)) + [-1] * 10
    assert torch.equal(ko[2, 3].cpu(), cache.rows_k[1][3]) and torch.all(ko[0] == 9.0)


def test_refusals_of_the_binding():
    """Tensors that are not as the call needs them, each named in the error."""
    from exact_io_aware_57_b200 import attn

    cache = Cache([40, 20], 2, 64, 16, BF, room=8)
    k, v, lens, table = cache.gpu()
    q = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    kn = torch.zeros(2, 3, 2, 64, dtype=BF, device="cuda")
    w = torch.zeros(2, 2, 64, device="cuda")
    lse = torch.zeros(2, 4, 3, device="cuda")
    i64 = lens.long()
    for match, call in [
        ("q must be contiguous", lambda: attn.attn_fwd_tree(q.transpose(1, 2).transpose(1, 2)[:, ::2], k, v, lens)),
        ("cache_lens must be torch.int32", lambda: attn.attn_fwd_tree(q, k, v, i64, block_table=table)),
        ("block_table must be torch.int32", lambda: attn.attn_fwd_tree(q, k, v, lens, block_table=table.long())),
        ("k_cache must be torch.bfloat16", lambda: attn.attn_fwd_tree(q, k.float(), v, lens, block_table=table)),
        ("v_cache must have shape", lambda: attn.attn_fwd_tree(q, k, v[:-1], lens, block_table=table)),
        ("k_new must have shape", lambda: attn.attn_fwd_tree(q, k, v, lens, k_new=kn[:, :2].contiguous(), v_new=kn)),
        ("k_cache must be \\[pages", lambda: attn.attn_fwd_tree(q[..., :32].contiguous(), k, v, lens)),
        ("tree_mask must be torch.int64", lambda: attn.attn_fwd_tree(q, k, v, lens, k_new=kn, v_new=kn, block_table=table,
                                                                    tree_mask=torch.zeros(3, 1, device="cuda"))),
        ("tree_mask must have shape", lambda: attn.attn_fwd_tree(q, k, v, lens, k_new=kn, v_new=kn, block_table=table,
                                                                 tree_mask=torch.zeros(3, 2, dtype=torch.int64,
                                                                                       device="cuda"))),
        ("row_lens is on cpu", lambda: attn.attn_fwd_tree(q, k, v, lens, block_table=table, row_lens=lens.cpu())),
        ("out must be torch.bfloat16", lambda: attn.attn_fwd_tree(q, k, v, lens, block_table=table, out=q.float())),
        ("error -3", lambda: attn.attn_fwd_tree(q, k, v, lens, block_table=table,
                                                workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))),
        ("unsupported dtype", lambda: attn.attn_fwd_tree(q.half(), k.half(), v.half(), lens, block_table=table)),
        ("error -1", lambda: attn.attn_fwd_tree(q[:, :, :3].contiguous(), k, v, lens, block_table=table)),
        ("lse must be torch.float32", lambda: attn.attn_cache_weights(q, lse.double(), k, lens, w, block_table=table)),
        ("weights must have shape", lambda: attn.attn_cache_weights(q, lse, k, lens, w[:, :1].contiguous(), out=w,
                                                                    block_table=table)),
        ("rows must have shape", lambda: attn.attn_cache_append(kn, kn, k, v, lens, block_table=table, rows=lens)),
        ("v_new must have shape", lambda: attn.attn_cache_append(kn, kn[:1], k, v, lens, block_table=table)),
        ("error -1", lambda: attn.attn_cache_append(kn, kn, k, v, lens, block_table=table, new_lens=lens)),
        ("error -1", lambda: attn.attn_cache_evict(k, v, w, lens, 4, k, v, block_table=table, out_table=table)),
        ("kept must have shape", lambda: attn.attn_cache_evict(k, v, w, lens, 4, k.clone(), v.clone(), block_table=table,
                                                               out_table=table, kept=torch.zeros(2, 2, 5,
                                                                                                 dtype=torch.int32,
                                                                                                 device="cuda"))),
    ]:
        with pytest.raises(attn.AttnError, match=match):
            call()
    status_ok()


def test_on_a_stream_of_the_callers():
    """stream=: the call runs there, and what it made lives until it has."""
    from exact_io_aware_57_b200 import attn

    cache = Cache([700, 900], 2, 128, 16, BF)
    k, v, lens, table = cache.gpu()
    q = torch.randn(2, 1, 8, 128, device="cuda").bfloat16()
    want, want_lse = attn.attn_fwd_tree(q, k, v, lens, block_table=table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [attn.attn_fwd_tree(q, k, v, lens, block_table=table, stream=side) for _ in range(5)]
    side.synchronize()
    for o, lse in got:  # the same work in the same order
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
