"""The key/value-cache calls where inputs are odd rather than wrong: rows that do not
count, values that are not finite or very large, the largest sizes, streams of the
caller's.  Definitions and tolerances are those of cache_parity.py."""
import math

import numpy as np
import pytest
import torch

from cache_parity import Cache, kept_ref, mask_words, random_tree, tree_ref, weights_ref, within
from parity import guarded_empty, guards_intact

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
BF, F32 = torch.bfloat16, torch.float32


def on_gpu(test):
    for mark in gpu:
        test = mark(test)
    return test


def status_ok():
    from exact_io_aware_57_b200 import attn

    torch.cuda.synchronize()
    assert attn.attn_device_status() == 0


# ------------------------------------------------- rows that do not count
def tree_bits(q, cache, row_lens=None):
    from exact_io_aware_57_b200 import attn

    k, v, lens, table = cache
    rl = None if row_lens is None else torch.tensor(row_lens, dtype=torch.int32).cuda()
    o, lse = attn.attn_fwd_tree(q, k, v, lens, block_table=table, row_lens=rl)
    status_ok()
    return o.view(torch.int16).cpu(), lse.view(torch.int32).cpu()


@on_gpu
@pytest.mark.parametrize("T,Hq", [(2, 8), (3, 10), (40, 8)])
def test_padding_rows_leave_the_others_bits(T, Hq):
    """Whatever finite values the rows t >= row_lens[b] hold."""
    g = torch.Generator().manual_seed(3)
    cache = Cache([700, 1300, 90], 2, 128, 16, BF).gpu()
    q, counts = torch.randn(3, T, Hq, 128, generator=g).to(BF).cuda(), [T - 1, 1, T]
    seen = []
    for fill in (0.0, 100.0, 1e30, -1e30):
        for b, r in enumerate(counts):
            q[b, r:] = fill * torch.sign(torch.randn(T - r, Hq, 128, generator=g)).cuda()
        seen.append(tree_bits(q, cache, counts))
    for o, lse in seen[1:]:
        assert torch.equal(o, seen[0][0]) and torch.equal(lse, seen[0][1])


@on_gpu
@pytest.mark.parametrize("d", [64, 128])
def test_results_do_not_depend_on_the_call_before(d):
    """A call of 16 rows per KV head leaves its rows in shared memory; one of fewer rows
    gives the same bits after any of them."""
    g = torch.Generator().manual_seed(4)
    cache = Cache([300 + 17 * i for i in range(40)], 2, d, 32, BF).gpu()
    q = torch.randn(40, 1, 8, d, generator=g).to(BF).cuda()
    before = torch.sign(torch.randn(40, 4, 8, d, generator=g)).to(BF).cuda()
    seen = []
    for fill in (0.0, 30.0, 1000.0):
        tree_bits(before * fill, cache)
        seen.append(tree_bits(q, cache))
    for o, lse in seen[1:]:
        assert torch.equal(o, seen[0][0]) and torch.equal(lse, seen[0][1])


# ------------------------------------------------- values that are not finite
def tree_call(q, rows, kn, vn, see):
    """A cache of the rows (lists of K, V per sequence), the call, O and LSE on the CPU."""
    from exact_io_aware_57_b200 import attn

    rows_k, rows_v = rows
    cache = Cache([x.shape[0] for x in rows_k], kn.shape[2], q.shape[3], 16, q.dtype)
    for b, x in enumerate(rows_k):
        for s in range(x.shape[0]):
            cache.k[cache.at(b, s)], cache.v[cache.at(b, s)] = x[s], rows_v[b][s]
    k, v, lens, table = cache.gpu()
    o, lse = attn.attn_fwd_tree(q.cuda(), k, v, lens, k_new=kn.cuda(), v_new=vn.cuda(), block_table=table,
                                tree_mask=mask_words(np.stack(see)).cuda())
    status_ok()
    return o.cpu().float(), lse.cpu()


def check_nan(got, ref, bad, lost=torch.isnan):
    """bad [B, T, Hq]: rows that are NaN (`lost`) throughout; the others within their bounds."""
    o, lse = got
    o_r, l_r, tol_o, tol_l = ref
    bl = bad.transpose(1, 2)
    assert torch.equal(lost(o), bad[..., None].expand_as(o))
    assert torch.equal(lost(lse), bl)
    within(torch.where(bad[..., None], 0.0, o), torch.where(bad[..., None], 0.0, o_r), tol_o.nan_to_num(1.0), "o")
    within(torch.where(bl, 0.0, lse), torch.where(bl, 0.0, l_r), tol_l.nan_to_num(1.0), "lse")


SIZES = [(3, 8, BF), (40, 8, BF), (70, 16, BF), (3, 8, F32), (20, 4, F32)]


def nan_case(T, Hq, dtype, lens=(900, 33, 130)):
    g, rng = torch.Generator().manual_seed(7), np.random.default_rng(7)
    B, Hkv, d = len(lens), 2, 64
    q = torch.randn(B, T, Hq, d, generator=g).to(dtype)
    kn, vn = (torch.randn(B, T, Hkv, d, generator=g).to(dtype) for _ in range(2))
    rows = [[torch.randn(n, Hkv, d, generator=g).to(dtype) for n in lens] for _ in range(2)]
    see = [random_tree(T, rng) for _ in range(B)]
    return q, rows, kn, vn, see, torch.zeros(B, T, Hq, dtype=torch.bool)


def ref_of(q, rows, kn, vn, see):
    B, T, _, d = q.shape
    return tree_ref(q, rows[0], rows[1], kn, vn, see, [T] * B, 1 / math.sqrt(d))


@on_gpu
@pytest.mark.parametrize("T,Hq,dtype", SIZES)
def test_nan_in_a_row_of_q(T, Hq, dtype):
    q, rows, kn, vn, see, bad = nan_case(T, Hq, dtype)
    ref = ref_of(q, rows, kn, vn, see)
    for b, t, h in ((0, 1, 2), (1, 0, 0), (2, T - 1, Hq - 1)):
        q[b, t, h, 5], bad[b, t, h] = math.nan, True
    check_nan(tree_call(q, rows, kn, vn, see), ref, bad)


@on_gpu
@pytest.mark.parametrize("T,Hq,dtype", SIZES)
def test_nan_in_cached_keys(T, Hq, dtype):
    """One slot, a whole tile's slots, all slots: every row that sees them is NaN."""
    q, rows, kn, vn, see, bad = nan_case(T, Hq, dtype)
    ref = ref_of(q, rows, kn, vn, see)
    rows[0][0][513, 0, 3] = math.nan
    rows[0][1][:, 1] = math.nan
    rows[0][2][0, 0, 0] = math.nan
    G = Hq // 2
    bad[0, :, :G] = bad[1, :, G:] = bad[2, :, :G] = True
    check_nan(tree_call(q, rows, kn, vn, see), ref, bad)


@on_gpu
@pytest.mark.parametrize("T,Hq,dtype", SIZES)
def test_nan_in_a_new_key(T, Hq, dtype):
    """Rows that do not see it are as ever."""
    q, rows, kn, vn, see, bad = nan_case(T, Hq, dtype, lens=(900, 0, 130))
    ref = ref_of(q, rows, kn, vn, see)
    for b in range(3):
        kn[b, 1, 1, 7] = math.nan
        bad[b, :, Hq // 2:] = torch.from_numpy(see[b][:, 1].copy())[:, None]
    assert bad.any() and not bad[:, :, Hq // 2:].all()
    check_nan(tree_call(q, rows, kn, vn, see), ref, bad)


@on_gpu
@pytest.mark.parametrize("T,Hq,dtype", SIZES)
def test_infinite_scores(T, Hq, dtype):
    """A key of one infinite component: score -inf weighs nothing, +inf leaves no answer."""
    q, rows, kn, vn, see, bad = nan_case(T, Hq, dtype)
    q[..., 9] = torch.where(q[..., 9] < 0, -0.5, 0.5).to(dtype)
    rows[0][0][700, 0, 9] = math.inf
    rows[0][1][2, 1, 9] = -math.inf
    G = Hq // 2
    bad[0, :, :G] = q[0, :, :G, 9] > 0
    bad[1, :, G:] = q[1, :, G:, 9] < 0
    # rows at -inf have the answer of a cache without that slot, the other heads any finite one
    whole = [[x.nan_to_num(posinf=0.0, neginf=0.0) for x in r] for r in rows]
    ref = ref_of(q, whole, kn, vn, see)
    for b, s, h0 in ((0, 700, 0), (1, 2, G)):
        less = [[torch.cat([x[:s], x[s + 1:]]) if i == b else x for i, x in enumerate(r)] for r in whole]
        for x, y in zip(ref, ref_of(q, less, kn, vn, see)):
            if x.shape[1] == T:
                x[b, :, h0:h0 + G] = y[b, :, h0:h0 + G]
            else:
                x[b, h0:h0 + G] = y[b, h0:h0 + G]
    check_nan(tree_call(q, rows, kn, vn, see), ref, bad, lambda x: ~torch.isfinite(x))


@on_gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_merge_keeps_nan(dtype):
    """A partial of NaN makes its row NaN; partials that saw nothing (whatever their O holds
    where all did) give zeros."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(5)
    o = torch.randn(3, 1, 4, 2, 64, generator=g)
    lse = torch.randn(3, 1, 2, 4, generator=g)
    want, want_lse = attn.attn_merge_partials(o.cuda(), lse.cuda(), out_dtype=dtype)
    lse[1, 0, 0, 1] = lse[:, 0, 1, 2] = lse[0, 0, 1, 0] = math.nan
    lse[1:, 0, 1, 0] = -math.inf
    lse[:, 0, 0, 3], o[:, 0, 3, 0] = -math.inf, math.nan
    got, got_lse = attn.attn_merge_partials(o.cuda(), lse.cuda(), out_dtype=dtype)
    status_ok()
    bad = torch.tensor([[False, True, False, False], [True, False, True, False]]).cuda()
    gone = torch.tensor([[False, False, False, True], [False] * 4]).cuda()
    assert torch.equal(torch.isnan(got_lse[0]), bad)
    assert torch.equal(torch.isnan(got[0]), bad.T[..., None].expand_as(got[0]))
    assert torch.all(got[0].transpose(0, 1)[gone] == 0) and torch.all(got_lse[0][gone] == -math.inf)
    keep = ~(bad | gone)
    assert torch.equal(got_lse[0][keep], want_lse[0][keep])
    assert torch.equal(got[0].transpose(0, 1)[keep], want[0].transpose(0, 1)[keep])


@on_gpu
@pytest.mark.parametrize("lens,T,Hq,Hkv,dtype", [([400, 250], 3, 4, 2, BF), ([700, 300], 200, 6, 2, BF), ([90], 9, 160, 1, BF),
                                                 ([400, 250], 3, 4, 2, F32), ([130, 200], 60, 4, 2, F32)])
def test_weights_of_rows_without_a_visible_key(lens, T, Hq, Hkv, dtype):
    """LSE = -inf: such a row adds nothing, whatever q holds there.  A NaN row or LSE makes
    the slots that see it NaN."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(6)
    cache, B = Cache(lens, Hkv, 64, 16, dtype), len(lens)
    k, _, cl, table = cache.gpu()
    q = torch.randn(B, T, Hq, 64, generator=g).to(dtype)
    lse = 6 + torch.rand(B, Hq, T, generator=g)
    w = torch.rand(B, Hkv, max(lens), generator=g)
    for b in range(B):
        for t, x in ((b, math.nan), (T - 1, math.inf)):
            q[b, t], lse[b, :, t] = x, -math.inf
    call = lambda: attn.attn_cache_weights(q.cuda(), lse.cuda(), k, cl, w.cuda(), block_table=table,
                                           out=torch.empty_like(w).cuda()).cpu()
    out = call()
    status_ok()
    ref, tol = weights_ref(q, lse, cache.rows_k, w, [list(range(T))] * B, [T] * B, 0.125)
    within(out, ref, tol, "weights")
    lse[0, Hq - 1, 1] = math.nan
    bad = call()
    status_ok()
    seen = torch.zeros_like(w, dtype=torch.bool)
    seen[0, Hkv - 1, :lens[0] - T + 2] = True
    assert torch.equal(torch.isnan(bad), seen) and torch.equal(bad[~seen], out[~seen])


# ------------------------------------------------- large values
@on_gpu
@pytest.mark.parametrize("T,Hq", [(1, 4), (4, 8), (40, 8)])
@pytest.mark.parametrize("rise", [6, 20, 40])
def test_large_values_after_a_low_first_score(T, Hq, rise):
    """|V| near 2^100 behind a first key whose scores are `rise` (log2 units) lower: the
    weights must not carry the sums out of fp32's range."""
    g = torch.Generator().manual_seed(12)
    n, d, Hkv = 600, 128, 2
    q = torch.full((1, T, Hq, d), 0.25).to(BF)
    rows_k = [0.02 * torch.randn(n, Hkv, d, generator=g)]
    # scores of 0 but the first: -rise ln 2
    rows_k[0][0] = -rise * math.log(2) * math.sqrt(d) / (0.25 * d)
    rows_k = [rows_k[0].to(BF)]
    rows_v = [(torch.randn(n, Hkv, d, generator=g) * 2.0 ** 100).to(BF)]
    kn, vn = torch.zeros(1, T, Hkv, d).to(BF), (torch.randn(1, T, Hkv, d, generator=g) * 2.0 ** 100).to(BF)
    see = [np.tril(np.ones((T, T), dtype=bool))]
    rows = (rows_k, rows_v)
    o, lse = tree_call(q, rows, kn, vn, see)
    o_r, l_r, tol_o, tol_l = ref_of(q, rows, kn, vn, see)
    within(o, o_r, tol_o, "o")
    within(lse, l_r, tol_l, "lse")


# ------------------------------------------------- many new tokens
@on_gpu
@pytest.mark.parametrize("T,Hq,Hkv,d,lens,row_lens", [
    (1000, 4, 2, 128, [300, 0], [1000, 700]),
    (4096, 1, 1, 64, [77], None),
    (2049, 2, 1, 64, [128, 1, 500], [2049, 64, 1025]),
])
@pytest.mark.parametrize("shape", ["chain", "tree"])
def test_long_chunks(T, Hq, Hkv, d, lens, row_lens, shape):
    """A chunk of a prompt, or a tree, of up to the most rows that a call takes."""
    from exact_io_aware_57_b200 import attn

    g, rng = torch.Generator().manual_seed(T), np.random.default_rng(T)
    B, counts = len(lens), row_lens or [T] * len(lens)
    cache = Cache(lens, Hkv, d, 32, BF)
    q, kn, vn = (torch.randn(B, T, h, d, generator=g).to(BF) for h in (Hq, Hkv, Hkv))
    for b, r in enumerate(counts):
        q[b, r:], kn[b, r:], vn[b, r:] = math.nan, math.nan, math.nan
    see = [random_tree(T, rng) if shape == "tree" else np.tril(np.ones((T, T), dtype=bool)) for _ in range(B)]
    mask = mask_words(np.stack(see)).cuda() if shape == "tree" else None
    k, v, cl, table = cache.gpu()
    ob, o = guarded_empty((B, T, Hq, d), BF)
    lb, lse = guarded_empty((B, Hq, T), F32)
    attn.attn_fwd_tree(q.cuda(), k, v, cl, k_new=kn.cuda(), v_new=vn.cuda(), block_table=table, tree_mask=mask,
                       row_lens=torch.tensor(counts, dtype=torch.int32).cuda(), out=o, lse=lse)
    status_ok()
    assert guards_intact(ob) and guards_intact(lb)
    o_r, l_r, tol_o, tol_l = tree_ref(q, cache.rows_k, cache.rows_v, kn, vn, see, counts, 1 / math.sqrt(d))
    within(lse, l_r, tol_l, "lse")
    within(o, o_r, tol_o, "o")


@on_gpu
def test_long_chunk_fp32():
    q, rows, kn, vn, see, bad = nan_case(700, 2, F32, lens=(100, 0))
    check_nan(tree_call(q, rows, kn, vn, see), ref_of(q, rows, kn, vn, see), bad)


# ------------------------------------------------- largest sizes
@on_gpu
@pytest.mark.parametrize("cap", [134215681, 1 << 28])
def test_weights_of_the_largest_capacity(cap):
    """Slots behind a short sequence's end, to the most that there can be."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(1)
    cache = Cache([5], 1, 64, 8, BF)
    k, _, cl, table = cache.gpu()
    q, lse = torch.randn(1, 1, 2, 64, generator=g).to(BF), torch.full((1, 2, 1), 2.0)
    w = torch.arange(cap, device="cuda", dtype=F32).remainder_(251).view(1, 1, cap)
    out = attn.attn_cache_weights(q.cuda(), lse.cuda(), k, cl, w, block_table=table, out=torch.empty_like(w))
    status_ok()
    assert torch.equal(out[..., 5:], w[..., 5:])
    ref, tol = weights_ref(q, lse, cache.rows_k, w[..., :5].cpu(), [[0]], [1], 0.125)
    within(out[..., :5], ref, tol, "weights")


def test_more_sequence_heads_than_a_grid_has_are_refused():
    from exact_io_aware_57_b200 import attn

    for dtype in (BF, F32):
        assert attn.attn_cache_weights_workspace_size(65535, 65535, 65535, 64, dtype) == 0
        assert attn.attn_cache_weights_workspace_size(65535, 32769, 32769, 64, dtype) == 0
        assert attn.attn_cache_weights_workspace_size(65535, 32768, 32768, 64, dtype) > 0


# ------------------------------------------------- row lists
@on_gpu
@pytest.mark.parametrize("n,bad", [(2, 0), (2, 1), (700, 699), (700, 300)])
@pytest.mark.parametrize("index", [-1, 9, 10 ** 9])
def test_append_with_a_row_that_does_not_exist(n, bad, index):
    """The sequence's length stays, the others are appended to."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(2)
    cache = Cache([3, 10, 0], 2, 64, 16, BF, room=n, stale=7.0)
    kn, vn = torch.randn(3, 9, 2, 64, generator=g).to(BF), torch.randn(3, 9, 2, 64, generator=g).to(BF)
    rows = torch.randint(0, 9, (3, n), generator=g, dtype=torch.int32)
    want = rows.clone()
    rows[1, bad] = index
    k, v, cl, table = cache.gpu()
    new = attn.attn_cache_append(kn.cuda(), vn.cuda(), k, v, cl, block_table=table, rows=rows.cuda())
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
    assert new.tolist() == [3 + n, 10, n]
    for b in (0, 2):
        for i in range(n):
            cache.k[cache.at(b, cache.lens[b] + i)] = kn[b, want[b, i]]
            cache.v[cache.at(b, cache.lens[b] + i)] = vn[b, want[b, i]]
    got_k, got_v = k.cpu(), v.cpu()
    for b, m in ((0, 3 + n), (1, 10), (2, n)):
        for s in range(m):
            at = cache.at(b, s)
            assert torch.equal(got_k[at], cache.k[at]) and torch.equal(got_v[at], cache.v[at])


@on_gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [3, 200])
def test_weights_with_a_row_that_does_not_exist(dtype, T):
    """It adds nothing; the other rows count as ever."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(6)
    cache = Cache([400, 250], 2, 64, 16, dtype)
    k, _, cl, table = cache.gpu()
    q = torch.randn(2, T, 4, 64, generator=g).to(dtype)
    lse = 6 + torch.rand(2, 4, T, generator=g)
    w = torch.rand(2, 2, 400, generator=g)
    rows = torch.arange(T, dtype=torch.int32).repeat(2, 1)
    rows[0, 1], rows[1, T - 1] = T, -1
    out = attn.attn_cache_weights(q.cuda(), lse.cuda(), k, cl, w.cuda(), block_table=table, rows=rows.cuda(),
                                  out=torch.empty_like(w).cuda())
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_ERR_INVALID
    gone = lse.clone()
    gone[0, :, 1] = gone[1, :, T - 1] = -math.inf
    ref, tol = weights_ref(q, gone, cache.rows_k, w, [list(range(T))] * 2, [T, T], 0.125)
    within(out, ref, tol, "weights")


# ------------------------------------------------- eviction within a pool
def evict_within(attn, **dst):
    """Return code of an eviction from k 4096, v 1 << 20 (never dereferenced) on the host."""
    import ctypes

    size = dict(num_pages=8, page_size=16, max_pages=4)
    src = attn.KVCache(k=4096, v=1 << 20, block_table=4096, lens=4096, **size)
    to = attn.KVCache(**{**dict(k=4096, v=1 << 20, block_table=8192, lens=None), **size, **dst})
    P = ctypes.c_void_p
    return attn.lib().attn_cache_evict(ctypes.byref(src), P(4096), 64, 8, 2, ctypes.byref(to), P(8192), P(4096), P(8192),
                                       2, 2, 64, 0, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses must not reach a GPU")
def test_eviction_within_a_pool_is_accepted_by_other_tables():
    """Accepted: the next answer is that there is no device to run on."""
    from exact_io_aware_57_b200 import attn

    for dst in (dict(), dict(v=1 << 21), dict(k=8192), dict(block_table=None), dict(k=8192, v=1 << 21, page_size=32)):
        assert evict_within(attn, **dst) == attn.ATTN_ERR_UNSUPPORTED
    for dst in (dict(block_table=4096), dict(block_table=4096, v=1 << 21), dict(page_size=32), dict(k=1 << 20, v=8192),
                dict(k=8192, v=4096)):
        assert evict_within(attn, **dst) == attn.ATTN_ERR_INVALID


@on_gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_evict_into_free_pages_of_the_same_pool(dtype):
    """There and, with more rows appended, back: the source's old pages are free by then."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(3)
    lens, keep, recent, page, Hkv, d = [150, 61, 30], 40, 8, 16, 2, 64
    cache = Cache(lens, Hkv, d, page, dtype, room=8, stale=7.0, spare=12)
    used = set(cache.table[cache.table >= 0].tolist())
    free = [p for p in range(cache.k.shape[0]) if p not in used]
    other = torch.full((3, 4), -9, dtype=torch.int32)
    for b in range(3):
        other[b, :4] = torch.tensor(free[4 * b:4 * b + 4])
    other = other.cuda()
    k, v, n, table = cache.gpu()
    keys, vals = [x.clone() for x in cache.rows_k], [x.clone() for x in cache.rows_v]
    for here, there in ((table, other), (other, table)):
        w = torch.rand(3, Hkv, 160, generator=g)
        counts = n.tolist()
        w_out, kept, n = attn.attn_cache_evict(k, v, w.cuda(), n, keep, k, v, recent=recent, block_table=here,
                                               out_table=there)
        status_ok()
        assert n.tolist() == [min(x, keep) for x in counts]
        at = there.cpu()
        for b, m in enumerate(n.tolist()):
            stay = [kept_ref(w[b, h], counts[b], keep, recent) for h in range(Hkv)]
            keys[b], vals[b] = (torch.stack([x[b][stay[h], h] for h in range(Hkv)], 1) for x in (keys, vals))
            for s in range(m):
                where = int(at[b, s // page]), s % page
                assert torch.equal(k[where].cpu(), keys[b][s]) and torch.equal(v[where].cpu(), vals[b][s])
        kn, vn = (torch.randn(3, 8, Hkv, d, generator=g).to(dtype) for _ in range(2))
        n = attn.attn_cache_append(kn.cuda(), vn.cuda(), k, v, n, block_table=there)
        keys, vals = [torch.cat([x, kn[b]]) for b, x in enumerate(keys)], [torch.cat([x, vn[b]]) for b, x in enumerate(vals)]
    status_ok()


# ------------------------------------------------- streams of the caller's
def cache_calls():
    """Name -> (a call of one operator on a given stream, outputs and workspace its own)."""
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(8)
    cache = Cache([700, 900], 2, 128, 16, BF, room=4)
    k, v, lens, table = cache.gpu()
    q, kn, vn = (torch.randn(2, 1, h, 128, generator=g).to(BF).cuda() for h in (8, 2, 2))
    lse = torch.randn(2, 8, 1, generator=g).cuda() + 7
    w = torch.rand(2, 2, 1000, generator=g).cuda()
    ko, vo = torch.zeros(2, 64, 2, 128, dtype=BF, device="cuda"), torch.zeros(2, 64, 2, 128, dtype=BF, device="cuda")
    return {
        "tree": lambda s: attn.attn_fwd_tree(q, k, v, lens, k_new=kn, v_new=vn, block_table=table, stream=s),
        "append": lambda s: (attn.attn_cache_append(kn, vn, k, v, lens, block_table=table, stream=s),),
        "weights": lambda s: (attn.attn_cache_weights(q, lse, k, lens, None, block_table=table, stream=s),),
        "evict": lambda s: attn.attn_cache_evict(k, v, w, lens, 64, ko, vo, block_table=table, stream=s),
    }


def check_streams(call, same=torch.equal):
    """No output or workspace of a call on a side stream lies in memory that work still
    pending on the current stream is about to write or read."""
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    warm = [call(side) for _ in range(8)]
    # blocks of every size, freed while the current stream has yet to write them
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 20, 1 << 22, 1 << 25)
            for _ in range(4)]
    for x in junk:
        x.fill_(1)  # (what is done for the first time may wait for the device)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    del warm
    torch.cuda._sleep(2_000_000_000)  # about a second
    for x in junk:
        x.fill_(255)
    spans = [(x.data_ptr(), x.data_ptr() + x.numel()) for x in junk]
    del junk, x
    got = call(side)
    for t in got:
        assert not any(lo < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < hi for lo, hi in spans)
    # what reads an output on the current stream is pending when the output is freed
    copies = [x.clone() for x in got]
    spans = [(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()) for x in got]
    del got, t
    again = [x for _ in range(3) for x in call(side)]
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    for t in again:
        assert not any(lo < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < hi for lo, hi in spans)
    torch.cuda.synchronize()
    for x, y in zip(copies, want):
        assert same(x, y)
    for i, x in enumerate(again):
        assert same(x, want[i % len(want)])


@on_gpu
@pytest.mark.parametrize("name", ["tree", "append", "weights", "evict"])
def test_memory_of_a_call_on_a_side_stream(name):
    check_streams(cache_calls()[name])
    status_ok()


def dense_calls():
    from exact_io_aware_57_b200 import attn

    g = torch.Generator().manual_seed(9)
    q, do = (torch.randn(1, 512, 4, 64, generator=g).to(BF).cuda() for _ in range(2))
    k, v = (torch.randn(1, 512, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    o, lse = attn.attn_fwd(q, k, v, causal=True)
    parts = [torch.stack(x) for x in zip(*(attn.attn_fwd_partial(q, k[:, i:i + 256].contiguous(),
                                                                 v[:, i:i + 256].contiguous()) for i in (0, 256)))]
    q3, k3, v3 = (x[0].contiguous() for x in (q, k, v))
    cu = torch.tensor([0, 200, 512], dtype=torch.int32).cuda()
    return {
        "fwd": lambda s: attn.attn_fwd(q, k, v, causal=True, stream=s),
        "dv": lambda s: attn.attn_fwd_dv(q, k, v, stream=s),
        "splitkv": lambda s: attn.attn_fwd_splitkv(q, k, v, num_splits=2, stream=s),
        "partial": lambda s: attn.attn_fwd_partial(q, k, v, stream=s),
        "merge": lambda s: attn.attn_merge_partials(*parts, stream=s),
        "varlen": lambda s: attn.attn_fwd_varlen(q3, k3, v3, cu, cu, 312, 312, causal=True, stream=s),
        "quantize": lambda s: attn.attn_quantize_e4m3(q, stream=s),
        "bwd": lambda s: attn.attn_bwd(q, k, v, o, lse, do, causal=True, stream=s),
        "bwd_varlen": lambda s: attn.attn_bwd_varlen(q3, k3, v3, o[0], lse[0], do[0], cu, cu, 312, 312, stream=s),
    }


@on_gpu
@pytest.mark.parametrize("name", ["fwd", "dv", "splitkv", "partial", "merge", "varlen", "quantize", "bwd", "bwd_varlen"])
def test_memory_of_a_dense_call_on_a_side_stream(name):
    # (dQ is summed in no fixed order in fp32, and rounded to bf16 once: a step apart at most)
    near = lambda x, y: torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=1e-4)
    check_streams(dense_calls()[name], near if name.startswith("bwd") else torch.equal)
    status_ok()


@on_gpu
def test_outputs_on_the_host_are_refused_on_a_side_stream():
    from exact_io_aware_57_b200 import attn

    k = torch.zeros(1, 8, 2, 64, dtype=BF, device="cuda")
    q, lens = torch.zeros(1, 1, 2, 64, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(attn.AttnError, match="out is on cpu"):
        attn.attn_fwd_tree(q, k, k, lens, out=torch.zeros(1, 1, 2, 64, dtype=BF), stream=torch.cuda.Stream())
    status_ok()


class FakeStream:
    device = torch.device("cuda", 1)


def test_stream_of_another_device_is_refused():
    """A tensor that says it is on device 0 and a stream of device 1, without a GPU."""
    from exact_io_aware_57_b200 import attn

    class OnDevice0:
        @staticmethod
        def get_device():
            return 0

    with pytest.raises(attn.AttnError, match="stream is on cuda:1, q on cuda:0"):
        attn._on(OnDevice0, "q", FakeStream)


def test_stream_of_another_device_is_refused_by_dense_calls(monkeypatch):
    from exact_io_aware_57_b200 import attn

    class Current:
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Current)
    for call in (lambda: attn.attn_fwd(None, None, None, stream=FakeStream),
                 lambda: attn.attn_selftest_ex2(None, FakeStream)):
        with pytest.raises(attn.AttnError, match="stream is on cuda:1, the current device is cuda:0"):
            call()
