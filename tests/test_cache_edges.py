"""The key/value-cache calls where inputs are odd rather than wrong: rows that do not
count, values that are not finite or very large, the largest sizes, streams of the
caller's.  Definitions and tolerances are those of cache_parity.py."""
import math

import numpy as np
import pytest
import torch

from cache_parity import Cache, mask_words, random_tree, tree_ref, weights_ref, within
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
