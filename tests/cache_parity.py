"""Key/value caches for the tests, and the cache operators' definitions in 64
bits, written slot by slot on the CPU.

Tolerances, fixed before any run.  A score is a dot product of d terms in fp32:
its error is at most (d + 2) 2^-24 scale sum |q_c k_c| =: e (products of bf16
are exact; every addition rounds once, and so do the two scalings).  exp turns
an absolute error of its argument into a relative one of its result; a base-2
argument of magnitude at most 64 adds 64 * 2^-23, the approximate exp2 2^-22.
So a weight p is off by a relative r = e + 1e-5 at most, and so is their sum:
  LSE      |err| <= r + 2^-23 |LSE|
  O        |err| <= 2 r A + h (A + |O|),  A = sum p |v|, where h is half a step
           of O's type (bf16 2^-8, fp32 2^-24): P is rounded to it before the
           product with V, and O once at the end
  weights  |err| <= r S + 2^-22 (S + |in|),  S the sum added: the LSE comes in
           fp32 (its rounding, 2^-24 |LSE|, is in the 1e-5), the sum's order
           adds a few roundings
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Cache:
    """Random pages in no order; slots behind a sequence's end hold NaN."""

    def __init__(self, lens, Hkv, d, page, dtype, room=0, seed=0, spare=3, stale=float("nan"), max_pages=None):
        g = torch.Generator().manual_seed(seed + 17)
        self.lens, self.page, self.B, self.Hkv, self.d, self.dtype = list(lens), page, len(lens), Hkv, d, dtype
        if page == 0:
            cap = max(max(lens) + room, 1)
            shape, self.table = (self.B, cap, Hkv, d), None
        else:
            need = [-(-(n + room) // page) for n in lens]
            total = sum(need) + spare
            order = torch.randperm(total, generator=g).int()
            # entries that no slot of the sequence uses name no page at all
            self.table, at = torch.full((self.B, max_pages or max(max(need), 1) + 1), -7, dtype=torch.int32), 0
            for b, n in enumerate(need):
                self.table[b, :n] = order[at:at + n]
                at += n
            shape = (total, page, Hkv, d)
        self.k = torch.full(shape, stale, dtype=dtype)
        self.v = torch.full(shape, stale, dtype=dtype)
        self.rows_k = [torch.randn(n, Hkv, d, generator=g).to(dtype) for n in lens]
        self.rows_v = [torch.randn(n, Hkv, d, generator=g).to(dtype) for n in lens]
        for b, n in enumerate(lens):
            for s in range(n):
                self.k[self.at(b, s)] = self.rows_k[b][s]
                self.v[self.at(b, s)] = self.rows_v[b][s]

    def at(self, b, s):
        return (b, s) if self.page == 0 else (int(self.table[b, s // self.page]), s % self.page)

    def gpu(self):
        t = None if self.table is None else self.table.cuda()
        return self.k.cuda(), self.v.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), t


def mask_words(see):
    """bool [..., T, T] -> int64 words [..., T, ceil(T / 64)]."""
    see = np.asarray(see, dtype=bool)
    T = see.shape[-1]
    words = (T + 63) // 64
    out = np.zeros(see.shape[:-1] + (words,), dtype=np.uint64)
    for j in range(T):
        out[..., j // 64] |= see[..., j].astype(np.uint64) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64))


def random_tree(T, rng):
    """Ancestors-or-self matrix of a random tree in topological order."""
    see = np.zeros((T, T), dtype=bool)
    for t in range(T):
        parent = rng.integers(-1, t) if t else -1
        if parent >= 0:
            see[t] = see[parent]
        see[t, t] = True
    return see


def tree_ref(q, rows_k, rows_v, k_new, v_new, see, row_lens, scale):
    """o, lse, and the bounds of their errors; see[b]: bool [T, T] or None (no new keys)."""
    B, T, Hq, d = q.shape
    Hkv = rows_k[0].shape[1]
    G, half = Hq // Hkv, HALF_STEP[q.dtype]
    o, lse = torch.zeros(B, T, Hq, d, dtype=torch.float64), torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        r = row_lens[b]
        if r == 0:
            continue
        k, v = rows_k[b].double(), rows_v[b].double()
        vis = torch.ones(r, k.shape[0], dtype=torch.bool)
        if see is not None:
            k, v = torch.cat([k, k_new[b, :r].double()]), torch.cat([v, v_new[b, :r].double()])
            vis = torch.cat([vis, torch.as_tensor(np.asarray(see[b])[:r, :r])], 1)
        for h in range(Hq):
            qh, kh, vh = q[b, :r, h].double(), k[:, h // G], v[:, h // G]
            s = (qh @ kh.T * scale).masked_fill(~vis, -math.inf)
            e = (d + 2) * 2.0 ** -24 * abs(scale) * (qh.abs() @ kh.abs().T).masked_fill(~vis, 0)
            rel = (e.amax(1) if e.shape[1] else e.new_zeros(r)) + 1e-5
            z = torch.logsumexp(s, 1) if s.shape[1] else s.new_full((r,), -math.inf)
            p = torch.where(vis, torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)
            A = p @ vh.abs()
            o[b, :r, h], lse[b, h, :r] = p @ vh, z
            tol_o[b, :r, h] = 2 * rel[:, None] * A + half * (A + o[b, :r, h].abs())
            tol_l[b, h, :r] = rel + 2.0 ** -23 * torch.where(z == -math.inf, 0.0, z.abs())
    return o, lse, tol_o, tol_l


def weights_ref(q, lse, rows_k, w_in, rows, counts, scale):
    """out [B, Hkv, cap] and the bound of its error; rows[b]: the counted rows of q in order."""
    B, T, Hq, d = q.shape
    Hkv = w_in.shape[1]
    G = Hq // Hkv
    out, tol = w_in.double().clone(), 2.0 ** -22 * w_in.double().abs()
    for b in range(B):
        n, c = rows_k[b].shape[0], counts[b]
        for i in range(c):
            t, last = rows[b][i], n - c + i
            for h in range(Hq):
                z = float(lse[b, h, t])
                if last < 0 or z == -math.inf:
                    continue
                kh, qh = rows_k[b][:last + 1, h // G].double(), q[b, t, h].double()
                p = torch.exp(kh @ qh * scale - z)
                e = (d + 2) * 2.0 ** -24 * abs(scale) * (kh.abs() @ qh.abs()) + 1e-5
                out[b, h // G, :last + 1] += p
                tol[b, h // G, :last + 1] += p * (e + 2.0 ** -22)
    return out, tol


def within(got, ref, tol, what=""):
    """Elementwise |got - ref| <= tol, infinities and NaN-freeness included."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert not torch.isnan(got).any(), f"{what}: NaN"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf), f"{what}: infinities differ"
    err = torch.where(inf, 0.0, (got - ref).abs())
    worst = float((err / tol.clamp(min=1e-300)).masked_fill(err == 0, 0).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound (max-abs {float(err.max()):.3e})"
    return worst


def kept_ref(w, n, keep, recent):
    """Slots that stay of one (sequence, head): by Python's own ordering."""
    if n <= keep:
        return list(range(n))
    key = [(-math.inf if math.isnan(x) else x) for x in w[:n - recent].tolist()]
    best = sorted(range(n - recent), key=lambda j: (-key[j], j))[:keep - recent]
    return sorted(best) + list(range(n - recent, n))
