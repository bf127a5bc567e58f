"""Measured cases of the key/value-cache operators: append, tree attention,
accumulated key weights and eviction.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, one sequence at a time, rounded once at the end) or, with ``own`` set,
calls the framework's entry points; ``exact`` states the definitions again in
64 bits.  Notation: a cache holds ``lens[b]`` slots of sequence b; slot s lies
on page ``table[b, s // page]`` at row ``s % page`` (``page`` 0 in a case: one
contiguous page for each sequence and no table).  Query head h reads KV head
h // (h_q // h_kv).
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _tree(name, batch, h_q, h_kv, d, page, len_min, len_max, drafts, shape, ragged=False, dtype="bf16", seed=1):
    """shape: "none" (rows see the cache only), "chain" (causal) or "tree"."""
    return dict(name=name, op="tree", batch=batch, h_q=h_q, h_kv=h_kv, d=d, page=page, len_min=len_min,
                len_max=len_max, drafts=drafts, shape=shape, ragged=ragged, dtype=dtype, plan_seed=seed)


def _weights(name, batch, h_q, h_kv, d, page, len_min, len_max, drafts, accepted, dtype="bf16", seed=1):
    """drafts rows of q, of which ``accepted`` (0: all of them) count."""
    return dict(name=name, op="weights", batch=batch, h_q=h_q, h_kv=h_kv, d=d, page=page, len_min=len_min,
                len_max=len_max, drafts=drafts, accepted=accepted, dtype=dtype, plan_seed=seed)


def _append(name, batch, h_kv, d, page, len_min, len_max, drafts, accepted, dtype="bf16", seed=1):
    return dict(name=name, op="append", batch=batch, h_kv=h_kv, d=d, page=page, len_min=len_min, len_max=len_max,
                drafts=drafts, accepted=accepted, dtype=dtype, plan_seed=seed)


def _evict(name, batch, h_kv, d, page, page_out, len_min, len_max, keep, recent, dtype="bf16", seed=1):
    return dict(name=name, op="evict", batch=batch, h_kv=h_kv, d=d, page=page, page_out=page_out, len_min=len_min,
                len_max=len_max, keep=keep, recent=recent, dtype=dtype, plan_seed=seed)


def listed():
    return [
        # one stream answering token by token on a short context: all latency
        _tree("tree_b1_len1000_t1", 1, 32, 8, 128, 64, 1000, 1000, 1, "chain"),
        # a serving batch in its ordinary decode step, lengths as they come
        _tree("tree_b64_len8191_t1_p16", 64, 32, 8, 128, 16, 300, 8191, 1, "chain", seed=2),
        # a batch that verifies drafted trees; the last rows of q are padding
        _tree("tree_b16_len12345_t61_p128", 16, 32, 8, 128, 128, 2000, 12345, 61, "tree", ragged=True, seed=3),
        # few very long contexts and a small tree: the largest read
        _tree("tree_b4_len131071_t13_p256", 4, 32, 8, 128, 256, 100000, 131071, 13, "tree", seed=4),
        # heads without sharing, d = 64, contiguous cache read only (no drafted keys)
        _tree("tree_b4_mha16_d64_len2047_t2", 4, 16, 16, 64, 0, 700, 2047, 2, "none", seed=5),
        # one decode step's weights over a batch
        _weights("weights_b32_len8191_t1_p64", 32, 32, 8, 128, 64, 1000, 8191, 1, 0, seed=6),
        # a whole prompt's weights over its own dense keys
        _weights("weights_prompt8192", 1, 32, 8, 128, 0, 8192, 8192, 8192, 0, seed=7),
        # the accepted path of a verified tree
        _weights("weights_b16_len6000_t61_acc5_p16", 16, 32, 8, 128, 16, 901, 6000, 61, 5, seed=8),
        # the step's accepted rows into a paged cache
        _append("append_b64_t61_acc5_p16", 64, 8, 128, 16, 100, 1001, 61, 5, seed=9),
        # a batch of prompts into a paged cache
        _append("append_b4_t4095_p64", 4, 8, 128, 64, 0, 37, 4095, 0, seed=10),
        # a long prompt's keys cut down to a budget
        _evict("evict_b1_len32768_keep4096", 1, 8, 128, 0, 64, 32768, 32768, 4096, 64, seed=11),
        # a running batch brought back to its budget, fp32
        _evict("evict_b16_len4500_keep4001_f32", 16, 8, 64, 32, 32, 3500, 4500, 4001, 257, dtype="f32", seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "append", "evict"])
    h_kv = rng.choice([1, 2, 4, 8, 16])
    h_q = h_kv * rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, 16, 16, 32, 64, 64, 128, 256])
    seed = rng.randrange(1 << 30)
    dtype = "f32" if rng.random() < 0.1 else "bf16"
    if op == "tree":
        batch = _log_int(rng, 1, 64)
        # slots in all bounded by what the largest listed case reads; fp32 runs on the CUDA cores
        cap = (2 ** 18 if dtype == "bf16" else 2 ** 13) * 8 // h_kv // batch
        len_max = _log_int(rng, 1, max(1, min(131072, cap)))
        drafts = rng.choice([1, 1, _log_int(rng, 2, 128)])
        if drafts * h_q * len_max * batch > 2 ** 27:
            drafts = 1
        shape = rng.choice(["chain", "tree", "tree", "none"])
        return {k: v for k, v in _tree("", batch, h_q, h_kv, d, page, rng.randint(0, len_max), len_max, drafts, shape,
                                       rng.random() < 0.5, dtype, seed).items() if k != "name"}
    if op == "weights":
        if rng.random() < 0.4:  # a prompt
            n = _log_int(rng, 16, int(6000 * math.sqrt(32 / max(h_q, 32))) if dtype == "bf16" else 700)
            c = _weights("", 1, h_q, h_kv, d, 0, n, n, n, 0, dtype, seed)
        else:
            batch = _log_int(rng, 1, 64)
            cap = (2 ** 18 if dtype == "bf16" else 2 ** 13) * 8 // h_kv // batch
            drafts = rng.choice([1, _log_int(rng, 2, 64)])
            acc = 0 if drafts == 1 else rng.randint(1, min(drafts, 8))
            len_max = _log_int(rng, 64, max(64, min(131072, cap)))
            c = _weights("", batch, h_q, h_kv, d, page, rng.randint(64, len_max), len_max, drafts, acc, dtype, seed)
        return {k: v for k, v in c.items() if k != "name"}
    if op == "append":
        drafts = _log_int(rng, 1, 4095)
        batch = _log_int(rng, 1, max(1, min(64, 16384 // drafts)))
        acc = rng.randint(1, drafts) if drafts <= 128 and rng.random() < 0.6 else 0
        len_max = _log_int(rng, 1, 2000)
        return {k: v for k, v in _append("", batch, h_kv, d, page, rng.randint(0, len_max), len_max, drafts, acc, dtype,
                                         seed).items() if k != "name"}
    batch = _log_int(rng, 1, 32)
    len_max = _log_int(rng, 2, max(2, 2 ** 17 * 8 // h_kv // batch // 2))
    keep = _log_int(rng, 1, min(len_max, 8192))
    return {k: v for k, v in _evict("", batch, h_kv, d, page, rng.choice([16, 32, 64, 256]), rng.randint(1, len_max),
                                    len_max, keep, rng.randint(0, keep), dtype, seed).items() if k != "name"}


# ------------------------------------- what a case's plan fixes (no tensor data)
def _plan(case):
    """Lengths, rows that count and trees: fixed by the case, not by the inputs' seed."""
    rng = random.Random(case["plan_seed"])
    B = case["batch"]
    lens = [rng.randint(case["len_min"], case["len_max"]) for _ in range(B)]
    lens[0] = case["len_max"]
    plan = {"lens": lens}
    T = case.get("drafts", 0)
    if case["op"] == "tree":
        plan["rows"] = [rng.randint(1, T) if case["ragged"] and b else T for b in range(B)]
        # parent of each drafted token among those before it; -1: the cache's end
        plan["parents"] = [[max(-1, t - 1 - int(rng.expovariate(0.4))) for t in range(T)] for _ in range(B)]
    elif case["op"] in ("weights", "append"):
        acc = case["accepted"]
        plan["count"] = [rng.randint(1, acc) if b else acc for b in range(B)] if acc else [T] * B
        plan["path"] = [sorted(rng.sample(range(T), c)) for c in plan["count"]] if acc else None
        if case["op"] == "weights":  # the rows counted are the sequence's last
            plan["lens"] = [max(n, c) for n, c in zip(lens, plan["count"])]
    return plan


def _visible(case, plan):
    """tree: for each sequence the drafted keys row t sees, as lists of index lists."""
    out = []
    for b in range(case["batch"]):
        rows = []
        for t in range(plan["rows"][b]):
            if case["shape"] == "none":
                rows.append([])
            elif case["shape"] == "chain":
                rows.append(list(range(t + 1)))
            else:
                p = plan["parents"][b][t]
                rows.append(([] if p < 0 else rows[p]) + [t])
        out.append(rows)
    return out


def work(case):
    plan = _plan(case)
    es = 2 if case["dtype"] == "bf16" else 4
    B, Hkv, d, lens = case["batch"], case["h_kv"], case["d"], plan["lens"]
    if case["op"] == "tree":
        Hq, rows = case["h_q"], plan["rows"]
        new = 0 if case["shape"] == "none" else sum(rows)
        seen = sum(len(r) for s in _visible(case, plan) for r in s)
        pairs = sum(n * r for n, r in zip(lens, rows)) + seen
        return {"bytes": (sum(lens) + new) * Hkv * d * 2 * es + sum(rows) * Hq * (2 * d * es + 4),
                "flops": 4 * pairs * Hq * d}
    if case["op"] == "weights":
        Hq, cnt = case["h_q"], plan["count"]
        pairs = sum(c * (n - c) + c * (c + 1) // 2 for n, c in zip(lens, cnt))
        return {"bytes": sum(lens) * Hkv * (d * es + 8) + sum(cnt) * Hq * (d * es + 4), "flops": 2 * pairs * Hq * d}
    if case["op"] == "append":
        return {"bytes": 4 * sum(plan["count"]) * Hkv * d * es, "flops": 0}
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": sum(lens) * Hkv * 4 + kept * Hkv * (4 * d * es + 8), "flops": 0}


# ------------------------------------------------------------------ the inputs
def _cache(case, lens, gen, dtype, page, fill=True):
    """Page pools of K and V with room for lens[b] slots, and the page table (None: contiguous)."""
    B, Hkv, d = case["batch"], case["h_kv"], case["d"]
    if page == 0:
        shape, table = (B, max(lens), Hkv, d), None
    else:
        per = -(-max(lens) // page)
        need = [-(-n // page) for n in lens]
        order = torch.randperm(sum(need), generator=gen, device="cuda").int()  # pages in no order
        table, at = torch.full((B, per), -1, dtype=torch.int32, device="cuda"), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        shape = (sum(need), page, Hkv, d)
    if not fill:
        return torch.zeros(shape, device="cuda", dtype=dtype), torch.zeros(shape, device="cuda", dtype=dtype), table
    # slots behind a sequence's end hold an earlier tenant's rows
    return (torch.randn(shape, device="cuda", dtype=dtype, generator=gen),
            torch.randn(shape, device="cuda", dtype=dtype, generator=gen), table)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + case["plan_seed"] % 1000003)
    plan, dtype, B = _plan(case), _DTYPES[case["dtype"]], case["batch"]
    lens, T, Hkv, d = plan["lens"], case.get("drafts", 0), case["h_kv"], case["d"]

    def randn(*shape):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    st = {"case": case, "plan": plan, "lens": _ints(lens)}
    if case["op"] == "tree":
        st["k"], st["v"], st["table"] = _cache(case, lens, gen, dtype, case["page"])
        st["q"] = randn(B, T, case["h_q"], d)
        new = case["shape"] != "none"
        st["k_new"], st["v_new"] = (randn(B, T, Hkv, d), randn(B, T, Hkv, d)) if new else (None, None)
        st["rows"] = _ints(plan["rows"]) if case["ragged"] else None
        st["mask"] = None
        if case["shape"] == "tree":  # bit j of row t: drafted key j is seen
            words = -(-T // 64)
            mask = [[[0] * words for _ in range(T)] for _ in range(B)]
            for b, seq in enumerate(_visible(case, plan)):
                for t, keys in enumerate(seq):
                    for j in keys:
                        mask[b][t][j // 64] |= 1 << (j % 64)
            mask = [[[w - (1 << 64) if w >> 63 else w for w in row] for row in seq] for seq in mask]
            st["mask"] = torch.tensor(mask, dtype=torch.int64, device="cuda")
    elif case["op"] == "weights":
        st["k"], _, st["table"] = _cache(case, lens, gen, dtype, case["page"])
        st["q"] = randn(B, T, case["h_q"], d)
        st["count"] = _ints(plan["count"]) if plan["path"] else None
        st["path"] = None
        seen = torch.ones(B, T, device="cuda")
        if plan["path"]:
            st["path"] = _ints([p + [0] * (case["accepted"] - len(p)) for p in plan["path"]])
        for b in range(B):
            rows = plan["path"][b] if plan["path"] else list(range(T))
            seen[b, rows] = torch.arange(lens[b] - len(rows) + 1, lens[b] + 1, device="cuda", dtype=torch.float32)
        # the log-sum-exp that attention over N(0, 1) keys comes to: ln n + |q|^2 / 2d
        qq = st["q"].float().square().sum(-1) / (2 * d)
        st["lse"] = (seen.log()[:, :, None] + qq).transpose(1, 2).contiguous()
        st["weights"] = torch.rand(B, Hkv, max(lens), device="cuda", generator=gen)
        st["out"] = torch.zeros_like(st["weights"])
    elif case["op"] == "append":
        full = [n + c for n, c in zip(lens, plan["count"])]
        st["k"], st["v"], st["table"] = _cache(case, full, gen, dtype, case["page"])
        st["k_new"], st["v_new"] = randn(B, T, Hkv, d), randn(B, T, Hkv, d)
        st["path"] = _ints([p + [0] * (case["accepted"] - len(p)) for p in plan["path"]]) if plan["path"] else None
        st["count"] = _ints(plan["count"]) if plan["path"] else None
    else:
        st["k"], st["v"], st["table"] = _cache(case, lens, gen, dtype, case["page"])
        kept = [min(n, case["keep"]) for n in lens]
        st["k_out"], st["v_out"], st["table_out"] = _cache(case, kept, gen, dtype, case["page_out"], fill=False)
        # a few keys hold most of the weight, many hold equal small amounts
        w = torch.rand(B, Hkv, max(lens), device="cuda", generator=gen).pow(8)
        st["weights"] = torch.where(w < 0.01, (w * 2000).floor() / 2000, w)
    return st


# ------------------------------------------------------------- one pass
def _slots(cache, table, b, lo, hi):
    """Page and row of slots lo .. hi - 1 of sequence b."""
    s = torch.arange(lo, hi, device=cache.device)
    if table is None:
        return torch.full_like(s, b), s
    page = cache.shape[1]
    return table[b].long()[s // page], s % page


def _plain_tree(st):
    case, plan = st["case"], st["plan"]
    B, T, Hq, d = st["q"].shape
    Hkv, G = case["h_kv"], Hq // case["h_kv"]
    o = torch.zeros(B, T, Hq, d, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, device="cuda")
    for b in range(B):
        n, r = plan["lens"][b], plan["rows"][b]
        at = _slots(st["k"], st["table"], b, 0, n)
        k, v = st["k"][at].float(), st["v"][at].float()
        q = st["q"][b, :r].float().reshape(r, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * r, d)
        if st["k_new"] is not None:
            k = torch.cat([k, st["k_new"][b, :r].float()])
            v = torch.cat([v, st["v_new"][b, :r].float()])
        s = q @ k.permute(1, 2, 0) / math.sqrt(d)
        if st["k_new"] is not None:
            j = torch.arange(r, device="cuda")
            if st["mask"] is None:
                see = j[None, :] <= j[:, None]
            else:
                see = (st["mask"][b, :r][:, j // 64] >> (j % 64)) & 1 == 1
            s[:, :, n:].masked_fill_(~see.repeat(G, 1), -math.inf)
        m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full((Hkv, G * r, 1), -math.inf)
        p = (s - m.masked_fill(m == -math.inf, 0)).exp()
        l = p.sum(-1, keepdim=True)
        ob = (p @ v.transpose(0, 1)) / l.masked_fill(l == 0, 1)
        o[b, :r] = ob.reshape(Hkv, G, r, d).permute(2, 0, 1, 3).reshape(r, Hq, d)
        lse[b, :, :r] = (m + l.log()).reshape(Hq, r)
    return o.to(st["q"].dtype), lse


def _plain_weights(st):
    case, plan = st["case"], st["plan"]
    B, T, Hq, d = st["q"].shape
    Hkv, G = case["h_kv"], Hq // case["h_kv"]
    out = st["weights"].clone()
    for b in range(B):
        n, c = plan["lens"][b], plan["count"][b]
        rows = st["path"][b, :c].long() if st["path"] is not None else torch.arange(T, device="cuda")
        at = _slots(st["k"], st["table"], b, 0, n)
        k = st["k"][at].float()
        q = st["q"][b, rows].float().reshape(c, Hkv, G, d).permute(1, 2, 0, 3)
        z = st["lse"][b][:, rows].reshape(Hkv, G, c, 1)
        piece = max(1, 2 ** 28 // (Hq * n))  # rows at a time: a prompt's scores are large
        for lo in range(0, c, piece):
            r = min(piece, c - lo)
            s = (q[:, :, lo:lo + r].reshape(Hkv, G * r, d) @ k.permute(1, 2, 0) / math.sqrt(d)).reshape(Hkv, G, r, n)
            p = (s - z[:, :, lo:lo + r]).exp()
            last = n - c + lo + torch.arange(r, device="cuda")
            p.masked_fill_(torch.arange(n, device="cuda")[None, :] > last[:, None], 0)
            out[b, :, :n] += p.sum((1, 2))
    return out


def _plain_append(st):
    plan = st["plan"]
    for b in range(st["case"]["batch"]):
        n, c = plan["lens"][b], plan["count"][b]
        rows = st["path"][b, :c].long() if st["path"] is not None else slice(None)
        at = _slots(st["k"], st["table"], b, n, n + c)
        st["k"][at] = st["k_new"][b, rows]
        st["v"][at] = st["v_new"][b, rows]
    count = st["count"] if st["count"] is not None else st["case"]["drafts"]
    return st["k"], st["v"], st["lens"] + count


def _plain_evict(st):
    case, plan = st["case"], st["plan"]
    B, Hkv, cap = st["weights"].shape
    keep = case["keep"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    w_out = torch.zeros_like(st["weights"])
    heads = torch.arange(Hkv, device="cuda")[:, None]
    for b in range(B):
        n = plan["lens"][b]
        if n > keep:
            old = n - case["recent"]  # slots that compete; the rest stay
            best = st["weights"][b, :, :old].sort(dim=-1, descending=True, stable=True).indices[:, :keep - case["recent"]]
            late = torch.arange(old, n, device="cuda").expand(Hkv, -1)
            idx = torch.cat([best.sort(-1).values, late], -1)
        else:
            idx = torch.arange(n, device="cuda").expand(Hkv, -1)
        m = idx.shape[1]
        kept[b, :, :m] = idx
        w_out[b, :, :m] = st["weights"][b].gather(1, idx)
        page, row = _slots(st["k"], st["table"], b, 0, n)
        to_page, to_row = _slots(st["k_out"], st["table_out"], b, 0, m)
        src = (page[idx], row[idx], heads)
        dst = (to_page[None, :], to_row[None, :], heads)
        st["k_out"][dst] = st["k"][src]
        st["v_out"][dst] = st["v"][src]
    return st["k_out"], st["v_out"], w_out, kept, st["lens"].clamp(max=keep)


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "weights": _plain_weights, "append": _plain_append, "evict": _plain_evict}[op](st)
    from exact_io_aware_57_b200 import attn

    if op == "tree":
        return attn.attn_fwd_tree(st["q"], st["k"], st["v"], st["lens"], k_new=st["k_new"], v_new=st["v_new"],
                                  block_table=st["table"], tree_mask=st["mask"], row_lens=st["rows"])
    if op == "weights":
        return attn.attn_cache_weights(st["q"], st["lse"], st["k"], st["lens"], st["weights"], block_table=st["table"],
                                       rows=st["path"], row_lens=st["count"], out=st["out"])
    if op == "append":
        new_lens = attn.attn_cache_append(st["k_new"], st["v_new"], st["k"], st["v"], st["lens"],
                                          block_table=st["table"], rows=st["path"], row_lens=st["count"])
        return st["k"], st["v"], new_lens
    weights, kept, new_lens = attn.attn_cache_evict(st["k"], st["v"], st["weights"], st["lens"], st["case"]["keep"],
                                                    st["k_out"], st["v_out"], recent=st["case"]["recent"],
                                                    block_table=st["table"], out_table=st["table_out"])
    return st["k_out"], st["v_out"], weights, kept, new_lens


# ------------------------------------------------- the definitions in 64 bits
def _dense64(cache, table, b, n):
    if table is None:
        return cache[b, :n].double()
    page = cache.shape[1]
    pages = [cache[int(p)] for p in table[b, :-(-n // page)].tolist()]
    return torch.cat(pages)[:n].double() if pages else cache[:0, 0].double()


def exact(case, seed):
    if case["op"] not in ("tree", "weights"):
        return None  # rows moved and slots chosen: nothing is computed
    st, plan = prepare(case, seed), _plan(case)
    B, T, Hq, d = st["q"].shape
    group = Hq // case["h_kv"]
    if case["op"] == "weights":
        out = st["weights"].double()
        for b in range(B):
            n, c = plan["lens"][b], plan["count"][b]
            k = _dense64(st["k"], st["table"], b, n)
            rows = plan["path"][b] if plan["path"] else range(T)
            rows = torch.tensor(list(rows), device="cuda")
            for lo in range(0, c, 2048):  # rows in pieces: 64-bit scores are large
                part = rows[lo:lo + 2048]
                last = n - c + lo + torch.arange(len(part), device="cuda")
                for h in range(Hq):
                    x = torch.einsum("id,jd->ij", st["q"][b, part, h].double(), k[:, h // group]) * d ** -0.5
                    e = torch.exp(x - st["lse"][b, h, part].double()[:, None])
                    out[b, h // group, :n] += torch.where(torch.arange(n, device="cuda") <= last[:, None], e, 0.0).sum(0)
        return out
    o = torch.zeros(B, T, Hq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, device="cuda", dtype=torch.float64)
    visible = _visible(case, plan)
    for b in range(B):
        n, r = plan["lens"][b], plan["rows"][b]
        k, v = _dense64(st["k"], st["table"], b, n), _dense64(st["v"], st["table"], b, n)
        see = torch.ones(r, n, dtype=torch.bool)
        if st["k_new"] is not None:
            k, v = torch.cat([k, st["k_new"][b, :r].double()]), torch.cat([v, st["v_new"][b, :r].double()])
            tail = torch.zeros(r, r, dtype=torch.bool)
            for t, keys in enumerate(visible[b]):
                tail[t, keys] = True
            see = torch.cat([see, tail], 1)
        see = see.cuda()
        if not see.any():
            continue
        for h in range(Hq):
            x = torch.einsum("td,jd->tj", st["q"][b, :r, h].double(), k[:, h // group]) * d ** -0.5
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[b, h, :r] = z
            o[b, :r, h] = torch.exp(x - z[:, None]).nan_to_num(0.0) @ v[:, h // group]
    return o, lse
