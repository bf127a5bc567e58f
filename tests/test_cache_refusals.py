"""What the cache calls refuse, before anything touches a GPU: the C entry points with
addresses that are never dereferenced, and the binding with tensors that are not on one."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


def ptr(x=4096):
    return P(x)


def cache(attn, **kw):
    args = dict(k=4096, v=4096, block_table=4096, lens=4096, num_pages=8, page_size=16, max_pages=4)
    args.update(kw)
    return attn.KVCache(**args)


def call(name, attn, c, **kw):
    """One entry point with acceptable arguments but for those in kw."""
    by = ctypes.byref(c) if c is not None else None
    a = dict(k_new=ptr(), v_new=ptr(), rows=None, max_rows=3, row_lens=None, new_lens=ptr(8192), batch=2, n_new=3, h_q=4,
             h_kv=2, d=64, dtype=0, q=ptr(), mask=None, mstride=0, o=ptr(), lse=ptr(), scale=0.1, ws=ptr(), ws_bytes=1 << 40,
             weights=ptr(), out=ptr(), cap=64, keep=8, recent=2, dst=None, kept=ptr())
    a.update(kw)
    L = attn.lib()
    if name == "append":
        return L.attn_cache_append(a["k_new"], a["v_new"], by, a["rows"], a["max_rows"], a["row_lens"], a["new_lens"],
                                   a["batch"], a["n_new"], a["h_kv"], a["d"], a["dtype"], None)
    if name == "tree":
        return L.attn_fwd_tree(a["q"], a["k_new"], a["v_new"], by, a["mask"], a["mstride"], a["row_lens"], a["o"], a["lse"],
                               a["batch"], a["h_q"], a["h_kv"], a["n_new"], a["d"], a["scale"], a["ws"], a["ws_bytes"],
                               a["dtype"], None)
    if name == "weights":
        return L.attn_cache_weights(a["q"], a["lse"], by, a["rows"], a["max_rows"], a["row_lens"], a["weights"], a["out"],
                                    a["cap"], a["batch"], a["h_q"], a["h_kv"], a["n_new"], a["d"], a["scale"], a["ws"],
                                    a["ws_bytes"], a["dtype"], None)
    dst = a["dst"] if a["dst"] is not None else cache(attn, k=1 << 20, v=1 << 21)
    out = a["out"] if a["out"].value != 4096 else ptr(8192)
    return L.attn_cache_evict(by, a["weights"], a["cap"], a["keep"], a["recent"], ctypes.byref(dst), out, a["kept"],
                              a["new_lens"], a["batch"], a["h_kv"], a["d"], a["dtype"], None)


ALL = ("append", "tree", "weights", "evict")
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3

CASES = [(n, c, {}, r) for n in ALL for c, r in (
    (dict(k=0), INVALID), (dict(k=4100), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=12), INVALID), (dict(max_pages=0), INVALID), (dict(block_table=None, num_pages=1), INVALID),
    (dict(block_table=4098), INVALID), (dict(lens=0), INVALID), (dict(page_size=(1 << 28) + 8), UNSUPPORTED))]
CASES += [(n, {}, kw, r) for n in ALL for kw, r in (
    (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(batch=0), INVALID), (dict(h_kv=0), INVALID),
    (dict(batch=65536), UNSUPPORTED))]
CASES += [(n, dict(v=0), {}, INVALID) for n in ("append", "tree", "evict")]
CASES += [
    ("append", {}, dict(k_new=None), INVALID), ("append", {}, dict(new_lens=ptr(4096)), INVALID),
    ("append", {}, dict(max_rows=4), INVALID), ("append", {}, dict(max_rows=0), INVALID),
    ("append", {}, dict(n_new=0), INVALID), ("append", {}, dict(v_new=ptr(4104)), INVALID),
    ("append", {}, dict(rows=ptr(4098)), INVALID),
    ("tree", {}, dict(q=None), INVALID), ("tree", {}, dict(k_new=None), INVALID), ("tree", {}, dict(h_q=3), INVALID),
    ("tree", {}, dict(n_new=4097), UNSUPPORTED), ("tree", {}, dict(mask=ptr(4100)), INVALID),
    ("tree", {}, dict(mask=ptr(), mstride=2), INVALID), ("tree", {}, dict(mask=ptr(), k_new=None, v_new=None), INVALID),
    ("tree", {}, dict(ws=None), WORKSPACE), ("tree", {}, dict(ws=ptr(4104)), WORKSPACE),
    ("weights", {}, dict(lse=None), INVALID), ("weights", {}, dict(out=None), INVALID),
    ("weights", {}, dict(cap=0), INVALID), ("weights", {}, dict(max_rows=4), INVALID),
    ("weights", {}, dict(h_q=5), INVALID), ("weights", {}, dict(ws_bytes=255), WORKSPACE),
    ("evict", {}, dict(weights=None), INVALID), ("evict", {}, dict(kept=None), INVALID),
    ("evict", {}, dict(keep=0), INVALID), ("evict", {}, dict(recent=9), INVALID), ("evict", {}, dict(recent=-1), INVALID),
    ("evict", {}, dict(out=ptr(4096 + 0), weights=ptr(8192)), INVALID), ("evict", {}, dict(new_lens=ptr(4096)), INVALID),
]


@pytest.mark.parametrize("name,cache_kw,kw,rc", CASES)
def test_refused(name, cache_kw, kw, rc):
    from exact_io_aware_57_b200 import attn

    assert call(name, attn, cache(attn, **cache_kw), **kw) == rc
    assert attn.attn_launch_count() == 0


def test_eviction_onto_itself_is_refused():
    from exact_io_aware_57_b200 import attn

    for kw in (dict(k=4096, v=1 << 20), dict(k=1 << 20, v=4096)):
        assert call("evict", attn, cache(attn), dst=cache(attn, **kw)) == INVALID
    assert call("append", attn, None) == INVALID


def test_acceptable_arguments_reach_the_device_check():
    """What the cases above vary is otherwise acceptable: without a GPU the next answer is
    that the device is not one the kernels are built for."""
    from exact_io_aware_57_b200 import attn

    if torch.cuda.is_available():
        pytest.skip("the addresses must not reach a GPU")
    for name in ALL:
        assert call(name, attn, cache(attn)) == UNSUPPORTED
        assert call(name, attn, cache(attn, block_table=None, page_size=77)) == UNSUPPORTED


def test_workspace_sizes():
    from exact_io_aware_57_b200 import attn

    one = attn.attn_fwd_tree_workspace_size(1, 32, 8, 1, 128)
    # a bf16 call's workspace goes by the rows of a (sequence, KV head), not by the batch
    assert 0 < one == attn.attn_fwd_tree_workspace_size(64, 32, 8, 1, 128)
    assert one < attn.attn_fwd_tree_workspace_size(1, 32, 8, 8, 128)
    assert attn.attn_fwd_tree_workspace_size(1, 32, 8, 0, 128) == 0
    assert attn.attn_fwd_tree_workspace_size(1, 32, 7, 1, 128) == 0
    assert attn.attn_cache_weights_workspace_size(1, 32, 8, 128) > 0
    assert attn.attn_cache_weights_workspace_size(1, 32, 8, 96) == 0


def test_binding_wants_gpu_tensors():
    from exact_io_aware_57_b200 import attn

    x = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(1, 2, 8)
    with pytest.raises(attn.AttnError, match="CUDA"):
        attn.attn_cache_append(x, x, x, x, lens)
    with pytest.raises(attn.AttnError, match="CUDA"):
        attn.attn_fwd_tree(x, x, x, lens)
    with pytest.raises(attn.AttnError, match="CUDA"):
        attn.attn_cache_weights(x, torch.zeros(1, 2, 8), x, lens, w)
    with pytest.raises(attn.AttnError, match="CUDA"):
        attn.attn_cache_evict(x, x, w, lens, 4, x, x)
    with pytest.raises(attn.AttnError, match="recent"):
        attn.attn_cache_evict(x, x, w, lens, 4, x, x, recent=5)
    with pytest.raises(attn.AttnError, match="together"):
        attn.attn_fwd_tree(x, x, x, lens, k_new=x)
    with pytest.raises(attn.AttnError, match="dimensions"):
        attn.attn_cache_append(x[0], x, x, x, lens)
