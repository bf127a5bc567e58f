"""Exact IO-aware attention for B200: thin Python binding of the C-ABI library
``libattn.so`` (declared in ``include/attn.h``).

This module only marshals arguments: it checks shapes/dtypes, allocates the
output tensors with PyTorch (device memory and streams are PyTorch's), and
calls the C entry points of the same names.  Every step of the attention path
runs in the library's CUDA kernels; there is no fallback.  If the library is
missing, importing this module raises.

``stream`` (default: the current one) is where a call runs.  Another stream than
the current one does not wait for it: the inputs have to be ready there, and the
outputs are, once it has been waited for.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import inspect
import math
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libattn.so"

ATTN_BF16 = 0
ATTN_F32 = 1
ATTN_OK = 0
ATTN_ERR_INVALID = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_WORKSPACE = -3
ATTN_ERR_CUDA = -4
ATTN_ERR_TIMEOUT = -5

# symbol -> (restype, argtypes)
_VP, _FP, _IP = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_I, _LL, _F, _SZ = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
EXPORTS = {
    "attn_fwd": (_I, [_VP, _VP, _VP, _FP, _LL, _VP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _I, _VP]),
    "attn_fwd_alibi": (_I, [_VP, _VP, _VP, _FP, _VP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _I, _VP]),
    "attn_bwd_alibi": (_I, [_VP, _VP, _VP, _FP, _VP, _FP, _VP, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I, _I,
                            _F, _I, _I, _VP]),
    "attn_fwd_local": (_I, [_VP, _VP, _VP, _FP, _VP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _I, _VP]),
    "attn_bwd_local": (_I, [_VP, _VP, _VP, _FP, _VP, _FP, _VP, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I, _I,
                            _F, _I, _I, _I, _I, _VP]),
    "attn_bwd_varlen": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP, _VP, _IP, _IP, _I, _I, _I, _I, _I, _I, _I, _I,
                             _F, _I, _VP, _SZ, _I, _VP]),
    "attn_fwd_dv": (_I, [_VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _VP]),
    "attn_bwd_dv": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I, _I, _I, _F,
                         _I, _I, _VP]),
    "attn_selftest_wait_timeout": (_I, [ctypes.c_longlong, _VP]),
    "attn_selftest_ex2": (_I, [_VP, _VP, ctypes.c_longlong, _VP]),
    "attn_splitkv_num_splits": (_I, [_I, _I, _I, _I]),
    "attn_splitkv_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "attn_fwd_splitkv": (_I, [_VP, _VP, _VP, _VP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _I, _VP, _SZ, _I, _VP]),
    "attn_merge_partials": (_I, [_FP, _FP, _I, _VP, _FP, _I, _I, _I, _I, _I, _VP]),
    "attn_fwd_partial": (_I, [_VP, _VP, _VP, _FP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _I, _VP]),
    "attn_quantize_e4m3": (_I, [_VP, _VP, _FP, _I, _I, _I, _I, _VP]),
    "attn_fwd_fp8": (_I, [_VP, _FP, _VP, _FP, _VP, _VP, _FP, _I, _I, _I, _I, _I, _I, _F, _I, _VP]),
    "attn_bwd_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "attn_bwd": (_I, [_VP, _VP, _VP, _FP, _LL, _VP, _FP, _VP, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I,
                      _I, _F, _I, _I, _VP]),
    "attn_bwd_noalloc": (_I, [_VP, _VP, _VP, _FP, _LL, _VP, _FP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                              _F, _I, _I, _VP]),
    "attn_fwd_varlen": (_I, [_VP, _VP, _VP, _VP, _FP, _IP, _IP, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                             _VP]),
    "attn_naive_scratch_size": (_SZ, [_I, _I]),
    "attn_fwd_naive": (_I, [_VP, _VP, _VP, _VP, _FP, _VP, _SZ, _I, _I, _I, _I, _I, _I, _F, _I, _VP]),
    "attn_cache_append": (_I, [_VP, _VP, _VP, _IP, _I, _IP, _IP, _I, _I, _I, _I, _I, _VP]),
    "attn_fwd_tree_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "attn_fwd_tree": (_I, [_VP, _VP, _VP, _VP, _VP, _LL, _IP, _VP, _FP, _I, _I, _I, _I, _I, _F, _VP, _SZ, _I, _VP]),
    "attn_cache_weights_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "attn_cache_weights": (_I, [_VP, _FP, _VP, _IP, _I, _IP, _FP, _FP, _I, _I, _I, _I, _I, _I, _F, _VP, _SZ, _I, _VP]),
    "attn_cache_evict": (_I, [_VP, _FP, _I, _I, _I, _VP, _FP, _IP, _IP, _I, _I, _I, _I, _VP]),
    "attn_strerror": (ctypes.c_char_p, [_I]),
    "attn_device_status": (_I, [_VP]),
    "attn_launch_count": (_LL, [_I]),
    "attn_set_kernel_events": (_I, [_I, _VP, _VP]),
}

ATTN_KERNEL_FWD = 0
ATTN_KERNEL_BWD = 1


class AttnError(RuntimeError):
    pass


def _load() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m exact_io_aware_57_b200.build`")
    lib = ctypes.CDLL(str(LIB_PATH))
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _check(rc: int) -> None:
    if rc != ATTN_OK:
        raise AttnError(f"libattn error {rc}: {_lib.attn_strerror(rc).decode()}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    if t.dtype == torch.float32:
        return ATTN_F32
    raise AttnError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise AttnError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise AttnError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on_its_stream(call):
    """A call that, given ``stream``, allocates its outputs and workspaces on that stream:
    memory of the current one may still be in use there by work that has not run.  Its
    outputs are not given out again before what uses them on the current stream has run."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def run(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return call(*args, **kwargs)
        caller = torch.cuda.current_stream()
        if stream.device != caller.device:
            raise AttnError(f"stream is on {stream.device}, the current device is {caller.device}")
        with torch.cuda.stream(stream):
            out = call(*args, **kwargs)
        for t in out if isinstance(out, tuple) else (out,):
            t.record_stream(stream)
            t.record_stream(caller)
        return out

    return run


def _bias_args(bias, B, Hq, Nq, Nk):
    if bias is None:
        return None, 0
    if bias.dtype != torch.float32:
        raise AttnError("bias must be fp32")
    per = Hq * Nq * Nk
    if bias.numel() == per:
        return _dev(bias, "bias"), 0
    if bias.numel() == B * per:
        return _dev(bias, "bias"), per
    raise AttnError("bias must be [Hq,Nq,Nk] or [B,Hq,Nq,Nk]")


def _slopes(alibi_slopes, Hq):
    if alibi_slopes.dtype != torch.float32 or alibi_slopes.numel() != Hq:
        raise AttnError("alibi_slopes must be fp32 [h_q]")
    return _dev(alibi_slopes, "alibi_slopes")


def _window_args(window, bias):
    if bias is not None:
        raise AttnError("a local window takes alibi_slopes, not a dense bias")
    wl, wr = window
    return (-1 if wl is None else int(wl)), (-1 if wr is None else int(wr))


@_on_its_stream
def attn_fwd(q, k, v, bias=None, causal=False, scale=None, out=None, lse=None, stream=None, alibi_slopes=None,
             window=None):
    """O, LSE = attention(q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d]); o like q, lse fp32 [B,Hq,Nq].
    bias: dense fp32 [Hq,Nq,Nk] or [B,Hq,Nq,Nk]; alibi_slopes: fp32 [Hq] (bias
    -slope_h |j - (i + Nk - Nq)| formed in the kernel); at most one of the two.
    window = (left, right): local attention, keys a - left .. a + right of the
    key a = i + Nk - Nq aligned with row i (None or negative: unbounded)."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32) if lse is None else lse
    if window is not None:
        wl, wr = _window_args(window, bias)
        _check(_lib.attn_fwd_local(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
                                   None if alibi_slopes is None else _slopes(alibi_slopes, Hq), _dev(o, "o"),
                                   _dev(lse, "lse"), B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)), wl, wr,
                                   _dtype_code(q), _stream(stream)))
        return o, lse
    if alibi_slopes is not None:
        if bias is not None:
            raise AttnError("pass either bias or alibi_slopes")
        _check(_lib.attn_fwd_alibi(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _slopes(alibi_slopes, Hq),
                                   _dev(o, "o"), _dev(lse, "lse"), B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)),
                                   _dtype_code(q), _stream(stream)))
        return o, lse
    bp, bs = _bias_args(bias, B, Hq, Nq, Nk)
    _check(_lib.attn_fwd(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), bp, bs, _dev(o, "o"), _dev(lse, "lse"),
                         B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)), _dtype_code(q), _stream(stream)))
    return o, lse


@_on_its_stream
def attn_fwd_dv(q, k, v, causal=False, scale=None, out=None, lse=None, stream=None):
    """Forward with V of its own width: q/k [..., d], v [B,Nk,Hkv,d_v] -> o [B,Nq,Hq,d_v]."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv, dv = k.shape[1], k.shape[2], v.shape[3]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty((B, Nq, Hq, dv), device=q.device, dtype=q.dtype) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32) if lse is None else lse
    _check(_lib.attn_fwd_dv(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"), B, Hq, Hkv,
                            Nq, Nk, d, dv, scale, int(bool(causal)), _dtype_code(q), _stream(stream)))
    return o, lse


@_on_its_stream
def attn_bwd_dv(q, k, v, o, lse, dout, causal=False, scale=None, workspace=None, dq=None, dk=None, dv=None,
                stream=None):
    """Backward of attn_fwd_dv: q/k/dq/dk width d, v/o/dout/dv width d_v."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv, d_v = k.shape[1], k.shape[2], v.shape[3]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(B, Hq, Nq, d), device=q.device, dtype=torch.uint8)
    _check(_lib.attn_bwd_dv(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"),
                            _dev(dout, "dout"), _dev(dq, "dq"), _dev(dk, "dk"), _dev(dv, "dv"),
                            _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), B, Hq, Hkv,
                            Nq, Nk, d, d_v, scale, int(bool(causal)), _dtype_code(q), _stream(stream)))
    return dq, dk, dv


def attn_selftest_wait_timeout(limit_cycles=1_000_000, stream=None) -> None:
    """Launch the bounded-wait self-test (a wait that gives up after limit_cycles)."""
    _check(_lib.attn_selftest_wait_timeout(int(limit_cycles), _stream(stream)))


@_on_its_stream
def attn_selftest_ex2(x, stream=None):
    """2^x by the kernels' FMA-pipe exponential (fp32 device tensor in, same out)."""
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp32 tensor")
    y = torch.empty_like(x)
    _check(_lib.attn_selftest_ex2(_dev(x, "x"), _dev(y, "y"), x.numel(), _stream(stream)))
    return y


def attn_splitkv_num_splits(batch, h_q, n_q, n_k) -> int:
    return int(_lib.attn_splitkv_num_splits(batch, h_q, n_q, n_k))


def attn_splitkv_workspace_size(batch, h_q, n_q, d, num_splits) -> int:
    return int(_lib.attn_splitkv_workspace_size(batch, h_q, n_q, d, num_splits))


@_on_its_stream
def attn_fwd_splitkv(q, k, v, causal=False, scale=None, num_splits=0, out=None, lse=None, workspace=None,
                     stream=None):
    """attn_fwd computed over num_splits key ranges and merged (bf16, dense)."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32) if lse is None else lse
    t = int(num_splits) if num_splits and num_splits > 0 else attn_splitkv_num_splits(B, Hq, Nq, Nk)
    if workspace is None:
        workspace = torch.empty(max(256, attn_splitkv_workspace_size(B, Hq, Nq, d, t)), device=q.device,
                                dtype=torch.uint8)
    _check(_lib.attn_fwd_splitkv(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"), B, Hq,
                                 Hkv, Nq, Nk, d, scale, int(bool(causal)), t, _dev(workspace, "workspace"),
                                 workspace.numel() * workspace.element_size(), _dtype_code(q), _stream(stream)))
    return o, lse


@_on_its_stream
def attn_fwd_partial(q, k, v, causal=False, scale=None, o_part=None, lse_part=None, stream=None):
    """Unmerged attention of q [B,Nq,Hq,d] over one key block k/v [B,Nk,Hkv,d] (bf16):
    o_part fp32 [B,Nq,Hq,d] (normalised over the block) and lse_part fp32 [B,Hq,Nq].
    Causal aligns the block bottom-right.  Partials of disjoint blocks combine
    with attn_merge_partials."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o_part = torch.empty((B, Nq, Hq, d), device=q.device, dtype=torch.float32) if o_part is None else o_part
    lse_part = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32) if lse_part is None else lse_part
    if o_part.dtype != torch.float32 or lse_part.dtype != torch.float32:
        raise AttnError("partials are fp32")
    _check(_lib.attn_fwd_partial(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o_part, "o_part"),
                                 _dev(lse_part, "lse_part"), B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)),
                                 _dtype_code(q), _stream(stream)))
    return o_part, lse_part


@_on_its_stream
def attn_quantize_e4m3(x, x8=None, scales=None, stream=None):
    """Per-(batch, head) e4m3 quantisation of x bf16 [B,N,H,d]: returns x8 (uint8
    e4m3 bytes, same layout) and scales fp32 [B,H] (amax / 448)."""
    if x.dtype != torch.bfloat16:
        raise AttnError("x must be bf16")
    B, N, H, d = x.shape
    x8 = torch.empty(x.shape, device=x.device, dtype=torch.uint8) if x8 is None else x8
    scales = torch.empty((B, H), device=x.device, dtype=torch.float32) if scales is None else scales
    _check(_lib.attn_quantize_e4m3(_dev(x, "x"), _dev(x8, "x8"), _dev(scales, "scales"), B, N, H, d,
                                   _stream(stream)))
    return x8, scales


@_on_its_stream
def attn_fwd_fp8(q8, q_scales, k8, k_scales, v, causal=False, scale=None, out=None, lse=None, stream=None):
    """Forward with S = Q8 K8^T on e4m3 tensor cores (see attn_quantize_e4m3), P V in
    bf16: o bf16 [B,Nq,Hq,d], lse fp32 [B,Hq,Nq].  d = 128."""
    B, Nq, Hq, d = q8.shape
    Nk, Hkv = k8.shape[1], k8.shape[2]
    if v.dtype != torch.bfloat16:
        raise AttnError("v must be bf16")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty((B, Nq, Hq, d), device=v.device, dtype=torch.bfloat16) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=v.device, dtype=torch.float32) if lse is None else lse
    _check(_lib.attn_fwd_fp8(_dev(q8, "q8"), _dev(q_scales, "q_scales"), _dev(k8, "k8"), _dev(k_scales, "k_scales"),
                             _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"), B, Hq, Hkv, Nq, Nk, d, scale,
                             int(bool(causal)), _stream(stream)))
    return o, lse


@_on_its_stream
def attn_merge_partials(o_parts, lse_parts, out=None, lse=None, out_dtype=torch.bfloat16, stream=None):
    """Merge fp32 partials o_parts [T,B,Nq,Hq,d], lse_parts [T,B,Hq,Nq] over disjoint key ranges."""
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise AttnError("partials must be fp32")
    T, B, Nq, Hq, d = o_parts.shape
    o = torch.empty((B, Nq, Hq, d), device=o_parts.device, dtype=out_dtype) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=o_parts.device, dtype=torch.float32) if lse is None else lse
    code = 0 if o.dtype == torch.bfloat16 else 1 if o.dtype == torch.float32 else None
    if code is None:
        raise AttnError("merge output must be bf16 or fp32")
    _check(_lib.attn_merge_partials(_dev(o_parts, "o_parts"), _dev(lse_parts, "lse_parts"), T, _dev(o, "o"),
                                    _dev(lse, "lse"), B, Hq, Nq, d, code, _stream(stream)))
    return o, lse


def attn_bwd_workspace_size(batch, h_q, n_q, d) -> int:
    return int(_lib.attn_bwd_workspace_size(batch, h_q, n_q, d))


@_on_its_stream
def attn_bwd(q, k, v, o, lse, dout, bias=None, causal=False, scale=None, workspace=None, dq=None, dk=None,
             dv=None, stream=None, alibi_slopes=None, window=None):
    """dq, dk, dv of attn_fwd for upstream gradient dout (layouts as q, k, v)."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = attn_bwd_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    if window is not None:
        wl, wr = _window_args(window, bias)
        _check(_lib.attn_bwd_local(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
                                   None if alibi_slopes is None else _slopes(alibi_slopes, Hq), _dev(o, "o"),
                                   _dev(lse, "lse"), _dev(dout, "dout"), _dev(dq, "dq"), _dev(dk, "dk"),
                                   _dev(dv, "dv"), _dev(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(), B, Hq, Hkv, Nq, Nk, d, scale,
                                   int(bool(causal)), wl, wr, _dtype_code(q), _stream(stream)))
        return dq, dk, dv
    if alibi_slopes is not None:
        if bias is not None:
            raise AttnError("pass either bias or alibi_slopes")
        _check(_lib.attn_bwd_alibi(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _slopes(alibi_slopes, Hq),
                                   _dev(o, "o"), _dev(lse, "lse"), _dev(dout, "dout"), _dev(dq, "dq"),
                                   _dev(dk, "dk"), _dev(dv, "dv"), _dev(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(), B, Hq, Hkv, Nq, Nk, d, scale,
                                   int(bool(causal)), _dtype_code(q), _stream(stream)))
        return dq, dk, dv
    bp, bs = _bias_args(bias, B, Hq, Nq, Nk)
    _check(_lib.attn_bwd(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), bp, bs, _dev(o, "o"), _dev(lse, "lse"),
                         _dev(dout, "dout"), _dev(dq, "dq"), _dev(dk, "dk"), _dev(dv, "dv"),
                         _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                         B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)), _dtype_code(q), _stream(stream)))
    return dq, dk, dv


@_on_its_stream
def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=False, scale=None,
                    out=None, lse=None, stream=None):
    """Packed forward: q [Tq,Hq,d], k/v [Tk,Hkv,d], cu_seqlens int32 device; lse [Hq,Tq]."""
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise AttnError("cu_seqlens must be int32")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((Hq, Tq), device=q.device, dtype=torch.float32) if lse is None else lse
    _check(_lib.attn_fwd_varlen(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"),
                                _dev(cu_seqlens_q, "cu_seqlens_q"), _dev(cu_seqlens_k, "cu_seqlens_k"),
                                cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), Tq, Tk, Hq, Hkv,
                                d, scale, int(bool(causal)), _dtype_code(q), _stream(stream)))
    return o, lse


@_on_its_stream
def attn_bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=False,
                    scale=None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Backward of attn_fwd_varlen: dq like q [Tq,Hq,d], dk/dv like k/v [Tk,Hkv,d]."""
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise AttnError("cu_seqlens must be int32")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(1, Hq, Tq, d), device=q.device, dtype=torch.uint8)
    _check(_lib.attn_bwd_varlen(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"),
                                _dev(dout, "dout"), _dev(dq, "dq"), _dev(dk, "dk"), _dev(dv, "dv"),
                                _dev(cu_seqlens_q, "cu_seqlens_q"), _dev(cu_seqlens_k, "cu_seqlens_k"),
                                cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), Tq, Tk, Hq, Hkv, d,
                                scale, int(bool(causal)), _dev(workspace, "workspace"),
                                workspace.numel() * workspace.element_size(), _dtype_code(q), _stream(stream)))
    return dq, dk, dv


class KVCache(ctypes.Structure):
    """attn_kv_cache of include/attn.h (device addresses and sizes)."""
    _fields_ = [("k", _VP), ("v", _VP), ("block_table", _IP), ("lens", _IP), ("num_pages", _I), ("page_size", _I),
                ("max_pages", _I)]


# A decode step makes several of these calls per layer, each of a few
# microseconds on the device, so their checks are few and cheap: one test per
# tensor, and the reasons only where it fails.  `dev` is a device index.
def _ptr(t, name, dtype, shape, dev):
    """Device address of t, a contiguous tensor of this dtype, shape and device."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise AttnError(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape:
        raise AttnError(f"{name} must have shape {list(shape)}, has {list(t.shape)}")
    if t.get_device() != dev:
        raise AttnError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise AttnError(f"{name} must be contiguous")


def _cache(k, v, lens, table, B, Hkv, d, dtype, dev, name="cache"):
    shape = k.shape
    if len(shape) != 4 or shape[2] != Hkv or shape[3] != d:
        raise AttnError(f"k_{name} must be [pages, page_size, {Hkv}, {d}], has {list(shape)}")
    tp, width = None, 1
    if table is not None:
        width = table.shape[-1]
        tp = _ptr(table, "block_table", torch.int32, (B, width), dev)
    return KVCache(_ptr(k, f"k_{name}", dtype, shape, dev), None if v is None else _ptr(v, f"v_{name}", dtype, shape, dev),
                   tp, None if lens is None else _ptr(lens, "cache_lens", torch.int32, (B,), dev), shape[0], shape[1],
                   width)


def _row_args(rows, row_lens, B, n, dev):
    """Addresses and width of the optional row list and row counts."""
    rp, width = None, n
    if rows is not None:
        width = rows.shape[-1]
        rp = _ptr(rows, "rows", torch.int32, (B, width), dev)
    return rp, width, None if row_lens is None else _ptr(row_lens, "row_lens", torch.int32, (B,), dev)


_HERE = contextlib.nullcontext()


def _on(t, name, stream):
    """t's device index, a context in which that device and the caller's `stream` (None:
    the current one) are current, and the stream that was current, where it is not that.

    What a call allocates it allocates inside: memory of the current stream may still be
    in use there by work that has not run, and the caller's stream does not wait for it."""
    dev = t.get_device()
    if dev < 0:
        raise AttnError(f"{name} must be a CUDA tensor")
    if stream is None:
        return dev, _HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev), None
    if stream.device.index != dev:
        raise AttnError(f"stream is on {stream.device}, {name} on cuda:{dev}")
    return dev, torch.cuda.stream(stream), torch.cuda.current_stream(dev)


def _dims(t, name, n):
    shape = t.shape
    if len(shape) != n:
        raise AttnError(f"{name} must have {n} dimensions, has {list(shape)}")
    return shape


def _stream_on(stream, dev) -> int:
    # (the handle alone: a Stream object takes 1.2 us to make)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _out(t, name, dtype, shape, dev, fresh):
    """Address of an output: the caller's, checked, or one made here."""
    return t.data_ptr() if fresh else _ptr(t, name, dtype, shape, dev)


def _used_on(stream, caller, *tensors):
    """Outputs and workspaces of a call on a stream of the caller's: their memory is not
    given out again before what uses them there, and on the stream that was current, has run."""
    if stream is not None:
        for t in tensors:
            if t.is_cuda:  # (what is not is refused with the other arguments)
                t.record_stream(stream)
                t.record_stream(caller)


def _scratch(workspace, like, dev, size_of, *args):
    """Address and bytes of the caller's workspace, or of a new one (returned to keep it alive)."""
    if workspace is None:
        n = size_of(dev, *args)
        workspace = like.new_empty(n, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), n
    if workspace.get_device() != dev:
        raise AttnError(f"workspace is on {workspace.device}, not on cuda:{dev}")
    return workspace, _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


# a size goes by the arguments and the device alone
@functools.lru_cache(maxsize=4096)
def _tree_size(dev, *args):
    return int(_lib.attn_fwd_tree_workspace_size(*args))


@functools.lru_cache(maxsize=4096)
def _weights_size(dev, *args):
    return int(_lib.attn_cache_weights_workspace_size(*args))


def attn_cache_append(k_new, v_new, k_cache, v_cache, cache_lens, block_table=None, rows=None, row_lens=None,
                      new_lens=None, stream=None):
    """Write rows of k_new / v_new [B,T,Hkv,d] behind the last slot of each sequence of a
    cache (k_cache / v_cache [pages, page_size, Hkv, d], cache_lens int32 [B], block_table
    int32 [B, max_pages]; without a table page b is sequence b's): slot cache_lens[b] + i
    takes row rows[b, i] (default i), i < row_lens[b] (default all).  Returns the new
    lengths, int32 [B], in a buffer of their own; cache_lens is not changed.  A sequence
    that is not acceptable (attn_device_status) keeps its length."""
    B, T, Hkv, d = shape = _dims(k_new, "k_new", 4)
    dt = k_new.dtype
    dev, here, caller = _on(k_new, "k_new", stream)
    with here:
        c = _cache(k_cache, v_cache, cache_lens, block_table, B, Hkv, d, dt, dev)
        rp, width, lp = _row_args(rows, row_lens, B, T, dev)
        fresh = new_lens is None
        if fresh:
            new_lens = torch.empty_like(cache_lens)
            _used_on(stream, caller, new_lens)
        _check(_lib.attn_cache_append(_ptr(k_new, "k_new", dt, shape, dev), _ptr(v_new, "v_new", dt, shape, dev),
                                      ctypes.byref(c), rp, width, lp,
                                      _out(new_lens, "new_lens", torch.int32, (B,), dev, fresh), B, T, Hkv, d,
                                      _dtype_code(k_new), _stream_on(stream, dev)))
    return new_lens


def attn_fwd_tree_workspace_size(batch, h_q, h_kv, n_q, d, dtype=torch.bfloat16) -> int:
    return int(_lib.attn_fwd_tree_workspace_size(batch, h_q, h_kv, n_q, d,
                                                 ATTN_F32 if dtype == torch.float32 else ATTN_BF16))


def attn_fwd_tree(q, k_cache, v_cache, cache_lens, k_new=None, v_new=None, block_table=None, tree_mask=None,
                  row_lens=None, scale=None, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of new tokens q [B,T,Hq,d] over a cache (see attn_cache_append) and their own
    keys k_new / v_new [B,T,Hkv,d]: row t sees every cached slot and the new keys j with bit
    j % 64 of tree_mask[(b,) t, j // 64] set (int64 [B,T,ceil(T/64)] or [T,ceil(T/64)];
    default j <= t).  Without k_new the rows see the cache only.  Rows t >= row_lens[b] and
    rows that see no key get O = 0, LSE = -inf.  T = 1 is a decode step."""
    B, T, Hq, d = shape = _dims(q, "q", 4)
    Hkv, dt = _dims(k_cache, "k_cache", 4)[2], q.dtype
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if (k_new is None) != (v_new is None):
        raise AttnError("pass k_new and v_new together")
    if tree_mask is not None and k_new is None:
        raise AttnError("tree_mask needs k_new and v_new")
    dev, here, caller = _on(q, "q", stream)
    with here:
        c = _cache(k_cache, v_cache, cache_lens, block_table, B, Hkv, d, dt, dev)
        new = (B, T, Hkv, d)
        kp = None if k_new is None else _ptr(k_new, "k_new", dt, new, dev)
        vp = None if v_new is None else _ptr(v_new, "v_new", dt, new, dev)
        mp, mstride = None, 0
        if tree_mask is not None:
            words = (T + 63) // 64
            if tree_mask.dim() == 3:
                mp, mstride = _ptr(tree_mask, "tree_mask", torch.int64, (B, T, words), dev), T * words
            else:
                mp = _ptr(tree_mask, "tree_mask", torch.int64, (T, words), dev)
        lp = None if row_lens is None else _ptr(row_lens, "row_lens", torch.int32, (B,), dev)
        qp = _ptr(q, "q", dt, shape, dev)
        fresh_o, fresh_lse = out is None, lse is None
        o = torch.empty_like(q) if fresh_o else out
        if fresh_lse:
            lse = q.new_empty((B, Hq, T), dtype=torch.float32)
        code = _dtype_code(q)
        workspace, wp, wbytes = _scratch(workspace, q, dev, _tree_size, B, Hq, Hkv, T, d, code)
        _used_on(stream, caller, o, lse, workspace)
        _check(_lib.attn_fwd_tree(qp, kp, vp, ctypes.byref(c), mp, mstride, lp,
                                  _out(o, "out", dt, shape, dev, fresh_o),
                                  _out(lse, "lse", torch.float32, (B, Hq, T), dev, fresh_lse), B, Hq, Hkv, T, d,
                                  scale, wp, wbytes, code, _stream_on(stream, dev)))
    return o, lse


def attn_cache_weights_workspace_size(batch, h_q, h_kv, d, dtype=torch.bfloat16) -> int:
    return int(_lib.attn_cache_weights_workspace_size(batch, h_q, h_kv, d,
                                                      ATTN_F32 if dtype == torch.float32 else ATTN_BF16))


def attn_cache_weights(q, lse, k_cache, cache_lens, weights, block_table=None, rows=None, row_lens=None, scale=None,
                       out=None, workspace=None, stream=None):
    """Add to weights fp32 [B,Hkv,cap] the attention weight each cached slot received from
    the sequences' last tokens: the rows rows[b, i] (default i), i < row_lens[b] (default
    all), of q [B,T,Hq,d] with their lse [B,Hq,T], each summed over the query heads of a
    group; row i sees the slots j <= cache_lens[b] - count + i.  weights None: zeros, of
    one page's or the table's capacity.  out: the result (default weights itself)."""
    B, T, Hq, d = shape = _dims(q, "q", 4)
    Hkv, dt = _dims(k_cache, "k_cache", 4)[2], q.dtype
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dev, here, caller = _on(q, "q", stream)
    with here:
        c = _cache(k_cache, None, cache_lens, block_table, B, Hkv, d, dt, dev)
        rp, width, lp = _row_args(rows, row_lens, B, T, dev)
        if out is None:
            out = weights
            if out is None:
                out = q.new_empty((B, Hkv, c.page_size * c.max_pages), dtype=torch.float32)
        cap = out.shape[-1]
        op = _ptr(out, "out", torch.float32, (B, Hkv, cap), dev)
        wp = None if weights is None else _ptr(weights, "weights", torch.float32, (B, Hkv, cap), dev)
        code = _dtype_code(q)
        workspace, sp, sbytes = _scratch(workspace, q, dev, _weights_size, B, Hq, Hkv, d, code)
        _used_on(stream, caller, out, workspace)
        _check(_lib.attn_cache_weights(_ptr(q, "q", dt, shape, dev), _ptr(lse, "lse", torch.float32, (B, Hq, T), dev),
                                       ctypes.byref(c), rp, width, lp, wp, op, cap, B, Hq, Hkv, T, d, scale, sp, sbytes,
                                       code, _stream_on(stream, dev)))
    return out


def attn_cache_evict(k_cache, v_cache, weights, cache_lens, keep, k_out, v_out, recent=0, block_table=None,
                     out_table=None, weights_out=None, kept=None, new_lens=None, stream=None):
    """Cut each sequence of a cache down to keep slots, per KV head: the last `recent` slots
    and the others of largest weight (fp32 [B,Hkv,cap]; ties: the lower slot).  They go in
    ascending order to the cache k_out / v_out (out_table), whose pages are others than the
    source's in use: another pool, or (out_table another table) free pages of the same one.
    Returns weights_out (like weights, zeros behind the last slot), kept int32
    [B,Hkv,keep] (source slots, -1 behind the last) and new_lens int32 [B]."""
    _, _, Hkv, d = _dims(k_cache, "k_cache", 4)
    B, _, cap = wshape = _dims(weights, "weights", 3)
    dt = k_cache.dtype
    keep, recent = int(keep), int(recent)
    if not 0 <= recent <= keep or keep == 0:
        raise AttnError("need 0 <= recent <= keep and keep > 0")
    dev, here, caller = _on(k_cache, "k_cache", stream)
    with here:
        src = _cache(k_cache, v_cache, cache_lens, block_table, B, Hkv, d, dt, dev)
        dst = _cache(k_out, v_out, None, out_table, B, Hkv, d, dt, dev, name="out")
        wp = _ptr(weights, "weights", torch.float32, (B, Hkv, cap), dev)
        fresh_w, fresh_kept, fresh_lens = weights_out is None, kept is None, new_lens is None
        if fresh_w:
            weights_out = torch.empty_like(weights)
        if fresh_kept:
            kept = weights.new_empty((B, Hkv, keep), dtype=torch.int32)
        if fresh_lens:
            new_lens = torch.empty_like(cache_lens)
        _used_on(stream, caller, weights_out, kept, new_lens)
        _check(_lib.attn_cache_evict(ctypes.byref(src), wp, cap, keep, recent, ctypes.byref(dst),
                                     _out(weights_out, "weights_out", torch.float32, wshape, dev, fresh_w),
                                     _out(kept, "kept", torch.int32, (B, Hkv, keep), dev, fresh_kept),
                                     _out(new_lens, "new_lens", torch.int32, (B,), dev, fresh_lens), B, Hkv, d,
                                     _dtype_code(k_cache), _stream_on(stream, dev)))
    return weights_out, kept, new_lens


def attn_naive_scratch_size(n_q, n_k) -> int:
    return int(_lib.attn_naive_scratch_size(n_q, n_k))


@_on_its_stream
def attn_fwd_naive(q, k, v, causal=False, scale=None, scratch=None, stream=None):
    """Materialising three-step forward (measurement comparator only)."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    if scratch is None:
        scratch = torch.empty(attn_naive_scratch_size(Nq, Nk), device=q.device, dtype=torch.uint8)
    _check(_lib.attn_fwd_naive(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o"), _dev(lse, "lse"),
                               _dev(scratch, "scratch"), scratch.numel(), B, Hq, Hkv, Nq, Nk, d, scale,
                               int(bool(causal)), _stream(stream)))
    return o, lse


def attn_device_status(stream=None) -> int:
    """Synchronise and return/clear the device status word: 0, ATTN_ERR_TIMEOUT
    (a bounded wait gave up) or ATTN_ERR_INVALID (packed offsets rejected)."""
    return int(_lib.attn_device_status(_stream(stream)))


def attn_launch_count(reset: bool = False) -> int:
    return int(_lib.attn_launch_count(int(bool(reset))))


def attn_set_kernel_events(which: int, start=None, stop=None) -> None:
    """Record torch.cuda.Event pair (start, stop) around launches of kernel `which`
    (ATTN_KERNEL_FWD / ATTN_KERNEL_BWD) from this thread; None clears."""
    sp = None if start is None else start.cuda_event
    ep = None if stop is None else stop.cuda_event
    if (start is not None and not sp) or (stop is not None and not ep):
        raise AttnError("record the events once (torch creates them lazily) before registering them")
    _check(_lib.attn_set_kernel_events(int(which), sp, ep))
