"""GB300 (sm_103a) fused scaled-dot-product attention, forward and backward.

A thin Python binding over the C ABI of ``libsdpa_tmem.so`` (declared in
``include/sdpa_tmem.h``): the functions below carry the same names and only
marshal torch tensors into device pointers and the current CUDA stream.  Every
step of the computation runs in the library's CUDA kernels; there is no other
path.  Importing this package does not load the library; the first call does,
and it raises if the library has not been built.

    from scaled_dot_product_tmem_gb300 import sdpa_forward, sdpa_backward
    o, lse = sdpa_forward(q, k, v, causal=True, window=1024)
    dq, dk, dv, d_off = sdpa_backward(q, k, v, o, dout, lse, causal=True, window=1024)

Tensors are BSHD bf16 on the GPU: q [B,S_q,H_q,d_qk], k [B,S_kv,H_kv,d_qk],
v [B,S_kv,H_kv,d_v]; lse fp32 [B,H_q,S_q]; softmax_offset fp32 [H_q].

Sequences of different lengths without padding rows, [T,H,d] with int32 offsets:

    o = attention_packed(q, k, v, cu_seqlens)

Serving over a 4-bit paged cache: attn_kv4_append fills it, sdpa_decode_kv4 attends over it,
attn_kv4_copy_pages forks and compacts it, kv4_gather reads it back:

    pool = kv4_pool(n_pages, H_kv, d, page_size)
    attn_kv4_append(k, v, cu_seqlens, pool, page_table, seq_lens)
    o, lse = sdpa_decode_kv4(q, pool, page_table, seq_lens + 1)

Rotary positions, by themselves (rope, differentiable), as an argument of attention and attention_packed,
or on the way into the cache (kv4_append_rope):

    inv_freq, gain = rope_frequencies(d)
    table = rope_table(inv_freq, positions, gain=gain)
    o = attention_packed(q, k, v, cu_seqlens, rope=table)

Drafted trees over the cache (speculative decoding):

    q = kv4_append_rope(q, k, v, table, cu_nodes, pool, page_table, seq_lens)
    o, lse = sdpa_tree_kv4(q, cu_nodes, parents, pool, page_table, seq_lens)
    attn_kv4_keep(pools, page_table, seq_lens, accepted, d)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

import torch

VANILLA, OFF_BY_ONE, LEARNABLE = 0, 1, 2
SOFTMAX_TYPES = {"vanilla": VANILLA, "off_by_one": OFF_BY_ONE, "learnable": LEARNABLE}
ATTN_OK = 0

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdpa_tmem.so")
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = attn_last_error_message()
        super().__init__(f"{what}: {attn_status_string(status)} (status {status})" + (f" [{detail}]" if detail else ""))


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m scaled_dot_product_tmem_gb300.build`"
                           " (or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, vp]
    lib.attn_fwd.restype = i
    lib.attn_bwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.attn_bwd_workspace_size.restype = sz
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, i, vp, sz,
                             vp]
    lib.attn_bwd.restype = i
    lib.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, vp, vp, vp]
    lib.attn_fwd_varlen.restype = i
    lib.attn_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, vp,
                                    vp, i, vp, sz, vp]
    lib.attn_bwd_varlen.restype = i
    lib.attn_status_string.argtypes = [i]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_last_error_message.argtypes = []
    lib.attn_last_error_message.restype = ctypes.c_char_p
    lib.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp,
                                     vp]
    lib.attn_bwd_noalloc.restype = i
    lib.attn_bwd_noalloc_max_scratch_bytes.argtypes = []
    lib.attn_bwd_noalloc_max_scratch_bytes.restype = sz
    lib.attn_bwd_noalloc_message.argtypes = []
    lib.attn_bwd_noalloc_message.restype = ctypes.c_char_p
    lib.attn_timing_enable.argtypes = [i]
    lib.attn_timing_enable.restype = i
    lib.attn_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int), i]
    lib.attn_timing_read.restype = i
    lib.attn_last_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.attn_last_device_error.restype = i
    lib.attn_selftest_wait_timeout.argtypes = [i, vp]
    lib.attn_selftest_wait_timeout.restype = i
    lib.attn_fwd_bias.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, i, i, vp, vp]
    lib.attn_fwd_bias.restype = i
    lib.attn_bwd_bias.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, vp, i, i, i, i, i, i, i, f, i, i,
                                  i, vp, i, vp, sz, vp]
    lib.attn_bwd_bias.restype = i
    lib.attn_fp8_amax.argtypes = [vp, sz, vp, vp]
    lib.attn_fp8_amax.restype = i
    lib.attn_fp8_quantize.argtypes = [vp, vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.attn_fp8_quantize.restype = i
    lib.attn_fp8_vt_row_bytes.argtypes = [i]
    lib.attn_fp8_vt_row_bytes.restype = i
    lib.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp, vp]
    lib.attn_fwd_fp8.restype = i
    lib.attn_fwd_varlen_bias.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, i, i, vp, vp, vp,
                                         vp]
    lib.attn_fwd_varlen_bias.restype = i
    lib.attn_bwd_varlen_bias.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, vp, i, i, i, i, i, i, i, f,
                                         i, i, i, vp, vp, vp, i, vp, sz, vp]
    lib.attn_bwd_varlen_bias.restype = i
    lib.attn_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, f, vp, vp]
    lib.attn_fwd_dropout.restype = i
    lib.attn_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, f,
                                     vp, i, vp, sz, vp]
    lib.attn_bwd_dropout.restype = i
    lib.attn_fp8_quantize_e5m2.argtypes = [vp, vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.attn_fp8_quantize_e5m2.restype = i
    lib.attn_fp8_quantize_both.argtypes = [vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.attn_fp8_quantize_both.restype = i
    lib.attn_bwd_fp8_workspace_size.argtypes = [i, i, i]
    lib.attn_bwd_fp8_workspace_size.restype = sz
    lib.attn_bwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i,
                                 i, i, i, f, i, i, i, vp, vp, sz, vp]
    lib.attn_bwd_fp8.restype = i
    lib.attn_packed_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.attn_packed_workspace_size.restype = sz
    lib.attn_fwd_packed.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i, vp, i, vp, sz, vp]
    lib.attn_fwd_packed.restype = i
    lib.attn_bwd_packed.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i,
                                    vp, i, vp, sz, vp]
    lib.attn_bwd_packed.restype = i
    ll = ctypes.c_longlong
    lib.attn_kv4_block_bytes.argtypes = [i, i]
    lib.attn_kv4_block_bytes.restype = i
    lib.attn_kv4_append.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, ll, ll, vp]
    lib.attn_kv4_append.restype = i
    lib.attn_kv4_gather.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp]
    lib.attn_kv4_gather.restype = i
    lib.attn_kv4_decode_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_kv4_decode_workspace_size.restype = sz
    lib.attn_kv4_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, i, vp, vp, sz, vp]
    lib.attn_kv4_decode.restype = i
    lib.attn_kv4_copy_pages.argtypes = [vp, i, i, sz, vp, vp, i, vp]
    lib.attn_kv4_copy_pages.restype = i
    lib.attn_rope_table.argtypes = [vp, vp, vp, i, i, f, vp]
    lib.attn_rope_table.restype = i
    lib.attn_rope.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, ll, ll, ll, ll, i, i, vp]
    lib.attn_rope.restype = i
    lib.attn_kv4_append_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, i, ll, ll, ll, ll,
                                         i, vp]
    lib.attn_kv4_append_rope.restype = i
    lib.attn_kv4_tree_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_kv4_tree_workspace_size.restype = sz
    lib.attn_kv4_tree.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, i, vp, i, vp, sz, vp]
    lib.attn_kv4_tree.restype = i
    lib.attn_kv4_keep.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp]
    lib.attn_kv4_keep.restype = i
    _lib = lib
    return lib


def library():
    """The loaded ctypes library (loads it on first use)."""
    return _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, ndim):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _stype(softmax_type):
    return SOFTMAX_TYPES[softmax_type] if isinstance(softmax_type, str) else int(softmax_type)


# ----------------------------------------------------------------------------- C ABI, same names


def attn_status_string(status: int) -> str:
    return _load().attn_status_string(int(status)).decode()


def attn_last_error_message() -> str:
    return _load().attn_last_error_message().decode()


def attn_last_device_error(stream=None):
    """Synchronise the stream; return (status, site) of the device error words and clear them."""
    site = ctypes.c_int(0)
    st = _load().attn_last_device_error(_stream(stream), ctypes.byref(site))
    return st, site.value


def attn_selftest_wait_timeout(site: int, stream=None) -> None:
    """Enqueue the failure-path self-test (a bounded wait that runs out; no fault)."""
    st = _load().attn_selftest_wait_timeout(int(site), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_selftest_wait_timeout")


def _check_lens(t, name, B):
    if t is not None:
        _check(t, name, torch.int32, 1)
        if t.shape[0] != B:
            raise ValueError(f"{name}: one length per batch entry ({B}), got {t.shape[0]}")


def _check_bias(bias, B, H_q, S_q, S_kv):
    _check(bias, "bias", torch.bfloat16, 4)
    Bb, Hb = bias.shape[0], bias.shape[1]
    if tuple(bias.shape[2:]) != (S_q, S_kv) or Bb not in (1, B) or Hb not in (1, H_q):
        raise ValueError(f"bias must be [1 or {B}, 1 or {H_q}, {S_q}, {S_kv}], got {tuple(bias.shape)}")
    return Bb, Hb


def _check_rng(rng_state):
    """rng_state: a CUDA int64 (or uint64) tensor of two values, seed then offset."""
    if rng_state is None:
        raise ValueError("dropout needs rng_state: a CUDA int64 tensor [seed, offset]")
    if rng_state.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise TypeError(f"rng_state must be int64 or uint64, got {rng_state.dtype}")
    if tuple(rng_state.shape) != (2,) or not rng_state.is_contiguous() or not rng_state.is_cuda:
        raise ValueError("rng_state must be a contiguous CUDA tensor of shape [2] (seed, offset)")


def attn_fwd(q, k, v, o, lse, *, causal=True, window=-1, softmax_type=VANILLA, softmax_offset=None, scale=0.0,
             seq_lens_q=None, seq_lens_kv=None, bias=None, dropout_p=0.0, rng_state=None, stream=None):
    """Forward into preallocated o [B,S_q,H_q,d_v] bf16 and lse [B,H_q,S_q] fp32.

    seq_lens_q / seq_lens_kv: optional int32 [B] device tensors for a padded batch
    (attn_fwd_varlen); None means full length.
    bias: optional bf16 [1 or B, 1 or H_q, S_q, S_kv] added to the scaled scores
    (attn_fwd_bias).
    dropout_p, rng_state: attention dropout (attn_fwd_dropout); rng_state is a CUDA
    int64 tensor [seed, offset], to be passed to the backward of the same step too.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _check(t, n, torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
    B, S_q, H_q, d_qk = q.shape
    _, S_kv, H_kv, d_v = v.shape
    _check_lens(seq_lens_q, "seq_lens_q", B)
    _check_lens(seq_lens_kv, "seq_lens_kv", B)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, S_q, S_kv, H_q, H_kv, d_qk, d_v, float(scale or 0.0),
            int(bool(causal)), int(window), _stype(softmax_type), _ptr(softmax_offset))
    if dropout_p:
        if bias is not None or seq_lens_q is not None or seq_lens_kv is not None:
            raise ValueError("dropout with a bias or padded batches is not supported")
        _check_rng(rng_state)
        st = _load().attn_fwd_dropout(*args, float(dropout_p), _ptr(rng_state), _stream(stream))
    elif bias is not None:
        Bb, Hb = _check_bias(bias, B, H_q, S_q, S_kv)
        if seq_lens_q is None and seq_lens_kv is None:
            st = _load().attn_fwd_bias(*args[:5], _ptr(bias), Bb, Hb, *args[5:], _stream(stream))
        else:
            st = _load().attn_fwd_varlen_bias(*args[:5], _ptr(bias), Bb, Hb, *args[5:], _ptr(seq_lens_q),
                                              _ptr(seq_lens_kv), _stream(stream))
    elif seq_lens_q is None and seq_lens_kv is None:
        st = _load().attn_fwd(*args, _stream(stream))
    else:
        st = _load().attn_fwd_varlen(*args, _ptr(seq_lens_q), _ptr(seq_lens_kv), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd")


def attn_bwd_workspace_size(B, S_q, S_kv, H_q, H_kv, d_qk, d_v, deterministic=True) -> int:
    return int(_load().attn_bwd_workspace_size(B, S_q, S_kv, H_q, H_kv, d_qk, d_v, int(bool(deterministic))))


def attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_offset=None, *, causal=True, window=-1, softmax_type=VANILLA,
             softmax_offset=None, scale=0.0, deterministic=True, workspace=None, seq_lens_q=None, seq_lens_kv=None,
             bias=None, dbias=None, dropout_p=0.0, rng_state=None, stream=None):
    """Backward into preallocated dq, dk, dv (bf16) and d_offset (fp32 [H_q], learnable).

    seq_lens_q / seq_lens_kv as for attn_fwd (attn_bwd_varlen).  bias as for attn_fwd,
    with dbias an optional preallocated fp32 tensor of the bias's shape
    (attn_bwd_bias).  dropout_p / rng_state as for attn_fwd (attn_bwd_dropout; the
    forward's values).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    B, S_q, H_q, d_qk = q.shape
    _, S_kv, H_kv, d_v = v.shape
    _check_lens(seq_lens_q, "seq_lens_q", B)
    _check_lens(seq_lens_kv, "seq_lens_kv", B)
    need = attn_bwd_workspace_size(B, S_q, S_kv, H_q, H_kv, d_qk, d_v, deterministic)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(d_offset),
            B, S_q, S_kv, H_q, H_kv, d_qk, d_v, float(scale or 0.0), int(bool(causal)), int(window),
            _stype(softmax_type), _ptr(softmax_offset))
    tail = (int(bool(deterministic)), _ptr(workspace), workspace.numel(), _stream(stream))
    if dropout_p:
        if bias is not None or seq_lens_q is not None or seq_lens_kv is not None:
            raise ValueError("dropout with a bias or padded batches is not supported")
        _check_rng(rng_state)
        st = _load().attn_bwd_dropout(*args, float(dropout_p), _ptr(rng_state), *tail)
    elif bias is not None:
        Bb, Hb = _check_bias(bias, B, H_q, S_q, S_kv)
        if dbias is not None:
            _check(dbias, "dbias", torch.float32, 4)
            if dbias.shape != bias.shape:
                raise ValueError("dbias must have the bias's shape")
        if seq_lens_q is None and seq_lens_kv is None:
            st = _load().attn_bwd_bias(*args[:10], _ptr(bias), Bb, Hb, _ptr(dbias), *args[10:], *tail)
        else:
            st = _load().attn_bwd_varlen_bias(*args[:10], _ptr(bias), Bb, Hb, _ptr(dbias), *args[10:],
                                              _ptr(seq_lens_q), _ptr(seq_lens_kv), *tail)
    elif seq_lens_q is None and seq_lens_kv is None:
        st = _load().attn_bwd(*args, *tail)
    else:
        st = _load().attn_bwd_varlen(*args, _ptr(seq_lens_q), _ptr(seq_lens_kv), *tail)
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd")


def attn_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, d_offset=None, *, causal=True, window=-1,
                     softmax_type=VANILLA, softmax_offset=None, scale=0.0, stream=None):
    """attn_bwd without a workspace: for callers that must not allocate device memory.

    The library keeps the scratch in a fixed built-in array (see
    attn_bwd_noalloc_max_scratch_bytes); this function allocates nothing either.
    Always the deterministic backward.  Calls that overlap on the GPU race on the
    shared array; the first call on a device must come before any stream capture.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    B, S_q, H_q, d_qk = q.shape
    _, S_kv, H_kv, d_v = v.shape
    st = _load().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                                  _ptr(dv), _ptr(d_offset), B, S_q, S_kv, H_q, H_kv, d_qk, d_v, float(scale or 0.0),
                                  int(bool(causal)), int(window), _stype(softmax_type), _ptr(softmax_offset),
                                  _stream(stream))
    if st != ATTN_OK:
        msg = _load().attn_bwd_noalloc_message().decode()
        raise AttnError(st, "attn_bwd_noalloc" + (f" ({msg})" if msg else ""))


def attn_bwd_noalloc_max_scratch_bytes() -> int:
    return int(_load().attn_bwd_noalloc_max_scratch_bytes())


def attn_bwd_noalloc_message() -> str:
    return _load().attn_bwd_noalloc_message().decode()


def attn_fwd_varlen(q, k, v, o, lse, seq_lens_q, seq_lens_kv, **kw):
    """attn_fwd on a padded batch: int32 [B] device tensors of query / key lengths."""
    attn_fwd(q, k, v, o, lse, seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv, **kw)


def attn_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, d_offset, seq_lens_q, seq_lens_kv, **kw):
    """attn_bwd on a padded batch (lengths as for attn_fwd_varlen)."""
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_offset, seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv, **kw)


def attn_fwd_varlen_bias(q, k, v, o, lse, bias, seq_lens_q, seq_lens_kv, **kw):
    """attn_fwd with an additive bias on a padded batch (entry b uses the top-left
    [Lq[b], Lkv[b]] corner of its bias planes)."""
    attn_fwd(q, k, v, o, lse, bias=bias, seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv, **kw)


def attn_bwd_varlen_bias(q, k, v, o, dout, lse, dq, dk, dv, d_offset, bias, dbias, seq_lens_q, seq_lens_kv, **kw):
    """attn_bwd with an additive bias on a padded batch; dbias is zero outside each
    entry's corner."""
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_offset, bias=bias, dbias=dbias, seq_lens_q=seq_lens_q,
             seq_lens_kv=seq_lens_kv, **kw)


def attn_fwd_dropout(q, k, v, o, lse, dropout_p, rng_state, **kw):
    """attn_fwd with attention dropout: probability dropout_p, rng_state a CUDA int64
    tensor [seed, offset]."""
    attn_fwd(q, k, v, o, lse, dropout_p=dropout_p, rng_state=rng_state, **kw)


def attn_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, d_offset, dropout_p, rng_state, **kw):
    """attn_bwd of a forward with attention dropout (the forward's dropout_p and rng_state)."""
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_offset, dropout_p=dropout_p, rng_state=rng_state, **kw)


def attn_fwd_bias(q, k, v, o, lse, bias, **kw):
    """attn_fwd with an additive bf16 bias [1 or B, 1 or H_q, S_q, S_kv]."""
    attn_fwd(q, k, v, o, lse, bias=bias, **kw)


def attn_bwd_bias(q, k, v, o, dout, lse, dq, dk, dv, d_offset, bias, dbias, **kw):
    """attn_bwd with an additive bias; dbias: fp32 tensor of the bias's shape, or None."""
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_offset, bias=bias, dbias=dbias, **kw)


KERNEL_CLASSES = ("fwd", "bwd_preprocess", "bwd_kv", "bwd_q", "bwd_dq_convert", "fp8_quantize", "kv4", "rope")


def attn_timing_enable(on: bool = True) -> None:
    _load().attn_timing_enable(int(bool(on)))


def attn_timing_read():
    """{class: (milliseconds, kernel launches)} accumulated since the last read."""
    n = len(KERNEL_CLASSES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    st = _load().attn_timing_read(ms, cnt, n)
    if st != ATTN_OK:
        raise AttnError(st, "attn_timing_read")
    return {name: (ms[k], cnt[k]) for k, name in enumerate(KERNEL_CLASSES)}


# ----------------------------------------------------------------------------- FP8 (E4M3) forward


def attn_fp8_vt_row_bytes(S: int) -> int:
    return int(_load().attn_fp8_vt_row_bytes(int(S)))


def attn_fp8_amax(x, amax, *, stream=None):
    """amax (fp32 [1], device) = max |x| over the bf16 tensor x."""
    if x.dtype != torch.bfloat16 or not x.is_contiguous() or not x.is_cuda:
        raise TypeError("x must be a contiguous bf16 CUDA tensor")
    _check(amax, "amax", torch.float32, 1)
    st = _load().attn_fp8_amax(_ptr(x), x.numel(), _ptr(amax), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fp8_amax")


def _fp8_quantize(name, x, x8, amax, descale, transpose, amax_out, stream):
    _check(x, "x", torch.bfloat16, 4)
    _check(x8, "x8", torch.uint8, 4)
    _check(amax, "amax", torch.float32, 1)
    _check(descale, "descale", torch.float32, 1)
    B, S, H, d = x.shape
    want = (B, H, d, attn_fp8_vt_row_bytes(S)) if transpose else (B, S, H, d)
    if tuple(x8.shape) != want:
        raise ValueError(f"x8 must have shape {want}, got {tuple(x8.shape)}")
    if amax_out is not None:
        _check(amax_out, "amax_out", torch.float32, 1)
    st = getattr(_load(), name)(_ptr(x), _ptr(x8), B, S, H, d, int(bool(transpose)), _ptr(amax), _ptr(descale),
                                _ptr(amax_out), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, name)


def attn_fp8_quantize(x, x8, amax, descale, *, transpose=False, amax_out=None, stream=None):
    """x8 (uint8 E4M3) = E4M3(x * 448 / amax); descale (fp32 [1]) = amax / 448 as 1 / scale.

    x bf16 BSHD [B,S,H,d]; x8 the same shape, or [B,H,d,S_pad] with transpose=True.
    amax_out (fp32 [1], optional): records max |x| during the same pass."""
    _fp8_quantize("attn_fp8_quantize", x, x8, amax, descale, transpose, amax_out, stream)


def attn_fp8_quantize_e5m2(x, x8, amax, descale, *, transpose=False, amax_out=None, stream=None):
    """attn_fp8_quantize with E5M2 codes: x8 = E5M2(x * 57344 / amax)."""
    _fp8_quantize("attn_fp8_quantize_e5m2", x, x8, amax, descale, transpose, amax_out, stream)


def attn_fp8_quantize_both(x, x8, x8t, amax, descale, *, e5m2=False, amax_out=None, stream=None):
    """One read of x, both layouts: x8 BSHD [B,S,H,d] and x8t [B,H,d,S_pad] (uint8), E4M3 or
    (e5m2=True) E5M2, with the same codes as the two separate casts."""
    _check(x, "x", torch.bfloat16, 4)
    _check(x8, "x8", torch.uint8, 4)
    _check(x8t, "x8t", torch.uint8, 4)
    _check(amax, "amax", torch.float32, 1)
    _check(descale, "descale", torch.float32, 1)
    B, S, H, d = x.shape
    if tuple(x8.shape) != (B, S, H, d):
        raise ValueError(f"x8 must have shape {(B, S, H, d)}, got {tuple(x8.shape)}")
    want = (B, H, d, attn_fp8_vt_row_bytes(S))
    if tuple(x8t.shape) != want:
        raise ValueError(f"x8t must have shape {want}, got {tuple(x8t.shape)}")
    if amax_out is not None:
        _check(amax_out, "amax_out", torch.float32, 1)
    st = _load().attn_fp8_quantize_both(_ptr(x), _ptr(x8), _ptr(x8t), B, S, H, d, int(bool(e5m2)), _ptr(amax),
                                        _ptr(descale), _ptr(amax_out), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fp8_quantize_both")


def fp8_quantize_both(x, *, amax=None, amax_out=None, fmt="e4m3", stream=None):
    """fp8_quantize in both layouts from one read: returns (x8, x8t, amax, descale)."""
    if fmt not in ("e4m3", "e5m2"):
        raise ValueError(f"fmt must be 'e4m3' or 'e5m2', got {fmt!r}")
    B, S, H, d = x.shape
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
        attn_fp8_amax(x, amax, stream=stream)
    x8 = torch.empty((B, S, H, d), dtype=torch.uint8, device=x.device)
    x8t = torch.empty((B, H, d, attn_fp8_vt_row_bytes(S)), dtype=torch.uint8, device=x.device)
    descale = torch.empty(1, dtype=torch.float32, device=x.device)
    attn_fp8_quantize_both(x, x8, x8t, amax, descale, e5m2=(fmt == "e5m2"), amax_out=amax_out, stream=stream)
    return x8, x8t, amax, descale


def attn_fwd_fp8(q8, k8, vt8, descale_q, descale_k, descale_v, o, lse, *, causal=True, window=-1,
                 softmax_type=VANILLA, softmax_offset=None, scale=0.0, stream=None):
    """E4M3 forward into preallocated o [B,S_q,H_q,d] bf16 and lse [B,H_q,S_q] fp32.

    q8 [B,S_q,H_q,d], k8 [B,S_kv,H_kv,d] uint8 E4M3 BSHD; vt8 [B,H_kv,d,S_pad] from
    attn_fp8_quantize(transpose=True); descale_* fp32 [1] device tensors."""
    for t, n in ((q8, "q8"), (k8, "k8"), (vt8, "vt8")):
        _check(t, n, torch.uint8, 4)
    for t, n in ((descale_q, "descale_q"), (descale_k, "descale_k"), (descale_v, "descale_v")):
        _check(t, n, torch.float32, 1)
    _check(o, "o", torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
    B, S_q, H_q, d = q8.shape
    _, S_kv, H_kv, _ = k8.shape
    if tuple(vt8.shape) != (B, H_kv, d, attn_fp8_vt_row_bytes(S_kv)):
        raise ValueError(f"vt8 must have shape {(B, H_kv, d, attn_fp8_vt_row_bytes(S_kv))}, got {tuple(vt8.shape)}")
    st = _load().attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(descale_q), _ptr(descale_k), _ptr(descale_v),
                              _ptr(o), _ptr(lse), B, S_q, S_kv, H_q, H_kv, d, float(scale or 0.0),
                              int(bool(causal)), int(window), _stype(softmax_type), _ptr(softmax_offset),
                              _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_fp8")


def fp8_quantize(x, *, transpose=False, amax=None, amax_out=None, fmt="e4m3", stream=None):
    """Per-tensor E4M3 (fmt="e5m2": E5M2) quantisation of a bf16 BSHD tensor: returns
    (x8, amax, descale).

    amax: an fp32 [1] device tensor holding the scaling statistic (for example the
    max of an amax history); None computes this tensor's own amax first (a second
    pass).  amax_out: optional fp32 [1] device tensor that records this tensor's
    amax during the cast (delayed scaling)."""
    if fmt not in ("e4m3", "e5m2"):
        raise ValueError(f"fmt must be 'e4m3' or 'e5m2', got {fmt!r}")
    B, S, H, d = x.shape
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
        attn_fp8_amax(x, amax, stream=stream)
    shape = (B, H, d, attn_fp8_vt_row_bytes(S)) if transpose else (B, S, H, d)
    x8 = torch.empty(shape, dtype=torch.uint8, device=x.device)
    descale = torch.empty(1, dtype=torch.float32, device=x.device)
    quant = attn_fp8_quantize_e5m2 if fmt == "e5m2" else attn_fp8_quantize
    quant(x, x8, amax, descale, transpose=transpose, amax_out=amax_out, stream=stream)
    return x8, amax, descale


def sdpa_forward_fp8(q, k, v, *, causal=True, window=-1, softmax_type=VANILLA, softmax_offset=None, scale=0.0,
                     stream=None):
    """bf16 in, bf16 out through the E4M3 forward: quantise Q, K (BSHD) and V
    (transposed) with their own amax, then run attn_fwd_fp8.  Returns (o, lse)."""
    q8, _, dq = fp8_quantize(q, stream=stream)
    k8, _, dk = fp8_quantize(k, stream=stream)
    vt8, _, dv = fp8_quantize(v, transpose=True, stream=stream)
    B, S_q, H_q, d = q.shape
    o = torch.empty((B, S_q, H_q, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H_q, S_q), dtype=torch.float32, device=q.device)
    attn_fwd_fp8(q8, k8, vt8, dq, dk, dv, o, lse, causal=causal, window=window, softmax_type=softmax_type,
                 softmax_offset=softmax_offset, scale=scale, stream=stream)
    return o, lse


def attn_bwd_fp8_workspace_size(B, S_q, H_q) -> int:
    return int(_load().attn_bwd_fp8_workspace_size(int(B), int(S_q), int(H_q)))


def attn_bwd_fp8(q8, k8, v8, do8, qt8, kt8, dot8, descale_q, descale_k, descale_v, descale_do, o, lse, ds_amax,
                 dq, dk, dv, d_offset=None, *, ds_amax_out=None, causal=True, window=-1, softmax_type=VANILLA,
                 softmax_offset=None, scale=0.0, workspace=None, stream=None):
    """FP8 backward into preallocated bf16 dq, dk, dv (BSHD) and d_offset (fp32 [H_q],
    learnable sinks).  q8, k8, v8 uint8 E4M3 BSHD; do8 uint8 E5M2 BSHD; qt8, dot8
    [B,H_q,d,S_pad(S_q)] and kt8 [B,H_kv,d,S_pad(S_kv)] the same codes transposed;
    o, lse the forward's outputs; descale_*, ds_amax (s = 57344 / ds_amax for dS) and
    ds_amax_out (receives max |dS|) fp32 [1] device tensors."""
    for t, n in ((q8, "q8"), (k8, "k8"), (v8, "v8"), (do8, "do8"), (qt8, "qt8"), (kt8, "kt8"), (dot8, "dot8")):
        _check(t, n, torch.uint8, 4)
    for t, n in ((descale_q, "descale_q"), (descale_k, "descale_k"), (descale_v, "descale_v"),
                 (descale_do, "descale_do"), (ds_amax, "ds_amax")):
        _check(t, n, torch.float32, 1)
    if ds_amax_out is not None:
        _check(ds_amax_out, "ds_amax_out", torch.float32, 1)
    for t, n in ((o, "o"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
    if d_offset is not None:
        _check(d_offset, "d_offset", torch.float32, 1)
    B, S_q, H_q, d = q8.shape
    _, S_kv, H_kv, _ = k8.shape
    want = {"qt8": (B, H_q, d, attn_fp8_vt_row_bytes(S_q)), "dot8": (B, H_q, d, attn_fp8_vt_row_bytes(S_q)),
            "kt8": (B, H_kv, d, attn_fp8_vt_row_bytes(S_kv))}
    for t, n in ((qt8, "qt8"), (dot8, "dot8"), (kt8, "kt8")):
        if tuple(t.shape) != want[n]:
            raise ValueError(f"{n} must have shape {want[n]}, got {tuple(t.shape)}")
    for t, n, shp in ((v8, "v8", k8.shape), (do8, "do8", q8.shape), (o, "o", q8.shape), (dq, "dq", q8.shape),
                      (dk, "dk", k8.shape), (dv, "dv", k8.shape)):
        if tuple(t.shape) != tuple(shp):
            raise ValueError(f"{n} must have shape {tuple(shp)}, got {tuple(t.shape)}")
    need = attn_bwd_fp8_workspace_size(B, S_q, H_q)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q8.device)
    st = _load().attn_bwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(do8), _ptr(qt8), _ptr(kt8), _ptr(dot8),
                              _ptr(descale_q), _ptr(descale_k), _ptr(descale_v), _ptr(descale_do), _ptr(o), _ptr(lse),
                              _ptr(ds_amax), _ptr(ds_amax_out), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(d_offset), B, S_q,
                              S_kv, H_q, H_kv, d, float(scale or 0.0), int(bool(causal)), int(window),
                              _stype(softmax_type), _ptr(softmax_offset), _ptr(workspace), workspace.numel(),
                              _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_fp8")


def sdpa_backward_fp8(q, k, v, o, dout, lse, *, ds_amax=None, ds_amax_out=None, causal=True, window=-1,
                      softmax_type=VANILLA, softmax_offset=None, scale=0.0, stream=None):
    """bf16 in, bf16 out through the FP8 backward: quantise Q, K, V (E4M3) and dO (E5M2)
    with their own amax, natural and transposed, then run attn_bwd_fp8.  ds_amax: the
    dS scaling statistic (fp32 [1] device tensor, e.g. the max of an amax history);
    None runs the backward twice, the first time only to record this step's max |dS|.
    Returns (dq, dk, dv, d_offset)."""
    q8, qt8, _, sq = fp8_quantize_both(q, stream=stream)
    k8, kt8, _, sk = fp8_quantize_both(k, stream=stream)
    v8, _, sv = fp8_quantize(v, stream=stream)
    do8, dot8, _, sdo = fp8_quantize_both(dout, fmt="e5m2", stream=stream)
    B, S_q, H_q, d = q.shape
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    d_offset = torch.empty(H_q, dtype=torch.float32, device=q.device)
    kw = dict(causal=causal, window=window, softmax_type=softmax_type, softmax_offset=softmax_offset, scale=scale,
              stream=stream)
    if ds_amax is None:
        ds_amax = torch.empty(1, dtype=torch.float32, device=q.device)
        first = torch.ones(1, dtype=torch.float32, device=q.device)
        attn_bwd_fp8(q8, k8, v8, do8, qt8, kt8, dot8, sq, sk, sv, sdo, o, lse, first, dq, dk, dv, d_offset,
                     ds_amax_out=ds_amax, **kw)
    attn_bwd_fp8(q8, k8, v8, do8, qt8, kt8, dot8, sq, sk, sv, sdo, o, lse, ds_amax, dq, dk, dv, d_offset,
                 ds_amax_out=ds_amax_out, **kw)
    return dq, dk, dv, d_offset


# ----------------------------------------------------------------------------- packed sequences


def _p(t):
    return 0 if t is None else t.data_ptr()


def _device_of(*tensors):
    """The one CUDA device of the tensors (None skipped), as its number."""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if dev >= 0 or i < 0:
                    raise ValueError(f"tensors on different devices, or not on a CUDA device: {t.device} and others")
                dev = i
    return dev


@contextlib.contextmanager
def _on(dev, stream):
    """Device `dev` current, and new tensors belonging to the stream that the call runs on."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _elsewhere(dev, stream):
    """Whether a call has to leave the current device or stream to allocate its tensors."""
    return stream is not None or dev != torch.cuda.current_device()


def _window(window):
    """The window as a C int: one past 32 bits must not wrap into a small one."""
    w = int(window)
    return w if -1 <= w <= 0x7fffffff else -1 if w < 0 else 0x7fffffff


def _raw_stream(dev, stream):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _check_cu(cu, name, B=None):
    _check(cu, name, torch.int32, 1)
    if cu.shape[0] < 1 or (B is not None and cu.shape[0] != B + 1):
        raise ValueError(f"{name} must hold one offset per sequence and the end"
                         + (f" ({B + 1} values)" if B is not None else "") + f", got {cu.shape[0]}")


@functools.lru_cache(maxsize=1024)
def attn_packed_workspace_size(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, backward=False) -> int:
    return int(_load().attn_packed_workspace_size(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, int(bool(backward))))


def _check_packed(q, k, v, cu_q, cu_kv, softmax_offset):
    """Checks shared by the packed calls; returns (B, T_q, T_kv, H_q, H_kv, d_qk, d_v)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 3)
    T_q, H_q, d_qk = q.shape
    T_kv, H_kv, d_v = v.shape
    if k.shape != (T_kv, H_kv, d_qk):
        raise ValueError(f"k must be {(T_kv, H_kv, d_qk)} (v's rows and heads, q's head dim), got {tuple(k.shape)}")
    _check_cu(cu_q, "cu_seqlens_q")
    B = cu_q.shape[0] - 1
    if cu_kv is not None:
        _check_cu(cu_kv, "cu_seqlens_kv", B)
    elif T_q != T_kv:
        raise ValueError(f"without cu_seqlens_kv the keys share the queries' offsets: {T_q} and {T_kv} rows")
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
        if softmax_offset.shape[0] != H_q:
            raise ValueError(f"softmax_offset must have one value per query head ({H_q})")
    return B, T_q, T_kv, H_q, H_kv, d_qk, d_v


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _check(workspace, "workspace", torch.uint8, 1)
    return workspace


def attn_fwd_packed(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv=None, *, causal=True, window=-1,
                    softmax_type=VANILLA, softmax_offset=None, scale=0.0, zero_rest=False, workspace=None,
                    stream=None):
    """Forward over packed sequences into preallocated o [T_q, H_q, d_v] bf16 and lse [H_q, T_q]
    fp32: q [T_q, H_q, d_qk], k [T_kv, H_kv, d_qk], v [T_kv, H_kv, d_v].

    cu_seqlens_q / cu_seqlens_kv: int32 [B+1] on the device, sequence b's rows are
    cu_seqlens[b] .. cu_seqlens[b+1] - 1 (cu_seqlens_kv None: the queries' offsets).  Rows of no
    sequence are left alone, or zeroed with zero_rest (lse -inf).  workspace: uint8 of
    attn_packed_workspace_size() bytes or more, not shared with a call that may run at the
    same time (None: a new one)."""
    sizes = _check_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset)
    _, T_q, _, H_q, _, _, d_v = sizes
    _check(o, "o", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    if tuple(o.shape) != (T_q, H_q, d_v) or tuple(lse.shape) != (H_q, T_q):
        raise ValueError(f"o must be {(T_q, H_q, d_v)} and lse {(H_q, T_q)}, got {tuple(o.shape)}, {tuple(lse.shape)}")
    dev = _device_of(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_fwd_packed(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, causal=causal, window=window,
                                   softmax_type=softmax_type, softmax_offset=softmax_offset, scale=scale,
                                   zero_rest=zero_rest, workspace=workspace)
    _run_fwd_packed(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, sizes, dev, causal, window, softmax_type,
                    softmax_offset, scale, zero_rest, workspace)


# The _run_* functions: the call itself, on the current stream of the current device `dev`, of checked
# arguments.  The calls that allocate their results come here too, past checks of tensors they made.
def _run_fwd_packed(q, k, v, o, lse, cu_q, cu_kv, sizes, dev, causal, window, softmax_type, softmax_offset, scale,
                    zero_rest, workspace):
    ws = _workspace(workspace, attn_packed_workspace_size(*sizes) if workspace is None else 0, q.device)
    st = _load().attn_fwd_packed(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_q), _p(cu_kv), *sizes,
                                 float(scale or 0.0), int(bool(causal)), _window(window), _stype(softmax_type),
                                 _p(softmax_offset), int(bool(zero_rest)), _p(ws), ws.numel(),
                                 _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_packed")


def _check_bwd_packed(q, k, v, o, dout, lse, cu_q, cu_kv, softmax_offset):
    sizes = _check_packed(q, k, v, cu_q, cu_kv, softmax_offset)
    _, T_q, _, H_q, _, _, d_v = sizes
    _check(lse, "lse", torch.float32, 2)
    if lse.shape != (H_q, T_q):
        raise ValueError(f"lse must be {(H_q, T_q)}, got {tuple(lse.shape)}")
    for t, n in ((o, "o"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 3)
        if t.shape != (T_q, H_q, d_v):
            raise ValueError(f"{n} must be {(T_q, H_q, d_v)}, got {tuple(t.shape)}")
    return sizes


def attn_bwd_packed(q, k, v, o, dout, lse, dq, dk, dv, d_offset, cu_seqlens_q, cu_seqlens_kv=None, *, causal=True,
                    window=-1, softmax_type=VANILLA, softmax_offset=None, scale=0.0, zero_rest=False, workspace=None,
                    stream=None):
    """Backward of attn_fwd_packed into preallocated dq, dk, dv (bf16, shapes of q, k, v) and
    d_offset (fp32 [H_q]; learnable sinks, else None).  Bitwise reproducible."""
    sizes = _check_bwd_packed(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv, softmax_offset)
    for t, n, of in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _check(t, n, torch.bfloat16, 3)
        if t.shape != of.shape:
            raise ValueError(f"{n} must be {tuple(of.shape)}, got {tuple(t.shape)}")
    if d_offset is not None:
        _check(d_offset, "d_offset", torch.float32, 1)
        if d_offset.shape[0] != q.shape[1]:
            raise ValueError(f"d_offset must have one value per query head ({q.shape[1]})")
    dev = _device_of(q, k, v, o, dout, lse, dq, dk, dv, d_offset, cu_seqlens_q, cu_seqlens_kv, softmax_offset,
                     workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_bwd_packed(q, k, v, o, dout, lse, dq, dk, dv, d_offset, cu_seqlens_q, cu_seqlens_kv,
                                   causal=causal, window=window, softmax_type=softmax_type,
                                   softmax_offset=softmax_offset, scale=scale, zero_rest=zero_rest,
                                   workspace=workspace)
    _run_bwd_packed(q, k, v, o, dout, lse, dq, dk, dv, d_offset, cu_seqlens_q, cu_seqlens_kv, sizes, dev, causal,
                    window, softmax_type, softmax_offset, scale, zero_rest, workspace)


def _run_bwd_packed(q, k, v, o, dout, lse, dq, dk, dv, d_offset, cu_q, cu_kv, sizes, dev, causal, window, softmax_type,
                    softmax_offset, scale, zero_rest, workspace):
    ws = _workspace(workspace, attn_packed_workspace_size(*sizes, True) if workspace is None else 0, q.device)
    st = _load().attn_bwd_packed(_p(q), _p(k), _p(v), _p(o), _p(dout), _p(lse), _p(dq), _p(dk), _p(dv), _p(d_offset),
                                 _p(cu_q), _p(cu_kv), *sizes, float(scale or 0.0), int(bool(causal)),
                                 _window(window), _stype(softmax_type), _p(softmax_offset), int(bool(zero_rest)), _p(ws),
                                 ws.numel(), _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_packed")


def sdpa_forward_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv=None, *, causal=True, window=-1, softmax_type=VANILLA,
                        softmax_offset=None, scale=0.0, workspace=None, stream=None):
    """Allocate O and LSE, run attn_fwd_packed, return (o, lse); rows of no sequence are zero (lse
    -inf)."""
    sizes = _check_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset)
    dev = _device_of(q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return sdpa_forward_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv, causal=causal, window=window,
                                       softmax_type=softmax_type, softmax_offset=softmax_offset, scale=scale,
                                       workspace=workspace)
    _, T_q, _, H_q, _, _, d_v = sizes
    o = torch.empty((T_q, H_q, d_v), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H_q, T_q), dtype=torch.float32, device=q.device)
    _run_fwd_packed(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, sizes, dev, causal, window, softmax_type,
                    softmax_offset, scale, True, workspace)
    return o, lse


def sdpa_backward_packed(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv=None, *, causal=True, window=-1,
                         softmax_type=VANILLA, softmax_offset=None, scale=0.0, workspace=None, stream=None):
    """Allocate dQ, dK, dV (and d_offset for the learnable sink), run attn_bwd_packed, return
    them; gradients of rows of no sequence are zero."""
    sizes = _check_bwd_packed(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv, softmax_offset)
    dev = _device_of(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return sdpa_backward_packed(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv, causal=causal,
                                        window=window, softmax_type=softmax_type, softmax_offset=softmax_offset,
                                        scale=scale, workspace=workspace)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    d_off = (torch.empty((q.shape[1],), dtype=torch.float32, device=q.device)
             if _stype(softmax_type) == LEARNABLE else None)
    _run_bwd_packed(q, k, v, o, dout, lse, dq, dk, dv, d_off, cu_seqlens_q, cu_seqlens_kv, sizes, dev, causal, window,
                    softmax_type, softmax_offset, scale, True, workspace)
    return dq, dk, dv, d_off


class SDPAPackedFunction(torch.autograd.Function):
    """autograd wrapper of the packed entry points."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset, causal, window, softmax_type, scale):
        ctx.kw = dict(causal=causal, window=window, softmax_type=softmax_type, scale=scale)
        o, lse = sdpa_forward_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset=softmax_offset, **ctx.kw)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, softmax_offset)
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse, cu_q, cu_kv, off = ctx.saved_tensors
        dq, dk, dv, d_off = sdpa_backward_packed(q, k, v, o, dout.contiguous(), lse, cu_q, cu_kv, softmax_offset=off,
                                                 **ctx.kw)
        return dq, dk, dv, None, None, d_off, None, None, None, None


def attention_packed(q, k, v, cu_seqlens_q, cu_seqlens_kv=None, softmax_offset=None, *, causal=True, window=-1,
                     softmax_type=VANILLA, scale=0.0, rope=None, rope_interleaved=False, rope_first_dim=0):
    """Differentiable attention over packed sequences: q [T_q, H_q, d_qk], k [T_kv, H_kv, d_qk],
    v [T_kv, H_kv, d_v]; q, k, v and the learnable offset receive gradients.  rope: a table of the rows'
    positions (rope_table), by which q and k (of the same rows) are rotated first."""
    if rope is not None:
        q, k = RopeFunction.apply(q, k, rope, bool(rope_interleaved), int(rope_first_dim))
    return SDPAPackedFunction.apply(q, k, v, cu_seqlens_q, cu_seqlens_kv, softmax_offset, causal, window,
                                    softmax_type, scale)


# ----------------------------------------------------------------------------- 4-bit paged cache


def kv4_pool(n_pages, H_kv, d, page_size, *, n_layers=None, device="cuda"):
    """A pool of pages of the 4-bit cache: uint8 [n_pages, H_kv, block] (with n_layers, one such
    pool per layer: [n_layers, n_pages, H_kv, block]).  Its contents need no initialisation."""
    block = kv4_block_bytes(page_size, d)
    shape = (n_pages, H_kv, block) if n_layers is None else (n_layers, n_pages, H_kv, block)
    return torch.empty(shape, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=64)
def attn_kv4_block_bytes(page_size, d) -> int:
    return int(_load().attn_kv4_block_bytes(int(page_size), int(d)))


def kv4_block_bytes(page_size, d) -> int:
    """Bytes of one page and kv head: page_size tokens of K and V at 4.5 bits a value."""
    n = attn_kv4_block_bytes(page_size, d)
    if n == 0:
        raise ValueError(f"page_size must be 16, 32, 64 or 128 and d 64 or 128, got {page_size} and {d}")
    return n


def _check_paged(pool, page_table, seq_lens, d):
    """Checks of a pool [n_pages, H_kv, block] with its page table and lengths; returns the
    sizes (B, n_pages, H_kv, page_size, max_pages)."""
    _check(pool, "pool", torch.uint8, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    n_pages, H_kv, block = pool.shape
    page_size = block * 8 // (9 * d) if d else 0
    if kv4_block_bytes(page_size, d) != block:
        raise ValueError(f"pool must be [n_pages, H_kv, kv4_block_bytes(page_size, {d})], got {tuple(pool.shape)}")
    B, max_pages = page_table.shape
    if seq_lens.shape[0] != B:
        raise ValueError(f"seq_lens: one length per row of page_table ({B}), got {seq_lens.shape[0]}")
    return B, n_pages, H_kv, page_size, max_pages


def _check_rows(t, name, H, d):
    """A packed bf16 tensor [T, H, d] whose rows may be apart (a slice of a fused projection)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != d:
        raise ValueError(f"{name} must be [T, {H}, {d}], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape[0] == 0:
        return H * d
    if (t.stride(2) != 1 and d > 1) or (t.stride(1) != d and H > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride = t.stride(0) if t.shape[0] > 1 else H * d
    if stride < H * d or stride % 8:
        raise ValueError(f"{name}: rows must not overlap and must be a multiple of 8 elements apart, got {stride}")
    return stride


def attn_kv4_append(k, v, cu_seqlens, pool, page_table, seq_lens, *, stream=None):
    """Quantise packed keys and values (bf16 [T, H_kv, d]) into the pages of a 4-bit cache.

    Rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (int32 [B+1] on the device) become tokens
    seq_lens[b], seq_lens[b] + 1, ... of sequence b (int32 [B]: its length before the call).
    pool: uint8 [n_pages, H_kv, block] (kv4_pool); page_table: int32 [B, max_pages].  The rows
    of k and v may be apart, as in a slice of a fused projection."""
    if k.dim() != 3:
        raise ValueError(f"k must be [T, H_kv, d], got shape {tuple(k.shape)}")
    T, _, d = k.shape
    B, n_pages, H_kv, page_size, max_pages = _check_paged(pool, page_table, seq_lens, d)
    ks, vs = _check_rows(k, "k", H_kv, d), _check_rows(v, "v", H_kv, d)
    if v.shape[0] != T:
        raise ValueError(f"k and v must have the same rows, got {T} and {v.shape[0]}")
    _check_cu(cu_seqlens, "cu_seqlens", B)
    dev = _device_of(k, v, cu_seqlens, pool, page_table, seq_lens)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_append(k, v, cu_seqlens, pool, page_table, seq_lens)
    st = _load().attn_kv4_append(_p(k), _p(v), _p(cu_seqlens), _p(pool), _p(page_table), _p(seq_lens), B, T, H_kv, d,
                                 n_pages, page_size, max_pages, ks, vs, _raw_stream(dev, stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_append")


def attn_kv4_gather(pool, page_table, cu_seqlens, seq_lens, k, v, *, zero_rest=False, stream=None):
    """Read tokens of a 4-bit cache back into preallocated packed k, v (bf16 [T, H_kv, d]): row
    cu_seqlens[b] + i is token seq_lens[b] + i of sequence b.  Rows past cu_seqlens[B] are left
    alone, or zeroed with zero_rest."""
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    T, _, d = k.shape
    B, n_pages, H_kv, page_size, max_pages = _check_paged(pool, page_table, seq_lens, d)
    for t, n in ((k, "k"), (v, "v")):
        if tuple(t.shape) != (T, H_kv, d):
            raise ValueError(f"{n} must be {(T, H_kv, d)}, got {tuple(t.shape)}")
    _check_cu(cu_seqlens, "cu_seqlens", B)
    dev = _device_of(k, v, cu_seqlens, pool, page_table, seq_lens)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_gather(pool, page_table, cu_seqlens, seq_lens, k, v, zero_rest=zero_rest)
    st = _load().attn_kv4_gather(_p(pool), _p(page_table), _p(cu_seqlens), _p(seq_lens), _p(k), _p(v), B, T, H_kv, d,
                                 n_pages, page_size, max_pages, int(bool(zero_rest)), _raw_stream(dev, stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_gather")


def kv4_gather(pool, page_table, cu_seqlens, seq_lens, total, d, *, stream=None):
    """attn_kv4_gather into new tensors of `total` rows: returns (k, v), zeros in the rows of no
    sequence."""
    dev = _device_of(pool)
    if dev >= 0 and _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv4_gather(pool, page_table, cu_seqlens, seq_lens, total, d)
    k = torch.empty((int(total), pool.shape[-2], int(d)), dtype=torch.bfloat16, device=pool.device)
    v = torch.empty_like(k)
    attn_kv4_gather(pool, page_table, cu_seqlens, seq_lens, k, v, zero_rest=True)
    return k, v


@functools.lru_cache(maxsize=1024)
def attn_kv4_decode_workspace_size(B, S_q, H_q, H_kv, d) -> int:
    return int(_load().attn_kv4_decode_workspace_size(B, S_q, H_q, H_kv, d))


def _check_decode(q, pool, page_table, seq_lens, softmax_offset):
    """Checks of a decode's inputs; returns (B, S_q, H_q, H_kv, d, n_pages, page_size, max_pages)."""
    _check(q, "q", torch.bfloat16, 4)
    B, S_q, H_q, d = q.shape
    Bt, n_pages, H_kv, page_size, max_pages = _check_paged(pool, page_table, seq_lens, d)
    if Bt != B:
        raise ValueError(f"page_table must have one row per batch entry ({B}), got {Bt}")
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
        if softmax_offset.shape[0] != H_q:
            raise ValueError(f"softmax_offset must have one value per query head ({H_q})")
    return B, S_q, H_q, H_kv, d, n_pages, page_size, max_pages


def attn_kv4_decode(q, pool, page_table, seq_lens, o, lse=None, *, window=-1, softmax_type=VANILLA,
                    softmax_offset=None, scale=0.0, workspace=None, stream=None):
    """Attention of the S_q newest tokens of every sequence over its 4-bit cache, into
    preallocated o (bf16, q's shape [B, S_q, H_q, d]) and, if given, lse (fp32 [B, H_q, S_q]).

    seq_lens: int32 [B] on the device, tokens in the cache (the S_q newest among them); query
    s sits at seq_lens[b] - S_q + s and sees the keys up to its own place, with window >= 0
    the last window + 1 of them.  workspace: uint8 of attn_kv4_decode_workspace_size() bytes
    or more, not shared with a call that may run at the same time (None: a new one)."""
    sizes = _check_decode(q, pool, page_table, seq_lens, softmax_offset)
    B, S_q, H_q = sizes[:3]
    _check(o, "o", torch.bfloat16, 4)
    if o.shape != q.shape:
        raise ValueError(f"o must have q's shape {tuple(q.shape)}, got {tuple(o.shape)}")
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
        if lse.shape != (B, H_q, S_q):
            raise ValueError(f"lse must be {(B, H_q, S_q)}, got {tuple(lse.shape)}")
    dev = _device_of(q, pool, page_table, seq_lens, o, lse, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_decode(q, pool, page_table, seq_lens, o, lse, window=window, softmax_type=softmax_type,
                                   softmax_offset=softmax_offset, scale=scale, workspace=workspace)
    _run_kv4_decode(q, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type, softmax_offset, scale,
                    workspace)


def _run_kv4_decode(q, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type, softmax_offset, scale,
                    workspace):
    ws = _workspace(workspace, attn_kv4_decode_workspace_size(*sizes[:5]) if workspace is None else 0, q.device)
    st = _load().attn_kv4_decode(_p(q), _p(pool), _p(page_table), _p(seq_lens), _p(o), _p(lse), *sizes,
                                 float(scale or 0.0), _window(window), _stype(softmax_type), _p(softmax_offset),
                                 _p(ws), ws.numel(), _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_decode")


def sdpa_decode_kv4(q, pool, page_table, seq_lens, *, window=-1, softmax_type=VANILLA, softmax_offset=None, scale=0.0,
                    workspace=None, stream=None):
    """Allocate O and LSE, run attn_kv4_decode, return (o, lse)."""
    sizes = _check_decode(q, pool, page_table, seq_lens, softmax_offset)
    dev = _device_of(q, pool, page_table, seq_lens, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return sdpa_decode_kv4(q, pool, page_table, seq_lens, window=window, softmax_type=softmax_type,
                                   softmax_offset=softmax_offset, scale=scale, workspace=workspace)
    o = torch.empty_like(q)
    lse = torch.empty((sizes[0], sizes[2], sizes[1]), dtype=torch.float32, device=q.device)
    _run_kv4_decode(q, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type, softmax_offset, scale,
                    workspace)
    return o, lse


def _host_pages(pages, name):
    t = pages if isinstance(pages, torch.Tensor) else torch.tensor(pages)
    if t.dim() == 1 and t.numel() == 0:
        t = t.to(torch.int32)
    if t.is_cuda:
        raise ValueError(f"{name}: page numbers are read on the host; pass a list or a CPU tensor")
    if t.dtype not in (torch.int32, torch.int64) or t.dim() != 1:
        raise ValueError(f"{name} must be a one-dimensional list of whole numbers")
    if t.dtype == torch.int64:  # a number past 32 bits must not wrap into a page
        if t.numel() and (int(t.max()) > 0x7fffffff or int(t.min()) < -0x80000000):
            raise ValueError(f"{name}: page number out of range")
        t = t.to(torch.int32)
    return t.contiguous()


def attn_kv4_copy_pages(pool, src, dst, *, stream=None):
    """Copy page src[i] to page dst[i] for every i, in the pool [n_pages, H_kv, block] or in
    each layer of [n_layers, n_pages, H_kv, block]: a fork's partly filled last page, or the
    moves of a compaction.  src, dst: lists or CPU tensors, checked before anything is
    launched: a destination named twice, a page that is both source and destination, or a page
    outside the pool is refused."""
    if pool.dim() not in (3, 4):
        raise ValueError(f"pool must be [n_pages, H_kv, block] or [n_layers, n_pages, H_kv, block], got "
                         f"{tuple(pool.shape)}")
    _check(pool, "pool", torch.uint8, pool.dim())
    src, dst = _host_pages(src, "src"), _host_pages(dst, "dst")
    if src.shape != dst.shape:
        raise ValueError(f"src and dst must have the same length, got {src.shape[0]} and {dst.shape[0]}")
    n_layers = pool.shape[0] if pool.dim() == 4 else 1
    n_pages, H_kv, block = pool.shape[-3:]
    dev = _device_of(pool)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_copy_pages(pool, src, dst)
    st = _load().attn_kv4_copy_pages(_p(pool), n_layers, n_pages, H_kv * block, _p(src), _p(dst), src.shape[0],
                                     _raw_stream(dev, stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_copy_pages")


# ----------------------------------------------------------------------------- rotary positions


def rope_frequencies(rot_dim, *, base=10000.0, scaling="none", factor=1.0, original_length=None, slow_turns=1.0,
                     fast_turns=32.0, gain=None, device="cuda"):
    """The frequencies of rot_dim / 2 pairs (fp64 [rot_dim / 2] on `device`, radians a position) and
    the gain of their cosines and sines: returns (inv_freq, gain), to be kept for all steps.

    Pair f of n turns by base^(-f / n) a position.  For contexts `factor` times as long as the
    model was trained for, scaling is "linear" (every frequency divided by the factor), "base" (the
    base multiplied by factor^(n / (n - 1)): the slowest pair slows down by the factor, the
    fastest stays) or "parts" (pairs that turn slow_turns times or less in original_length positions are
    divided by the factor, those that turn fast_turns times or more stay, those between are
    blended by the logarithm of their turns, not rounded to whole pairs; the gain is 0.1 ln(factor) + 1).
    gain: another one.  A model whose frequencies are blended otherwise (linearly in the turns, or with whole pairs
    as bounds) brings its own inv_freq."""
    n = int(rot_dim) // 2
    if rot_dim != 2 * n or n <= 0 or n % 8 or n > 128:
        raise ValueError(f"rot_dim must be a multiple of 16 and at most 256, got {rot_dim}")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError(f"base and factor must be positive, got {base} and {factor}")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError(f'scaling must be "none", "linear", "base" or "parts", got {scaling!r}')
    f = torch.arange(n, dtype=torch.float64) / n
    if scaling == "base":
        base = base * factor ** (n / (n - 1))
    w = torch.as_tensor(base, dtype=torch.float64) ** -f
    if scaling == "linear":
        w = w / factor
    if scaling == "parts":
        if original_length is None or original_length <= 0 or not 0 < slow_turns < fast_turns:
            raise ValueError("scaling by parts needs the original_length, and 0 < slow_turns < fast_turns")
        turns = original_length * w / (2 * math.pi)
        keep = (torch.log(turns / slow_turns) / math.log(fast_turns / slow_turns)).clamp(0.0, 1.0)
        w = w * keep + w / factor * (1 - keep)
        if gain is None:
            gain = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return w.to(device), 1.0 if gain is None else float(gain)


def _written(*tensors):
    """Tells autograd that a kernel wrote tensors of the caller's: a gradient that still needs what they held
    is then refused instead of wrong."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def attn_rope_table(inv_freq, positions, table, *, gain=1.0, stream=None):
    """Cosines and sines of positions into the preallocated table (fp32 [T, 2, n]): table[t, 0] =
    gain cos(p_t inv_freq), table[t, 1] = gain sin(p_t inv_freq).  inv_freq: fp64 [n] on the device;
    positions: int32 of T values.  Angles are reduced without rounding, also those of far positions.  (A
    gradient of a rotation by what the table held before is refused afterwards.)"""
    _check(inv_freq, "inv_freq", torch.float64, 1)
    _check(positions, "positions", torch.int32, positions.dim())
    _check(table, "table", torch.float32, 3)
    T, n = positions.numel(), inv_freq.shape[0]
    if tuple(table.shape) != (T, 2, n):
        raise ValueError(f"table must be {(T, 2, n)}, got {tuple(table.shape)}")
    dev = _device_of(inv_freq, positions, table)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_rope_table(inv_freq, positions, table, gain=gain)
    _run_rope_table(inv_freq, positions, table, T, n, dev, gain)
    _written(table)


def _run_rope_table(inv_freq, positions, table, T, n, dev, gain):
    if T > 0x7FFFFFFF:
        raise ValueError(f"at most 2^31 - 1 positions, got {T}")
    st = _load().attn_rope_table(_p(inv_freq), _p(positions), _p(table), T, n, float(gain), _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_rope_table")


def rope_table(inv_freq, positions, *, gain=1.0, stream=None):
    """attn_rope_table into a new table [T, 2, n], T the positions' count: made once a step, for
    the rotations of all its layers."""
    _check(inv_freq, "inv_freq", torch.float64, 1)
    _check(positions, "positions", torch.int32, positions.dim())
    dev = _device_of(inv_freq, positions)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rope_table(inv_freq, positions, gain=gain)
    T, n = positions.numel(), inv_freq.shape[0]
    table = torch.empty((T, 2, n), dtype=torch.float32, device=inv_freq.device)
    _run_rope_table(inv_freq, positions, table, T, n, dev, gain)
    return table


def _row_stride(t, name):
    """Elements between the rows of a bf16 tensor [.., H, d], which must be evenly apart."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() < 3:
        raise ValueError(f"{name} must be [rows, H, d] or [B, S, H, d], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, strides = t.shape, t.stride()
    H, d = shape[-2:]
    if t.is_contiguous() or t.numel() == 0:
        return H * d
    if (strides[-1] != 1 and d > 1) or (strides[-2] != d and H > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride, reach = None, 0  # of the innermost rows; what the rows so far span
    for size, step in zip(shape[-3::-1], strides[-3::-1]):
        if size == 1:
            continue
        if stride is None:
            stride, reach = step, step * size
        elif step != reach:
            raise ValueError(f"{name}: the rows must be evenly apart, got strides {t.stride()}")
        else:
            reach *= size
    if stride is None:
        return H * d
    if stride < H * d or stride % 8:
        raise ValueError(f"{name}: rows must not overlap and must be a multiple of 8 elements apart, got {stride}")
    return stride


def _check_rope(q, k, table):
    """Checks of heads and their table; returns (T, H_q, H_k, d, n, table rows)."""
    _check(table, "table", torch.float32, 3)
    R, two, n = table.shape
    if two != 2:
        raise ValueError(f"table must be [rows, 2, n], got {tuple(table.shape)}")
    shape = q.shape
    dims = len(shape)
    if dims < 3:
        raise ValueError(f"q must be [rows, H, d] or [B, S, H, d], got {tuple(shape)}")
    T, H, d = shape[0] if dims == 3 else math.prod(shape[:-2]), shape[-2], shape[-1]
    if T > 0x7FFFFFFF:
        raise ValueError(f"at most 2^31 - 1 rows, got {T}")
    H_k = 0
    if k is not None:
        other = k.shape
        if len(other) != dims or other[-1] != d or (other[0] != T if dims == 3 else other[:-2] != shape[:-2]):
            raise ValueError(f"k must have q's rows and head dim, got {tuple(other)} and {tuple(shape)}")
        H_k = other[-2]
    if R != T and not (dims == 4 and R == shape[1]):
        raise ValueError(f"table must have one row per row of q ({T})"
                         + (f" or per position ({shape[1]})" if dims == 4 else "") + f", got {R}")
    return T, H, H_k, d, n, R


def attn_rope(q, k, table, q_out, k_out, *, interleaved=False, first_dim=0, inverse=False, stream=None):
    """Rotate the heads of q and k (bf16 [T, H, d] or [B, S, H, d]; k may be None) by their rows'
    positions into q_out, k_out of the same shapes; q_out may be q (in place).

    table: fp32 [T, 2, n] (rope_table), one row per row of q; for [B, S, H, d] it may be [S, 2, n],
    shared by the batch.  Dims first_dim .. first_dim + 2n of every head are turned, as pairs (f, n + f) or,
    interleaved, (2f, 2f + 1); the others are copied.  inverse: the transposed rotation, which
    takes the gradient of the results to that of q and k.  Rows may be apart (a slice of a fused
    projection), evenly and by a multiple of 8 elements.  Not differentiable (rope is): results that are part of
    a graph, as q of a projection in training rotated in place, are refused."""
    T, H, H_k, d, n, R = _check_rope(q, k, table)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q_out, k_out)):
        raise ValueError("q_out and k_out must not require gradients: rope() is the differentiable rotation")
    if q_out is None or q_out.shape != q.shape or (k is not None and (k_out is None or k_out.shape != k.shape)):
        raise ValueError("q_out and k_out must have the shapes of q and k")
    strides = [_row_stride(q, "q"), 0 if k is None else _row_stride(k, "k"), _row_stride(q_out, "q_out"),
               0 if k is None else _row_stride(k_out, "k_out")]
    dev = _device_of(q, k, table, q_out, k_out)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_rope(q, k, table, q_out, k_out, interleaved=interleaved, first_dim=first_dim, inverse=inverse)
    _run_rope(q, k, table, q_out, k_out, (T, H, H_k, d, n), R, strides, dev, interleaved, first_dim, inverse)
    _written(q_out, k_out)


def _run_rope(q, k, table, q_out, k_out, sizes, R, strides, dev, interleaved, first_dim, inverse):
    st = _load().attn_rope(_p(q), _p(k), _p(table), _p(q_out), _p(k_out), *sizes, int(first_dim), R, *strides,
                           int(bool(interleaved)), int(bool(inverse)), _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_rope")


def _rope_new(q, k, table, interleaved, first_dim, inverse, stream):
    sizes = _check_rope(q, k, table)
    dev = _device_of(q, k, table)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _rope_new(q, k, table, interleaved, first_dim, inverse, None)
    H, H_k, d = sizes[1:4]
    strides = [_row_stride(q, "q"), 0 if k is None else _row_stride(k, "k"), H * d, H_k * d]
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _run_rope(q, k, table, q_out, k_out, sizes[:5], sizes[5], strides, dev, interleaved, first_dim, inverse)
    return q_out, k_out


def rope_forward(q, k, table, *, interleaved=False, first_dim=0, stream=None):
    """attn_rope into new tensors: returns (q, k) rotated."""
    return _rope_new(q, k, table, interleaved, first_dim, False, stream)


def rope_backward(dq, dk, table, *, interleaved=False, first_dim=0, stream=None):
    """Gradients of rope_forward's inputs from those of its results: returns (dq, dk)."""
    return _rope_new(dq, dk, table, interleaved, first_dim, True, stream)


def _evenly(t):
    """A gradient as autograd hands it over, copied if its rows are not as a kernel can read them."""
    try:
        _row_stride(t, "gradient")
        return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)
    except ValueError:
        return t.contiguous()


class RopeFunction(torch.autograd.Function):
    """autograd wrapper of the rotation; its gradient is the transposed rotation, differentiable in turn."""

    @staticmethod
    def forward(ctx, q, k, table, interleaved, first_dim, inverse=False):
        ctx.set_materialize_grads(False)
        ctx.args = interleaved, first_dim, inverse
        ctx.save_for_backward(table)
        return _rope_new(q, k, table, *ctx.args, None)

    @staticmethod
    def backward(ctx, dq, dk):
        (table,) = ctx.saved_tensors
        interleaved, first_dim, inverse = ctx.args
        dq, dk = (None if g is None else _evenly(g) for g in (dq, dk))
        if dq is None and dk is None:
            return None, None, None, None, None, None
        rest = table, interleaved, first_dim, not inverse
        turn = RopeFunction.apply if torch.is_grad_enabled() else lambda *a: _rope_new(*a, None)
        if dq is None:
            return None, turn(dk, None, *rest)[0], None, None, None, None
        return (*turn(dq, dk, *rest), None, None, None, None)


def rope(q, k, table, *, interleaved=False, first_dim=0):
    """Differentiable rotation of q and k (k may be None) by positions: returns (q, k); arguments as
    for attn_rope.  The table receives no gradient.

    A step captured into a CUDA graph (this or any other differentiable call): no result of an eager call whose
    gradient still leads to the same leaves may be alive, or autograd ends the capture."""
    return RopeFunction.apply(q, k, table, bool(interleaved), int(first_dim))


def _check_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens):
    """Checks shared by the appends with a rotation; returns the sizes and strides as the C call takes them."""
    if k.dim() != 3:
        raise ValueError(f"k must be [T, H_kv, d], got shape {tuple(k.shape)}")
    T, _, d = k.shape
    B, n_pages, H_kv, page_size, max_pages = _check_paged(pool, page_table, seq_lens, d)
    ks, vs = _check_rows(k, "k", H_kv, d), _check_rows(v, "v", H_kv, d)
    if v.shape[0] != T:
        raise ValueError(f"k and v must have the same rows, got {T} and {v.shape[0]}")
    _check_cu(cu_seqlens, "cu_seqlens", B)
    _check(table, "table", torch.float32, 3)
    if table.shape[0] != T or table.shape[1] != 2:
        raise ValueError(f"table must be [{T}, 2, n], got {tuple(table.shape)}")
    H_q = qs = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T:
            raise ValueError(f"q must be [{T}, H_q, {d}], got {tuple(q.shape)}")
        H_q = q.shape[1]
        qs = _check_rows(q, "q", H_q, d)
    return (B, T, H_q, H_kv, d, n_pages, page_size, max_pages, table.shape[2]), (qs, ks, vs)


def _run_append_rope(q, k, v, table, cu, pool, page_table, seq_lens, q_out, sizes, strides, qos, dev, interleaved, first_dim):
    st = _load().attn_kv4_append_rope(_p(q), _p(k), _p(v), _p(table), _p(q_out), _p(cu), _p(pool), _p(page_table),
                                      _p(seq_lens), *sizes, int(first_dim), *strides, qos, int(bool(interleaved)),
                                      _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_append_rope")


def attn_kv4_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, q_out, *, interleaved=False, first_dim=0,
                         stream=None):
    """attn_kv4_append of keys rotated on the way, and the queries rotated in the same launch.

    k, v (bf16 [T, H_kv, d]), cu_seqlens, pool, page_table, seq_lens as for attn_kv4_append; table: fp32
    [T, 2, n], one row per row of k; q, q_out: bf16 [T, H_q, d], or None.  Results and cache are bit for
    bit those of attn_rope and attn_kv4_append."""
    sizes, strides = _check_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens)
    qos = 0
    if q is not None:
        if q_out is None or q_out.shape != q.shape:
            raise ValueError(f"q_out must have q's shape {tuple(q.shape)}")
        qos = _check_rows(q_out, "q_out", q.shape[1], q.shape[2])
    dev = _device_of(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, q_out)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, q_out,
                                        interleaved=interleaved, first_dim=first_dim)
    _run_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, q_out, sizes, strides, qos, dev, interleaved,
                     first_dim)


def kv4_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, *, interleaved=False, first_dim=0, stream=None):
    """attn_kv4_append_rope with the rotated queries in a new tensor, which is returned (None
    without q)."""
    sizes, strides = _check_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens)
    dev = _device_of(q, k, v, table, cu_seqlens, pool, page_table, seq_lens)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv4_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, interleaved=interleaved,
                                   first_dim=first_dim)
    q_out = None if q is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _run_append_rope(q, k, v, table, cu_seqlens, pool, page_table, seq_lens, q_out, sizes, strides,
                     sizes[2] * sizes[4], dev, interleaved, first_dim)
    return q_out


# ----------------------------------------------------------------------------- drafted trees


@functools.lru_cache(maxsize=1024)
def attn_kv4_tree_workspace_size(B, T, H_q, H_kv, d) -> int:
    return int(_load().attn_kv4_tree_workspace_size(B, T, H_q, H_kv, d))


def _check_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, softmax_offset):
    """Checks of a tree's inputs; returns (B, T, H_q, H_kv, d, n_pages, page_size, max_pages)."""
    _check(q, "q", torch.bfloat16, 3)
    T, H_q, d = q.shape
    B, n_pages, H_kv, page_size, max_pages = _check_paged(pool, page_table, seq_lens, d)
    _check_cu(cu_seqlens, "cu_seqlens", B)
    if parents is not None:
        _check(parents, "parents", torch.int32, 1)
        if parents.shape[0] != T:
            raise ValueError(f"parents: one per row of q ({T}), got {parents.shape[0]}")
    if softmax_offset is not None:
        _check(softmax_offset, "softmax_offset", torch.float32, 1)
        if softmax_offset.shape[0] != H_q:
            raise ValueError(f"softmax_offset must have one value per query head ({H_q})")
    return B, T, H_q, H_kv, d, n_pages, page_size, max_pages


def attn_kv4_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, o, lse=None, *, window=-1, softmax_type=VANILLA,
                  softmax_offset=None, scale=0.0, zero_rest=False, workspace=None, stream=None):
    """Attention of drafted trees over their sequences' 4-bit caches, into preallocated o (bf16, q's
    shape [T, H_q, d]) and, if given, lse (fp32 [H_q, T]).

    Rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (int32 [B+1] on the device) are the nodes of sequence b's
    tree, already in the cache as its tokens seq_lens[b], seq_lens[b] + 1, ... (seq_lens: int32 [B], the
    tokens before the tree).  parents: int32 [T], the number of a node's parent within its sequence,
    below its own; negative: a child of the last token before the tree.  None: a chain (tokens in
    causal order, any number of them; much faster than a long chain given as parents).  A node sees the tokens before the tree, its ancestors and
    itself, with window >= 0 those of the last window + 1 positions.  Rows of no sequence are left
    alone, or zeroed with zero_rest (lse -inf).  workspace: as for attn_kv4_decode.

    The kernel is chosen by the rows on average, T / B: a large tree or chain among many single tokens, idle sequences or
    spare rows of q is read several times over, and is faster in a call of its own."""
    sizes = _check_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, softmax_offset)
    T, H_q = sizes[1:3]
    _check(o, "o", torch.bfloat16, 3)
    if o.shape != q.shape:
        raise ValueError(f"o must have q's shape {tuple(q.shape)}, got {tuple(o.shape)}")
    if lse is not None:
        _check(lse, "lse", torch.float32, 2)
        if lse.shape != (H_q, T):
            raise ValueError(f"lse must be {(H_q, T)}, got {tuple(lse.shape)}")
    dev = _device_of(q, cu_seqlens, parents, pool, page_table, seq_lens, o, lse, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, o, lse, window=window,
                                 softmax_type=softmax_type, softmax_offset=softmax_offset, scale=scale,
                                 zero_rest=zero_rest, workspace=workspace)
    _run_kv4_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type,
                  softmax_offset, scale, zero_rest, workspace)


def _run_kv4_tree(q, cu, parents, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type, softmax_offset,
                  scale, zero_rest, workspace):
    ws = _workspace(workspace, attn_kv4_tree_workspace_size(*sizes[:5]) if workspace is None else 0, q.device)
    st = _load().attn_kv4_tree(_p(q), _p(cu), _p(parents), _p(pool), _p(page_table), _p(seq_lens), _p(o), _p(lse), *sizes,
                               float(scale or 0.0), _window(window), _stype(softmax_type), _p(softmax_offset),
                               int(bool(zero_rest)), _p(ws), ws.numel(), _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_tree")


def sdpa_tree_kv4(q, cu_seqlens, parents, pool, page_table, seq_lens, *, window=-1, softmax_type=VANILLA,
                  softmax_offset=None, scale=0.0, workspace=None, stream=None):
    """Allocate O and LSE, run attn_kv4_tree, return (o, lse); rows of no sequence are zero (lse -inf)."""
    sizes = _check_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, softmax_offset)
    dev = _device_of(q, cu_seqlens, parents, pool, page_table, seq_lens, softmax_offset, workspace)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return sdpa_tree_kv4(q, cu_seqlens, parents, pool, page_table, seq_lens, window=window,
                                 softmax_type=softmax_type, softmax_offset=softmax_offset, scale=scale,
                                 workspace=workspace)
    o = torch.empty_like(q)
    lse = torch.empty((sizes[2], sizes[1]), dtype=torch.float32, device=q.device)
    _run_kv4_tree(q, cu_seqlens, parents, pool, page_table, seq_lens, o, lse, sizes, dev, window, softmax_type,
                  softmax_offset, scale, True, workspace)
    return o, lse


def attn_kv4_keep(pool, page_table, seq_lens, kept, d, *, stream=None):
    """Keep accepted nodes: token seq_lens[b] + kept[b, i] of sequence b becomes its token seq_lens[b] + i,
    for i in order until the first negative entry, in the pool [n_pages, H_kv, block] or in each
    layer of [n_layers, n_pages, H_kv, block].  kept: int32 [B, most] on the device, the numbers of
    the accepted nodes, usually ascending (a path from the root); d: the head dim.  The caller
    then adds the count of each row to seq_lens."""
    if pool.dim() not in (3, 4):
        raise ValueError(f"pool must be [n_pages, H_kv, block] or [n_layers, n_pages, H_kv, block], got "
                         f"{tuple(pool.shape)}")
    _check(pool, "pool", torch.uint8, pool.dim())
    n_layers = pool.shape[0] if pool.dim() == 4 else 1
    n_pages, H_kv, block = pool.shape[-3:]
    _check(page_table, "page_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _check(kept, "kept", torch.int32, 2)
    d = int(d)
    page_size = block * 8 // (9 * d) if d > 0 else 0
    if kv4_block_bytes(page_size, d) != block:
        raise ValueError(f"pool's blocks must be kv4_block_bytes(page_size, {d}) bytes, got {block}")
    B, max_pages = page_table.shape
    if seq_lens.shape[0] != B or kept.shape[0] != B:
        raise ValueError(f"seq_lens and kept: one row per row of page_table ({B}), got {seq_lens.shape[0]} and "
                         f"{kept.shape[0]}")
    dev = _device_of(pool, page_table, seq_lens, kept)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_kv4_keep(pool, page_table, seq_lens, kept, d)
    st = _load().attn_kv4_keep(_p(pool), _p(page_table), _p(seq_lens), _p(kept), B, kept.shape[1], n_layers, H_kv, d,
                               n_pages, page_size, max_pages, _raw_stream(dev, None))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv4_keep")


# ----------------------------------------------------------------------------- conveniences


def sdpa_forward(q, k, v, *, causal=True, window=-1, softmax_type=VANILLA, softmax_offset=None, scale=0.0,
                 seq_lens_q=None, seq_lens_kv=None, bias=None, dropout_p=0.0, rng_state=None, stream=None):
    """Allocate O and LSE, run attn_fwd, return (o, lse)."""
    B, S_q, H_q, _ = q.shape
    d_v = v.shape[3]
    o = torch.empty((B, S_q, H_q, d_v), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H_q, S_q), dtype=torch.float32, device=q.device)
    attn_fwd(q, k, v, o, lse, causal=causal, window=window, softmax_type=softmax_type,
             softmax_offset=softmax_offset, scale=scale, seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv,
             bias=bias, dropout_p=dropout_p, rng_state=rng_state, stream=stream)
    return o, lse


def sdpa_backward(q, k, v, o, dout, lse, *, causal=True, window=-1, softmax_type=VANILLA, softmax_offset=None,
                  scale=0.0, deterministic=True, workspace=None, seq_lens_q=None, seq_lens_kv=None, bias=None,
                  dropout_p=0.0, rng_state=None, stream=None):
    """Allocate dQ, dK, dV (and d_offset for the learnable sink), run attn_bwd, return them;
    with a bias, also dbias (fp32, the bias's shape) as a fifth output."""
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    st = _stype(softmax_type)
    d_off = torch.empty((q.shape[2],), dtype=torch.float32, device=q.device) if st == LEARNABLE else None
    dbias = torch.empty(bias.shape, dtype=torch.float32, device=q.device) if bias is not None else None
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, d_off, causal=causal, window=window, softmax_type=st,
             softmax_offset=softmax_offset, scale=scale, deterministic=deterministic, workspace=workspace,
             seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv, bias=bias, dbias=dbias, dropout_p=dropout_p,
             rng_state=rng_state, stream=stream)
    return (dq, dk, dv, d_off) if bias is None else (dq, dk, dv, d_off, dbias)


class SDPAFunction(torch.autograd.Function):
    """autograd wrapper: forward and backward both run in the library's kernels (the
    plain, padded-batch, bias and dropout entry points, chosen by the arguments)."""

    @staticmethod
    def forward(ctx, q, k, v, softmax_offset, bias, causal, window, softmax_type, scale, deterministic,
                seq_lens_q, seq_lens_kv, dropout_p, rng_state):
        kw = dict(causal=causal, window=window, softmax_type=softmax_type, scale=scale, seq_lens_q=seq_lens_q,
                  seq_lens_kv=seq_lens_kv, dropout_p=dropout_p, rng_state=rng_state)
        o, lse = sdpa_forward(q, k, v, softmax_offset=softmax_offset, bias=bias, **kw)
        ctx.save_for_backward(q, k, v, o, lse, softmax_offset, bias)
        ctx.kw = dict(kw, deterministic=deterministic)
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse, off, bias = ctx.saved_tensors
        res = sdpa_backward(q, k, v, o, dout.contiguous(), lse, softmax_offset=off, bias=bias, **ctx.kw)
        dq, dk, dv, d_off = res[:4]
        dbias = None
        if bias is not None and ctx.needs_input_grad[4]:
            dbias = res[4] if bias.dtype == torch.float32 else res[4].to(bias.dtype)  # autograd wants bias's dtype
        return dq, dk, dv, d_off, dbias, None, None, None, None, None, None, None, None, None


def new_rng_state(device=None):
    """A fresh dropout rng_state: a CUDA int64 [seed, offset] with a seed drawn from
    torch's default generator and offset 0."""
    seed = int(torch.randint(0, 2 ** 62, (1,)).item())
    return torch.tensor([seed, 0], dtype=torch.int64, device=device or "cuda")


def attention(q, k, v, softmax_offset=None, *, causal=True, window=-1, softmax_type=VANILLA, scale=0.0,
              deterministic=True, bias=None, seq_lens_q=None, seq_lens_kv=None, dropout_p=0.0, rng_state=None,
              rope=None, rope_interleaved=False, rope_first_dim=0):
    """Differentiable fused attention. q, k, v, the learnable offset and the bias receive
    gradients. seq_lens_q / seq_lens_kv (int32 [B] on the device) make it a padded batch;
    dropout_p > 0 applies attention dropout with rng_state (a fresh one when None; the
    backward regenerates the same decisions from it).  rope: a table of positions (rope_table, one
    row per position or per row), by which q and k (of the same rows) are rotated first."""
    if rope is not None:
        q, k = RopeFunction.apply(q, k, rope, bool(rope_interleaved), int(rope_first_dim))
    if dropout_p and rng_state is None:
        rng_state = new_rng_state(q.device)
    return SDPAFunction.apply(q, k, v, softmax_offset, bias, causal, window, softmax_type, scale, deterministic,
                              seq_lens_q, seq_lens_kv, dropout_p, rng_state)
