"""fp8_kv_cache_write_gb300 -- Python binding of libfp8kv (FP8 paged KV cache and
attention over it, hand-written CUDA for GB300 / sm_103a).

This module only marshals arguments: it checks dtypes/devices, allocates outputs
and workspaces with torch when the caller does not pass them, and calls the C
ABI declared in include/fp8kv.h with raw device pointers and the current CUDA
stream.  Every step of the computation runs in the library's kernels; there is
no CPU fallback, and every call raises if libfp8kv.so is missing.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8kv.so")

PAGE_SIZE = 16
KV_E4M3, KV_BF16 = 0, 1
SCALE_PER_TENSOR, SCALE_PER_HEAD, SCALE_PER_TOKEN_HEAD = 0, 1, 2
OUT_F32, OUT_BF16 = 0, 1
# decode flags (include/fp8kv.h): what may run before the preceding kernel ends
DECODE_EARLY_SETUP, DECODE_EARLY_PAGES = 1, 2
# prefill flags: two-level accumulation, operand precision of the e4m3 path
PREFILL_TWO_LEVEL, PREFILL_SPLIT_ALWAYS, PREFILL_SPLIT_NEVER = 1, 2, 4

# frequency scalings of rope_freqs, and the latent cache's rotary values a row
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = 0, 1, 2, 3, 4
LATENT_ROPE = 64

STATUS = {0: "FP8KV_OK", -1: "FP8KV_ERR_INVALID", -2: "FP8KV_ERR_UNSUPPORTED",
          -3: "FP8KV_ERR_WORKSPACE", -4: "FP8KV_ERR_CUDA", -5: "FP8KV_ERR_TIMEOUT",
          -6: "FP8KV_ERR_BAD_INDEX"}

EXPORTS = ("fp8kv_kv_cache_write", "fp8kv_decode_plan", "fp8kv_paged_decode_attn",
           "fp8kv_decode_step", "fp8kv_paged_decode_attn_noalloc", "fp8kv_prefill_attn",
           "fp8kv_prefill_attn_ws", "fp8kv_prefill_workspace_bytes", "fp8kv_quantize_e4m3",
           "fp8kv_resolve_scales", "fp8kv_rope_freqs", "fp8kv_rope_kv_cache_write",
           "fp8kv_kv_cache_read", "fp8kv_latent_cache_write", "fp8kv_latent_cache_read",
           "fp8kv_latent_attn_plan", "fp8kv_latent_decode_attn", "fp8kv_status_string",
           "fp8kv_last_warning")
NOALLOC_DECODE_SCRATCH_BYTES = 8 << 20

_lib = None


class Fp8kvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_string(status)})")


def build(force: bool = False) -> str:
    """Compile libfp8kv.so in-tree (nvcc, sm_103a)."""
    from . import _build
    return _build.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libfp8kv.so not found at {LIB_PATH}: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
        u32 = ctypes.c_uint
        L.fp8kv_kv_cache_write.argtypes = [P, P, P, i64, i32, i32, P, P, i64, i32, i32, P, P, P,
                                           P, P, P]
        L.fp8kv_kv_cache_write.restype = i32
        L.fp8kv_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32,
                                        ctypes.POINTER(i32), ctypes.POINTER(sz)]
        L.fp8kv_decode_plan.restype = i32
        L.fp8kv_paged_decode_attn.argtypes = [P, P, P, i32, i32, P, P, P, P, P, i32, P, i32, i32,
                                              i32, i32, i64, f32, i32, i32, P, sz, P, i32, u32, P,
                                              P]
        L.fp8kv_paged_decode_attn.restype = i32
        L.fp8kv_decode_step.argtypes = [P, P, P, P, P, i32, i32, P, P, P, P, P, i32, P, i32, i32,
                                        i32, i32, i64, f32, i32, i32, P, sz, P, i32, u32, P, P]
        L.fp8kv_decode_step.restype = i32
        L.fp8kv_paged_decode_attn_noalloc.argtypes = [P, P, P, i32, i32, P, P, P, P, P, i32, P,
                                                      i32, i32, i32, i32, i64, f32, i32, i32, P,
                                                      i32, P, P]
        L.fp8kv_paged_decode_attn_noalloc.restype = i32
        L.fp8kv_prefill_attn.argtypes = [P, P, i32, P, P, i32, i32, P, P, P, P, f32, f32, P, i32, P,
                                         i32, i32, i32, i32, i64, f32, i32, P, i32, P, P]
        L.fp8kv_prefill_attn.restype = i32
        L.fp8kv_prefill_attn_ws.argtypes = [P, P, i32, P, P, i32, i32, P, P, P, P, f32, f32, P,
                                            i32, P, i32, i32, i32, i32, i64, f32, i32, P, sz, P,
                                            i32, P, P]
        L.fp8kv_prefill_attn_ws.restype = i32
        L.fp8kv_prefill_workspace_bytes.argtypes = [i32, ctypes.POINTER(sz)]
        L.fp8kv_prefill_workspace_bytes.restype = i32
        L.fp8kv_quantize_e4m3.argtypes = [P, f32, P, i64, P]
        L.fp8kv_quantize_e4m3.restype = i32
        FP = ctypes.POINTER(f32)
        L.fp8kv_resolve_scales.argtypes = [i32, i32, i32, FP, FP, f32, f32, FP, FP, FP, FP]
        L.fp8kv_resolve_scales.restype = i32
        f64 = ctypes.c_double
        L.fp8kv_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, P, FP]
        L.fp8kv_rope_freqs.restype = i32
        L.fp8kv_rope_kv_cache_write.argtypes = [P, i64, P, i64, P, i64, P, P, P, i32, i32, f32,
                                                i64, i32, i32, i32, P, i64, P, P, i64, i32, i32,
                                                P, P, P, P, P, P]
        L.fp8kv_rope_kv_cache_write.restype = i32
        L.fp8kv_kv_cache_read.argtypes = [P, P, i64, i32, i32, P, P, P, P, P, i64, i32, i32, P, P,
                                          i32, P, P]
        L.fp8kv_kv_cache_read.restype = i32
        L.fp8kv_latent_cache_write.argtypes = [P, i64, P, i64, P, P, i32, f32, P, i64, i32, P,
                                               i64, i32, i32, P, P, P, i64, i64, P, i64, i64, i32,
                                               P, P]
        L.fp8kv_latent_cache_write.restype = i32
        L.fp8kv_latent_cache_read.argtypes = [P, i64, i32, i32, P, P, P, i64, i32, P, i32, P, P]
        L.fp8kv_latent_cache_read.restype = i32
        L.fp8kv_latent_attn_plan.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                             ctypes.POINTER(sz)]
        L.fp8kv_latent_attn_plan.restype = i32
        L.fp8kv_latent_decode_attn.argtypes = [P, P, i32, i32, P, P, P, i32, P, i32, i32, i32,
                                               i32, i64, f32, i32, P, sz, P, i32, P, P]
        L.fp8kv_latent_decode_attn.restype = i32
        L.fp8kv_status_string.argtypes = [i32]
        L.fp8kv_status_string.restype = ctypes.c_char_p
        L.fp8kv_last_warning.argtypes = []
        L.fp8kv_last_warning.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fp8kv_status_string(int(status)).decode()


def last_warning() -> str:
    return lib().fp8kv_last_warning().decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype=None, device=True, contiguous=True, pinned_ok=False):
    """dtype / contiguity / placement check.  pinned_ok: pinned host memory is
    accepted too (the kernels read or write it directly over the host link)."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if device and not t.is_cuda and not (pinned_ok and t.is_pinned()):
        raise ValueError(f"{name}: expected a CUDA tensor" +
                         (" or pinned host memory" if pinned_ok else ""))
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def _raise(st, what):
    if st != 0:
        raise Fp8kvError(st, what)


def kv_cache_write(k, v, slot_mapping, k_cache, v_cache, *, kv_dtype, scale_mode=SCALE_PER_TENSOR,
                   k_scale=None, v_scale=None, k_scale_cache=None, v_scale_cache=None,
                   err_flag=None, stream=None) -> None:
    """Store bf16 K/V rows [T][Hkv][D] at slot_mapping into the paged cache
    (uint8 e4m3 or bf16 [num_blocks][Hkv][16][D]); see fp8kv_kv_cache_write."""
    _check(k, "k", torch.bfloat16, pinned_ok=True)
    _check(v, "v", torch.bfloat16, pinned_ok=True)
    _check(slot_mapping, "slot_mapping", torch.int64, pinned_ok=True)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(t, n, torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16)
    for n, t in (("k_scale", k_scale), ("v_scale", v_scale), ("k_scale_cache", k_scale_cache),
                 ("v_scale_cache", v_scale_cache)):
        _check(t, n, torch.float32)
    _check(err_flag, "err_flag", torch.int32)
    T, Hkv, D = k.shape
    st = lib().fp8kv_kv_cache_write(
        _ptr(k), _ptr(v), _ptr(slot_mapping), T, Hkv, D, _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], kv_dtype, scale_mode, _ptr(k_scale), _ptr(v_scale),
        _ptr(k_scale_cache), _ptr(v_scale_cache), _ptr(err_flag), _stream(stream))
    _raise(st, "kv_cache_write")


def decode_plan(B, Hq, Hkv, D, max_blocks_per_seq, window=0, num_splits=0):
    """(num_splits, workspace_bytes) that paged_decode_attn will use."""
    s = ctypes.c_int(0)
    w = ctypes.c_size_t(0)
    st = lib().fp8kv_decode_plan(B, Hq, Hkv, D, max_blocks_per_seq, window, num_splits,
                                 ctypes.byref(s), ctypes.byref(w))
    _raise(st, "decode_plan")
    return s.value, w.value


def paged_decode_attn(q, k_cache, v_cache, block_table, context_lens, *, kv_dtype,
                      scale_mode=SCALE_PER_TENSOR, k_scale=None, v_scale=None,
                      k_scale_cache=None, v_scale_cache=None, softmax_scale=None, window=0,
                      num_splits=0, workspace=None, out=None, out_dtype=OUT_F32, flags=0,
                      err_flag=None, stream=None):
    """Decode attention of q [B][Hq][D] (bf16) over the paged cache; returns out
    [B][Hq][D] (fp32 or bf16).  flags: 0 or DECODE_EARLY_SETUP / DECODE_EARLY_PAGES.
    See fp8kv_paged_decode_attn."""
    _check(q, "q", torch.bfloat16, pinned_ok=True)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(t, n, torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16)
    _check(block_table, "block_table", torch.int32)
    _check(context_lens, "context_lens", torch.int32, pinned_ok=True)
    for n, t in (("k_scale", k_scale), ("v_scale", v_scale), ("k_scale_cache", k_scale_cache),
                 ("v_scale_cache", v_scale_cache)):
        _check(t, n, torch.float32)
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    mbs = block_table.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    splits, ws_bytes = decode_plan(B, Hq, Hkv, D, mbs, window, num_splits)
    if ws_bytes > 0 and (workspace is None or workspace.numel() * workspace.element_size()
                         < ws_bytes):
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=k_cache.device)
    if out is None:
        out = torch.empty(B, Hq, D, device=k_cache.device,
                          dtype=torch.float32 if out_dtype == OUT_F32 else torch.bfloat16)
    _check(out, "out", torch.float32 if out_dtype == OUT_F32 else torch.bfloat16,
           pinned_ok=True)
    st = lib().fp8kv_paged_decode_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), kv_dtype, scale_mode, _ptr(k_scale),
        _ptr(v_scale), _ptr(k_scale_cache), _ptr(v_scale_cache), _ptr(block_table), mbs,
        _ptr(context_lens), B, Hq, Hkv, D, k_cache.shape[0], float(softmax_scale), int(window),
        int(num_splits), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(out),
        out_dtype, int(flags), _ptr(err_flag), _stream(stream))
    _raise(st, "paged_decode_attn")
    return out


def decode_step(q, k_new, v_new, k_cache, v_cache, block_table, context_lens, *, kv_dtype,
                scale_mode=SCALE_PER_TENSOR, k_scale=None, v_scale=None, k_scale_cache=None,
                v_scale_cache=None, softmax_scale=None, window=0, num_splits=0, workspace=None,
                out=None, out_dtype=OUT_F32, flags=0, err_flag=None, stream=None):
    """One decode step in one call: stores the new token k_new / v_new [B][Hkv][D]
    (bf16) of every sequence at position context_lens[b] - 1 of its page table
    (quantized as kv_cache_write does), then attends q [B][Hq][D] over all its
    keys.  Returns out [B][Hq][D].  See fp8kv_decode_step."""
    _check(q, "q", torch.bfloat16, pinned_ok=True)
    _check(k_new, "k_new", torch.bfloat16, pinned_ok=True)
    _check(v_new, "v_new", torch.bfloat16, pinned_ok=True)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(t, n, torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16)
    _check(block_table, "block_table", torch.int32)
    _check(context_lens, "context_lens", torch.int32, pinned_ok=True)
    for n, t in (("k_scale", k_scale), ("v_scale", v_scale), ("k_scale_cache", k_scale_cache),
                 ("v_scale_cache", v_scale_cache)):
        _check(t, n, torch.float32)
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
        raise ValueError(f"k_new / v_new: expected shape {(B, Hkv, D)}")
    mbs = block_table.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    splits, ws_bytes = decode_plan(B, Hq, Hkv, D, mbs, window, num_splits)
    if ws_bytes > 0 and (workspace is None or workspace.numel() * workspace.element_size()
                         < ws_bytes):
        workspace = torch.empty(ws_bytes // 4, dtype=torch.float32, device=k_cache.device)
    if out is None:
        out = torch.empty(B, Hq, D, device=k_cache.device,
                          dtype=torch.float32 if out_dtype == OUT_F32 else torch.bfloat16)
    _check(out, "out", torch.float32 if out_dtype == OUT_F32 else torch.bfloat16,
           pinned_ok=True)
    st = lib().fp8kv_decode_step(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), kv_dtype, scale_mode,
        _ptr(k_scale), _ptr(v_scale), _ptr(k_scale_cache), _ptr(v_scale_cache),
        _ptr(block_table), mbs, _ptr(context_lens), B, Hq, Hkv, D, k_cache.shape[0],
        float(softmax_scale), int(window), int(num_splits), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(out),
        out_dtype, int(flags), _ptr(err_flag), _stream(stream))
    _raise(st, "decode_step")
    return out


def paged_decode_attn_noalloc(q, k_cache, v_cache, block_table, context_lens, *, kv_dtype,
                              scale_mode=SCALE_PER_TENSOR, k_scale=None, v_scale=None,
                              k_scale_cache=None, v_scale_cache=None, softmax_scale=None,
                              window=0, num_splits=0, out, out_dtype=OUT_F32, err_flag=None,
                              stream=None):
    """paged_decode_attn without a workspace, for callers that cannot allocate
    device memory: the split partials live in the library's static device array
    (NOALLOC_DECODE_SCRATCH_BYTES per GPU).  `out` must be passed.  Calls that
    overlap on the GPU race on that array; the first call on a device should
    come before any stream capture."""
    _check(q, "q", torch.bfloat16, pinned_ok=True)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(t, n, torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16)
    _check(block_table, "block_table", torch.int32)
    _check(context_lens, "context_lens", torch.int32, pinned_ok=True)
    _check(out, "out", torch.float32 if out_dtype == OUT_F32 else torch.bfloat16,
           pinned_ok=True)
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    mbs = block_table.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    st = lib().fp8kv_paged_decode_attn_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), kv_dtype, scale_mode, _ptr(k_scale),
        _ptr(v_scale), _ptr(k_scale_cache), _ptr(v_scale_cache), _ptr(block_table), mbs,
        _ptr(context_lens), B, Hq, Hkv, D, k_cache.shape[0], float(softmax_scale), int(window),
        int(num_splits), _ptr(out), out_dtype, _ptr(err_flag), _stream(stream))
    if st == -3:
        if num_splits == 0:
            raise Fp8kvError(st, f"paged_decode_attn_noalloc: one split slot per (sequence, KV "
                                 f"head) already needs B*Hq*(D+2)*4 = {B * Hq * (D + 2) * 4} "
                                 f"bytes, more than the static array's "
                                 f"{NOALLOC_DECODE_SCRATCH_BYTES}; use paged_decode_attn with "
                                 f"a workspace")
        _, need = decode_plan(B, Hq, Hkv, D, mbs, window, num_splits)
        raise Fp8kvError(st, f"paged_decode_attn_noalloc: the split plan needs {need} bytes of "
                             f"scratch but the static array holds "
                             f"{NOALLOC_DECODE_SCRATCH_BYTES}; pass fewer num_splits (or 0) or "
                             f"use paged_decode_attn with a workspace")
    _raise(st, "paged_decode_attn_noalloc")
    return out


def prefill_workspace_bytes(D):
    """Bytes of the workspace fp8kv_prefill_attn_ws takes at head_dim D."""
    n = ctypes.c_size_t(0)
    _raise(lib().fp8kv_prefill_workspace_bytes(int(D), ctypes.byref(n)), "prefill_workspace_bytes")
    return n.value


# zero-filled prefill workspaces, one per (device, stream, D): the kernel leaves
# its counters zero after each call, and calls on one stream never overlap
_prefill_ws = {}


def prefill_workspace(device, stream, D):
    """The cached zero-initialised workspace prefill_attn uses on `stream` (a
    torch stream; None: the current one)."""
    key = (torch.device(device).index, _stream(stream).value or 0, int(D))
    ws = _prefill_ws.get(key)
    if ws is None:
        ws = torch.zeros(prefill_workspace_bytes(D), dtype=torch.uint8, device=device)
        _prefill_ws[key] = ws
    return ws


def prefill_attn(q, cu_seqlens_q, max_seqlen_q, k_cache, v_cache, block_table, context_lens,
                 *, kv_dtype=KV_E4M3, scale_mode=SCALE_PER_TENSOR, k_scale=None, v_scale=None,
                 k_scale_cache=None, v_scale_cache=None, q_scale=1.0, prob_scale=1.0,
                 softmax_scale=None, two_level=False, split="auto", out=None, out_dtype=OUT_F32,
                 err_flag=None, stream=None, workspace="auto"):
    """Chunked causal FP8 prefill of q [Tq][Hq][D] (bf16) over the paged cache;
    returns out [Tq][Hq][D].  split: "auto" (split e4m3 operands for blocks of
    rows under 8192 keys), "always" or "never".  workspace: "auto" (a cached
    zeroed workspace per device and stream, so that launches with more query
    tiles than SMs run balanced over persistent CTAs), a zeroed uint8 tensor of
    prefill_workspace_bytes(D), or None (one CTA per query tile).  See
    fp8kv_prefill_attn and fp8kv_prefill_attn_ws."""
    if split not in ("auto", "always", "never"):
        raise ValueError("split: 'auto', 'always' or 'never'")
    flags = (PREFILL_TWO_LEVEL if two_level else 0) | {
        "auto": 0, "always": PREFILL_SPLIT_ALWAYS, "never": PREFILL_SPLIT_NEVER}[split]
    _check(q, "q", torch.bfloat16)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(t, n, torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16)
    _check(block_table, "block_table", torch.int32)
    _check(context_lens, "context_lens", torch.int32)
    for n, t in (("k_scale", k_scale), ("v_scale", v_scale), ("k_scale_cache", k_scale_cache),
                 ("v_scale_cache", v_scale_cache)):
        _check(t, n, torch.float32)
    Tq, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty(Tq, Hq, D, device=q.device,
                          dtype=torch.float32 if out_dtype == OUT_F32 else torch.bfloat16)
    _check(out, "out", torch.float32 if out_dtype == OUT_F32 else torch.bfloat16)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace: 'auto', a uint8 tensor or None")
        workspace = prefill_workspace(q.device, stream, D)
    _check(workspace, "workspace", torch.uint8)
    st = lib().fp8kv_prefill_attn_ws(
        _ptr(q), _ptr(cu_seqlens_q), int(max_seqlen_q), _ptr(k_cache), _ptr(v_cache), kv_dtype,
        scale_mode, _ptr(k_scale), _ptr(v_scale), _ptr(k_scale_cache), _ptr(v_scale_cache),
        float(q_scale), float(prob_scale),
        _ptr(block_table), block_table.shape[1], _ptr(context_lens), cu_seqlens_q.numel() - 1,
        Hq, Hkv, D, k_cache.shape[0], float(softmax_scale), flags, _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _ptr(out),
        out_dtype, _ptr(err_flag), _stream(stream))
    _raise(st, "prefill_attn")
    return out


def quantize_e4m3(x, scale=1.0, out=None, stream=None):
    """e4m3 codes (uint8) of fp32 x / scale, computed on the GPU."""
    _check(x, "x", torch.float32)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(out, "out", torch.uint8)
    st = lib().fp8kv_quantize_e4m3(_ptr(x), float(scale), _ptr(out), x.numel(), _stream(stream))
    _raise(st, "quantize_e4m3")
    return out


def _floats(x):
    if x is None:
        return []
    if isinstance(x, torch.Tensor):
        return [float(e) for e in x.detach().cpu().reshape(-1).tolist()]
    if isinstance(x, (int, float)):
        return [float(x)]
    return [float(e) for e in x]


def resolve_scales(kv_dtype, scale_mode, k_loaded=None, v_loaded=None, q_loaded=-1.0,
                   prob_loaded=-1.0):
    """Scales to use from what a checkpoint loader found; -1.0 (any negative
    value) means "not loaded".  k_loaded / v_loaded: one float (per-tensor) or a
    sequence of Hkv floats (per-head); unused for per-token-head and bf16 caches.
    Returns (k_scales, v_scales, q_scale, prob_scale) with k/v as lists (None
    where the mode has no per-tensor scale).  Host-only (no GPU needed); the
    rules are those of fp8kv_resolve_scales in include/fp8kv.h."""
    per_tensor_like = kv_dtype == KV_E4M3 and scale_mode in (SCALE_PER_TENSOR, SCALE_PER_HEAD)
    if per_tensor_like:
        ks, vs = _floats(k_loaded), _floats(v_loaded)
        if len(ks) != len(vs):
            raise ValueError("k_loaded and v_loaded differ in length")
    else:
        ks = vs = []
    n = len(ks)
    FA = ctypes.c_float * max(n, 1)
    kin, vin, kout, vout = FA(*ks), FA(*vs), FA(), FA()
    q, pr = ctypes.c_float(), ctypes.c_float()
    st = lib().fp8kv_resolve_scales(kv_dtype, scale_mode, n, kin, vin, float(q_loaded),
                                    float(prob_loaded), kout, vout, ctypes.byref(q),
                                    ctypes.byref(pr))
    _raise(st, "resolve_scales")
    if not per_tensor_like:
        return None, None, q.value, pr.value
    return list(kout[:n]), list(vout[:n]), q.value, pr.value


# ---------------------------------------------------------------- rotary and latent calls
# These calls sit in a decode step's launch path, so their checks are one expression of
# plain attribute reads; only when it fails do the slower functions below find out what
# was wrong and say so.
_bf16, _u8, _i64, _i32, _f32 = (torch.bfloat16, torch.uint8, torch.int64, torch.int32,
                                torch.float32)


class _On:
    """Makes a device current for a call (the library launches on the current device)."""

    def __init__(self, device):
        self.device = device
        self.back = torch.cuda.current_device()

    def __enter__(self):
        if self.back != self.device:
            torch.cuda.set_device(self.device)

    def __exit__(self, *exc):
        if self.back != self.device:
            torch.cuda.set_device(self.back)


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_this_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(name, device, stream, *args):
    """Calls the library on `device`, with `stream` (a torch stream; None: that device's
    current one) as the last argument; raises its status."""
    handle = _raw_stream(device) if stream is None else stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if _this_device() == device:
        st = fn(*args, handle)
    else:
        with _On(device):
            st = fn(*args, handle)
    if st != 0:
        raise Fp8kvError(st, name[6:])


def _new(like, shape, dtype, stream):
    """An output or a workspace of a call.  On another stream than the current one it is
    that stream's memory, and the current stream (whose program gets it) may keep it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _p(t):
    return None if t is None else t.data_ptr()


def _rows_ok(t, T, H, D):
    """bf16 [T][H][D] with contiguous heads (any token stride)."""
    if t.dtype is not _bf16 or t.shape != (T, H, D):
        return False
    st = t.stride()
    return st[2] == 1 and (H == 1 or st[1] == D)


def _vec_ok(t, n):
    return t.dtype is _i64 and t.shape == (n,) and t.is_contiguous()


def _dense_ok(t, dtype, shape):
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _scale_ok(kv_dtype, scale_mode, given, cached, rows, heads):
    """The scales that the cache's mode reads are there (the others are ignored)."""
    if kv_dtype == KV_BF16:
        return True
    if scale_mode == SCALE_PER_TOKEN_HEAD:
        return cached is not None and _dense_ok(cached, _f32, rows)
    return (given is not None and given.dtype is _f32 and given.is_contiguous() and
            given.numel() >= (heads if scale_mode == SCALE_PER_HEAD else 1))


def _on_device(device, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != device:
            return False
    return device >= 0


def _say_vector(t, name, n):
    _check(t, name, torch.int64)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name}: expected {n} values")


def _say_rows(t, name, shape):
    _check(t, name, torch.bfloat16, contiguous=False)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1 or (t.dim() == 3 and t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name}: expected contiguous heads (only the token stride may differ)")


def _say_dense(t, name, dtype, shape):
    _check(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _say_scales(kv_dtype, scale_mode, rows, heads, **kw):
    if kv_dtype not in (KV_E4M3, KV_BF16):
        raise ValueError("kv_dtype: KV_E4M3 or KV_BF16")
    if kv_dtype == KV_BF16:
        return
    if scale_mode not in (SCALE_PER_TENSOR, SCALE_PER_HEAD, SCALE_PER_TOKEN_HEAD):
        raise ValueError("scale_mode: one of the SCALE_ constants")
    for n, t in kw.items():
        cached = n.endswith("cache")
        if cached != (scale_mode == SCALE_PER_TOKEN_HEAD):
            continue
        if t is None:
            raise ValueError(f"{n}: needed by this scale_mode")
        _check(t, n, torch.float32)
        if cached and tuple(t.shape) != tuple(rows):
            raise ValueError(f"{n}: expected shape {tuple(rows)}, got {tuple(t.shape)}")
        if not cached and t.numel() < (heads if scale_mode == SCALE_PER_HEAD else 1):
            raise ValueError(f"{n}: too few scales")


def _say_device(device, **tensors):
    for n, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError(f"{n}: expected a CUDA tensor on the same device as the others, "
                             f"got {t.device}")
    raise ValueError("expected CUDA tensors, of shapes and types as documented")


def _out_type(out_dtype):
    if out_dtype == OUT_BF16:
        return _bf16
    if out_dtype == OUT_F32:
        return _f32
    raise ValueError("out_dtype: OUT_F32 or OUT_BF16")


def rope_freqs(rotary_dim, base=10000.0, *, scaling=ROPE_NONE, factor=1.0, original_context=0,
               low=1.0, high=None, device=None):
    """(freqs, mscale) for the rotary calls: freqs int64 [rotary_dim / 2] on `device`
    (None: the CPU), turns per position in 2^-64ths.  low / high: the turns over
    original_context between which YARN (default high 32) and BANDS (default 4) blend.
    See fp8kv_rope_freqs."""
    if high is None:
        high = 32.0 if scaling == ROPE_YARN else 4.0
    freqs = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.int64)
    m = ctypes.c_float(0.0)
    st = lib().fp8kv_rope_freqs(int(rotary_dim), float(base), int(scaling), float(factor),
                                float(original_context), float(low), float(high),
                                ctypes.c_void_p(freqs.data_ptr()), ctypes.byref(m))
    _raise(st, "rope_freqs")
    return (freqs if device is None else freqs.to(device)), m.value


def rope_kv_cache_write(q, k, v, positions, slot_mapping, rope_freqs, k_cache, v_cache, *,
                        kv_dtype, scale_mode=SCALE_PER_TENSOR, interleaved=False, mscale=1.0,
                        k_scale=None, v_scale=None, k_scale_cache=None, v_scale_cache=None,
                        q_out=None, err_flag=None, stream=None):
    """Rotary positions of q [T][Hq][D] and k [T][Hkv][D] (bf16; views of one
    projection's output are fine) and the store of k and v at slot_mapping into the
    paged cache, in one kernel.  Returns the rotated q (q_out, which may be q itself;
    None q: None).  rope_freqs: int64 [rotary_dim / 2] (see rope_freqs()).  See
    fp8kv_rope_kv_cache_write."""
    T, Hkv, D = k.shape
    Hq = 0 if q is None else q.shape[1]
    nb = k_cache.shape[0]
    dev = k.get_device()
    cdt = _u8 if kv_dtype == KV_E4M3 else _bf16
    pages, rows = (nb, Hkv, PAGE_SIZE, D), (nb, Hkv, PAGE_SIZE)
    if not (_rows_ok(k, T, Hkv, D) and _rows_ok(v, T, Hkv, D) and
            (q is None or _rows_ok(q, T, Hq, D)) and
            (q_out is None or q is not None and _rows_ok(q_out, T, Hq, D)) and
            _vec_ok(positions, T) and _vec_ok(slot_mapping, T) and
            rope_freqs.dtype is _i64 and rope_freqs.is_contiguous() and
            _dense_ok(k_cache, cdt, pages) and _dense_ok(v_cache, cdt, pages) and
            _scale_ok(kv_dtype, scale_mode, k_scale, k_scale_cache, rows, Hkv) and
            _scale_ok(kv_dtype, scale_mode, v_scale, v_scale_cache, rows, Hkv) and
            (err_flag is None or err_flag.dtype is _i32) and
            _on_device(dev, q, v, positions, slot_mapping, rope_freqs, k_cache, v_cache, k_scale,
                       v_scale, k_scale_cache, v_scale_cache, q_out, err_flag)):
        _say_rows(k, "k", (T, Hkv, D))
        _say_rows(v, "v", (T, Hkv, D))
        if q is not None:
            _say_rows(q, "q", (T, Hq, D))
        if q_out is not None:
            _say_rows(q_out, "q_out", (T, Hq, D))
        _say_vector(positions, "positions", T)
        _say_vector(slot_mapping, "slot_mapping", T)
        _check(rope_freqs, "rope_freqs", torch.int64)
        _say_dense(k_cache, "k_cache", cdt, pages)
        _say_dense(v_cache, "v_cache", cdt, pages)
        _say_scales(kv_dtype, scale_mode, rows, Hkv, k_scale=k_scale, v_scale=v_scale,
                    k_scale_cache=k_scale_cache, v_scale_cache=v_scale_cache)
        _check(err_flag, "err_flag", torch.int32)
        _say_device(dev, q=q, v=v, positions=positions, slot_mapping=slot_mapping,
                    rope_freqs=rope_freqs, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale,
                    v_scale=v_scale, k_scale_cache=k_scale_cache, v_scale_cache=v_scale_cache,
                    q_out=q_out, err_flag=err_flag)
    if q is not None and q_out is None:
        q_out = _new(q, (T, Hq, D), _bf16, stream)
    _launch("fp8kv_rope_kv_cache_write", dev, stream, _p(q), 0 if q is None else q.stride(0),
            k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), positions.data_ptr(),
            slot_mapping.data_ptr(), rope_freqs.data_ptr(), 2 * rope_freqs.numel(), interleaved,
            mscale, T, Hq, Hkv, D, _p(q_out), 0 if q is None else q_out.stride(0),
            k_cache.data_ptr(), v_cache.data_ptr(), nb, kv_dtype, scale_mode, _p(k_scale),
            _p(v_scale), _p(k_scale_cache), _p(v_scale_cache), _p(err_flag))
    return q_out


def kv_cache_read(k_cache, v_cache, slot_mapping, *, kv_dtype, scale_mode=SCALE_PER_TENSOR,
                  k_scale=None, v_scale=None, k_scale_cache=None, v_scale_cache=None, k_out=None,
                  v_out=None, out_dtype=OUT_BF16, err_flag=None, stream=None):
    """The rows at slot_mapping as values: (k, v), each [T][Hkv][D] bf16 or fp32.
    Negative slots give zero rows.  See fp8kv_kv_cache_read."""
    nb, Hkv, _, D = k_cache.shape
    T = slot_mapping.shape[0]
    dev = k_cache.get_device()
    cdt, dt = _u8 if kv_dtype == KV_E4M3 else _bf16, _out_type(out_dtype)
    pages, rows, shape = (nb, Hkv, PAGE_SIZE, D), (nb, Hkv, PAGE_SIZE), (T, Hkv, D)
    if not (_dense_ok(k_cache, cdt, pages) and _dense_ok(v_cache, cdt, pages) and
            _vec_ok(slot_mapping, T) and
            _scale_ok(kv_dtype, scale_mode, k_scale, k_scale_cache, rows, Hkv) and
            _scale_ok(kv_dtype, scale_mode, v_scale, v_scale_cache, rows, Hkv) and
            (k_out is None or _dense_ok(k_out, dt, shape)) and
            (v_out is None or _dense_ok(v_out, dt, shape)) and
            (err_flag is None or err_flag.dtype is _i32) and
            _on_device(dev, v_cache, slot_mapping, k_scale, v_scale, k_scale_cache, v_scale_cache,
                       k_out, v_out, err_flag)):
        _say_dense(k_cache, "k_cache", cdt, pages)
        _say_dense(v_cache, "v_cache", cdt, pages)
        _say_vector(slot_mapping, "slot_mapping", T)
        _say_scales(kv_dtype, scale_mode, rows, Hkv, k_scale=k_scale, v_scale=v_scale,
                    k_scale_cache=k_scale_cache, v_scale_cache=v_scale_cache)
        for n, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                _say_dense(t, n, dt, shape)
        _check(err_flag, "err_flag", torch.int32)
        _say_device(dev, v_cache=v_cache, slot_mapping=slot_mapping, k_scale=k_scale,
                    v_scale=v_scale, k_scale_cache=k_scale_cache, v_scale_cache=v_scale_cache,
                    k_out=k_out, v_out=v_out, err_flag=err_flag)
    if k_out is None:
        k_out = _new(k_cache, shape, dt, stream)
    if v_out is None:
        v_out = _new(k_cache, shape, dt, stream)
    _launch("fp8kv_kv_cache_read", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), nb,
            kv_dtype, scale_mode, _p(k_scale), _p(v_scale), _p(k_scale_cache), _p(v_scale_cache),
            slot_mapping.data_ptr(), T, Hkv, D, k_out.data_ptr(), v_out.data_ptr(), out_dtype,
            _p(err_flag))
    return k_out, v_out


def latent_cache_write(c, k_pe, slot_mapping, cache, *, kv_dtype, scale_mode=SCALE_PER_TENSOR,
                       scale=None, scale_cache=None, positions=None, rope_freqs=None,
                       interleaved=False, mscale=1.0, q_pe=None, q_pe_out=None, err_flag=None,
                       stream=None):
    """Store latent rows [c | rotated k_pe] (bf16 [T][L] and [T][64]) at slot_mapping
    into the latent cache [num_blocks][16][L + 64], and rotate q_pe [T][H][64] in the
    same launch.  positions / rope_freqs None: nothing is rotated.  q_pe_out: None
    allocates it; q_pe itself, or a view such as q[..., L:].  Returns q_pe_out (None
    without q_pe).  See fp8kv_latent_cache_write."""
    T, L = c.shape
    nb = cache.shape[0]
    dev = c.get_device()
    cdt = _u8 if kv_dtype == KV_E4M3 else _bf16
    H = 0 if q_pe is None else q_pe.shape[1]
    q_shape = (T, H, LATENT_ROPE)
    if not (c.dtype is _bf16 and c.stride(1) == 1 and k_pe.dtype is _bf16 and
            k_pe.shape == (T, LATENT_ROPE) and k_pe.stride(1) == 1 and _vec_ok(slot_mapping, T) and
            _dense_ok(cache, cdt, (nb, PAGE_SIZE, L + LATENT_ROPE)) and
            _scale_ok(kv_dtype, scale_mode, scale, scale_cache, (nb, PAGE_SIZE), 1) and
            (positions is None and rope_freqs is None or
             positions is not None and rope_freqs is not None and _vec_ok(positions, T) and
             _vec_ok(rope_freqs, LATENT_ROPE // 2)) and
            (q_pe is None and q_pe_out is None or
             q_pe is not None and q_pe.dtype is _bf16 and q_pe.shape == q_shape and
             q_pe.stride(2) == 1) and
            (q_pe_out is None or q_pe_out.dtype is _bf16 and q_pe_out.shape == q_shape and
             q_pe_out.stride(2) == 1) and
            (err_flag is None or err_flag.dtype is _i32) and
            _on_device(dev, k_pe, slot_mapping, cache, scale, scale_cache, positions, rope_freqs,
                       q_pe, q_pe_out, err_flag)):
        _say_rows(c, "c", (T, L))
        _say_rows(k_pe, "k_pe", (T, LATENT_ROPE))
        _say_vector(slot_mapping, "slot_mapping", T)
        _say_dense(cache, "cache", cdt, (nb, PAGE_SIZE, L + LATENT_ROPE))
        _say_scales(kv_dtype, scale_mode, (nb, PAGE_SIZE), 1, scale=scale, scale_cache=scale_cache)
        if (positions is None) != (rope_freqs is None):
            raise ValueError("positions and rope_freqs: both or neither")
        if positions is not None:
            _say_vector(positions, "positions", T)
            _say_vector(rope_freqs, "rope_freqs", LATENT_ROPE // 2)
        if q_pe is None and q_pe_out is not None:
            raise ValueError("q_pe_out without q_pe")
        for n, t in (("q_pe", q_pe), ("q_pe_out", q_pe_out)):
            if t is not None:
                _check(t, n, torch.bfloat16, contiguous=False)
                if tuple(t.shape) != q_shape or t.stride(2) != 1:
                    raise ValueError(f"{n}: expected rows of shape {q_shape}")
        _check(err_flag, "err_flag", torch.int32)
        _say_device(dev, k_pe=k_pe, slot_mapping=slot_mapping, cache=cache, scale=scale,
                    scale_cache=scale_cache, positions=positions, rope_freqs=rope_freqs,
                    q_pe=q_pe, q_pe_out=q_pe_out, err_flag=err_flag)
    qs = os_ = (0, 0)
    if q_pe is not None:
        if q_pe_out is None:
            q_pe_out = _new(q_pe, q_shape, _bf16, stream)
        qs, os_ = q_pe.stride(), q_pe_out.stride()
    _launch("fp8kv_latent_cache_write", dev, stream, c.data_ptr(), c.stride(0), k_pe.data_ptr(),
            k_pe.stride(0), _p(positions), _p(rope_freqs), interleaved, mscale,
            slot_mapping.data_ptr(), T, L, cache.data_ptr(), nb, kv_dtype, scale_mode, _p(scale),
            _p(scale_cache), _p(q_pe), qs[0], qs[1], _p(q_pe_out), os_[0], os_[1], H, _p(err_flag))
    return q_pe_out


def latent_cache_read(cache, slot_mapping, *, kv_dtype, scale_mode=SCALE_PER_TENSOR, scale=None,
                      scale_cache=None, out=None, out_dtype=OUT_BF16, err_flag=None, stream=None):
    """The latent rows at slot_mapping as values [T][L + 64] (bf16 or fp32), e.g. for
    the up-projection to per-head keys and values.  See fp8kv_latent_cache_read."""
    nb, _, W = cache.shape
    T = slot_mapping.shape[0]
    dev = cache.get_device()
    cdt, dt = _u8 if kv_dtype == KV_E4M3 else _bf16, _out_type(out_dtype)
    if not (_dense_ok(cache, cdt, (nb, PAGE_SIZE, W)) and _vec_ok(slot_mapping, T) and
            _scale_ok(kv_dtype, scale_mode, scale, scale_cache, (nb, PAGE_SIZE), 1) and
            (out is None or _dense_ok(out, dt, (T, W))) and
            (err_flag is None or err_flag.dtype is _i32) and
            _on_device(dev, slot_mapping, scale, scale_cache, out, err_flag)):
        _say_dense(cache, "cache", cdt, (nb, PAGE_SIZE, W))
        _say_vector(slot_mapping, "slot_mapping", T)
        _say_scales(kv_dtype, scale_mode, (nb, PAGE_SIZE), 1, scale=scale, scale_cache=scale_cache)
        if out is not None:
            _say_dense(out, "out", dt, (T, W))
        _check(err_flag, "err_flag", torch.int32)
        _say_device(dev, slot_mapping=slot_mapping, scale=scale, scale_cache=scale_cache, out=out,
                    err_flag=err_flag)
    if out is None:
        out = _new(cache, (T, W), dt, stream)
    _launch("fp8kv_latent_cache_read", dev, stream, cache.data_ptr(), nb, kv_dtype, scale_mode,
            _p(scale), _p(scale_cache), slot_mapping.data_ptr(), T, W - LATENT_ROPE,
            out.data_ptr(), out_dtype, _p(err_flag))
    return out


def latent_attn_plan(B, S, H, latent_dim, max_blocks_per_seq, num_splits=0):
    """(workers, workspace_bytes) that latent_decode_attn will use on the current device."""
    s, w = ctypes.c_int(0), ctypes.c_size_t(0)
    st = lib().fp8kv_latent_attn_plan(B, S, H, latent_dim, max_blocks_per_seq, num_splits,
                                      ctypes.byref(s), ctypes.byref(w))
    _raise(st, "latent_attn_plan")
    return s.value, w.value


@functools.lru_cache(maxsize=256)
def _latent_workspace_bytes(device, *shape):
    with _On(device):
        return latent_attn_plan(*shape)[1]


def latent_decode_attn(q, cache, block_table, context_lens, *, latent_dim, kv_dtype,
                       softmax_scale, scale_mode=SCALE_PER_TENSOR, scale=None, scale_cache=None,
                       num_splits=0, workspace=None, out=None, out_dtype=OUT_F32, err_flag=None,
                       stream=None):
    """Absorbed latent attention of q [B][S][H][L + 64] (bf16; [B][H][L + 64] for one
    token a sequence) over the paged latent cache; returns [B][S][H][L] (or [B][H][L]).
    Query s sees the keys up to position context_lens - S + s.  softmax_scale is the
    model's (1 / sqrt of its expanded head dimension), so it has no default.  A workspace
    under latent_attn_plan()'s bytes for the same sizes and num_splits is not used: one is
    allocated for the call.  See fp8kv_latent_decode_attn."""
    L, W = latent_dim, latent_dim + LATENT_ROPE
    qs = q.shape
    B, H = qs[0], qs[-2]
    S = qs[1] if len(qs) == 4 else 1
    nb, mbs = cache.shape[0], block_table.shape[1]
    dev = cache.get_device()
    cdt, dt = _u8 if kv_dtype == KV_E4M3 else _bf16, _out_type(out_dtype)
    shape = (B, S, H, L) if len(qs) == 4 else (B, H, L)
    if not (q.dtype is _bf16 and 3 <= len(qs) <= 4 and qs[-1] == W and q.is_contiguous() and
            _dense_ok(cache, cdt, (nb, PAGE_SIZE, W)) and
            _dense_ok(block_table, _i32, (B, mbs)) and _dense_ok(context_lens, _i32, (B,)) and
            _scale_ok(kv_dtype, scale_mode, scale, scale_cache, (nb, PAGE_SIZE), 1) and
            (out is None or _dense_ok(out, dt, shape)) and
            (workspace is None or workspace.is_contiguous()) and
            (err_flag is None or err_flag.dtype is _i32) and
            _on_device(dev, q, block_table, context_lens, scale, scale_cache, workspace, out,
                       err_flag)):
        _check(q, "q", torch.bfloat16)
        if not 3 <= q.dim() <= 4 or q.shape[-1] != W:
            raise ValueError(f"q: expected [B][S][H][{W}] or [B][H][{W}]")
        _say_dense(cache, "cache", cdt, (nb, PAGE_SIZE, W))
        _say_dense(block_table, "block_table", torch.int32, (B, mbs))
        _say_dense(context_lens, "context_lens", torch.int32, (B,))
        _say_scales(kv_dtype, scale_mode, (nb, PAGE_SIZE), 1, scale=scale, scale_cache=scale_cache)
        if out is not None:
            _say_dense(out, "out", dt, shape)
        _check(workspace, "workspace")
        _check(err_flag, "err_flag", torch.int32)
        _say_device(dev, q=q, block_table=block_table, context_lens=context_lens, scale=scale,
                    scale_cache=scale_cache, workspace=workspace, out=out, err_flag=err_flag)
    need = _latent_workspace_bytes(dev, B, S, H, L, mbs, num_splits)
    have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if have < need:
        workspace, have = _new(cache, (need,), _u8, stream), need
    if out is None:
        out = _new(cache, shape, dt, stream)
    _launch("fp8kv_latent_decode_attn", dev, stream, q.data_ptr(), cache.data_ptr(), kv_dtype,
            scale_mode, _p(scale), _p(scale_cache), block_table.data_ptr(), mbs,
            context_lens.data_ptr(), B, S, H, L, nb, softmax_scale, num_splits,
            workspace.data_ptr(), have, out.data_ptr(), out_dtype, _p(err_flag))
    return out
