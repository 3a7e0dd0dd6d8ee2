"""K3 DFlash drafter block attention on sm_103a: thin Python binding.

The compute lives in ``libk3da.so`` (hand-written CUDA, C ABI declared in
``include/k3da.h``).  This module only marshals torch tensors into that ABI:
pointers (device memory, or pinned host memory where the ABI allows it),
sizes, dtype codes and the current CUDA stream.  There is no
CPU fallback: if the library is missing, every call raises.

Operation (page "[None][feat] Share Kimi K3 FP4 modeling and add NVFP4
support on SM103", NVIDIA/TensorRT-LLM PR #20532, commit adding
k3_drafter_attn / k3_drafter_attn_qknorm): each of R <= 8 requests brings a
block of B <= 8 draft tokens; every block token attends densely to its
request's paged context (HND pages of 64) and to its own block's K/V, taken
from qkv and never written to the pool; GQA 6:1 (6/1 or 24/4 heads),
head_dim 64.  ``k3da_attn_qknorm`` first applies per-head q/k RMSNorm and
NeoX RoPE.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

__all__ = [
    "K3daError", "library_path", "load_library", "workspace_bytes", "k3da_attn",
    "k3da_attn_qknorm", "STATUS_BAD_LENGTH", "STATUS_BAD_PAGE", "STATUS_TIMEOUT",
    "k3da_kv_append", "k3da_kv_append_qknorm", "k3da_kv_gather", "k3da_chunk_attn",
    "chunk_workspace_bytes", "alloc_chunk_workspace", "alloc_cache",
    "k3da_token_probs", "k3da_verify", "k3da_pages_resize", "k3da_pages_fork", "k3da_pages_compact", "k3da_kv_copy",
    "alloc_pages", "compact_workspace_bytes", "alloc_compact_workspace",
    "STATUS_BAD_TOKEN", "STATUS_NO_PAGES", "STATUS_BAD_COUNT", "STATUS_BAD_REQUEST",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libk3da.so")
_lock = threading.Lock()
_lib = None

OK, EINVAL, EUNSUPPORTED, ECUDA, EWORKSPACE = 0, -1, -2, -3, -4
STATUS_BAD_LENGTH, STATUS_BAD_PAGE, STATUS_TIMEOUT = 1, 2, 4
STATUS_BAD_TOKEN, STATUS_NO_PAGES, STATUS_BAD_COUNT, STATUS_BAD_REQUEST = 8, 16, 32, 64
POS_I32, POS_I64 = 0, 1
CACHE_BF16, CACHE_E4M3 = 0, 1
MASKS = {"causal": 0, "full": 1, "context": 2}
LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_CHUNK_REQUESTS = 1024
EXPORTED = ["k3da_workspace_bytes", "k3da_attn", "k3da_attn_qknorm", "k3da_attn_qknorm_noalloc",
            "k3da_noalloc_scratch_bytes", "k3da_split_grid", "k3da_set_phase_event",
            "k3da_error_string", "k3da_version", "k3da_qk_norm_rope", "k3da_attn_qknorm_yarn",
            "k3da_qk_norm_rope_yarn", "k3da_selftest_wait_timeout", "k3da_kv_append",
            "k3da_kv_append_qknorm", "k3da_kv_gather", "k3da_chunk_workspace_bytes", "k3da_chunk_attn",
            "k3da_packed_call", "k3da_token_probs", "k3da_verify", "k3da_pages_resize", "k3da_pages_fork",
            "k3da_compact_workspace_bytes", "k3da_pages_compact", "k3da_kv_copy"]
# k3da_packed_call: a call's number, how many words it has, and what they are.
_PACKED = {what: (number, len(words), struct.Struct(words).pack) for number, (what, words) in enumerate((
    ("k3da_kv_append", "q" * 16), ("k3da_kv_append_qknorm", "q" * 18 + "dd" + "q" * 4), ("k3da_kv_gather", "q" * 16),
    ("k3da_chunk_attn", "q" * 18 + "d" + "q" * 4), ("k3da_token_probs", "q" * 12), ("k3da_verify", "q" * 15),
    ("k3da_pages_resize", "q" * 10), ("k3da_pages_fork", "q" * 11), ("k3da_pages_compact", "q" * 13),
    ("k3da_kv_copy", "q" * 11)))}


class Yarn(ctypes.Structure):
    """k3da_yarn: YaRN RoPE scaling (factor, original_max_position, beta_fast,
    beta_slow, mscale).  mscale 0 asks the library for the YaRN paper's
    default multiplier."""
    _fields_ = [("factor", ctypes.c_float), ("original_max_position", ctypes.c_float),
                ("beta_fast", ctypes.c_float), ("beta_slow", ctypes.c_float), ("mscale", ctypes.c_float)]

    @classmethod
    def of(cls, factor: float, original_max_position: float, beta_fast: float = 32.0,
           beta_slow: float = 1.0, mscale: float = 0.0):
        return cls(factor, original_max_position, beta_fast, beta_slow, mscale)

    def as_dict(self):
        return {k: float(getattr(self, k)) for k, _ in self._fields_}


class K3daError(ValueError):
    """A call refused by the library (host-side check) or a device status."""


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libk3da.so (ctypes) and declare its signatures; raise if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -m speculative_decoding_drafter_k3_gb300.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(_LIB_PATH)
        c_int, c_i64, c_sz, vp, c_f = (ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                                       ctypes.c_void_p, ctypes.c_float)
        lib.k3da_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.k3da_workspace_bytes.restype = c_sz
        common = [vp, vp, vp, c_i64, vp, c_int, vp, c_int, c_int, c_int, c_int, c_int, c_f]
        lib.k3da_attn.argtypes = common + [vp, c_sz, vp, vp]
        lib.k3da_attn.restype = c_int
        lib.k3da_attn_qknorm.argtypes = common + [vp, c_int, vp, vp, c_f, c_f, vp, c_sz, vp, vp]
        lib.k3da_attn_qknorm.restype = c_int
        lib.k3da_error_string.argtypes = [c_int]
        lib.k3da_error_string.restype = ctypes.c_char_p
        lib.k3da_attn_qknorm_noalloc.argtypes = common + [vp, c_int, vp, vp, c_f, c_f, vp, vp]
        lib.k3da_attn_qknorm_noalloc.restype = c_int
        lib.k3da_noalloc_scratch_bytes.argtypes = []
        lib.k3da_noalloc_scratch_bytes.restype = c_sz
        lib.k3da_split_grid.argtypes = [c_int]
        lib.k3da_split_grid.restype = c_int
        lib.k3da_set_phase_event.argtypes = [vp]
        lib.k3da_set_phase_event.restype = c_int
        lib.k3da_version.argtypes = []
        lib.k3da_version.restype = c_int
        lib.k3da_qk_norm_rope.argtypes = [vp, c_int, c_int, c_int, c_int, vp, c_int, vp, vp, c_f, c_f, vp]
        lib.k3da_qk_norm_rope.restype = c_int
        yp = ctypes.POINTER(Yarn)
        lib.k3da_attn_qknorm_yarn.argtypes = common + [vp, c_int, vp, vp, c_f, c_f, yp, vp, c_sz, vp, vp]
        lib.k3da_attn_qknorm_yarn.restype = c_int
        lib.k3da_qk_norm_rope_yarn.argtypes = [vp, c_int, c_int, c_int, c_int, vp, c_int, vp, vp, c_f, c_f, yp, vp]
        lib.k3da_qk_norm_rope_yarn.restype = c_int
        lib.k3da_selftest_wait_timeout.argtypes = [vp, ctypes.c_ulonglong, vp]
        lib.k3da_selftest_wait_timeout.restype = c_int
        cache = [vp, c_int, vp, c_i64, vp, c_int, vp, vp, c_int]
        lib.k3da_kv_append.argtypes = cache + [vp, c_int, c_int, c_int, c_int, vp, vp]
        lib.k3da_kv_append.restype = c_int
        lib.k3da_kv_append_qknorm.argtypes = cache + [vp, c_int, c_int, c_int, c_int, vp, c_int, vp, vp, c_f, c_f,
                                                      yp, vp, vp, vp]
        lib.k3da_kv_append_qknorm.restype = c_int
        lib.k3da_kv_gather.argtypes = [vp, vp] + cache + [c_int, c_int, c_int, vp, vp]
        lib.k3da_kv_gather.restype = c_int
        lib.k3da_chunk_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.k3da_chunk_workspace_bytes.restype = c_sz
        lib.k3da_chunk_attn.argtypes = [vp, vp, vp, c_i64, c_int] + cache + [c_int, c_int, c_int, c_int, c_f, vp, c_sz,
                                                                             vp, vp]
        lib.k3da_chunk_attn.restype = c_int
        lib.k3da_token_probs.argtypes = [vp, c_i64, vp, c_int, c_i64, c_int, c_int, vp, vp, c_int, vp, vp]
        lib.k3da_token_probs.restype = c_int
        lib.k3da_verify.argtypes = [vp, vp, vp, c_int, vp, c_i64, vp, c_i64, vp, c_int, c_int, vp, c_int, vp, vp]
        lib.k3da_verify.restype = c_int
        book = [vp, c_int, vp, c_int, vp, c_i64]
        lib.k3da_pages_resize.argtypes = book + [vp, vp, vp, vp]
        lib.k3da_pages_resize.restype = c_int
        lib.k3da_pages_fork.argtypes = book + [vp, vp, c_int, vp, vp]
        lib.k3da_pages_fork.restype = c_int
        lib.k3da_compact_workspace_bytes.argtypes = [c_i64]
        lib.k3da_compact_workspace_bytes.restype = c_sz
        lib.k3da_pages_compact.argtypes = book + [vp, c_int, vp, vp, c_sz, vp, vp]
        lib.k3da_pages_compact.restype = c_int
        lib.k3da_kv_copy.argtypes = [vp, c_int, vp, c_i64, c_int, c_int, vp, c_int, vp, vp, vp]
        lib.k3da_kv_copy.restype = c_int
        lib.k3da_packed_call.argtypes = [c_int, ctypes.c_char_p, c_int]
        lib.k3da_packed_call.restype = c_int
        _lib = lib
        return lib


def error_string(code: int) -> str:
    return load_library().k3da_error_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise K3daError(f"{what}: {error_string(rc)} (code {rc})")


def workspace_bytes(num_requests: int, block_len: int, num_q_heads: int, num_kv_heads: int,
                    page_stride: int) -> int:
    n = load_library().k3da_workspace_bytes(num_requests, block_len, num_q_heads, num_kv_heads,
                                            page_stride)
    if n == 0:
        raise K3daError("workspace_bytes: sizes out of contract")
    return int(n)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _device_or_pinned(name, t):
    """out, qkv, page_table, ctx_lens and positions may live in pinned host
    memory, which the kernels read (or write) across the host link."""
    if not (t.is_cuda or t.is_pinned()) or not t.is_contiguous():
        raise K3daError(f"{name} must be a contiguous CUDA tensor or a contiguous pinned host tensor")


def _device_scratch(workspace, status):
    """The workspace and the status word are always device memory."""
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise K3daError("workspace must be a contiguous CUDA tensor")
    if status is not None and (not status.is_cuda or status.dtype != torch.int32):
        raise K3daError("status must be an int32 CUDA tensor")


def _shape_args(out, qkv, kv_pool, page_table, ctx_lens, block_len, num_q_heads, num_kv_heads):
    for name, t in [("out", out), ("qkv", qkv), ("page_table", page_table), ("ctx_lens", ctx_lens)]:
        _device_or_pinned(name, t)
    if not kv_pool.is_cuda or not kv_pool.is_contiguous():
        raise K3daError("kv_pool must be a contiguous CUDA tensor")
    if qkv.dtype != torch.bfloat16 or out.dtype != torch.bfloat16 or kv_pool.dtype != torch.bfloat16:
        raise K3daError("qkv, out and kv_pool must be bf16")
    if page_table.dtype != torch.int32 or ctx_lens.dtype != torch.int32:
        raise K3daError("page_table and ctx_lens must be int32")
    if page_table.dim() != 2 or kv_pool.dim() != 5:
        raise K3daError("page_table must be [R, S] and kv_pool [pages, 2, Hkv, 64, 64]")
    R = page_table.shape[0]
    T = R * block_len
    D = kv_pool.shape[-1]
    if (tuple(kv_pool.shape[1:]) != (2, num_kv_heads, 64, D) or ctx_lens.numel() != R
            or tuple(qkv.shape) != (T, (num_q_heads + 2 * num_kv_heads) * D)
            or tuple(out.shape) != (T, num_q_heads * D)):
        raise K3daError("tensor shapes disagree with (R, B, Hq, Hkv, head_dim)")
    return R, kv_pool.shape[0], page_table.shape[1], D


def _qknorm_args(positions, q_norm_w, k_norm_w, T, D):
    """Checks the fused variant's extra tensors; returns the positions' dtype code."""
    if positions.dtype not in (torch.int32, torch.int64) or positions.numel() != T:
        raise K3daError("positions must be [T] int32 or int64")
    _device_or_pinned("positions", positions)
    for name, t in [("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)]:
        if not t.is_cuda or not t.is_contiguous():
            raise K3daError(f"{name} must be a contiguous CUDA tensor")
    if q_norm_w.dtype != torch.bfloat16 or k_norm_w.dtype != torch.bfloat16 or \
            q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise K3daError("norm weights must be [64] bf16")
    return POS_I64 if positions.dtype == torch.int64 else POS_I32


def k3da_attn(out, qkv, kv_pool, page_table, ctx_lens, *, block_len: int, num_q_heads: int,
              num_kv_heads: int, softmax_scale: float = 0.125, workspace, status=None,
              stream=None):
    """Block attention on already normalised and roped q/k (C: k3da_attn)."""
    lib = load_library()
    R, num_pages, S, D = _shape_args(out, qkv, kv_pool, page_table, ctx_lens, block_len,
                                     num_q_heads, num_kv_heads)
    _device_scratch(workspace, status)
    rc = lib.k3da_attn(_ptr(out), _ptr(qkv), _ptr(kv_pool), num_pages, _ptr(page_table), S,
                       _ptr(ctx_lens), R, block_len, num_q_heads, num_kv_heads, D,
                       float(softmax_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
                       _ptr(status), _stream(stream))
    _check(rc, "k3da_attn")
    return out


def k3da_attn_qknorm(out, qkv, kv_pool, page_table, ctx_lens, positions, q_norm_w, k_norm_w, *,
                     block_len: int, num_q_heads: int, num_kv_heads: int,
                     softmax_scale: float = 0.125, eps: float = 1e-5, rope_base: float = 10000.0,
                     workspace, status=None, stream=None, yarn=None):
    """Block attention with fused q/k RMSNorm + NeoX RoPE (C: k3da_attn_qknorm);
    with ``yarn`` (a ``Yarn``), YaRN RoPE (C: k3da_attn_qknorm_yarn)."""
    lib = load_library()
    R, num_pages, S, D = _shape_args(out, qkv, kv_pool, page_table, ctx_lens, block_len,
                                     num_q_heads, num_kv_heads)
    _device_scratch(workspace, status)
    pos_code = _qknorm_args(positions, q_norm_w, k_norm_w, R * block_len, D)
    args = [_ptr(out), _ptr(qkv), _ptr(kv_pool), num_pages, _ptr(page_table), S, _ptr(ctx_lens), R,
            block_len, num_q_heads, num_kv_heads, D, float(softmax_scale), _ptr(positions), pos_code,
            _ptr(q_norm_w), _ptr(k_norm_w), float(eps), float(rope_base)]
    tail = [_ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)]
    if yarn is None:
        rc = lib.k3da_attn_qknorm(*args, *tail)
        _check(rc, "k3da_attn_qknorm")
    else:
        rc = lib.k3da_attn_qknorm_yarn(*args, ctypes.byref(yarn), *tail)
        _check(rc, "k3da_attn_qknorm_yarn")
    return out


def k3da_qk_norm_rope(qkv, positions, q_norm_w, k_norm_w, *, num_q_heads: int, num_kv_heads: int,
                      eps: float = 1e-5, rope_base: float = 10000.0, stream=None, yarn=None):
    """The fused q/k RMSNorm + NeoX RoPE cell, in place on the q and k heads
    of ``qkv`` ``[T, (Hq+2Hkv)*64]`` bf16 (C: k3da_qk_norm_rope); with
    ``yarn`` (a ``Yarn``), YaRN RoPE (C: k3da_qk_norm_rope_yarn)."""
    lib = load_library()
    for name, t in [("qkv", qkv), ("positions", positions), ("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)]:
        if not t.is_cuda or not t.is_contiguous():
            raise K3daError(f"{name} must be a contiguous CUDA tensor")
    if qkv.dtype != torch.bfloat16 or qkv.dim() != 2:
        raise K3daError("qkv must be [T, (Hq+2Hkv)*64] bf16")
    D = qkv.shape[1] // (num_q_heads + 2 * num_kv_heads)
    T = qkv.shape[0]
    if positions.dtype not in (torch.int32, torch.int64) or positions.numel() != T:
        raise K3daError("positions must be [T] int32 or int64")
    if q_norm_w.dtype != torch.bfloat16 or k_norm_w.dtype != torch.bfloat16 or \
            q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise K3daError("norm weights must be [head_dim] bf16")
    pos_code = POS_I64 if positions.dtype == torch.int64 else POS_I32
    args = [_ptr(qkv), T, num_q_heads, num_kv_heads, D, _ptr(positions), pos_code, _ptr(q_norm_w),
            _ptr(k_norm_w), float(eps), float(rope_base)]
    if yarn is None:
        rc = lib.k3da_qk_norm_rope(*args, _stream(stream))
        _check(rc, "k3da_qk_norm_rope")
    else:
        rc = lib.k3da_qk_norm_rope_yarn(*args, ctypes.byref(yarn), _stream(stream))
        _check(rc, "k3da_qk_norm_rope_yarn")
    return qkv


def alloc_workspace(num_requests: int, block_len: int, num_q_heads: int, num_kv_heads: int,
                    page_stride: int, device=None) -> torch.Tensor:
    """A workspace tensor (uint8, 256-byte aligned by torch) for these sizes."""
    device = torch.device("cuda") if device is None else torch.device(device)
    n = workspace_bytes(num_requests, block_len, num_q_heads, num_kv_heads, page_stride)
    return torch.empty(n, dtype=torch.uint8, device=device)


def case_workspace(case) -> torch.Tensor:
    return alloc_workspace(case.R, case.B, case.Hq, case.Hkv, case.page_stride, case.pool.device)


def run_case(case, out=None, workspace=None, status=None, stream=None, yarn=None):
    """Run the op on a ``workloads.Case`` whose pool and norm weights are on
    the GPU; its qkv, page table, lengths and positions may be pinned host
    tensors (``yarn``: YaRN RoPE for the fused variant)."""
    if out is None:
        out = torch.empty(case.T, case.Hq * case.D, dtype=torch.bfloat16, device=case.pool.device)
    if workspace is None:
        workspace = case_workspace(case)
    kw = dict(block_len=case.B, num_q_heads=case.Hq, num_kv_heads=case.Hkv,
              softmax_scale=case.scale, workspace=workspace, status=status, stream=stream)
    if case.qknorm:
        return k3da_attn_qknorm(out, case.qkv, case.pool, case.page_table, case.ctx_lens,
                                case.positions, case.q_norm_w, case.k_norm_w, eps=case.eps,
                                rope_base=case.rope_base, yarn=yarn, **kw)
    return k3da_attn(out, case.qkv, case.pool, case.page_table, case.ctx_lens, **kw)


def set_phase_event(event):
    """Record ``event`` (a torch.cuda.Event) between the split pass and the
    combine of every later call from this thread; None turns it off."""
    if event is None:
        handle = None
    else:
        handle = ctypes.c_void_p(event.cuda_event)
    _check(load_library().k3da_set_phase_event(handle), "k3da_set_phase_event")


def split_grid(device: int = -1) -> int:
    """CTAs the split pass launches on ``device`` (SMs x CTAs per SM)."""
    return int(load_library().k3da_split_grid(device))


def k3da_attn_qknorm_noalloc(out, qkv, kv_pool, page_table, ctx_lens, positions, q_norm_w, k_norm_w, *,
                             block_len: int, num_q_heads: int, num_kv_heads: int,
                             softmax_scale: float = 0.125, eps: float = 1e-5,
                             rope_base: float = 10000.0, status=None, stream=None):
    """k3da_attn_qknorm without a workspace argument, for callers that cannot
    allocate: the library's fixed per-GPU scratch array is used instead
    (C: k3da_attn_qknorm_noalloc; calls that overlap on the GPU race on it)."""
    lib = load_library()
    R, num_pages, S, D = _shape_args(out, qkv, kv_pool, page_table, ctx_lens, block_len,
                                     num_q_heads, num_kv_heads)
    _device_scratch(None, status)
    pos_code = _qknorm_args(positions, q_norm_w, k_norm_w, R * block_len, D)
    rc = lib.k3da_attn_qknorm_noalloc(_ptr(out), _ptr(qkv), _ptr(kv_pool), num_pages, _ptr(page_table),
                                      S, _ptr(ctx_lens), R, block_len, num_q_heads, num_kv_heads, D,
                                      float(softmax_scale), _ptr(positions), pos_code, _ptr(q_norm_w),
                                      _ptr(k_norm_w), float(eps), float(rope_base), _ptr(status),
                                      _stream(stream))
    _check(rc, "k3da_attn_qknorm_noalloc")
    return out


# ---- the paged cache: append, gather, chunk attention ----------------------

def alloc_cache(num_pages: int, num_kv_heads: int, *, quantised: bool = False, device=None):
    """(kv_pool, kv_scales): a zeroed paged cache, bf16 (kv_scales None) or
    e4m3 codes with e8m0 scales."""
    device = torch.device("cuda") if device is None else torch.device(device)
    shape = (num_pages, 2, num_kv_heads, 64)
    if not quantised:
        return torch.zeros(*shape, 64, dtype=torch.bfloat16, device=device), None
    pool = torch.zeros(*shape, 64, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    return pool, torch.zeros(*shape, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)


def _on(dev, **tensors):
    """Every tensor is contiguous and on device ``dev``."""
    for name, t in tensors.items():
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise K3daError(f"{name} must be contiguous and on the cache's device (cuda:{dev})")


def _cache_args(kv_pool, kv_scales, page_table, lens, cu_seqlens, num_kv_heads, status):
    """Checks a cache call's common tensors.  Returns the cache's device index,
    head_dim and the C arguments from kv_pool to num_requests.  (Calls on
    small inputs are bound by this code: it asks each tensor for no more than
    it needs.)"""
    dev = kv_pool.get_device()
    if dev < 0 or not kv_pool.is_contiguous():
        raise K3daError("kv_pool must be a contiguous CUDA tensor")
    shape = kv_pool.shape
    if len(shape) != 5 or shape[1] != 2 or shape[2] != num_kv_heads or shape[3] != 64:
        raise K3daError("kv_pool must be [pages, 2, Hkv, 64, 64]")
    dtype = kv_pool.dtype
    scales = 0
    if dtype is torch.bfloat16:
        code = CACHE_BF16
        if kv_scales is not None:
            raise K3daError("a bf16 cache has no scales")
    elif dtype is torch.float8_e4m3fn:
        code = CACHE_E4M3
        if kv_scales is None or kv_scales.dtype is not torch.float8_e8m0fnu or kv_scales.shape != shape[:-1]:
            raise K3daError("an e4m3 cache needs kv_scales [pages, 2, Hkv, 64] float8_e8m0fnu")
        if kv_scales.get_device() != dev or not kv_scales.is_contiguous():
            raise K3daError(f"kv_scales must be contiguous and on the cache's device (cuda:{dev})")
        scales = kv_scales.data_ptr()
    else:
        raise K3daError("kv_pool must be bfloat16 or float8_e4m3fn")
    table_shape = page_table.shape
    if page_table.dtype is not torch.int32 or len(table_shape) != 2:
        raise K3daError("page_table must be [R, S] int32")
    R, S = table_shape
    if lens.dtype is not torch.int32 or lens.numel() != R or cu_seqlens.dtype is not torch.int32 or \
            cu_seqlens.numel() != R + 1:
        raise K3daError("lengths must be [R] and cu_seqlens [R + 1], both int32")
    for t in (page_table, lens, cu_seqlens):
        if t.get_device() != dev or not t.is_contiguous():
            raise K3daError(f"page_table, lengths and cu_seqlens must be contiguous and on the cache's device (cuda:{dev})")
    if status is not None:
        _on(dev, status=status)
        if status.dtype is not torch.int32 or status.numel() < 1:
            raise K3daError("status must be an int32 CUDA tensor")
    return dev, shape[4], (kv_pool.data_ptr(), code, scales, shape[0], page_table.data_ptr(), S, lens.data_ptr(),
                           cu_seqlens.data_ptr(), R)


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _enqueue(what, dev, stream, status, *args):
    """Calls the library's ``what`` with ``args``, the status word and the
    stream, on device ``dev``.  (As a packed call: 1.3 us less than two dozen
    converted arguments.)"""
    call = (_lib or load_library()).k3da_packed_call
    number, count, pack = _PACKED[what]
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index == dev:
        handle = stream.cuda_stream
    else:
        raise K3daError("stream must be one of the cache's device")
    try:
        words = pack(*args, 0 if status is None else status.data_ptr(), handle)
    except struct.error as e:
        raise K3daError(f"{what}: {e}") from None
    if torch._C._cuda_getDevice() == dev:
        rc = call(number, words, count)
    else:
        with torch.cuda.device(dev):
            rc = call(number, words, count)
    if rc != OK:
        _check(rc, what)


def _qkv_rows(qkv, num_q_heads, num_kv_heads, D, dev):
    shape = qkv.shape
    if qkv.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != (num_q_heads + 2 * num_kv_heads) * D or \
            qkv.get_device() != dev or not qkv.is_contiguous():
        raise K3daError("qkv must be [T, (Hq+2Hkv)*64] bf16, contiguous and on the cache's device")
    return shape[0]


def k3da_kv_append(kv_pool, qkv, page_table, ctx_lens, cu_seqlens, *, num_q_heads: int, num_kv_heads: int,
                   kv_scales=None, status=None, stream=None):
    """Write the k and v heads of the packed rows ``qkv`` (k already
    normalised and roped) into the paged cache at tokens ``ctx_lens[r] + i``
    (C: k3da_kv_append).  Returns ``kv_pool``."""
    dev, D, args = _cache_args(kv_pool, kv_scales, page_table, ctx_lens, cu_seqlens, num_kv_heads, status)
    T = _qkv_rows(qkv, num_q_heads, num_kv_heads, D, dev)
    _enqueue("k3da_kv_append", dev, stream, status, *args, qkv.data_ptr(), T, num_q_heads, num_kv_heads, D)
    return kv_pool


def k3da_kv_append_qknorm(kv_pool, qkv, page_table, ctx_lens, cu_seqlens, positions, q_norm_w, k_norm_w, *,
                          num_q_heads: int, num_kv_heads: int, q_out=None, eps: float = 1e-5,
                          rope_base: float = 10000.0, yarn=None, kv_scales=None, status=None, stream=None):
    """``k3da_kv_append`` of raw k: RMSNorm + NeoX RoPE (with ``yarn``, YaRN
    RoPE) on the way into the cache, and of q into ``q_out`` [T, Hq*64] when
    given (C: k3da_kv_append_qknorm).  Returns ``kv_pool``."""
    dev, D, args = _cache_args(kv_pool, kv_scales, page_table, ctx_lens, cu_seqlens, num_kv_heads, status)
    T = _qkv_rows(qkv, num_q_heads, num_kv_heads, D, dev)
    for t in (positions, q_norm_w, k_norm_w):
        if t.get_device() != dev or not t.is_contiguous():
            raise K3daError(f"positions and norm weights must be contiguous and on the cache's device (cuda:{dev})")
    if positions.dtype is torch.int64:
        code = POS_I64
    elif positions.dtype is torch.int32:
        code = POS_I32
    else:
        raise K3daError("positions must be [T] int32 or int64")
    if positions.numel() != T:
        raise K3daError("positions must be [T] int32 or int64")
    if q_norm_w.dtype is not torch.bfloat16 or k_norm_w.dtype is not torch.bfloat16 or \
            q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise K3daError("norm weights must be [64] bf16")
    if q_out is not None and (q_out.dtype is not torch.bfloat16 or q_out.shape != (T, num_q_heads * D) or
                              q_out.get_device() != dev or not q_out.is_contiguous()):
        raise K3daError("q_out must be [T, Hq*64] bf16, contiguous and on the cache's device")
    _enqueue("k3da_kv_append_qknorm", dev, stream, status, *args, qkv.data_ptr(), T, num_q_heads, num_kv_heads, D,
             positions.data_ptr(), code, q_norm_w.data_ptr(), k_norm_w.data_ptr(), eps, rope_base,
             0 if yarn is None else ctypes.addressof(yarn), _addr(q_out))
    return kv_pool


def k3da_kv_gather(k_out, v_out, kv_pool, page_table, starts, cu_seqlens, *, num_kv_heads: int, kv_scales=None,
                   status=None, stream=None):
    """Read cache tokens ``starts[r] + i`` back into the packed rows of
    ``k_out`` and ``v_out`` [T, Hkv*64] bf16 (C: k3da_kv_gather).  Returns
    both."""
    dev, D, args = _cache_args(kv_pool, kv_scales, page_table, starts, cu_seqlens, num_kv_heads, status)
    _on(dev, k_out=k_out, v_out=v_out)
    shape = k_out.shape
    if k_out.dtype is not torch.bfloat16 or v_out.dtype is not torch.bfloat16 or len(shape) != 2 or \
            shape[1] != num_kv_heads * D or v_out.shape != shape:
        raise K3daError("k_out and v_out must be [T, Hkv*64] bf16")
    _enqueue("k3da_kv_gather", dev, stream, status, k_out.data_ptr(), v_out.data_ptr(), *args, shape[0], num_kv_heads, D)
    return k_out, v_out


def chunk_workspace_bytes(num_tokens: int, num_requests: int, num_q_heads: int, num_kv_heads: int,
                          page_stride: int) -> int:
    n = load_library().k3da_chunk_workspace_bytes(num_tokens, num_requests, num_q_heads, num_kv_heads, page_stride)
    if n == 0:
        raise K3daError("chunk_workspace_bytes: sizes out of contract")
    return int(n)


def alloc_chunk_workspace(num_tokens: int, num_requests: int, num_q_heads: int, num_kv_heads: int,
                          page_stride: int, device=None) -> torch.Tensor:
    """A workspace tensor for ``k3da_chunk_attn`` calls of these sizes."""
    device = torch.device("cuda") if device is None else torch.device(device)
    n = chunk_workspace_bytes(num_tokens, num_requests, num_q_heads, num_kv_heads, page_stride)
    return torch.empty(n, dtype=torch.uint8, device=device)


def k3da_chunk_attn(out, q, kv_pool, page_table, ctx_lens, cu_seqlens, *, num_q_heads: int, num_kv_heads: int,
                    softmax_scale: float = 0.125, mask: str = "causal", kv_scales=None, lse=None, workspace,
                    status=None, stream=None):
    """Attention of ragged chunks of new tokens over the paged cache (C:
    k3da_chunk_attn).  ``q`` [T, Hq*64] bf16 may be a view whose rows are
    further apart (``qkv[:, :Hq*64]``); ``mask`` is "causal", "full" or
    "context"; ``lse`` [T, Hq] fp32 is optional.  Returns ``out``."""
    dev, D, args = _cache_args(kv_pool, kv_scales, page_table, ctx_lens, cu_seqlens, num_kv_heads, status)
    shape = q.shape
    if q.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != num_q_heads * D or q.get_device() != dev or \
            (shape[0] and q.stride(1) != 1):
        raise K3daError("q must be [T, Hq*64] bf16 on the cache's device, each row contiguous")
    T = shape[0]
    for t in (out, workspace) if lse is None else (out, workspace, lse):
        if t.get_device() != dev or not t.is_contiguous():
            raise K3daError(f"out, lse and workspace must be contiguous and on the cache's device (cuda:{dev})")
    if out.dtype is not torch.bfloat16 or out.shape != shape:
        raise K3daError("out must be [T, Hq*64] bf16")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, num_q_heads)):
        raise K3daError("lse must be [T, Hq] fp32")
    code = MASKS.get(mask)
    if code is None:
        raise K3daError(f"mask must be one of {', '.join(MASKS)}")
    _enqueue("k3da_chunk_attn", dev, stream, status, out.data_ptr(), _addr(lse), q.data_ptr(),
             q.stride(0) if T > 1 else shape[1], T, *args, num_q_heads, num_kv_heads, D, code, softmax_scale,
             workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


_I32, _F32 = torch.int32, torch.float32


def _ints(dev, *tensors):
    """Each is int32, contiguous and on device ``dev``."""
    for t in tensors:
        if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
            raise K3daError(f"page tables, lengths, counts, lists and cu_seqlens must be int32, contiguous and on one CUDA device (cuda:{dev})")


def _status_word(status, dev):
    _on(dev, status=status)
    if status.dtype is not _I32 or status.numel() < 1:
        raise K3daError("status must be an int32 CUDA tensor")


# ---- around the drafts: probabilities and verification ---------------------

def _rows(name, t, dev, shape):
    """``t`` is [T, V] = shape, each row contiguous, on device ``dev``;
    returns its address and its rows' distance."""
    if t.get_device() != dev or dev < 0 or len(shape) != 2 or t.shape != shape:
        raise K3daError(f"{name} must be [T, V], on one CUDA device (cuda:{dev})")
    row, step = t.stride()
    if step != 1 and shape[1] > 1 and shape[0]:
        raise K3daError(f"{name} must have contiguous rows")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def k3da_token_probs(probs, logits, cu_seqlens, *, temperatures=None, status=None, stream=None):
    """Probabilities [T, V] fp32 of ``logits`` [T, V] (bf16, fp16 or fp32) at
    each request's temperature, ``temperatures`` [R] fp32 (C:
    k3da_token_probs).  Rows of either may be further apart than V.  Returns
    ``probs``."""
    dev = logits.get_device()
    code = LOGITS.get(logits.dtype)
    if code is None or probs.dtype is not _F32:
        raise K3daError("logits must be bf16, fp16 or fp32, and probs fp32")
    shape = logits.shape
    x, x_stride = _rows("logits", logits, dev, shape)
    out, out_stride = _rows("probs", probs, dev, shape)
    _ints(dev, cu_seqlens)
    R = cu_seqlens.numel() - 1
    if temperatures is not None and (temperatures.dtype is not _F32 or temperatures.numel() != R or
                                     temperatures.get_device() != dev or not temperatures.is_contiguous()):
        raise K3daError("temperatures must be [R] fp32, contiguous and on the logits' device")
    if status is not None:
        _status_word(status, dev)
    T, V = shape
    _enqueue("k3da_token_probs", dev, stream, status, out, out_stride, x, code, x_stride, T, V, _addr(temperatures),
             cu_seqlens.data_ptr(), R)
    return probs


def k3da_verify(out_tokens, num_out, tokens, target_probs, uniforms, cu_seqlens, *, draft_probs=None, status=None,
                stream=None):
    """Which of the drafts ``tokens[cu[r] + 1:cu[r + 1]]`` stay, and the token
    that follows them, from ``uniforms`` [T] (C: k3da_verify).  ``target_probs``
    and ``draft_probs`` are [T, V] fp32, row i's those of the token behind row
    i (of a drafter whose rows predict their own position: ``q[1:]`` of a ``q``
    of one row more).  Returns ``out_tokens`` [T] and ``num_out`` [R]."""
    dev = target_probs.get_device()
    shape = target_probs.shape
    p, p_stride = _rows("target_probs", target_probs, dev, shape)
    q = q_stride = 0
    if draft_probs is not None:
        q, q_stride = _rows("draft_probs", draft_probs, dev, shape)
        if draft_probs.dtype is not _F32:
            raise K3daError("draft_probs must be fp32")
    if target_probs.dtype is not _F32 or uniforms.dtype is not _F32:
        raise K3daError("target_probs and uniforms must be fp32")
    T, V = shape
    kind = tokens.dtype
    if kind is _I32:
        code = POS_I32
    elif kind is torch.int64:
        code = POS_I64
    else:
        raise K3daError("tokens must be [T] int32 or int64")
    if out_tokens.dtype is not kind:
        raise K3daError("out_tokens must be of the tokens' type")
    for t in (tokens, out_tokens, uniforms):
        if t.numel() != T or t.get_device() != dev or not t.is_contiguous():
            raise K3daError(f"tokens, out_tokens and uniforms must be [T], contiguous and on one CUDA device (cuda:{dev})")
    _ints(dev, cu_seqlens, num_out)
    R = cu_seqlens.numel() - 1
    if num_out.numel() != R:
        raise K3daError("cu_seqlens must be [R + 1] and num_out [R]")
    if status is not None:
        _status_word(status, dev)
    _enqueue("k3da_verify", dev, stream, status, out_tokens.data_ptr(), num_out.data_ptr(), tokens.data_ptr(), code, p, p_stride,
             q, q_stride, uniforms.data_ptr(), T, V, cu_seqlens.data_ptr(), R)
    return out_tokens, num_out


# ---- the pages of a cache ---------------------------------------------------

def alloc_pages(num_requests: int, page_stride: int, num_pages: int, device=None):
    """(page_table, lens, refs) of a cache that nobody uses yet."""
    device = torch.device("cuda") if device is None else torch.device(device)
    return (torch.full((num_requests, page_stride), -1, dtype=torch.int32, device=device),
            torch.zeros(num_requests, dtype=torch.int32, device=device),
            torch.zeros(num_pages, dtype=torch.int32, device=device))


def _book_args(page_table, lens, refs, status, *others):
    """Checks the pages' state; returns its device index, R and the C
    arguments."""
    dev = page_table.get_device()
    shape = page_table.shape
    if dev < 0 or len(shape) != 2:
        raise K3daError("page_table must be an [R, S] CUDA tensor")
    _ints(dev, page_table, lens, refs, *others)
    R, S = shape
    if lens.numel() != R:
        raise K3daError("lens must be [R]")
    if status is not None:
        _status_word(status, dev)
    return dev, R, (page_table.data_ptr(), S, lens.data_ptr(), R, refs.data_ptr(), refs.numel())


def k3da_pages_resize(page_table, lens, refs, new_lens, copies, *, status=None, stream=None):
    """Room for ``new_lens`` [R] tokens: pages are given back and taken, pages
    that others hold too and that are written into next are parted (C:
    k3da_pages_resize).  Changes ``page_table``, ``lens`` and ``refs``; the pages to
    copy are listed in ``copies`` [3, R] (see k3da_kv_copy), which is returned."""
    dev, R, args = _book_args(page_table, lens, refs, status, new_lens, copies)
    if new_lens.numel() != R or copies.shape != (3, R):
        raise K3daError("new_lens must be [R] and copies [3, R]")
    _enqueue("k3da_pages_resize", dev, stream, status, *args, new_lens.data_ptr(), copies.data_ptr())
    return copies


def k3da_pages_fork(page_table, lens, refs, parents, children, *, status=None, stream=None):
    """Requests ``children`` [N], which hold nothing, become copies of
    requests ``parents`` [N] on the same pages (C: k3da_pages_fork).  Changes
    and returns ``page_table``, ``lens`` and ``refs``."""
    dev, _, args = _book_args(page_table, lens, refs, status, parents, children)
    n = parents.numel()
    if children.numel() != n:
        raise K3daError("parents and children must be [N]")
    _enqueue("k3da_pages_fork", dev, stream, status, *args, parents.data_ptr(), children.data_ptr(), n)
    return page_table, lens, refs


def compact_workspace_bytes(num_pages: int) -> int:
    n = load_library().k3da_compact_workspace_bytes(num_pages)
    if n == 0:
        raise K3daError("compact_workspace_bytes: sizes out of contract")
    return int(n)


def alloc_compact_workspace(num_pages: int, device=None) -> torch.Tensor:
    """A workspace tensor for ``k3da_pages_compact`` of a pool of this size."""
    device = torch.device("cuda") if device is None else torch.device(device)
    return torch.empty(compact_workspace_bytes(num_pages), dtype=torch.uint8, device=device)


def k3da_pages_compact(page_table, lens, refs, copies, num_copies, *, workspace, status=None, stream=None):
    """Pages move together at the pool's start, at most ``copies.shape[1]`` of
    them (C: k3da_pages_compact).  Changes ``page_table`` and ``refs``; the
    moves are listed in ``copies`` [3, N], their number in ``num_copies`` [1],
    which are returned."""
    dev, _, args = _book_args(page_table, lens, refs, status, copies, num_copies)
    shape = copies.shape
    if len(shape) != 2 or shape[0] != 3 or num_copies.numel() != 1:
        raise K3daError("copies must be [3, N] and num_copies [1]")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise K3daError(f"workspace must be contiguous and on the page table's device (cuda:{dev})")
    _enqueue("k3da_pages_compact", dev, stream, status, *args, copies.data_ptr(), shape[1], num_copies.data_ptr(),
             workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return copies, num_copies


def k3da_kv_copy(kv_pool, copies, *, kv_scales=None, num_copies=None, status=None, stream=None):
    """Copies pages as ``copies`` [3, N] (from, to, tokens) lists them, the
    first ``num_copies`` [1] columns of it if given (C: k3da_kv_copy).
    Returns ``kv_pool``."""
    dev = kv_pool.get_device()
    shape = kv_pool.shape
    if dev < 0 or not kv_pool.is_contiguous() or len(shape) != 5 or shape[1] != 2 or shape[3] != 64:
        raise K3daError("kv_pool must be a contiguous [pages, 2, Hkv, 64, 64] CUDA tensor")
    if kv_pool.dtype is torch.bfloat16 and kv_scales is None:
        code = CACHE_BF16
    elif kv_pool.dtype is torch.float8_e4m3fn and kv_scales is not None:
        code = CACHE_E4M3
        _on(dev, kv_scales=kv_scales)
        if kv_scales.dtype is not torch.float8_e8m0fnu or kv_scales.shape != shape[:-1]:
            raise K3daError("kv_scales must be [pages, 2, Hkv, 64] float8_e8m0fnu")
    else:
        raise K3daError("kv_pool must be bfloat16 without scales or float8_e4m3fn with them")
    _ints(dev, copies)
    list_shape = copies.shape
    if len(list_shape) != 2 or list_shape[0] != 3:
        raise K3daError("copies must be [3, N]")
    if num_copies is not None:
        _ints(dev, num_copies)
        if num_copies.numel() != 1:
            raise K3daError("num_copies must be [1]")
    if status is not None:
        _status_word(status, dev)
    _enqueue("k3da_kv_copy", dev, stream, status, kv_pool.data_ptr(), code, _addr(kv_scales), shape[0], shape[2], shape[4],
             copies.data_ptr(), list_shape[1], _addr(num_copies))
    return kv_pool
