"""Exact attention forward for NVIDIA B200 (sm_100a): Python binding of ``libfa_b200.so``.

The functions here only marshal arguments (pointers, sizes, the current CUDA stream) into the C ABI
of include/fa.h; every step of the attention runs in the library's CUDA kernels.  PyTorch supplies
device memory and streams.  There is no fallback: if the library is missing or the device is not
an sm_100 GPU, calls raise.

    o, lse = fa_fwd(q, k, v, causal=True)            # q, k, v: bf16 [B, H, N, d] on cuda
    o, lse = fa_decode_paged(q, k_pool, v_pool, block_table, seq_lens)

A serving step over an 8-bit cache writes its tokens and then attends to them:

    freqs, amp = rope_frequencies(rot)
    q = fa_cache_append(k, v, k_pool, v_pool, slots, k_scale=ks, v_scale=vs, positions=pos,
                        freqs=freqs, amplitude=amp, q=q)
    o, lse = fa_decode_paged_q8(q, k_pool, v_pool, ks, vs, block_table, seq_lens)
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

from . import build as _build

__all__ = ["fa_fwd", "fa_bwd", "fa_decode_paged", "fa_decode_paged_noalloc", "fa_prefill_paged",
           "fa_tree_attention", "fa_fwd_keyrange", "fa_merge_partials",
           "fa_decode_workspace_size",
           "rope_frequencies", "fa_rope", "fa_cache_append", "fa_cache_read",
           "fa_decode_paged_q8", "fa_prefill_paged_q8", "fa_tree_attention_q8",
           "fa_q8_workspace_size",
           "NOALLOC_SCRATCH_BYTES", "device_status",
           "FaError", "library_path", "load_library", "EXPORTED_SYMBOLS", "STATUS"]

STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_ALIGNMENT",
          4: "FA_ERR_LAUNCH", 5: "FA_ERR_TIMEOUT", 6: "FA_ERR_WORKSPACE"}
FA_OUT_BF16, FA_OUT_F32 = 0, 1

EXPORTED_SYMBOLS = ("fa_fwd", "fa_decode_workspace_size", "fa_decode_paged",
                    "fa_decode_paged_noalloc", "fa_prefill_paged", "fa_tree_attention",
                    "fa_fwd_keyrange", "fa_merge_partials",
                    "fa_bwd_workspace_size",
                    "fa_bwd", "fa_get_device_status",
                    "fa_status_string",
                    "fa_last_error_string", "fa_version", "fa_selftest_wait_timeout",
                    "fa_probe_ex2_rate", "fa_probe_read_rate", "fa_fwd_schedule",
                    "fa_rope", "fa_cache_append", "fa_cache_read", "fa_q8_workspace_size",
                    "fa_decode_paged_q8", "fa_prefill_paged_q8", "fa_tree_attention_q8")

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if _lib is not None:
            msg = f"{where}: {_lib.fa_status_string(status).decode()}"
            if status == 4:
                msg += f" ({_lib.fa_last_error_string().decode()})"
        super().__init__(msg)


def library_path() -> str:
    return _build.LIB_PATH


def load_library():
    """Load the in-tree shared library (build it first with ``python -m exact_attention_158_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"CUDA library not built: {path} is missing "
                          "(run `python -m exact_attention_158_b200.build`)")
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, vp]
    lib.fa_fwd.restype = i32
    lib.fa_decode_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.fa_decode_workspace_size.restype = sz
    lib.fa_decode_paged.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, f32,
                                    vp, sz, vp]
    lib.fa_decode_paged.restype = i32
    lib.fa_prefill_paged.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                     i32, f32, vp]
    lib.fa_prefill_paged.restype = i32
    lib.fa_fwd_keyrange.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32,
                                    i32, f32, vp]
    lib.fa_fwd_keyrange.restype = i32
    lib.fa_merge_partials.argtypes = [vp, vp, i32, ctypes.c_longlong, i32, vp, i32, vp, vp]
    lib.fa_merge_partials.restype = i32
    lib.fa_tree_attention.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, i32, vp, i32, i32, i32,
                                      i32, f32, vp]
    lib.fa_tree_attention.restype = i32
    lib.fa_bwd_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.fa_bwd_workspace_size.restype = ctypes.c_size_t
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                           f32, vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = i32
    i64, i64p = ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)
    lib.fa_rope.argtypes = [vp, i64p, vp, i64p, vp, i64p, vp, i64p, i32, i32, vp, i64, vp, i32, i32,
                            f32, i32, i32, i32, i32, i32, i32, vp]
    lib.fa_rope.restype = i32
    lib.fa_cache_append.argtypes = [vp, i64p, vp, i64p, vp, vp, vp, vp, i32, vp, i32, vp, i64p, vp,
                                    i64p, vp, vp, i32, i32, f32, i32, i32, i32, i32, vp]
    lib.fa_cache_append.restype = i32
    lib.fa_cache_read.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, vp]
    lib.fa_cache_read.restype = i32
    lib.fa_q8_workspace_size.argtypes = [i32] * 6
    lib.fa_q8_workspace_size.restype = sz
    lib.fa_decode_paged_q8.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, vp, i32,
                                       i32, i32, i32, f32, vp, sz, vp]
    lib.fa_decode_paged_q8.restype = i32
    lib.fa_prefill_paged_q8.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, vp, i32,
                                        i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.fa_prefill_paged_q8.restype = i32
    lib.fa_tree_attention_q8.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, vp, i32, vp,
                                         i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.fa_tree_attention_q8.restype = i32
    lib.fa_get_device_status.argtypes = [vp]
    lib.fa_get_device_status.restype = i32
    lib.fa_status_string.argtypes = [i32]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_last_error_string.argtypes = []
    lib.fa_last_error_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i32
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise FaError(status, where)


def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _require(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out_code(out_dtype) -> int:
    if out_dtype == torch.bfloat16:
        return FA_OUT_BF16
    if out_dtype == torch.float32:
        return FA_OUT_F32
    raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None,
           out_dtype=torch.bfloat16, out=None, lse=None, return_lse: bool = True, stream=None):
    """Exact attention forward.  q, k, v: bf16 [B, H, N, d] contiguous on one CUDA device.

    Returns (o [B, H, N, d] in out_dtype, lse fp32 [B, H, N] or None)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n)
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one shape [B, H, N, d]")
    B, H, N, d = q.shape
    code = _out_code(out_dtype)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    else:
        _require(out, "out", out_dtype)
        if out.shape != q.shape:
            raise ValueError("out has the wrong shape")
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    elif lse is not None:
        _require(lse, "lse", torch.float32)
        if lse.shape != (B, H, N):
            raise ValueError("lse has the wrong shape")
    with torch.cuda.device(q.device):
        st = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), code,
                        lse.data_ptr() if lse is not None else None, B, H, N, d, int(causal),
                        float(scale) if scale is not None else 0.0, _stream_handle(stream))
    _check(st, "fa_fwd")
    return out, lse


def fa_decode_workspace_size(num_seqs: int, H: int, d: int, max_blocks_per_seq: int) -> int:
    return int(load_library().fa_decode_workspace_size(num_seqs, H, d, max_blocks_per_seq))


def fa_decode_paged(q, k_pool, v_pool, block_table, seq_lens, scale: float | None = None,
                    out_dtype=torch.bfloat16, out=None, lse=None, return_lse: bool = True,
                    workspace=None, stream=None):
    """One decode step over a paged KV cache.

    q bf16 [S, H, d]; k_pool, v_pool bf16 [num_blocks, H, 16, d]; block_table int32
    [S, max_blocks]; seq_lens int32 [S].  Returns (o [S, H, d], lse fp32 [S, H] or None)."""
    lib = load_library()
    for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _require(t, n)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    S, H, d = q.shape
    P = k_pool.shape[0]
    if k_pool.shape != (P, H, 16, d) or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool / v_pool must be [num_blocks, H, 16, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_table must be [S, max_blocks] and seq_lens [S]")
    maxb = block_table.shape[1]
    code = _out_code(out_dtype)
    if out is None:
        out = torch.empty((S, H, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
    need = lib.fa_decode_workspace_size(S, H, d, maxb)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        st = lib.fa_decode_paged(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                 block_table.data_ptr(), maxb, seq_lens.data_ptr(), P,
                                 out.data_ptr(), code,
                                 lse.data_ptr() if lse is not None else None, S, H, d,
                                 float(scale) if scale is not None else 0.0,
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_handle(stream))
    _check(st, "fa_decode_paged")
    return out, lse


def fa_bwd(q, k, v, o, dout, lse, causal: bool = False, scale: float | None = None,
           grad_dtype=torch.bfloat16, workspace=None, stream=None):
    """Attention backward: q, k, v, dout bf16 [B, H, N, d]; o (bf16 or fp32) and lse (fp32
    [B, H, N]) from fa_fwd with the same causal and scale.  Returns (dq, dk, dv) in grad_dtype."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _require(t, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"o must be bf16 or fp32, got {o.dtype}")
    _require(o, "o", o.dtype)
    _require(lse, "lse", torch.float32)
    B, H, N, d = q.shape
    for t, n in ((k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if lse.shape != (B, H, N):
        raise ValueError("lse must be [B, H, N]")
    code = _out_code(grad_dtype)
    need = int(lib.fa_bwd_workspace_size(B, H, N, d))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    dq, dk, dv = (torch.empty(q.shape, dtype=grad_dtype, device=q.device) for _ in range(3))
    with torch.cuda.device(q.device):
        st = lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _out_code(o.dtype),
                        dout.data_ptr(),
                        lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), code, B, H, N,
                        d, int(causal), float(scale) if scale is not None else 0.0,
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        _stream_handle(stream))
    _check(st, "fa_bwd")
    return dq, dk, dv


def fa_fwd_keyrange(q, k, v, q_row0: int = 0, k_pos0: int = 0, causal: bool = False,
                    scale: float | None = None, out_dtype=torch.float32, out=None, lse=None,
                    stream=None):
    """Partial attention of the query rows q_row0.. of q [B, H, Nq, d] (row i at position i) over
    the keys k, v [B, H, Nk, d] at positions k_pos0...  Rows that see no key get O = 0,
    LSE = -inf; rows before q_row0 of out / lse are left as they are.  Returns (o, lse)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n)
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B, H, Nk, d] with q's B, H, d")
    code = _out_code(out_dtype)
    if out is None:
        out = torch.empty((B, H, Nq, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_keyrange(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), code,
                                 lse.data_ptr(), B, H, Nq, q_row0, Nk, k_pos0, d, int(causal),
                                 float(scale) if scale is not None else 0.0, _stream_handle(stream))
    _check(st, "fa_fwd_keyrange")
    return out, lse


def fa_merge_partials(o_parts, lse_parts, out_dtype=torch.bfloat16, stream=None):
    """o_parts fp32 [G, ..., d], lse_parts fp32 [G, ...]: partials of the same rows over disjoint
    key ranges.  Returns the merged (o [..., d], lse [...])."""
    lib = load_library()
    _require(o_parts, "o_parts", torch.float32)
    _require(lse_parts, "lse_parts", torch.float32)
    G, d = o_parts.shape[0], o_parts.shape[-1]
    if lse_parts.shape != o_parts.shape[:-1]:
        raise ValueError("lse_parts must be o_parts' shape without the last dimension")
    rows = lse_parts[0].numel()
    code = _out_code(out_dtype)
    o = torch.empty(o_parts.shape[1:], dtype=out_dtype, device=o_parts.device)
    lse = torch.empty(lse_parts.shape[1:], dtype=torch.float32, device=o_parts.device)
    with torch.cuda.device(o_parts.device):
        st = lib.fa_merge_partials(o_parts.data_ptr(), lse_parts.data_ptr(), G, rows, d,
                                   o.data_ptr(), code, lse.data_ptr(), _stream_handle(stream))
    _check(st, "fa_merge_partials")
    return o, lse


def fa_tree_attention(q, k_pool, v_pool, block_table, seq_lens, tree_mask,
                      scale: float | None = None, out_dtype=torch.bfloat16, out=None, lse=None,
                      return_lse: bool = True, stream=None):
    """Tree verification: q bf16 [S, H, T, d] holds the T draft nodes, the last T cached tokens of
    each sequence; tree_mask int64 [S, T] (uint64 bit patterns: bit u of entry t set when node t
    sees node u; T <= 64).  Pools, table and lengths as for fa_prefill_paged.
    Returns (o [S, H, T, d], lse fp32 [S, H, T] or None)."""
    lib = load_library()
    for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _require(t, n)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    _require(tree_mask, "tree_mask", torch.int64)
    S, H, T, d = q.shape
    P = k_pool.shape[0]
    if k_pool.shape != (P, H, 16, d) or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool / v_pool must be [num_blocks, H, 16, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_table must be [S, max_blocks] and seq_lens [S]")
    if tree_mask.shape != (S, T):
        raise ValueError("tree_mask must be [S, T]")
    code = _out_code(out_dtype)
    if out is None:
        out = torch.empty((S, H, T, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, H, T), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        st = lib.fa_tree_attention(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                   block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
                                   P, tree_mask.data_ptr(), out.data_ptr(), code,
                                   lse.data_ptr() if lse is not None else None, S, H, T, d,
                                   float(scale) if scale is not None else 0.0,
                                   _stream_handle(stream))
    _check(st, "fa_tree_attention")
    return out, lse


def fa_prefill_paged(q, k_pool, v_pool, block_table, seq_lens, causal: bool = True,
                     scale: float | None = None, out_dtype=torch.bfloat16, out=None, lse=None,
                     return_lse: bool = True, stream=None):
    """Chunked prefill over a paged KV cache: q bf16 [S, H, Lq, d] holds the last Lq positions of
    each sequence (their keys/values already in the cache); k_pool, v_pool bf16
    [num_blocks, H, 16, d]; block_table int32 [S, max_blocks]; seq_lens int32 [S] (each >= Lq).
    Returns (o [S, H, Lq, d], lse fp32 [S, H, Lq] or None)."""
    lib = load_library()
    for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _require(t, n)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    S, H, Lq, d = q.shape
    P = k_pool.shape[0]
    if k_pool.shape != (P, H, 16, d) or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool / v_pool must be [num_blocks, H, 16, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_table must be [S, max_blocks] and seq_lens [S]")
    code = _out_code(out_dtype)
    if out is None:
        out = torch.empty((S, H, Lq, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, H, Lq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        st = lib.fa_prefill_paged(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                  block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
                                  P, out.data_ptr(), code,
                                  lse.data_ptr() if lse is not None else None, S, H, Lq, d,
                                  int(causal), float(scale) if scale is not None else 0.0,
                                  _stream_handle(stream))
    _check(st, "fa_prefill_paged")
    return out, lse


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the library's device status word."""
    return int(load_library().fa_get_device_status(_stream_handle(stream)))


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # FA_NOALLOC_SCRATCH_BYTES in include/fa.h


def fa_decode_paged_noalloc(q, k_pool, v_pool, block_table, seq_lens, out, lse=None,
                            scale: float | None = None, stream=None):
    """fa_decode_paged for callers that cannot allocate device memory at decode time.

    The caller passes every buffer, ``out`` included (bf16 or fp32 [S, H, d]; ``lse`` fp32
    [S, H] or None); the split-context scratch is the library's static 32 MiB device array, so
    nothing is allocated here or in the library.  Calls that overlap on the GPU share that array
    and race: serialise them.  Sizes needing more scratch than the array holds raise FaError."""
    lib = load_library()
    f = lib.fa_decode_paged_noalloc
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    f.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp]
    f.restype = i32
    for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _require(t, n)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    if q.dim() != 3:
        raise ValueError("q must be [S, H, d]")
    S, H, d = q.shape
    P = k_pool.shape[0]
    if k_pool.shape != (P, H, 16, d) or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool / v_pool must be [num_blocks, H, 16, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_table must be [S, max_blocks] and seq_lens [S]")
    code = _out_code(out.dtype) if isinstance(out, torch.Tensor) else None
    if code is None:
        raise ValueError("out must be a bf16 or fp32 CUDA tensor")
    _require(out, "out", out.dtype)
    if out.shape != (S, H, d):
        raise ValueError("out must be [S, H, d]")
    if lse is not None:
        _require(lse, "lse", torch.float32)
        if lse.shape != (S, H):
            raise ValueError("lse must be [S, H]")
    for t, n in ((k_pool, "k_pool"), (v_pool, "v_pool"), (block_table, "block_table"),
                 (seq_lens, "seq_lens"), (out, "out")) + (((lse, "lse"),) if lse is not None else ()):
        if t.device != q.device:
            raise ValueError(f"{n} must be on q's device ({q.device})")
    # the library resolves its scratch array, and launches, on the current device
    with torch.cuda.device(q.device):
        st = f(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
               block_table.shape[1], seq_lens.data_ptr(), P, out.data_ptr(), code,
               lse.data_ptr() if lse is not None else None, S, H, d,
               float(scale) if scale is not None else 0.0, _stream_handle(stream))
    _check(st, "fa_decode_paged_noalloc")
    return out, lse


# ------------------------------------------------------------------------------------------------
# rotary positions, the paged cache's writer and reader, attention over an 8-bit cache
# ------------------------------------------------------------------------------------------------

_ROPE_LAYOUT = {"half": 0, "interleaved": 1}
_CACHE_TYPE = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original_len: int = 4096, fast: float = 32.0,
                     slow: float = 1.0, device="cuda"):
    """Frequencies of fa_rope's rot / 2 pairs, in radians per position, and the amplitude that goes
    with them: (float64 [rot / 2] on `device`, float).

    f_j = base^(-2j / rot).  For contexts `factor` times as long as the trained ones, scaling is
      "linear"  all positions are shrunk: f_j / factor (position interpolation, Chen et al. 2023);
      "base"    the base grows to base * factor^(rot / (rot - 2)), which keeps the fastest pair and
                slows the slowest by `factor`;
      "ramp"    pairs that turn more than `fast` times in `original_len` positions keep their
                frequency, those that turn less than `slow` times take f_j / factor, with a linear
                ramp in the number of turns between, and the amplitude is 0.1 ln(factor) + 1 (YaRN,
                Peng et al. 2023)."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if not (base > 0 and factor >= 1.0):
        raise ValueError("base must be positive and factor at least 1")
    if scaling == "base":
        if rot <= 2:
            raise ValueError("scaling 'base' needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if not fast > slow:
            raise ValueError("scaling 'ramp' needs fast > slow")
        turns = original_len * f / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'ramp', got {scaling!r}")
    return f.to(device), amplitude


# A decode step makes these calls once per layer, so their own time counts.  Arguments are checked in
# one expression each and explained only when it fails; the stream is read as a raw handle and the
# device switched only when it is not the current one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_stride_arrays: dict = {}


def _strides(t, n):
    """The first n strides as a C array (shared by calls with the same strides, never written)."""
    key = t.stride()[:n]
    arr = _stride_arrays.get(key)
    if arr is None:
        if len(_stride_arrays) >= 4096:
            _stride_arrays.clear()
        arr = _stride_arrays[key] = (ctypes.c_longlong * n)(*key)
    return arr


def _stream_on(index, stream):
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is not None:
        return _raw_stream(index)
    return int(torch.cuda.current_stream(index).cuda_stream)


def _new(like, shape, dtype, stream):
    """Memory for a call on `stream`, on like's device: it comes from that stream's pool, so whatever
    the current stream still does to freed memory, or does with it next, cannot meet the kernel.
    shape None: like's own (like is then contiguous; this is the quicker of torch's two calls)."""
    if stream is None:
        return torch.empty_like(like, dtype=dtype) if shape is None else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return _new(like, shape, dtype, None)


def _on_device(index, where, fn, *args):
    if torch.cuda.current_device() == index:
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st != 0:
        raise FaError(st, where)


def _require_rows(t, name, dims, dtypes, index=None):
    """A CUDA tensor whose last dimension is contiguous; the others may have any strides."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == dims
            and (t.stride(-1) == 1 or t.numel() == 0)
            and (t.get_device() == index if index is not None else t.is_cuda)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    raise ValueError(f"{name} must be on cuda:{index}")


def _require_flat(t, name, dtype, shape, index=None):
    """A contiguous CUDA tensor of the given type and shape (None: any), on the given device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)
            and (t.get_device() == index if index is not None else t.is_cuda)):
        return
    _require(t, name, dtype)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{index}")


def _rope_args(freqs, positions, layout, index):
    """(freqs pointer, rot, layout code) after the checks both rotating calls share."""
    code = _ROPE_LAYOUT.get(layout)
    if code is None:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if freqs is None:
        return None, 0, code
    _require_flat(freqs, "freqs", torch.float64, None, index)
    if freqs.dim() != 1:
        raise ValueError("freqs must be [rot / 2]")
    if positions is None:
        raise ValueError("positions are needed with freqs")
    return freqs.data_ptr(), 2 * freqs.numel(), code


_ROPE_IO = (torch.bfloat16, torch.float32)
_BF16 = (torch.bfloat16,)


def fa_rope(q, k, positions, freqs, layout: str = "half", amplitude: float = 1.0,
            inverse: bool = False, out_dtype=None, q_out=None, k_out=None, stream=None):
    """Rotary positions.  q [B, Hq, N, d] and k [B, Hk, N, d] (or None), bf16 or fp32, any strides
    with the features contiguous (a projection's [B, N, heads, d] goes in as its transpose(1, 2));
    positions int32 [N] or [B, N]; freqs float64 [rot / 2], see rope_frequencies; layout "half"
    (pairs j, j + rot/2) or "interleaved" (2j, 2j + 1).  inverse=True turns back: the gradient.

    Returns (q_out, k_out): the tensors passed, which may be q and k themselves, or new contiguous
    [B, H, N, d] ones in out_dtype (default: the input's)."""
    lib = load_library()
    _require_rows(q, "q", 4, _ROPE_IO)
    dev = q.get_device()
    B, Hq, N, d = q.shape
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else q.dtype
    out_code = _out_code(out_dtype)
    if q_out is None:
        q_out = _new(q, (B, Hq, N, d), out_dtype, stream)
    else:
        _require_rows(q_out, "q_out", 4, (out_dtype,), dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    Hk, kp, ks, kop, kos = 0, None, None, None, None
    if k is not None:
        _require_rows(k, "k", 4, (q.dtype,), dev)
        Hk = k.shape[1]
        if k.shape != (B, Hk, N, d):
            raise ValueError("k must be [B, Hk, N, d] with q's B, N, d")
        if k_out is None:
            k_out = _new(q, (B, Hk, N, d), out_dtype, stream)
        else:
            _require_rows(k_out, "k_out", 4, (out_dtype,), dev)
            if k_out.shape != k.shape:
                raise ValueError("k_out must have k's shape")
        if Hk:
            kp, ks, kop, kos = k.data_ptr(), _strides(k, 3), k_out.data_ptr(), _strides(k_out, 3)
    elif k_out is not None:
        raise ValueError("k_out without k")
    fptr, rot, code = _rope_args(freqs, positions, layout, dev)
    pos_ptr, pos_stride = None, 0
    if positions is not None:
        _require_flat(positions, "positions", torch.int32, None, dev)
        pos_stride = N if positions.dim() == 2 else 0
        if positions.shape != ((B, N) if positions.dim() == 2 else (N,)):
            raise ValueError("positions must be [N] or [B, N]")
        pos_ptr = positions.data_ptr()
    _on_device(dev, "fa_rope", lib.fa_rope, q.data_ptr(), _strides(q, 3), q_out.data_ptr(),
               _strides(q_out, 3), kp, ks, kop, kos, _out_code(q.dtype), out_code, pos_ptr, pos_stride,
               fptr, rot, code, float(amplitude), int(inverse), B, Hq, Hk, N, d, _stream_on(dev, stream))
    return q_out, k_out


def _require_pools(k_pool, v_pool, k_scale, v_scale):
    """(cache type code, num_blocks, heads, d, scale pointers, device index) of a paged pool."""
    code = _CACHE_TYPE.get(getattr(k_pool, "dtype", None))
    if code is None:
        raise ValueError("k_pool must be a bfloat16, float8_e4m3fn or int8 tensor")
    _require_flat(k_pool, "k_pool", k_pool.dtype, None)
    if k_pool.dim() != 4 or k_pool.shape[2] != 16:
        raise ValueError("k_pool / v_pool must be [num_blocks, H, 16, d]")
    P, H, _, d = k_pool.shape
    index = k_pool.get_device()
    _require_flat(v_pool, "v_pool", k_pool.dtype, k_pool.shape, index)
    if not code:
        return code, P, H, d, None, None, index
    _require_flat(k_scale, "k_scale", torch.float32, (P, H, 16), index)
    _require_flat(v_scale, "v_scale", torch.float32, (P, H, 16), index)
    return code, P, H, d, k_scale.data_ptr(), v_scale.data_ptr(), index


def fa_cache_append(k, v, k_pool, v_pool, slots, k_scale=None, v_scale=None, positions=None,
                    freqs=None, layout: str = "half", amplitude: float = 1.0, q=None, q_out=None,
                    stream=None):
    """Write T tokens' keys and values to their slots of the paged cache, in place.

    k, v bf16 [T, Hk, d] (any strides, features contiguous); k_pool, v_pool [num_blocks, Hk, 16, d]
    in bfloat16, float8_e4m3fn or int8, the 8-bit types with k_scale, v_scale fp32
    [num_blocks, Hk, 16]; slots int64 [T] (block * 16 + row; negative: not written).  With freqs
    (float64 [rot / 2]) and positions (int32 [T]) the keys are rotated first, and q bf16 [T, Hq, d]
    beside them.  Returns q_out (new and contiguous unless passed), or None without q."""
    lib = load_library()
    code, P, Hk, d, ksp, vsp, dev = _require_pools(k_pool, v_pool, k_scale, v_scale)
    _require_rows(k, "k", 3, _BF16, dev)
    _require_rows(v, "v", 3, _BF16, dev)
    T = k.shape[0]
    if k.shape != (T, Hk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hk, d] with the pools' heads and features")
    _require_flat(slots, "slots", torch.int64, (T,), dev)
    fptr, rot, lcode = _rope_args(freqs, positions, layout, dev)
    pos_ptr = None
    if positions is not None:
        _require_flat(positions, "positions", torch.int32, (T,), dev)
        pos_ptr = positions.data_ptr()
    Hq, qp, qs, qop, qos = 0, None, None, None, None
    if q is not None:
        _require_rows(q, "q", 3, _BF16, dev)
        Hq = q.shape[1]
        if q.shape != (T, Hq, d):
            raise ValueError("q must be [T, Hq, d]")
        if q_out is None:
            q_out = _new(q, (T, Hq, d), q.dtype, stream)
        else:
            _require_rows(q_out, "q_out", 3, _BF16, dev)
            if q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
        if Hq:
            qp, qs, qop, qos = q.data_ptr(), _strides(q, 2), q_out.data_ptr(), _strides(q_out, 2)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _on_device(dev, "fa_cache_append", lib.fa_cache_append, k.data_ptr(), _strides(k, 2), v.data_ptr(),
               _strides(v, 2), k_pool.data_ptr(), v_pool.data_ptr(), ksp, vsp, code, slots.data_ptr(),
               P, qp, qs, qop, qos, pos_ptr, fptr, rot, lcode, float(amplitude), T, Hq, Hk, d,
               _stream_on(dev, stream))
    return q_out


def fa_cache_read(k_pool, v_pool, slots, k_scale=None, v_scale=None, k_out=None, v_out=None,
                  stream=None):
    """Read the rows at slots (int64 [T]; negative: zeros) of a paged cache back as bf16: returns
    (k, v), each [T, H, d].  Pools and scales as for fa_cache_append."""
    lib = load_library()
    code, P, H, d, ksp, vsp, dev = _require_pools(k_pool, v_pool, k_scale, v_scale)
    _require_flat(slots, "slots", torch.int64, None, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    T = slots.shape[0]
    if k_out is None:
        k_out = _new(k_pool, (T, H, d), torch.bfloat16, stream)
    else:
        _require_flat(k_out, "k_out", torch.bfloat16, (T, H, d), dev)
    if v_out is None:
        v_out = _new(k_out, None, torch.bfloat16, stream)
    else:
        _require_flat(v_out, "v_out", torch.bfloat16, (T, H, d), dev)
    _on_device(dev, "fa_cache_read", lib.fa_cache_read, k_pool.data_ptr(), v_pool.data_ptr(), ksp, vsp,
               code, slots.data_ptr(), P, k_out.data_ptr(), v_out.data_ptr(), T, H, d,
               _stream_on(dev, stream))
    return k_out, v_out


@functools.lru_cache(maxsize=1024)
def fa_q8_workspace_size(S: int, Hq: int, Hk: int, Lq: int, d: int, max_blocks_per_seq: int) -> int:
    """Bytes of workspace fa_decode_paged_q8 (Lq = 1), fa_prefill_paged_q8 and fa_tree_attention_q8
    need; 0 when none."""
    return int(load_library().fa_q8_workspace_size(S, Hq, Hk, Lq, d, max_blocks_per_seq))


def _attend_q8(where, q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, tree_mask, causal,
               scale, out_dtype, out, lse, return_lse, workspace, stream):
    lib = load_library()
    code, P, Hk, d, ksp, vsp, dev = _require_pools(k_pool, v_pool, k_scale, v_scale)
    if not code:
        raise ValueError("k_pool / v_pool must be float8_e4m3fn or int8")
    _require_flat(q, "q", torch.bfloat16, None, dev)
    shape = q.shape
    if len(shape) != (3 if causal is None else 4):
        raise ValueError("q must be [S, Hq, d]" if causal is None else "q must be [S, Hq, Lq, d]")
    S, Hq, Lq = shape[0], shape[1], 1 if causal is None else shape[2]
    if shape[-1] != d or Hk == 0 or Hq % Hk:
        raise ValueError("q must have the pools' d and a multiple of their heads")
    _require_flat(block_table, "block_table", torch.int32, None, dev)
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [S, max_blocks]")
    _require_flat(seq_lens, "seq_lens", torch.int32, (S,), dev)
    if tree_mask is not None:
        _require_flat(tree_mask, "tree_mask", torch.int64, (S, Lq), dev)
    code_o = _out_code(out_dtype)
    if out is None:
        out = _new(q, None, out_dtype, stream)
    else:
        _require_flat(out, "out", out_dtype, shape, dev)
    if lse is not None:
        _require_flat(lse, "lse", torch.float32, shape[:-1], dev)
    elif return_lse:
        lse = _new(q, shape[:-1], torch.float32, stream)
    maxb = block_table.shape[1]
    ws, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = fa_q8_workspace_size(S, Hq, Hk, Lq, d, maxb)
        if ws_bytes:
            workspace = _new(q, (ws_bytes,), torch.uint8, stream)
            ws = workspace.data_ptr()
    else:
        _require_flat(workspace, "workspace", workspace.dtype, None, dev)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    head = (q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), ksp, vsp, code,
            block_table.data_ptr(), maxb, seq_lens.data_ptr(), P)
    outs = (out.data_ptr(), code_o, None if lse is None else lse.data_ptr(), S, Hq, Hk)
    tail = (0.0 if scale is None else float(scale), ws, ws_bytes, _stream_on(dev, stream))
    if causal is None:
        _on_device(dev, where, lib.fa_decode_paged_q8, *head, *outs, d, *tail)
    elif tree_mask is not None:
        _on_device(dev, where, lib.fa_tree_attention_q8, *head, tree_mask.data_ptr(), *outs, Lq, d, *tail)
    else:
        _on_device(dev, where, lib.fa_prefill_paged_q8, *head, *outs, Lq, d, int(causal), *tail)
    return out, lse


def fa_decode_paged_q8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                       scale: float | None = None, out_dtype=torch.bfloat16, out=None, lse=None,
                       return_lse: bool = True, workspace=None, stream=None):
    """One decode step over an 8-bit paged cache (see fa_cache_append), query heads sharing key
    heads: q bf16 [S, Hq, d]; pools float8_e4m3fn or int8 [num_blocks, Hk, 16, d]; scales fp32
    [num_blocks, Hk, 16]; block_table int32 [S, max_blocks]; seq_lens int32 [S] (0: an empty slot).
    Returns (o [S, Hq, d], lse fp32 [S, Hq] or None)."""
    return _attend_q8("fa_decode_paged_q8", q, k_pool, v_pool, k_scale, v_scale, block_table,
                      seq_lens, None, None, scale, out_dtype, out, lse, return_lse, workspace, stream)


def fa_prefill_paged_q8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                        causal: bool = True, scale: float | None = None, out_dtype=torch.bfloat16,
                        out=None, lse=None, return_lse: bool = True, workspace=None, stream=None):
    """Chunked prefill over an 8-bit paged cache: q bf16 [S, Hq, Lq, d] holds the last Lq positions
    of each sequence, already in the cache; the rest as for fa_decode_paged_q8.
    Returns (o [S, Hq, Lq, d], lse fp32 [S, Hq, Lq] or None)."""
    return _attend_q8("fa_prefill_paged_q8", q, k_pool, v_pool, k_scale, v_scale, block_table,
                      seq_lens, None, bool(causal), scale, out_dtype, out, lse, return_lse, workspace,
                      stream)


def fa_tree_attention_q8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, tree_mask,
                         scale: float | None = None, out_dtype=torch.bfloat16, out=None, lse=None,
                         return_lse: bool = True, workspace=None, stream=None):
    """Tree verification over an 8-bit paged cache: q bf16 [S, Hq, T, d] holds the T <= 64 nodes, the
    last T cached tokens; tree_mask int64 [S, T] as for fa_tree_attention; the rest as for
    fa_decode_paged_q8.  Returns (o [S, Hq, T, d], lse fp32 [S, Hq, T] or None)."""
    if tree_mask is None:
        raise ValueError("tree_mask must be [S, T]")
    return _attend_q8("fa_tree_attention_q8", q, k_pool, v_pool, k_scale, v_scale, block_table,
                      seq_lens, tree_mask, False, scale, out_dtype, out, lse, return_lse, workspace,
                      stream)


def selftest_wait_timeout(limit_us: int = 50_000, stream=None) -> int:
    """Launch the bounded-wait self-test and return the device status it leaves (expect 5,
    FA_ERR_TIMEOUT); the status word is read and cleared."""
    lib = load_library()
    f = lib.fa_selftest_wait_timeout
    f.argtypes = [ctypes.c_uint, ctypes.c_void_p]
    f.restype = ctypes.c_int
    _check(f(limit_us, _stream_handle(stream)), "fa_selftest_wait_timeout")
    return device_status(stream)


def probe_ex2_rate(iters: int = 200_000, stream=None) -> tuple[int, float]:
    """Run the exponential-throughput probe once on the current device; returns (exponentials
    launched, device milliseconds from CUDA events on the stream)."""
    lib = load_library()
    f = lib.fa_probe_ex2_rate
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_longlong), ctypes.c_void_p]
    f.restype = ctypes.c_int
    s = stream if stream is not None else torch.cuda.current_stream()
    sink = torch.zeros(1, dtype=torch.float32, device="cuda")
    n = ctypes.c_longlong(0)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(s)
    _check(f(sink.data_ptr(), int(iters), ctypes.byref(n), int(s.cuda_stream)), "fa_probe_ex2_rate")
    b.record(s)
    b.synchronize()
    return int(n.value), a.elapsed_time(b)


def probe_read_rate(buf: torch.Tensor, stream=None) -> float:
    """Read every byte of the contiguous CUDA tensor `buf` once with the decode's streaming loads;
    returns the device milliseconds (CUDA events on the stream)."""
    lib = load_library()
    f = lib.fa_probe_read_rate
    f.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]
    f.restype = ctypes.c_int
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    s = stream if stream is not None else torch.cuda.current_stream()
    sink = torch.zeros(1, dtype=torch.float32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(s)
    _check(f(buf.data_ptr(), nbytes, sink.data_ptr(), int(s.cuda_stream)), "fa_probe_read_rate")
    b.record(s)
    b.synchronize()
    return a.elapsed_time(b)


def fwd_schedule(B: int, H: int, N: int, d: int, num_ctas: int):
    """The unit-to-CTA assignment of a causal fa_fwd launch of this shape on `num_ctas` SMs (host
    only).  Returns (start, unit) int32 numpy arrays, CTA c running unit[start[c]:start[c+1]] in
    order, or None when the launch deals its units in snake order instead."""
    import numpy as np
    lib = load_library()
    f = lib.fa_fwd_schedule
    ip = ctypes.POINTER(ctypes.c_int)
    f.argtypes = [ctypes.c_int] * 5 + [ip, ip, ctypes.c_int, ip]
    f.restype = ctypes.c_int
    units = B * H * ((N + 255) // 256)
    start = np.zeros(num_ctas + 1, dtype=np.int32)
    unit = np.zeros(max(units, 1), dtype=np.int32)
    count = ctypes.c_int(0)
    _check(f(B, H, N, d, num_ctas, start.ctypes.data_as(ip), unit.ctypes.data_as(ip), unit.size,
             ctypes.byref(count)), "fa_fwd_schedule")
    return (start, unit[:count.value]) if count.value > 0 else None
