"""ctypes binding of ``libmla.so`` (declared in ``include/mla.h``) over torch tensors.

Argument marshalling only: every step of the decode runs in the library's kernels.
torch supplies device memory and the current CUDA stream. The library is loaded on
first use; if it is missing this raises — there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

KV_BF16 = 0
KV_FP8_E4M3 = 1
D_QK = 576
D_V = 512
D_INDEX = 128

MLA_OK = 0
STATUS = {0: "MLA_OK", -1: "MLA_ERR_INVALID_ARG", -2: "MLA_ERR_UNSUPPORTED",
          -3: "MLA_ERR_WORKSPACE_TOO_SMALL", -4: "MLA_ERR_CUDA", -5: "MLA_ERR_TIMEOUT",
          -6: "MLA_ERR_DEVICE_INDEX"}
EXPORTS = ("mla_abi_version", "mla_status_string", "mla_decode_workspace_size", "mla_decode",
           "mla_decode_check", "mla_cache_write", "mla_decode_noalloc", "mla_decode_noalloc_check",
           "mla_profile_begin", "mla_profile_end", "mla_test_set_hooks", "mla_decode_with_cache_write",
           "mla_rope_cache_write", "mla_chunk_workspace_size", "mla_chunk_attention", "mla_merge_states",
           "mla_index_cache_write", "mla_index_scores", "mla_select_blocks", "mla_sparse_workspace_size",
           "mla_sparse_attention")
NOALLOC_SCRATCH_BYTES = 32 << 20

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla.so")
_lib = None


class MLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_string(status)})")


class DecodeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("s_q", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("causal", ctypes.c_int32)]


class ChunkParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("causal", ctypes.c_int32)]


class IndexParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "num_tokens", "num_heads", "page_size", "num_pages",
                                              "max_blocks_per_seq", "max_seq_len", "block_size", "causal")]


class SparseParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "num_tokens", "num_heads", "page_size", "num_pages",
                                              "max_blocks_per_seq", "max_seq_len", "block_size", "top_k", "kv_dtype",
                                              "causal")]


def lib() -> ctypes.CDLL:
    """The loaded library (loads it on first call; raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build(); "
                               "this package has no non-CUDA implementation")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.mla_abi_version.restype = i32
        L.mla_status_string.restype = ctypes.c_char_p
        L.mla_status_string.argtypes = [i32]
        L.mla_decode_workspace_size.restype = sz
        L.mla_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams), i32]
        L.mla_decode.restype = i32
        L.mla_decode.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, ctypes.c_float, vp,
                                 vp, vp, vp, sz, vp]
        L.mla_decode_check.restype = i32
        L.mla_decode_check.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.mla_decode_noalloc.restype = i32
        L.mla_decode_noalloc.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, ctypes.c_float,
                                         vp, vp, vp, vp]
        L.mla_decode_noalloc_check.restype = i32
        L.mla_decode_noalloc_check.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        L.mla_cache_write.restype = i32
        L.mla_cache_write.argtypes = [vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp]
        L.mla_decode_with_cache_write.restype = i32
        L.mla_decode_with_cache_write.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, i32, vp, vp, vp, vp,
                                                  ctypes.c_float, vp, vp, vp, vp, sz, vp]
        L.mla_test_set_hooks.restype = i32
        L.mla_test_set_hooks.argtypes = [ctypes.c_uint64, i32]
        L.mla_profile_begin.restype = i32
        L.mla_profile_begin.argtypes = [i32]
        L.mla_profile_end.restype = i32
        L.mla_profile_end.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32)]
        i64 = ctypes.c_int64
        L.mla_rope_cache_write.restype = i32
        L.mla_rope_cache_write.argtypes = [vp, i64, vp, i64, vp, vp, i32, i32, vp, i32, vp, i32, i32, i32, vp, vp,
                                           i64, i64, i32, vp, vp, vp]
        L.mla_chunk_workspace_size.restype = sz
        L.mla_chunk_workspace_size.argtypes = [ctypes.POINTER(ChunkParams), i32]
        L.mla_chunk_attention.restype = i32
        L.mla_chunk_attention.argtypes = [ctypes.POINTER(ChunkParams), vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                          vp, sz, vp]
        L.mla_merge_states.restype = i32
        L.mla_merge_states.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp]
        L.mla_index_cache_write.restype = i32
        L.mla_index_cache_write.argtypes = [vp, i64, vp, vp, i32, i32, vp, i32, vp, vp, i32, i32, vp, i64, i64, vp, i32,
                                            vp, vp, vp, vp]
        L.mla_index_scores.restype = i32
        L.mla_index_scores.argtypes = [ctypes.POINTER(IndexParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.mla_select_blocks.restype = i32
        L.mla_select_blocks.argtypes = [vp, i64, i32, i32, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
        L.mla_sparse_workspace_size.restype = sz
        L.mla_sparse_workspace_size.argtypes = [ctypes.POINTER(SparseParams), i32]
        L.mla_sparse_attention.restype = i32
        L.mla_sparse_attention.argtypes = [ctypes.POINTER(SparseParams), vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                           vp, vp, sz, vp]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mla_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_params(batch, s_q, num_heads, page_size, num_pages, max_blocks_per_seq, max_seq_len,
                kv_dtype, causal=True) -> DecodeParams:
    return DecodeParams(int(batch), int(s_q), int(num_heads), int(page_size), int(num_pages),
                        int(max_blocks_per_seq), int(max_seq_len), int(kv_dtype), int(bool(causal)))


def workspace_size(params: DecodeParams, num_sms: int = 0) -> int:
    n = lib().mla_decode_workspace_size(ctypes.byref(params), int(num_sms))
    if n == 0:
        raise MLAError(-1, "mla_decode_workspace_size")
    return int(n)


def alloc_workspace(params: DecodeParams, device=None) -> torch.Tensor:
    return torch.empty(workspace_size(params), dtype=torch.uint8, device=device or "cuda")


def _kv_dtype_of(kv_cache: torch.Tensor) -> int:
    if kv_cache.dtype == torch.bfloat16:
        return KV_BF16
    if kv_cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        return KV_FP8_E4M3
    raise TypeError(f"kv_cache dtype {kv_cache.dtype}: expected bfloat16, uint8 or float8_e4m3fn")


def _decode_inputs(q, kv_cache, block_table, seq_lens, kv_scale, max_seq_len, causal, out, lse):
    """Check the decode inputs (the library reads them asynchronously, so they are used as
    given: no temporary copies), allocate missing outputs, and build the parameters."""
    B, s_q, H, d = q.shape
    if d != D_QK or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [B, s_q, H, 576] tensor")
    Np, P, d2 = kv_cache.shape
    if d2 != D_QK or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [Np, P, 576] tensor")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_table and seq_lens must be int32")
    if not block_table.is_contiguous() or not seq_lens.is_contiguous():
        raise ValueError("block_table and seq_lens must be contiguous")
    if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_table must be [B, MB] and seq_lens [B]")
    kvd = _kv_dtype_of(kv_cache)
    if kvd == KV_FP8_E4M3 and (kv_scale is None or kv_scale.dtype != torch.float32):
        raise ValueError("the FP8 cache needs kv_scale as a float32 device tensor")
    params = make_params(B, s_q, H, P, Np, block_table.shape[1], max_seq_len, kvd, causal)
    if out is None:
        out = torch.empty((B, s_q, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=q.device)
    return params, kvd, out, lse


def decode(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
           seq_lens: torch.Tensor, softmax_scale: float, kv_scale: torch.Tensor | None = None,
           *, max_seq_len: int, causal: bool = True, out: torch.Tensor | None = None,
           lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
           stream=None):
    """Paged MLA decode. q [B, s_q, H, 576] bf16; kv_cache [Np, P, 576] (bf16, or uint8 /
    float8_e4m3fn bytes); block_table [B, MB] int32; seq_lens [B] int32; kv_scale a
    1-element float32 device tensor for the FP8 cache. Returns (out, lse)."""
    params, kvd, out, lse = _decode_inputs(q, kv_cache, block_table, seq_lens, kv_scale, max_seq_len,
                                           causal, out, lse)
    if workspace is None:
        workspace = alloc_workspace(params, q.device)
    st = lib().mla_decode(ctypes.byref(params), _ptr(q), _ptr(kv_cache), _ptr(block_table),
                          _ptr(seq_lens), ctypes.c_float(softmax_scale),
                          _ptr(kv_scale) if kvd == KV_FP8_E4M3 else None, _ptr(out), _ptr(lse),
                          _ptr(workspace), workspace.numel(), _stream(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode")
    return out, lse


def decode_with_cache_write(latent: torch.Tensor, rope: torch.Tensor, slot_mapping: torch.Tensor,
                            q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                            seq_lens: torch.Tensor, softmax_scale: float,
                            kv_scale: torch.Tensor | None = None, *, max_seq_len: int,
                            causal: bool = True, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            stream=None):
    """cache_write() of a step's new tokens followed by decode(), in one launch chain (the
    scheduler kernel writes the new rows). Returns (out, lse)."""
    n = latent.shape[0]
    if latent.shape != (n, 512) or rope.shape != (n, 64) or latent.dtype != torch.bfloat16 \
            or rope.dtype != torch.bfloat16 or not latent.is_contiguous() or not rope.is_contiguous():
        raise ValueError("latent [N,512] and rope [N,64] must be contiguous bf16")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 [N] tensor")
    params, kvd, out, lse = _decode_inputs(q, kv_cache, block_table, seq_lens, kv_scale, max_seq_len,
                                           causal, out, lse)
    if workspace is None:
        workspace = alloc_workspace(params, q.device)
    st = lib().mla_decode_with_cache_write(ctypes.byref(params), _ptr(latent), _ptr(rope), _ptr(slot_mapping), n,
                                           _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
                                           ctypes.c_float(softmax_scale),
                                           _ptr(kv_scale) if kvd == KV_FP8_E4M3 else None, _ptr(out), _ptr(lse),
                                           _ptr(workspace), workspace.numel(), _stream(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_with_cache_write")
    return out, lse


def decode_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                   seq_lens: torch.Tensor, softmax_scale: float, kv_scale: torch.Tensor | None = None,
                   *, max_seq_len: int, causal: bool = True, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, stream=None):
    """decode() without a workspace, for callers that cannot allocate device memory: the
    library's own static scratch array (NOALLOC_SCRATCH_BYTES) is used instead. Calls
    must not overlap on the GPU; pass out and lse to allocate nothing here either."""
    params, kvd, out, lse = _decode_inputs(q, kv_cache, block_table, seq_lens, kv_scale, max_seq_len,
                                           causal, out, lse)
    st = lib().mla_decode_noalloc(ctypes.byref(params), _ptr(q), _ptr(kv_cache), _ptr(block_table),
                                  _ptr(seq_lens), ctypes.c_float(softmax_scale),
                                  _ptr(kv_scale) if kvd == KV_FP8_E4M3 else None, _ptr(out),
                                  _ptr(lse), _stream(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_noalloc")
    return out, lse


def decode_noalloc_check(stream=None):
    """Synchronise and read the device error word of the last decode_noalloc: (status, bits)."""
    bits = ctypes.c_uint32(0)
    st = lib().mla_decode_noalloc_check(_stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


def decode_check(workspace: torch.Tensor, stream=None):
    """Synchronise and read the device error word: returns (status, bits)."""
    bits = ctypes.c_uint32(0)
    st = lib().mla_decode_check(_ptr(workspace), _stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


def test_set_hooks(wait_limit_ns: int = 0, stall: bool = False) -> None:
    """Tests only: bound of the kernels' pipeline waits (0 = the default 2 s) and the stall
    that makes the first softmax wait run out."""
    st = lib().mla_test_set_hooks(int(wait_limit_ns), int(bool(stall)))
    if st != 0:
        raise MLAError(st, "mla_test_set_hooks")


def profile_begin(max_launches: int) -> None:
    """Time the decode kernel of each of the next `max_launches` decode calls (CUDA events
    around its launch, recorded by the library on the call's stream)."""
    st = lib().mla_profile_begin(int(max_launches))
    if st != 0:
        raise MLAError(st, "mla_profile_begin")


def profile_end():
    """Stop timing; returns (summed decode-kernel milliseconds, number of timed launches)."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int32(0)
    st = lib().mla_profile_end(ctypes.byref(ms), ctypes.byref(n))
    if st != 0:
        raise MLAError(st, "mla_profile_end")
    return float(ms.value), int(n.value)


def cache_write(latent: torch.Tensor, rope: torch.Tensor, slot_mapping: torch.Tensor,
                kv_cache: torch.Tensor, kv_scale: torch.Tensor | None = None,
                device_error: torch.Tensor | None = None, stream=None) -> None:
    """Write token rows concat(latent[t], rope[t]) into the paged cache at slot_mapping[t]."""
    n = latent.shape[0]
    if latent.shape != (n, 512) or rope.shape != (n, 64) or latent.dtype != torch.bfloat16 \
            or rope.dtype != torch.bfloat16 or not latent.is_contiguous() or not rope.is_contiguous():
        raise ValueError("latent [N,512] and rope [N,64] must be contiguous bf16")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 [N] tensor")
    Np, P, _ = kv_cache.shape
    kvd = _kv_dtype_of(kv_cache)
    st = lib().mla_cache_write(_ptr(latent), _ptr(rope), _ptr(slot_mapping), n,
                               _ptr(kv_cache), Np, P, kvd,
                               _ptr(kv_scale) if kvd == KV_FP8_E4M3 else None,
                               _ptr(device_error), _stream(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_write")


def _addresses(stream, *tensors):
    """(stream handle, addresses of the tensors). The library launches on the current device and
    dereferences these there, so all of them have to live on it. (The checks of the calls below
    cost as much as a small kernel: they look at each property once.)"""
    dev = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else 0
    at = []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        if t.get_device() != dev:            # -1: not on a GPU
            raise ValueError("every tensor must be on the current device" if t.is_cuda else
                             "every tensor must be on the GPU")
        at.append(t.data_ptr())
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream, at


def _allocated(stream, shape, dtype, device) -> torch.Tensor:
    """A tensor of the current stream's that a kernel on `stream` uses, whenever it is freed."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        t.record_stream(stream)
    return t


def _rows_of(t: torch.Tensor, n: int, width: int, name: str) -> int:
    """Row stride of a bf16 [n, width] tensor whose rows are contiguous and 16-byte aligned."""
    if t.dtype is not torch.bfloat16 or t.shape != (n, width):
        raise ValueError(f"{name} must be a bf16 [N, {width}] tensor with contiguous rows")
    stride, inner = t.stride()
    if n > 0 and inner != 1:
        raise ValueError(f"{name} must be a bf16 [N, {width}] tensor with contiguous rows")
    if n <= 1:
        stride = width
    if stride < width or stride % 8 != 0:
        raise ValueError(f"the rows of {name} must be apart by a multiple of 8 elements, {width} at least")
    return stride


def rope_cache_write(latent: torch.Tensor, rope: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                     slot_mapping: torch.Tensor, kv_cache: torch.Tensor, kv_scale: torch.Tensor | None = None, *,
                     q_rope: torch.Tensor | None = None, q: torch.Tensor | None = None, interleaved: bool = True,
                     device_error: torch.Tensor | None = None, stream=None) -> None:
    """cache_write() with the position rotation applied on the way: token t's row
    concat(latent[t], rotated rope[t]) goes to slot_mapping[t], and q_rope [N, H, 64] rotated
    into q[..., 512:] (q [N, H, 576] contiguous). cos_sin [max_pos, 64] float32 holds the
    cosines and sines of every position; pairs are neighbours (interleaved) or a half apart.
    latent, rope and q_rope may be strided views of projections. Negative positions mark
    padding tokens."""
    n = latent.shape[0]
    ls = _rows_of(latent, n, 512, "latent")
    rs = _rows_of(rope, n, 64, "rope")
    i64 = torch.int64
    if positions.dtype is not i64 or positions.shape != (n,) or not positions.is_contiguous() or \
            slot_mapping.dtype is not i64 or slot_mapping.shape != (n,) or not slot_mapping.is_contiguous():
        raise ValueError("positions and slot_mapping must be contiguous int64 [N] tensors")
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 [max_pos, 64] tensor")
    max_pos, width = cos_sin.shape
    if width != 64:
        raise ValueError("cos_sin must be a contiguous float32 [max_pos, 64] tensor")
    if kv_cache.dim() != 3 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [Np, P, 576] tensor")
    Np, P, width = kv_cache.shape
    if width != D_QK:
        raise ValueError("kv_cache must be a contiguous [Np, P, 576] tensor")
    kvd = _kv_dtype_of(kv_cache)
    if kvd == KV_FP8_E4M3 and (kv_scale is None or kv_scale.dtype != torch.float32 or kv_scale.numel() < 1):
        raise ValueError("the FP8 cache needs kv_scale as a float32 device tensor")
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q are given together or not at all")
    H, qt, qh = 0, 0, 0
    if q is not None:
        if q.dtype is not torch.bfloat16 or q.dim() != 3 or not q.is_contiguous():
            raise ValueError("q must be a contiguous bf16 [N, H, 576] tensor")
        qn, H, width = q.shape
        if qn != n or width != D_QK:
            raise ValueError("q must be a contiguous bf16 [N, H, 576] tensor")
        if q_rope.dtype is not torch.bfloat16 or q_rope.shape != (n, H, 64):
            raise ValueError("q_rope must be a bf16 [N, H, 64] tensor with contiguous last dimension")
        qt, qh, inner = q_rope.stride()
        if inner != 1 and n > 0 and H > 0:
            raise ValueError("q_rope must be a bf16 [N, H, 64] tensor with contiguous last dimension")
        if n <= 1:
            qt = 0
        if H <= 1:
            qh = 0
        if H < 1 or qt % 8 != 0 or qh % 8 != 0:
            raise ValueError("q_rope's tokens and heads must be apart by a multiple of 8 elements")
    if device_error is not None and device_error.dtype not in (torch.int32, torch.uint32):
        raise ValueError("device_error must be a 32-bit integer tensor")
    handle, at = _addresses(stream, latent, rope, positions, cos_sin, slot_mapping, kv_cache,
                            kv_scale if kvd == KV_FP8_E4M3 else None, q_rope if n > 0 else None, q if n > 0 else None,
                            device_error)
    st = lib().mla_rope_cache_write(at[0], ls, at[1], rs, at[2], at[3], max_pos, 1 if interleaved else 0, at[4], n,
                                    at[5], Np, P, kvd, at[6], at[7], qt, qh, H, at[8], at[9], handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_rope_cache_write")


def make_chunk_params(batch, num_tokens, num_heads, page_size, num_pages, max_blocks_per_seq, max_seq_len,
                      kv_dtype, causal=True) -> ChunkParams:
    if max_seq_len > 0x7FFFFFFF:             # the structure's field would keep its low 32 bits
        raise ValueError("max_seq_len must be at most 2^20")
    return ChunkParams(int(batch), int(num_tokens), int(num_heads), int(page_size), int(num_pages),
                       int(max_blocks_per_seq), int(max_seq_len), int(kv_dtype), int(bool(causal)))


def chunk_workspace_size(params: ChunkParams, num_sms: int = 0) -> int:
    n = lib().mla_chunk_workspace_size(ctypes.byref(params), int(num_sms))
    if n == 0:
        raise MLAError(-1, "mla_chunk_workspace_size")
    return int(n)


def alloc_chunk_workspace(params: ChunkParams, device=None) -> torch.Tensor:
    return torch.empty(chunk_workspace_size(params), dtype=torch.uint8, device=device or "cuda")


def chunk_attention(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    cu_q_lens: torch.Tensor, softmax_scale: float, kv_scale: torch.Tensor | None = None, *,
                    max_seq_len: int, causal: bool = True, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of a ragged batch of new tokens over the paged cache. q [T, H, 576] bf16, rows
    cu_q_lens[b] .. cu_q_lens[b+1] being the last positions of sequence b; cu_q_lens [B + 1] and
    seq_lens [B] int32; the rest as decode(). Rows that belong to no sequence are left as they
    are in out and lse (uninitialised when these are allocated here). Returns (out, lse)."""
    if q.dim() != 3 or q.shape[2] != D_QK or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [T, H, 576] tensor")
    T, H, _ = q.shape
    if kv_cache.dim() != 3 or kv_cache.shape[2] != D_QK or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [Np, P, 576] tensor")
    Np, P, _ = kv_cache.shape
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens), ("cu_q_lens", cu_q_lens)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    B = seq_lens.numel()
    if seq_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != B or cu_q_lens.shape != (B + 1,):
        raise ValueError("block_table must be [B, MB], seq_lens [B] and cu_q_lens [B + 1]")
    kvd = _kv_dtype_of(kv_cache)
    if kvd == KV_FP8_E4M3 and (kv_scale is None or kv_scale.dtype != torch.float32 or kv_scale.numel() < 1):
        raise ValueError("the FP8 cache needs kv_scale as a float32 device tensor")
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != (T, H, D_V) or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 [T, H, 512] tensor")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, H) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [T, H] tensor")
    if workspace is not None and not workspace.is_contiguous():     # its size is taken from its elements
        raise ValueError("workspace must be contiguous")
    scale = kv_scale if kvd == KV_FP8_E4M3 else None
    params = make_chunk_params(B, T, H, P, Np, block_table.shape[1], max_seq_len, kvd, causal)
    handle, at = _addresses(stream, q, kv_cache, block_table, seq_lens, cu_q_lens, scale, out, lse, workspace)
    if out is None:
        out = _allocated(stream, (T, H, D_V), torch.bfloat16, q.device)
        at[6] = out.data_ptr()
    if lse is None:
        lse = _allocated(stream, (T, H), torch.float32, q.device)
        at[7] = lse.data_ptr()
    if workspace is None:
        workspace = _allocated(stream, (chunk_workspace_size(params),), torch.uint8, q.device)
        at[8] = workspace.data_ptr()
    st = lib().mla_chunk_attention(ctypes.byref(params), at[0], at[1], at[2], at[3], at[4], softmax_scale, at[5], at[6],
                                   at[7], at[8], workspace.numel() * workspace.element_size(), handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_chunk_attention")
    return out, lse


def merge_states(out_a: torch.Tensor, lse_a: torch.Tensor, out_b: torch.Tensor, lse_b: torch.Tensor, *,
                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Join two attention results over disjoint keys: out_* [..., 512] bf16 and lse_* [...]
    float32 as decode() and chunk_attention() return them. out and lse may be given, in place
    of one of the inputs among others. Returns (out, lse)."""
    shape = lse_a.shape
    full = shape + (D_V,)
    for t in (out_a, out_b) if out is None else (out_a, out_b, out):
        if t.dtype is not torch.bfloat16 or t.shape != full or not t.is_contiguous():
            raise ValueError("out_a, out_b and out must be contiguous bf16 [..., 512] tensors of the shape of lse_a")
    for t in (lse_a, lse_b) if lse is None else (lse_a, lse_b, lse):
        if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
            raise ValueError("lse_a, lse_b and lse must be contiguous float32 tensors of one shape")
    handle, at = _addresses(stream, out_a, lse_a, out_b, lse_b, out, lse)
    if out is None:
        out = _allocated(stream, full, torch.bfloat16, out_a.device)
        at[4] = out.data_ptr()
    if lse is None:
        lse = _allocated(stream, shape, torch.float32, out_a.device)
        at[5] = lse.data_ptr()
    st = lib().mla_merge_states(at[0], at[1], at[2], at[3], lse_a.numel(), at[4], at[5], handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_merge_states")
    return out, lse


_I32_MAX = 0x7FFFFFFF        # a structure's or an argument's 32-bit field would keep the low bits of a larger number
_CODES = (torch.float8_e4m3fn, torch.uint8)


def _ragged(seq_lens, cu_q_lens, block_table=None) -> int:
    """Checks the offsets, lengths and block table of a ragged batch; its number of sequences."""
    i32, shape = torch.int32, seq_lens.shape
    if len(shape) != 1 or cu_q_lens.shape != (shape[0] + 1,):
        raise ValueError("seq_lens must be [B] and cu_q_lens [B + 1]")
    if seq_lens.dtype is not i32 or cu_q_lens.dtype is not i32 or not seq_lens.is_contiguous() or not cu_q_lens.is_contiguous():
        raise ValueError("seq_lens and cu_q_lens must be contiguous int32 tensors")
    if block_table is not None:
        table = block_table.shape
        if len(table) != 2 or table[0] != shape[0] or block_table.dtype is not i32 or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [B, MB] tensor")
        if table[1] > _I32_MAX:
            raise ValueError("the columns of block_table must fit 32 bits")
    if shape[0] > _I32_MAX:
        raise ValueError("the number of sequences must fit 32 bits")
    return shape[0]


def _error_word(device_error) -> None:
    if device_error.dtype not in (torch.int32, torch.uint32) or device_error.numel() < 1:
        raise ValueError("device_error must be a 32-bit integer tensor")


def _index_pool(index_cache, index_scale):
    """(pages, rows of a page) of an index cache and its scales."""
    shape = index_cache.shape
    if len(shape) != 3 or shape[2] != D_INDEX or index_cache.dtype not in _CODES or not index_cache.is_contiguous():
        raise ValueError("index_cache must be a contiguous uint8 or float8_e4m3fn [Np, P, 128] tensor")
    if index_scale.dtype is not torch.float32 or index_scale.shape != shape[:2] or not index_scale.is_contiguous():
        raise ValueError("index_scale must be a contiguous float32 [Np, P] tensor")
    return shape[0], shape[1]


def index_cache_write(keys: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, slot_mapping: torch.Tensor,
                      index_cache: torch.Tensor, index_scale: torch.Tensor, *, queries: torch.Tensor | None = None,
                      weights: torch.Tensor | None = None, q_index: torch.Tensor | None = None,
                      q_weights: torch.Tensor | None = None, interleaved: bool = True,
                      device_error: torch.Tensor | None = None, stream=None) -> None:
    """New tokens' index keys [N, 128] bf16, their last 64 values rotated, as E4M3 codes into
    index_cache [Np, P, 128] and a float32 scale each into index_scale [Np, P], at
    slot_mapping[t]; and their index queries [N, H, 128] bf16, rotated, as codes into q_index
    [N, H, 128], with weights [N, H] float32 times each query's scale in q_weights [N, H].
    positions, cos_sin, slot_mapping and interleaved as rope_cache_write(). keys and queries may be
    strided views of projections. Negative positions mark padding tokens."""
    n = keys.shape[0]
    stride = _rows_of(keys, n, D_INDEX, "keys")
    i64, f32, rows = torch.int64, torch.float32, (n,)
    if positions.dtype is not i64 or positions.shape != rows or not positions.is_contiguous() or \
            slot_mapping.dtype is not i64 or slot_mapping.shape != rows or not slot_mapping.is_contiguous():
        raise ValueError("positions and slot_mapping must be contiguous int64 [N] tensors")
    table = cos_sin.shape
    if len(table) != 2 or table[1] != 64 or cos_sin.dtype is not f32 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 [max_pos, 64] tensor")
    Np, P = _index_pool(index_cache, index_scale)
    H, qt, qh = 0, 0, 0
    if queries is not None:
        if weights is None or q_index is None or q_weights is None:
            raise ValueError("queries, weights, q_index and q_weights are given together or not at all")
        shape = queries.shape
        if len(shape) != 3 or shape[0] != n or shape[2] != D_INDEX or queries.dtype is not torch.bfloat16:
            raise ValueError("queries must be a bf16 [N, H, 128] tensor with contiguous last dimension")
        H = shape[1]
        qt, qh, inner = queries.stride()
        if H < 1 or (inner != 1 and n > 0):
            raise ValueError("queries must be a bf16 [N, H, 128] tensor with contiguous last dimension")
        if n <= 1:
            qt = 0
        if H <= 1:
            qh = 0
        if qt % 8 != 0 or qh % 8 != 0:
            raise ValueError("the tokens and heads of queries must be apart by a multiple of 8 elements")
        if q_index.dtype not in _CODES or q_index.shape != shape or not q_index.is_contiguous():
            raise ValueError("q_index must be a contiguous uint8 or float8_e4m3fn [N, H, 128] tensor")
        heads = shape[:2]
        if weights.dtype is not f32 or weights.shape != heads or not weights.is_contiguous() or \
                q_weights.dtype is not f32 or q_weights.shape != heads or not q_weights.is_contiguous():
            raise ValueError("weights and q_weights must be contiguous float32 [N, H] tensors")
    elif weights is not None or q_index is not None or q_weights is not None:
        raise ValueError("queries, weights, q_index and q_weights are given together or not at all")
    if device_error is not None:
        _error_word(device_error)
    if n == 0:
        keys = queries = weights = q_index = q_weights = None
    handle, at = _addresses(stream, keys, positions, cos_sin, slot_mapping, index_cache, index_scale, queries, weights,
                            q_index, q_weights, device_error)
    st = lib().mla_index_cache_write(at[0], stride, at[1], at[2], table[0], 1 if interleaved else 0, at[3], n,
                                     at[4], at[5], Np, P, at[6], qt, qh, at[7], H, at[8], at[9], at[10], handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_index_cache_write")


def index_scores(q_index: torch.Tensor, q_weights: torch.Tensor, index_cache: torch.Tensor, index_scale: torch.Tensor,
                 block_table: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor, *, max_seq_len: int,
                 block_size: int, causal: bool = True, out: torch.Tensor | None = None,
                 device_error: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scores [T, ceil(max_seq_len / block_size)] float32 of the blocks of each new token's context:
    the largest, over the block's keys that the token sees, of the key's scale times the sum over
    the index heads of q_weights times the positive part of q_index . key; -inf without such a key.
    q_index [T, H, 128] and q_weights [T, H] as index_cache_write() leaves them; the ragged batch as
    chunk_attention(). Rows that belong to no sequence are left as they are in out (uninitialised when
    it is allocated here)."""
    shape = q_index.shape
    if len(shape) != 3 or shape[2] != D_INDEX or q_index.dtype not in _CODES or not q_index.is_contiguous():
        raise ValueError("q_index must be a contiguous uint8 or float8_e4m3fn [T, H, 128] tensor")
    T, H, _ = shape
    if q_weights.dtype is not torch.float32 or q_weights.shape != shape[:2] or not q_weights.is_contiguous():
        raise ValueError("q_weights must be a contiguous float32 [T, H] tensor")
    Np, P = _index_pool(index_cache, index_scale)
    B = _ragged(seq_lens, cu_q_lens, block_table)
    if device_error is not None:
        _error_word(device_error)
    if not 0 < max_seq_len <= _I32_MAX or not 0 < block_size <= _I32_MAX:
        raise ValueError("max_seq_len and block_size must be positive and fit 32 bits")
    shape = (T, (max_seq_len + block_size - 1) // block_size)
    if out is not None and (out.dtype is not torch.float32 or out.shape != shape or not out.is_contiguous()):
        raise ValueError("out must be a contiguous float32 [T, ceil(max_seq_len / block_size)] tensor")
    handle, at = _addresses(stream, q_index, q_weights, index_cache, index_scale, block_table, seq_lens, cu_q_lens, out,
                            device_error)
    if out is None:
        out = _allocated(stream, shape, torch.float32, q_index.device)
        at[7] = out.data_ptr()
    params = IndexParams(B, T, H, P, Np, block_table.shape[1], max_seq_len, block_size, 1 if causal else 0)
    st = lib().mla_index_scores(ctypes.byref(params), at[0], at[1], at[2], at[3], at[4], at[5], at[6], at[7], at[8], handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_index_scores")
    return out


def select_blocks(scores: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor, top_k: int, *, block_size: int,
                  keep_first: int = 0, keep_last: int = 0, causal: bool = True, out: torch.Tensor | None = None,
                  device_error: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Selected blocks [T, top_k] int32 of each new token: its first keep_first and latest keep_last
    blocks, then those with the largest scores (ties to the lower index), ascending, -1 behind them.
    scores [T, blocks] float32 as index_scores() returns them (rows may be apart). Rows that belong to no
    sequence are left as they are in out (uninitialised when it is allocated here)."""
    shape = scores.shape
    if len(shape) != 2 or scores.dtype is not torch.float32:
        raise ValueError("scores must be a float32 [T, blocks] tensor with contiguous rows")
    T, C = shape
    if T > _I32_MAX or C > _I32_MAX:
        raise ValueError("the rows and columns of scores must fit 32 bits")
    stride, inner = scores.stride()
    if inner != 1 and T > 0 and C > 1:
        raise ValueError("scores must be a float32 [T, blocks] tensor with contiguous rows")
    if T <= 1:
        stride = max(stride, C)
    if stride < C:
        raise ValueError("the rows of scores must not overlap")
    B = _ragged(seq_lens, cu_q_lens)
    if device_error is not None:
        _error_word(device_error)
    if keep_first < 0 or keep_last < 0 or not 0 < top_k <= _I32_MAX or keep_first + keep_last > top_k:
        raise ValueError("top_k must be positive and hold keep_first + keep_last blocks")
    if not 0 < block_size <= _I32_MAX:
        raise ValueError("block_size must be positive and fit 32 bits")
    if out is not None and (out.dtype is not torch.int32 or out.shape != (T, top_k) or not out.is_contiguous()):
        raise ValueError("out must be a contiguous int32 [T, top_k] tensor")
    handle, at = _addresses(stream, scores, seq_lens, cu_q_lens, out, device_error)
    if out is None:
        out = _allocated(stream, (T, top_k), torch.int32, scores.device)
        at[3] = out.data_ptr()
    st = lib().mla_select_blocks(at[0], stride, T, C, at[1], at[2], B, block_size, top_k, keep_first, keep_last,
                                 1 if causal else 0, at[3], at[4], handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_select_blocks")
    return out


def make_sparse_params(batch, num_tokens, num_heads, page_size, num_pages, max_blocks_per_seq, max_seq_len, block_size,
                       top_k, kv_dtype, causal=True) -> SparseParams:
    fields = [int(v) for v in (batch, num_tokens, num_heads, page_size, num_pages, max_blocks_per_seq, max_seq_len,
                               block_size, top_k, kv_dtype, bool(causal))]
    for (name, _), value in zip(SparseParams._fields_, fields):
        if not -_I32_MAX <= value <= _I32_MAX:
            raise ValueError(f"{name} must fit 32 bits")
    return SparseParams(*fields)


def sparse_workspace_size(params: SparseParams, num_sms: int = 0) -> int:
    n = lib().mla_sparse_workspace_size(ctypes.byref(params), int(num_sms))
    if n == 0:
        raise MLAError(-1, "mla_sparse_workspace_size")
    return int(n)


def alloc_sparse_workspace(params: SparseParams, device=None) -> torch.Tensor:
    return torch.empty(sparse_workspace_size(params), dtype=torch.uint8, device=device or "cuda")


def sparse_attention(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     cu_q_lens: torch.Tensor, selected: torch.Tensor, softmax_scale: float,
                     kv_scale: torch.Tensor | None = None, *, max_seq_len: int, block_size: int, causal: bool = True,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """chunk_attention() of which each new token sees only the keys of its selected blocks of
    block_size tokens. selected [T, K] int32, as select_blocks() returns it, is a set for each token:
    order and repetitions do not matter, entries that name no block with a visible key (-1 among them)
    are left out. A token without any key gets out 0 and lse -inf. Returns (out, lse)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != D_QK or q.dtype is not torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [T, H, 576] tensor")
    T, H, _ = shape
    shape = kv_cache.shape
    if len(shape) != 3 or shape[2] != D_QK or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [Np, P, 576] tensor")
    Np, P, _ = shape
    B = _ragged(seq_lens, cu_q_lens, block_table)
    shape = selected.shape
    if len(shape) != 2 or shape[0] != T or selected.dtype is not torch.int32 or not selected.is_contiguous():
        raise ValueError("selected must be a contiguous int32 [T, K] tensor")
    if shape[1] > _I32_MAX:
        raise ValueError("the columns of selected must fit 32 bits")
    kvd = _kv_dtype_of(kv_cache)
    if kvd == KV_FP8_E4M3 and (kv_scale is None or kv_scale.dtype != torch.float32 or kv_scale.numel() < 1):
        raise ValueError("the FP8 cache needs kv_scale as a float32 device tensor")
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != (T, H, D_V) or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 [T, H, 512] tensor")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, H) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [T, H] tensor")
    if workspace is not None and not workspace.is_contiguous():     # its size is taken from its elements
        raise ValueError("workspace must be contiguous")
    scale = kv_scale if kvd == KV_FP8_E4M3 else None
    if not 0 < max_seq_len <= _I32_MAX or not 0 < block_size <= _I32_MAX:
        raise ValueError("max_seq_len and block_size must be positive and fit 32 bits")
    params = SparseParams(B, T, H, P, Np, block_table.shape[1], max_seq_len, block_size, shape[1], kvd, 1 if causal else 0)
    handle, at = _addresses(stream, q, kv_cache, block_table, seq_lens, cu_q_lens, selected, scale, out, lse, workspace)
    if out is None:
        out = _allocated(stream, (T, H, D_V), torch.bfloat16, q.device)
        at[7] = out.data_ptr()
    if lse is None:
        lse = _allocated(stream, (T, H), torch.float32, q.device)
        at[8] = lse.data_ptr()
    if workspace is None:
        workspace = _allocated(stream, (sparse_workspace_size(params),), torch.uint8, q.device)
        at[9] = workspace.data_ptr()
    st = lib().mla_sparse_attention(ctypes.byref(params), at[0], at[1], at[2], at[3], at[4], at[5], softmax_scale, at[6],
                                    at[7], at[8], at[9], workspace.numel() * workspace.element_size(), handle)
    if st != MLA_OK:
        raise MLAError(st, "mla_sparse_attention")
    return out, lse
