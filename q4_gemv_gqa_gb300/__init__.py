"""Python binding of the GB300 decoder-step library (libgem.so, include/gem.h).

Each function marshals torch CUDA tensors into the C ABI call of the same name and
raises GemError on a non-zero status.  All computation runs in the CUDA library; torch
only provides device memory and the current stream.  Importing this package fails if
libgem.so is missing, and every call fails if the tensors are not on a CUDA device.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import LayerDesc

lib = _lib.load()

GEM_OK = 0
ACT_SILU = 0
ACT_GELU_TANH = 1
DEVFLAG_POS_RANGE = 1
DEVFLAG_TIMEOUT = 2
DEVFLAG_PAGE_RANGE = 4
DEVFLAG_NO_ROOM = 8

__all__ = ["GemError", "q4_0_gemv", "q4_0_gemv_workspace", "q4_0_gemv_fused", "q8_0_gemv", "argmax", "argmax_workspace", "rmsnorm", "rmsnorm_qknorm_rope", "gqa_decode_attn",
           "gqa_decode_attn_workspace", "gqa_decode_attn_fused", "swiglu", "decode_layer", "decode_layer_workspace",
           "kv4_page_bytes", "kv_block_tables", "qknorm_mrope", "kv4_append", "kv4_gather", "kv4_attn",
           "kv4_attn_workspace", "rmsnorm_fp8", "quant_fp8", "fp8_gemm", "logprobs", "DeviceLayer", "device_status", "status_from_flags", "set_wait_limit",
           "set_test_injection", "LayerDesc"]


class GemError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib.gem_status_string(status).decode()
        if status == 4:
            msg += " (cudaError %d)" % lib.gem_last_cuda_error()
        super().__init__("%s: %s [status %d]" % (what, msg, status))


def _check(st: int, what: str) -> None:
    if st != GEM_OK:
        raise GemError(st, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """Bytes for a call on `stream` (None: the current one), of that stream's memory: a block of another
    stream's may still be in use by work pending there, and would be given back to it at the end of the call."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


_HALF_BITS = (torch.int16, torch.uint16)   # binary16 bit patterns


def _dev(t: torch.Tensor | None, dtype, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    ok = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
    if not ok:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _cache_shape(k: torch.Tensor | None, v: torch.Tensor, B: int, n_kv: int, d: int) -> int:
    """Caches must be [B, n_kv, cap, d] (the kernels address them from these sizes); k may be
    None for a compact (V-only) cache."""
    for name, c in (("k_cache", k), ("v_cache", v)):
        if c is None and name == "k_cache":
            continue
        if c.dim() != 4 or c.shape[0] != B or c.shape[1] != n_kv or c.shape[3] != d:
            raise ValueError("%s must be [B=%d, n_kv=%d, cap, d=%d], got %s" % (name, B, n_kv, d, tuple(c.shape)))
    if k is not None and v.shape != k.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    return int(v.shape[2])


def _q4_bytes(W: torch.Tensor, N: int, K: int) -> None:
    # K % 32 != 0 is left to the library, which rejects it with GEM_ERR_BAD_SHAPE
    if K % 32 == 0 and W.numel() < N * (K // 32) * 18:
        raise ValueError("W must hold N x K Q4_0 weights (%d bytes), has %d" % (N * (K // 32) * 18, W.numel()))


def version() -> int:
    return lib.gem_version()


def device_status(reset: bool = False) -> int:
    v = C.c_int32(0)
    _check(lib.gem_device_status(C.byref(v), int(reset)), "gem_device_status")
    return v.value


def status_from_flags(flags: int) -> int:
    """gem_status that a set of GEM_DEVFLAG_* bits stands for (host only)."""
    return int(lib.gem_status_from_flags(flags))


INJECT_RING_SHORTFALL = 1
INJECT_GRID_ARRIVAL = 2


def set_wait_limit(ns: int) -> None:
    """Wall-time limit of every device-side wait on the current device (0: default 1 s)."""
    _check(lib.gem_set_wait_limit(int(ns)), "gem_set_wait_limit")


def set_test_injection(mask: int) -> None:
    """GEM_INJECT_* bits: make one bounded wait run out (tests of the timeout path)."""
    _check(lib.gem_set_test_injection(int(mask)), "gem_set_test_injection")


def q4_0_gemv_workspace(B: int, K: int) -> int:
    return int(lib.gem_q4_0_gemv_workspace(B, K))


def q4_0_gemv(W: torch.Tensor, N: int, K: int, x: torch.Tensor, y: torch.Tensor,
              residual: torch.Tensor | None = None, stream=None,
              workspace: torch.Tensor | None = None, shared_records: bool = False) -> torch.Tensor:
    """y[b] = deq(W) @ x[b] (+ residual[b]).  x: [B, >=K] fp32, y: [B, >=N] fp32.

    With B >= 2 the call goes through gem_q4_0_gemv_ws with `workspace` (a uint8 device tensor
    of q4_0_gemv_workspace(B, K) bytes; allocated here when not given), so concurrent calls
    share no state.  shared_records=True calls gem_q4_0_gemv instead, whose records live in
    the library's own per-device array."""
    B = x.shape[0] if x.dim() == 2 else 1
    _q4_bytes(W, N, K)
    if x.shape[-1] < K or y.shape[-1] < N:
        raise ValueError("x must have >= K columns and y >= N")
    need = q4_0_gemv_workspace(B, K) if K % 32 == 0 else 0
    if shared_records or need == 0:
        st = lib.gem_q4_0_gemv(_dev(W, torch.uint8, "W"), N, K, _dev(x, torch.float32, "x"),
                               x.shape[-1], B, _dev(y, torch.float32, "y"), y.shape[-1],
                               _dev(residual, torch.float32, "residual"), _stream(stream))
        _check(st, "gem_q4_0_gemv")
        return y
    if workspace is None:
        workspace = _scratch(need, x.device, stream)
    st = lib.gem_q4_0_gemv_ws(_dev(W, torch.uint8, "W"), N, K, _dev(x, torch.float32, "x"),
                              x.shape[-1], B, _dev(y, torch.float32, "y"), y.shape[-1],
                              _dev(residual, torch.float32, "residual"),
                              _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
                              _stream(stream))
    _check(st, "gem_q4_0_gemv_ws")
    return y


def q4_0_gemv_fused(W0: torch.Tensor, W1: torch.Tensor | None, N: int, K: int, x: torch.Tensor,
                    y: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6,
                    act: int = ACT_SILU, residual: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Pre-norm (gamma) + Q4_0 GEMV, or the gate/up pair (W1) with the gated activation.
    x: [B, >=K] fp32, y: [B, >=N] fp32; workspace as for q4_0_gemv (allocated when needed)."""
    B = x.shape[0] if x.dim() == 2 else 1
    _q4_bytes(W0, N, K)
    if W1 is not None:
        _q4_bytes(W1, N, K)
    if x.shape[-1] < K or y.shape[-1] < N:
        raise ValueError("x must have >= K columns and y >= N")
    need = q4_0_gemv_workspace(B, K) if K % 32 == 0 else 0
    if need and workspace is None:
        workspace = _scratch(need, x.device, stream)
    st = lib.gem_q4_0_gemv_fused(_dev(W0, torch.uint8, "W0"), _dev(W1, torch.uint8, "W1"), N, K,
                                 _dev(x, torch.float32, "x"), x.shape[-1], B,
                                 _dev(gamma, torch.float32, "gamma"), eps, act,
                                 _dev(y, torch.float32, "y"), y.shape[-1],
                                 _dev(residual, torch.float32, "residual"),
                                 _dev(workspace, torch.uint8, "workspace") if need else None,
                                 workspace.numel() if need else 0, _stream(stream))
    _check(st, "gem_q4_0_gemv_fused")
    return y


def q4_0_gemm_workspace(M: int, K: int) -> int:
    return int(lib.gem_q4_0_gemm_workspace(M, K))


def q4_0_gemm(W0: torch.Tensor, W1: torch.Tensor | None, N: int, K: int, x: torch.Tensor,
              y: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6,
              act: int = ACT_SILU, residual: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Batched prefill GEMM: M = x.shape[0] (<= 32) prompt rows through W0 (or the W0/W1 pair),
    each weight read once.  Same options as q4_0_gemv_fused; workspace allocated when needed."""
    M = x.shape[0] if x.dim() == 2 else 1
    _q4_bytes(W0, N, K)
    if W1 is not None:
        _q4_bytes(W1, N, K)
    if x.shape[-1] < K or y.shape[-1] < N:
        raise ValueError("x must have >= K columns and y >= N")
    need = q4_0_gemm_workspace(M, K) if K % 32 == 0 else 0
    if need and workspace is None:
        workspace = _scratch(need, x.device, stream)
    st = lib.gem_q4_0_gemm(_dev(W0, torch.uint8, "W0"), _dev(W1, torch.uint8, "W1"), N, K,
                           _dev(x, torch.float32, "x"), x.shape[-1], M,
                           _dev(gamma, torch.float32, "gamma"), eps, act,
                           _dev(y, torch.float32, "y"), y.shape[-1],
                           _dev(residual, torch.float32, "residual"),
                           _dev(workspace, torch.uint8, "workspace") if need else None,
                           workspace.numel() if need else 0, _stream(stream))
    _check(st, "gem_q4_0_gemm")
    return y


def q8_0_gemv(W: torch.Tensor, N: int, K: int, x: torch.Tensor, y: torch.Tensor,
              stream=None) -> torch.Tensor:
    """Tied Q8_0 embedding / logit projection: y[b] = deq(W) @ x[b].  W: N x (K/32*34) bytes."""
    B = x.shape[0] if x.dim() == 2 else 1
    if K % 32 == 0 and W.numel() < N * (K // 32) * 34:
        raise ValueError("W must hold N x K Q8_0 weights (%d bytes), has %d" % (N * (K // 32) * 34, W.numel()))
    if x.shape[-1] < K or y.shape[-1] < N:
        raise ValueError("x must have >= K columns and y >= N")
    st = lib.gem_q8_0_gemv(_dev(W, torch.uint8, "W"), N, K, _dev(x, torch.float32, "x"), x.shape[-1], B,
                           _dev(y, torch.float32, "y"), y.shape[-1], _stream(stream))
    _check(st, "gem_q8_0_gemv")
    return y


def argmax_workspace(B: int, N: int) -> int:
    return int(lib.gem_argmax_workspace(B, N))


def argmax(y: torch.Tensor, idx: torch.Tensor, workspace: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """idx[b] = index of the largest y[b][n] (lowest index on ties; NaN never chosen)."""
    B = y.shape[0] if y.dim() == 2 else 1
    N = y.shape[-1]
    if idx.numel() < B:
        raise ValueError("idx must hold B indices")
    need = argmax_workspace(B, N)
    if workspace is None:
        workspace = _scratch(max(need, 1), y.device, stream)
    st = lib.gem_argmax(_dev(y, torch.float32, "y"), N, B, N, _dev(idx, torch.int32, "idx"),
                        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "gem_argmax")
    return idx


def topk_workspace(B: int, N: int, k: int) -> int:
    return int(lib.gem_topk_workspace(B, N, k))


def topk(y: torch.Tensor, k: int, idx: torch.Tensor, val: torch.Tensor,
         workspace: torch.Tensor | None = None, stream=None):
    """The k largest entries of each row of y [B, N] fp32, largest first (ties: lowest index;
    NaN after every number): idx int32 [B, k], val fp32 [B, k]."""
    B = y.shape[0] if y.dim() == 2 else 1
    N = y.shape[-1]
    need = topk_workspace(B, N, k)
    if workspace is None and need:
        workspace = _scratch(need, y.device, stream)
    st = lib.gem_topk(_dev(y, torch.float32, "y"), N, B, N, k, _dev(idx, torch.int32, "idx"),
                      _dev(val, torch.float32, "val"), _dev(workspace, torch.uint8, "workspace"),
                      workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(st, "gem_topk")
    return idx, val


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor | None, eps: float, out: torch.Tensor,
            stream=None) -> torch.Tensor:
    B = x.shape[0] if x.dim() == 2 else 1
    st = lib.gem_rmsnorm(_dev(x, torch.float32, "x"), B, x.shape[-1],
                         _dev(gamma, torch.float32, "gamma"), eps,
                         _dev(out, torch.float32, "out"), _stream(stream))
    _check(st, "gem_rmsnorm")
    return out


def rmsnorm_qknorm_rope(qkv: torch.Tensor, n_q: int, n_kv: int, d: int,
                        gamma_q: torch.Tensor | None, gamma_k: torch.Tensor | None, v_mode: int,
                        eps: float, pos: torch.Tensor, theta: float, rope_dim: int,
                        k_cache: torch.Tensor | None, v_cache: torch.Tensor, window: int = 0,
                        status: torch.Tensor | None = None, stream=None) -> None:
    """qkv [B, ldqkv] fp32 in place; caches binary16 bits (int16/uint16) [B, n_kv, cap, d]; pos int32 [B].

    k_cache None with v_mode 1 appends the V row only (a compact full-attention cache)."""
    B = qkv.shape[0]
    cap = _cache_shape(k_cache, v_cache, B, n_kv, d)
    st = lib.gem_rmsnorm_qknorm_rope(
        _dev(qkv, torch.float32, "qkv"), qkv.shape[-1], B, n_q, n_kv, d,
        _dev(gamma_q, torch.float32, "gamma_q"), _dev(gamma_k, torch.float32, "gamma_k"),
        v_mode, eps, _dev(pos, torch.int32, "pos"), theta, rope_dim,
        _dev(k_cache, _HALF_BITS, "k_cache"), _dev(v_cache, _HALF_BITS, "v_cache"), cap,
        window, _dev(status, torch.int32, "status"), _stream(stream))
    _check(st, "gem_rmsnorm_qknorm_rope")


def gqa_decode_attn_workspace(B: int, n_q: int, n_kv: int, d: int, cache_cap: int,
                              window: int = 0) -> int:
    return int(lib.gem_gqa_decode_attn_workspace(B, n_q, n_kv, d, cache_cap, window))


def gqa_decode_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, n_q: int,
                    n_kv: int, d: int, pos: torch.Tensor, window: int, scale: float,
                    out: torch.Tensor, workspace: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [B, ldq] fp32 (head h at column h*d); caches uint16 [B, n_kv, cap, d]."""
    B = q.shape[0]
    cap = _cache_shape(k_cache, v_cache, B, n_kv, d)
    ws_ptr = _dev(workspace, torch.uint8, "workspace")
    ws_bytes = workspace.numel() if workspace is not None else 0
    st = lib.gem_gqa_decode_attn(
        _dev(q, torch.float32, "q"), q.shape[-1], _dev(k_cache, _HALF_BITS, "k_cache"),
        _dev(v_cache, _HALF_BITS, "v_cache"), B, n_q, n_kv, d, cap,
        _dev(pos, torch.int32, "pos"), window, scale, _dev(out, torch.float32, "out"),
        out.shape[-1], ws_ptr, ws_bytes, _dev(status, torch.int32, "status"), _stream(stream))
    _check(st, "gem_gqa_decode_attn")
    return out


def gqa_decode_attn_fused(qkv: torch.Tensor, n_q: int, n_kv: int, d: int,
                          gamma_q: torch.Tensor | None, gamma_k: torch.Tensor | None, v_mode: int,
                          eps: float, pos: torch.Tensor, theta: float, rope_dim: int,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, window: int, scale: float,
                          out: torch.Tensor, workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """QK-norm + RoPE + KV append + attention from the raw QKV projection row (qkv [B, ldqkv])."""
    B = qkv.shape[0]
    cap = _cache_shape(k_cache, v_cache, B, n_kv, d)
    st = lib.gem_gqa_decode_attn_fused(
        _dev(qkv, torch.float32, "qkv"), qkv.shape[-1], B, n_q, n_kv, d,
        _dev(gamma_q, torch.float32, "gamma_q"), _dev(gamma_k, torch.float32, "gamma_k"), v_mode, eps,
        _dev(pos, torch.int32, "pos"), theta, rope_dim, _dev(k_cache, _HALF_BITS, "k_cache"),
        _dev(v_cache, _HALF_BITS, "v_cache"), cap, window, scale, _dev(out, torch.float32, "out"),
        out.shape[-1], _dev(workspace, torch.uint8, "workspace"),
        workspace.numel() if workspace is not None else 0, _dev(status, torch.int32, "status"),
        _stream(stream))
    _check(st, "gem_gqa_decode_attn_fused")
    return out


def gqa_decode_attn_compact_workspace(B: int, n_q: int, n_kv: int, d: int, cache_cap: int,
                                      rope_dim: int) -> int:
    return int(lib.gem_gqa_decode_attn_compact_workspace(B, n_q, n_kv, d, cache_cap, rope_dim))


def gqa_decode_attn_compact(q: torch.Tensor, v_cache: torch.Tensor, n_q: int, n_kv: int, d: int,
                            pos: torch.Tensor, scale: float, gamma_k: torch.Tensor, rope_dim: int,
                            theta: float, out: torch.Tensor, workspace: torch.Tensor | None = None,
                            status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention over a V-only cache; K_j = RoPE_j(V_j * gamma_k) is rebuilt inside the kernel."""
    B = q.shape[0]
    cap = _cache_shape(None, v_cache, B, n_kv, d)
    st = lib.gem_gqa_decode_attn_compact(
        _dev(q, torch.float32, "q"), q.shape[-1], _dev(v_cache, _HALF_BITS, "v_cache"), B, n_q, n_kv,
        d, cap, _dev(pos, torch.int32, "pos"), scale, _dev(gamma_k, torch.float32, "gamma_k"),
        rope_dim, theta, _dev(out, torch.float32, "out"), out.shape[-1],
        _dev(workspace, torch.uint8, "workspace"), workspace.numel() if workspace is not None else 0,
        _dev(status, torch.int32, "status"), _stream(stream))
    _check(st, "gem_gqa_decode_attn_compact")
    return out


NOALLOC_SCRATCH_BYTES = 8 << 20  # GEM_ATTN_NOALLOC_SCRATCH_BYTES


def gqa_decode_attn_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            n_q: int, n_kv: int, d: int, pos: torch.Tensor, window: int,
                            scale: float, out: torch.Tensor, status: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """gqa_decode_attn with the split partials in the library's own per-device array.

    For callers that must not allocate device memory while decoding.  Allocates nothing;
    calls that may run concurrently on one device race on the shared array; shapes whose
    partials exceed NOALLOC_SCRATCH_BYTES raise GemError (GEM_ERR_WORKSPACE)."""
    B = q.shape[0]
    cap = _cache_shape(k_cache, v_cache, B, n_kv, d)
    st = lib.gem_gqa_decode_attn_noalloc(
        _dev(q, torch.float32, "q"), q.shape[-1], _dev(k_cache, _HALF_BITS, "k_cache"),
        _dev(v_cache, _HALF_BITS, "v_cache"), B, n_q, n_kv, d, cap,
        _dev(pos, torch.int32, "pos"), window, scale, _dev(out, torch.float32, "out"),
        out.shape[-1], _dev(status, torch.int32, "status"), _stream(stream))
    _check(st, "gem_gqa_decode_attn_noalloc")
    return out


def swiglu(gate: torch.Tensor, up: torch.Tensor, act: int, out: torch.Tensor,
           stream=None) -> torch.Tensor:
    B = gate.shape[0] if gate.dim() == 2 else 1
    st = lib.gem_swiglu(_dev(gate, torch.float32, "gate"), _dev(up, torch.float32, "up"), B,
                        gate.shape[-1], act, _dev(out, torch.float32, "out"), _stream(stream))
    _check(st, "gem_swiglu")
    return out


# ---- paged 4-bit KV cache -------------------------------------------------------------------


def _here(t: torch.Tensor, dtype, name: str, shape, device: int):
    """Pointer of a contiguous tensor of this type and shape on the current device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError("%s must be contiguous %s %s on the current CUDA device, got %s %s on %s" % (
            name, dtype, tuple(shape), t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _rows(t: torch.Tensor, cols: int, name: str, device: int):
    """(pointer, row stride, rows) of an fp32 [rows, >= cols] tensor whose rows are contiguous; a column
    range of a wider tensor will do."""
    if t.dim() != 2 or t.dtype is not torch.float32 or t.get_device() != device:
        raise ValueError("%s must be fp32 [rows, >= %d] on the current CUDA device, got %s %s on %s" % (
            name, cols, t.dtype, tuple(t.shape), t.device))
    rows, have = t.shape
    ld, step = t.stride()
    if have < cols or (step != 1 and have > 1 and rows):
        raise ValueError("%s must be fp32 [rows, >= %d] with contiguous rows, got %s strides %s" % (
            name, cols, tuple(t.shape), t.stride()))
    return t.data_ptr(), (ld if rows > 1 else (have + 3) // 4 * 4), rows


def _stream_on(stream, device: int) -> int:
    """Handle of `stream`, or of the current stream of `device` (the current one)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _status(status: torch.Tensor | None, device: int):
    return None if status is None else _here(status, torch.int32, "status", status.shape, device)


def _pool(pool: torch.Tensor, n_kv: int, d: int, page: int, device: int):
    """(pointer, pages) of a pool [n_pages, kv4_page_bytes(n_kv, d, page)]; the library rejects the sizes
    that have no pages."""
    n_pages = pool.shape[0]
    return _here(pool, torch.uint8, "pool", (n_pages, n_kv * d * page * 9 // 8), device), n_pages


def kv4_page_bytes(n_kv: int, d: int, page: int) -> int:
    """Bytes of one page of the 4-bit KV cache; 0 for sizes that the calls reject."""
    return int(lib.gem_kv4_page_bytes(n_kv, d, page))


def kv_block_tables(cached: torch.Tensor, fresh: torch.Tensor, page: int, table: torch.Tensor, ring: torch.Tensor,
                    ring_in: torch.Tensor, ring_out: torch.Tensor, kv_len: torch.Tensor, cu_tokens: torch.Tensor,
                    slot: torch.Tensor, pos: torch.Tensor, seq: torch.Tensor, status: torch.Tensor | None = None,
                    stream=None) -> None:
    """Pages for the new tokens of B requests (or back from ended ones, fresh -1), and every token's
    slot, position and request.  int32 tensors cached, fresh, kv_len [B], cu_tokens [B + 1],
    table [B, max_pages], ring [n_pages], slot, pos, seq [T_cap]; int64 ring_in, ring_out [2]."""
    dev = torch.cuda.current_device()
    i32, i64 = torch.int32, torch.int64
    B, T, n_pages, max_pages = cached.shape[0], slot.shape[0], ring.shape[0], table.shape[-1]
    st = lib.gem_kv_block_tables(
        _here(cached, i32, "cached", (B,), dev), _here(fresh, i32, "fresh", (B,), dev), B, page,
        _here(table, i32, "table", (B, max_pages), dev), max_pages, _here(ring, i32, "ring", (n_pages,), dev), n_pages,
        _here(ring_in, i64, "ring_in", (2,), dev), _here(ring_out, i64, "ring_out", (2,), dev),
        _here(kv_len, i32, "kv_len", (B,), dev), _here(cu_tokens, i32, "cu_tokens", (B + 1,), dev),
        _here(slot, i32, "slot", (T,), dev), _here(pos, i32, "pos", (T,), dev), _here(seq, i32, "seq", (T,), dev), T,
        _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_kv_block_tables")


def qknorm_mrope(qkv: torch.Tensor, n_q: int, n_kv: int, d: int, gamma_q: torch.Tensor | None,
                 gamma_k: torch.Tensor | None, eps: float, pos: torch.Tensor, sections, theta: float,
                 out: torch.Tensor, interleaved: bool = False, status: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """QK-norm and RoPE of the Q and K heads of T rows.  qkv, out: fp32 [T, >= (n_q + n_kv) * d] (out may
    be qkv); pos int32 [n_axes, T]; sections: the number of frequencies of each axis (their sum is half
    of the rotated dims); interleaved: the axes take turns along the frequencies."""
    dev = torch.cuda.current_device()
    cols, axes = (n_q + n_kv) * d, len(sections)
    xp, ldx, T = _rows(qkv, cols, "qkv", dev)
    op, ldo, rows = _rows(out, cols, "out", dev)
    if rows != T:
        raise ValueError("out must have T=%d rows, got %d" % (T, rows))
    st = lib.gem_qknorm_mrope(
        xp, ldx, T, n_q, n_kv, d, None if gamma_q is None else _here(gamma_q, torch.float32, "gamma_q", (d,), dev),
        None if gamma_k is None else _here(gamma_k, torch.float32, "gamma_k", (d,), dev), eps,
        _here(pos, torch.int32, "pos", (axes, T), dev), T, axes, (C.c_int32 * axes)(*sections), int(interleaved), theta,
        op, ldo, _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_qknorm_mrope")
    return out


def kv4_append(k: torch.Tensor, v: torch.Tensor, n_kv: int, d: int, slot: torch.Tensor, pool: torch.Tensor,
               page: int, status: torch.Tensor | None = None, stream=None) -> None:
    """Quantise the rows of k and v (fp32 [T, >= n_kv * d], columns of a wider tensor will do) into the
    slots int32 [T] (-1: none) of pool (uint8 [n_pages, kv4_page_bytes(n_kv, d, page)])."""
    dev = torch.cuda.current_device()
    kp, ldk, T = _rows(k, n_kv * d, "k", dev)
    vp, ldv, rows = _rows(v, n_kv * d, "v", dev)
    pp, n_pages = _pool(pool, n_kv, d, page, dev)
    if rows != T:
        raise ValueError("k and v must have the same number of rows, got %d and %d" % (T, rows))
    st = lib.gem_kv4_append(kp, ldk, vp, ldv, T, n_kv, d, _here(slot, torch.int32, "slot", (T,), dev), pp, n_pages,
                            page, _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_kv4_append")


def kv4_gather(pool: torch.Tensor, page: int, n_kv: int, d: int, slot: torch.Tensor, k: torch.Tensor | None,
               v: torch.Tensor | None, status: torch.Tensor | None = None, stream=None):
    """Read the rows at the slots int32 [T] back into k and v (fp32 [T, >= n_kv * d], either may be None)."""
    dev = torch.cuda.current_device()
    pp, n_pages = _pool(pool, n_kv, d, page, dev)
    T = slot.shape[0]
    kp, ldk, k_rows = (None, 0, T) if k is None else _rows(k, n_kv * d, "k", dev)
    vp, ldv, v_rows = (None, 0, T) if v is None else _rows(v, n_kv * d, "v", dev)
    if k_rows != T or v_rows != T:
        raise ValueError("k and v must have one row for each of the %d slots" % T)
    st = lib.gem_kv4_gather(pp, n_pages, page, n_kv, d, _here(slot, torch.int32, "slot", (T,), dev), T, kp, ldk, vp,
                            ldv, _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_kv4_gather")
    return k, v


def kv4_attn_workspace(T: int, B: int, n_q: int, n_kv: int, d: int) -> int:
    return int(lib.gem_kv4_attn_workspace(T, B, n_q, n_kv, d))


def kv4_attn(q: torch.Tensor, n_q: int, n_kv: int, d: int, cu_tokens: torch.Tensor, kv_len: torch.Tensor,
             table: torch.Tensor, pool: torch.Tensor, page: int, window: int, scale: float, out: torch.Tensor,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Attention of the rows of q (fp32 [T, >= n_q * d]) over the paged 4-bit cache: request b's rows are
    cu_tokens[b] .. cu_tokens[b + 1] (int32 [B + 1]), the last positions of its kv_len[b] (int32 [B]);
    table int32 [B, max_pages].  workspace: uint8, at least kv4_attn_workspace(...) bytes (allocated when
    not given)."""
    dev = torch.cuda.current_device()
    qp, ldq, T = _rows(q, n_q * d, "q", dev)
    op, ldo, rows = _rows(out, n_q * d, "out", dev)
    pp, n_pages = _pool(pool, n_kv, d, page, dev)
    B, max_pages = kv_len.shape[0], table.shape[-1]
    if rows != T:
        raise ValueError("out must have T=%d rows, got %d" % (T, rows))
    if workspace is None:
        workspace = _scratch(lib.gem_kv4_attn_workspace(T, B, n_q, n_kv, d), q.device, stream)
    ws_bytes = workspace.shape[0]
    st = lib.gem_kv4_attn(qp, ldq, T, _here(cu_tokens, torch.int32, "cu_tokens", (B + 1,), dev),
                          _here(kv_len, torch.int32, "kv_len", (B,), dev), B, n_q, n_kv, d,
                          _here(table, torch.int32, "table", (B, max_pages), dev), max_pages, pp, n_pages, page, window,
                          scale, op, ldo, _here(workspace, torch.uint8, "workspace", (ws_bytes,), dev), ws_bytes,
                          _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_kv4_attn")
    return out


# ---- 8-bit floating point, scores -----------------------------------------------------------


_E4M3 = (torch.uint8, torch.float8_e4m3fn)   # e4m3 codes


def _codes(t: torch.Tensor, cols: int, name: str, device: int):
    """(pointer, row stride, rows) of e4m3 codes [rows, >= cols] (uint8 or float8_e4m3fn) whose rows are contiguous."""
    if t.dim() != 2 or t.dtype not in _E4M3 or t.get_device() != device:
        raise ValueError("%s must be uint8 or float8_e4m3fn [rows, >= %d] on the current CUDA device, got %s %s on %s" % (
            name, cols, t.dtype, tuple(t.shape), t.device))
    rows, have = t.shape
    ld, step = t.stride()
    if have < cols or (step != 1 and have > 1 and rows):
        raise ValueError("%s must be [rows, >= %d] with contiguous rows, got %s strides %s" % (
            name, cols, tuple(t.shape), t.stride()))
    return t.data_ptr(), (ld if rows > 1 else (have + 15) // 16 * 16), rows


def _same_rows(rows: int, **others: int) -> None:
    for name, n in others.items():
        if n != rows:
            raise ValueError("%s must have %d rows, got %d" % (name, rows, n))


def rmsnorm_fp8(x: torch.Tensor, gamma: torch.Tensor | None, eps: float, codes: torch.Tensor, scales: torch.Tensor,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """RMSNorm of x (+ residual) in 8 bits: x fp32 [T, H], codes uint8 or float8_e4m3fn [T, >= H], scales fp32
    [T, >= ceil(H / 128)].  out (may be x or residual) receives x + residual."""
    dev = torch.cuda.current_device()
    H = x.shape[-1]
    xp, ldx, T = _rows(x, H, "x", dev)
    rp, ldr, r_rows = (None, 0, T) if residual is None else _rows(residual, H, "residual", dev)
    op, ldo, o_rows = (None, 0, T) if out is None else _rows(out, H, "out", dev)
    cp, ldc, c_rows = _codes(codes, H, "codes", dev)
    sp, lds, s_rows = _rows(scales, -(-H // 128), "scales", dev)
    if not T == r_rows == o_rows == c_rows == s_rows:
        _same_rows(T, residual=r_rows, out=o_rows, codes=c_rows, scales=s_rows)
    st = lib.gem_rmsnorm_fp8(xp, ldx, rp, ldr, op, ldo, T, H, None if gamma is None else _here(gamma, torch.float32, "gamma", (H,), dev),
                             eps, cp, ldc, sp, lds, _stream_on(stream, dev))
    _check(st, "gem_rmsnorm_fp8")
    return codes, scales


def quant_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, up: torch.Tensor | None = None,
              act: int = ACT_SILU, stream=None):
    """act(x) * up, or x itself (up None), in 8 bits; x, up fp32 [T, H] (column ranges of a wider tensor will
    do), codes and scales as rmsnorm_fp8."""
    dev = torch.cuda.current_device()
    H = x.shape[-1]
    xp, ldx, T = _rows(x, H, "x", dev)
    up_p, ldu, u_rows = (None, 0, T) if up is None else _rows(up, H, "up", dev)
    cp, ldc, c_rows = _codes(codes, H, "codes", dev)
    sp, lds, s_rows = _rows(scales, -(-H // 128), "scales", dev)
    if not T == u_rows == c_rows == s_rows:
        _same_rows(T, up=u_rows, codes=c_rows, scales=s_rows)
    st = lib.gem_quant_fp8(xp, ldx, up_p, ldu, T, H, act, cp, ldc, sp, lds, _stream_on(stream, dev))
    _check(st, "gem_quant_fp8")
    return codes, scales


def fp8_gemm(W: torch.Tensor, w_scales: torch.Tensor, x: torch.Tensor, x_scales: torch.Tensor, y: torch.Tensor,
             residual: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x @ W.T (+ residual) of 8-bit rows: W [N, K] e4m3 (uint8 or float8_e4m3fn) with w_scales fp32
    [ceil(N / 128), ceil(K / 128)], x [M, >= K] with x_scales fp32 [M, >= ceil(K / 128)], y and residual (which
    may be y) fp32 [M, >= N] of the same row stride.  W is read while the kernel before this one on the stream may still run:
    a kernel that writes it must not be that one (a synchronisation or another launch between them will do)."""
    dev = torch.cuda.current_device()
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be contiguous [N, K], got %s strides %s" % (tuple(W.shape), W.stride()))
    N, K = W.shape
    wp, _, _ = _codes(W, K, "W", dev)
    xp, ldx, M = _codes(x, K, "x", dev)
    sp, lds, s_rows = _rows(x_scales, -(-K // 128), "x_scales", dev)
    yp, ldy, y_rows = _rows(y, N, "y", dev)
    rp, ldr, r_rows = (None, ldy, M) if residual is None else _rows(residual, N, "residual", dev)
    if not M == s_rows == y_rows == r_rows:
        _same_rows(M, x_scales=s_rows, y=y_rows, residual=r_rows)
    if ldr != ldy and M > 1:
        raise ValueError("residual must have y's row stride %d, got %d" % (ldy, ldr))
    st = lib.gem_fp8_gemm(wp, _here(w_scales, torch.float32, "w_scales", (-(-N // 128), -(-K // 128)), dev), N, K, xp, ldx,
                          sp, lds, M, yp, ldy, rp, _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_fp8_gemm")
    return y


def logprobs(y: torch.Tensor, tokens: torch.Tensor | None, logp: torch.Tensor | None, entropy: torch.Tensor | None = None,
             rank: torch.Tensor | None = None, idx: torch.Tensor | None = None, val: torch.Tensor | None = None,
             scale: float = 1.0, status: torch.Tensor | None = None, stream=None,
             workspace: torch.Tensor | None = None) -> None:
    """Scores of the logit rows y (fp32 [T, N]): logp, entropy fp32 and rank int32 [T] of the tokens int32 [T]
    (-1: none), and the k alternatives idx int32, val fp32 [T, k] with their log probabilities.  Outputs that are
    None are not computed.  workspace: uint8 bytes, as for the other calls with scratch; the call needs none and leaves
    them as they are."""
    dev = torch.cuda.current_device()
    N = y.shape[-1]
    yp, ldy, T = _rows(y, N, "y", dev)
    f32, i32 = torch.float32, torch.int32
    if (idx is None) != (val is None):
        raise ValueError("idx and val come together")
    if workspace is not None:
        _here(workspace, torch.uint8, "workspace", workspace.shape, dev)
    k = 0 if idx is None else idx.shape[-1]
    st = lib.gem_logprobs(yp, ldy, T, N, scale, None if tokens is None else _here(tokens, i32, "tokens", (T,), dev),
                          None if logp is None else _here(logp, f32, "logp", (T,), dev), None if rank is None else _here(rank, i32, "rank", (T,), dev),
                          None if entropy is None else _here(entropy, f32, "entropy", (T,), dev), k, _here(idx, i32, "idx", (T, k), dev) if k else None,
                          _here(val, f32, "val", (T, k), dev) if k else None, _status(status, dev), _stream_on(stream, dev))
    _check(st, "gem_logprobs")


class DeviceLayer:
    """Device-resident weights of one decoder layer plus its gem_layer_desc."""

    def __init__(self, shape, tensors, device="cuda"):
        def up(a, dt):
            return None if a is None else torch.from_numpy(a).to(device=device, dtype=dt).contiguous()

        self.shape = shape
        self.w_qkv = up(tensors.w_qkv, torch.uint8)
        self.w_o = up(tensors.w_o, torch.uint8)
        self.w_gate = up(tensors.w_gate, torch.uint8)
        self.w_up = up(tensors.w_up, torch.uint8)
        self.w_down = up(tensors.w_down, torch.uint8)
        self.g_attn = up(tensors.g_attn, torch.float32)
        self.g_ffn = up(tensors.g_ffn, torch.float32)
        self.g_q = up(tensors.g_q, torch.float32)
        self.g_k = up(tensors.g_k, torch.float32)
        self.g_post_attn = up(tensors.g_post_attn, torch.float32)
        self.g_post_ffn = up(tensors.g_post_ffn, torch.float32)
        self._make_desc()

    _TENSORS = ("w_qkv", "w_o", "w_gate", "w_up", "w_down", "g_attn", "g_ffn", "g_q", "g_k",
                "g_post_attn", "g_post_ffn")

    @classmethod
    def clone(cls, src: "DeviceLayer") -> "DeviceLayer":
        """A layer with its own device copies of src's weights (same values, new buffers)."""
        obj = cls.__new__(cls)
        obj.shape = src.shape
        for name in cls._TENSORS:
            t = getattr(src, name)
            setattr(obj, name, None if t is None else t.clone())
        obj._make_desc()
        return obj

    def _make_desc(self):
        ptr = lambda t: None if t is None else t.data_ptr()
        s = self.shape
        self.desc = LayerDesc(
            H=s.H, n_q=s.n_q, n_kv=s.n_kv, d=s.d, F=s.F, eps=s.eps, theta=s.theta,
            scale=float(s.scale), rope_dim=s.rope_dim, window=s.window, act=s.act,
            qk_norm=int(s.qk_norm), v_from_k=int(s.v_from_k), post_norms=int(s.post_norms),
            w_qkv=ptr(self.w_qkv), w_o=ptr(self.w_o), w_gate=ptr(self.w_gate),
            w_up=ptr(self.w_up), w_down=ptr(self.w_down), g_attn=ptr(self.g_attn),
            g_ffn=ptr(self.g_ffn), g_q=ptr(self.g_q), g_k=ptr(self.g_k),
            g_post_attn=ptr(self.g_post_attn), g_post_ffn=ptr(self.g_post_ffn),
            compact_kv=int(getattr(s, "compact_kv", False)))

    def weight_bytes(self) -> int:
        return sum(t.numel() for t in (self.w_qkv, self.w_o, self.w_gate, self.w_up, self.w_down))


def decode_layer_workspace(layer: DeviceLayer, B: int, cache_cap: int) -> int:
    return int(lib.gem_decode_layer_workspace(C.byref(layer.desc), B, cache_cap))


def decode_layer(layer: DeviceLayer, x: torch.Tensor, k_cache: torch.Tensor | None,
                 v_cache: torch.Tensor, pos: torch.Tensor, workspace: torch.Tensor,
                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One layer step, in place on x [B, H] fp32; caches uint16 [B, n_kv, cap, d] (a compact_kv
    layer keeps the V cache alone: k_cache may be None)."""
    B = x.shape[0]
    s = layer.shape
    cap = _cache_shape(k_cache, v_cache, B, s.n_kv, s.d)
    if x.dim() != 2 or x.shape[1] != s.H:
        raise ValueError("x must be [B, H=%d], got %s" % (s.H, tuple(x.shape)))
    st = lib.gem_decode_layer(C.byref(layer.desc), B, _dev(x, torch.float32, "x"),
                              _dev(k_cache, _HALF_BITS, "k_cache"),
                              _dev(v_cache, _HALF_BITS, "v_cache"), cap,
                              _dev(pos, torch.int32, "pos"), _dev(workspace, torch.uint8, "workspace"),
                              workspace.numel(), _dev(status, torch.int32, "status"),
                              _stream(stream))
    _check(st, "gem_decode_layer")
    return x


class StepPlan:
    """Every layer of a decode step in one persistent launch (gem_step_plan).

    layers: DeviceLayer list; k_caches, v_caches: per-layer uint16 [B, n_kv, cap, d]
    tensors, kept referenced by the plan."""

    def __init__(self, layers, B: int, k_caches, v_caches):
        n = len(layers)
        if len(k_caches) != n or len(v_caches) != n:
            raise ValueError("one K and one V cache per layer")
        for dl, k, v in zip(layers, k_caches, v_caches):
            _cache_shape(k, v, B, dl.shape.n_kv, dl.shape.d)
        self._keep = (list(layers), list(k_caches), list(v_caches))
        descs = (LayerDesc * n)(*[dl.desc for dl in layers])
        kp = (C.c_void_p * n)(*[_dev(k, _HALF_BITS, "k_cache") for k in k_caches])
        vp = (C.c_void_p * n)(*[_dev(v, _HALF_BITS, "v_cache") for v in v_caches])
        caps = (C.c_int64 * n)(*[int(k.shape[2]) for k in k_caches])
        h = C.c_void_p()
        st = lib.gem_step_plan_create(descs, n, B, kp, vp, caps, C.byref(h))
        _check(st, "gem_step_plan_create")
        self._h = h
        self.B = B

    def step(self, x: torch.Tensor, pos: torch.Tensor, status: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
        H = self._keep[0][0].shape.H
        if x.dim() != 2 or x.shape[0] != self.B or x.shape[1] != H:
            raise ValueError("x must be [B=%d, H=%d], got %s" % (self.B, H, tuple(x.shape)))
        if pos.numel() < self.B:
            raise ValueError("pos must hold B positions")
        st = lib.gem_decode_step(self._h, _dev(x, torch.float32, "x"), _dev(pos, torch.int32, "pos"),
                                 _dev(status, torch.int32, "status"), _stream(stream))
        _check(st, "gem_decode_step")
        return x

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib.gem_step_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
