"""B200 (sm_100a) matrix products with GGUF block-quantized weights.

A thin Python binding over the C ABI in ``include/kq.h`` (shared library
``_lib/libkq.so``, built by ``python -m gguf_quant_dequant_q4_b200.build``).
This module only marshals arguments: torch provides device memory and the
current CUDA stream, every step of the computation runs in the library's
kernels.  There is no CPU fallback; calling an op without the built library or
without a CUDA device raises.

Codecs (ggml type ids): ``Q4_0 = 2``, ``Q8_0 = 8``, ``Q4_K = 12``, ``Q5_K = 13``,
``Q6_K = 14`` (q5_K and q4_0: dequantize and the tensor-core products).  Weights are
wire bytes ``uint8 [N, row_bytes]`` ("transpose=True" layout: y = x @ W.T),
activations ``bfloat16 [M, K]``, outputs ``float32``.

KV cache (``kv_plan``, ``kv_append``, ``kv_attention``): pools of keys and of
values are ``uint8 [pages, kv_heads, page_size, row_bytes(Q4_0, head_dim)]``, rows
of q4_0 blocks as ``dequantize`` reads them.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

Q4_0, Q8_0, Q4_K, Q5_K, Q6_K = 2, 8, 12, 13, 14
NAMES = {Q4_0: "q4_0", Q8_0: "q8_0", Q4_K: "q4_K", Q5_K: "q5_K", Q6_K: "q6_K"}
_BLOCK = {Q4_0: (32, 18), Q8_0: (32, 34), Q4_K: (256, 144), Q5_K: (256, 176), Q6_K: (256, 210)}
TILE_ROWS = 64

DEV_BAD_EXPERT, DEV_BAD_ROWS, DEV_BAD_RANGE, DEV_UNSORTED = 0x1, 0x2, 0x4, 0x8
DEV_TIMEOUT, DEV_TOO_MANY, DEV_X_RANGE = 0x10, 0x20, 0x40

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libkq.so")

# Every entry point declared in include/kq.h: name -> (restype, argtypes)
_vp, _i64, _i32, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
SIGNATURES = {
    "kq_block_info": (_int, [_int, ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "kq_status_string": (ctypes.c_char_p, [_int]),
    "kq_last_cuda_error": (_int, []),
    "kq_read_device_status": (_int, [ctypes.POINTER(_i32), _int]),
    "kq_set_wait_limit": (_int, [_i64]),
    "kq_dequantize": (_int, [_int, _vp, _i64, _i64, _vp, _vp]),
    "kq_quantize": (_int, [_int, _vp, _i64, _i64, _vp, _vp]),
    "kq_qmv": (_int, [_int, _vp, _i64, _i64, _vp, _i64, _vp, _vp]),
    "kq_qmm": (_int, [_int, _vp, _i64, _i64, _vp, _i64, _vp, _vp]),
    "kq_moe_sort": (_int, [_vp, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "kq_expert_tile_map": (_int, [_vp, _i64, _i32, _vp, _i64, _vp, _vp, _vp]),
    "kq_gather_qmm": (_int, [_int, _vp, _i32, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp]),
    "kq_gather_qmv": (_int, [_int, _vp, _i32, _i64, _i64, _vp, _i32, _vp, _i64, _i32, _vp, _vp, _vp]),
    "kq_gather_mix": (_int, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _vp]),
    "kq_moe_glu_gather": (_int, [_int, _vp, _vp, _i32, _i64, _i64, _vp, _vp, _i64, _i32, _i32, ctypes.c_float,
                                 _vp, _vp, _vp]),
    "kq_kv_plan": (_int, [_vp, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "kq_kv_append": (_int, [_int, _vp, _vp, _int, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _i32, _vp, _vp]),
    "kq_kv_attention_workspace": (_int, [_i32, _i32, _i32, _i32, ctypes.POINTER(_i64)]),
    "kq_kv_attention": (_int, [_int, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp,
                               _i64, ctypes.c_float, _i32, _i32, _vp, _vp, _i64, _vp, _vp]),
}
ACT_SILU, ACT_GELU_TANH, ACT_SILU_LIMIT = 0, 1, 2

_lib = None


class KQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().kq_status_string(status).decode()
        if status == 4:
            msg += f" (cudaError {lib().kq_last_cuda_error()})"
        super().__init__(f"{what}: {msg} [status {status}]")


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m gguf_quant_dequant_q4_b200.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise KQError(rc, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need_cuda(*ts):
    # contiguity first: a strided view (say, some rows of every expert of a
    # bank) would otherwise be walked with the packed stride
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")


def _need(t, what: str, size: int, count: int | None = None, exact: bool = False) -> None:
    """Tensor ``t`` (if given) holds elements of ``size`` bytes, and at least
    (or exactly) ``count`` of them: the C ABI takes bare pointers, so a buffer
    shorter than the call's sizes would be read or written past its end."""
    if t is None:
        return
    if t.element_size() != size:
        raise TypeError(f"{what}: {size}-byte elements expected, got {t.dtype}")
    if count is not None and (t.numel() != count if exact else t.numel() < count):
        raise ValueError(f"{what}: {'exactly' if exact else 'at least'} {count} elements expected, got {t.numel()}")


def _whole_blocks(qtype: int, k: int) -> bool:
    # sizes the library accepts; anything else it rejects with its own status
    return qtype in _BLOCK and k > 0 and k % _BLOCK[qtype][0] == 0


def _need_bank(w, what: str, qtype: int, k: int, dims: int) -> None:
    """Weight bytes with ``dims`` dimensions whose rows hold ``k`` values."""
    _need(w, what, 1)
    if w.dim() != dims:
        raise ValueError(f"{what}: {dims} dimensions expected, got {w.dim()}")
    if _whole_blocks(qtype, k) and w.shape[-1] != row_bytes(qtype, k):
        raise ValueError(f"{what}: rows of {row_bytes(qtype, k)} bytes expected for k = {k}, got {w.shape[-1]}")


def block_info(qtype: int) -> tuple[int, int]:
    v, b = _int(), _int()
    _check(lib().kq_block_info(qtype, ctypes.byref(v), ctypes.byref(b)), "kq_block_info")
    return v.value, b.value


def row_bytes(qtype: int, k: int) -> int:
    vpb, bpb = _BLOCK[qtype]
    return k // vpb * bpb


def read_device_status(clear: bool = False) -> int:
    v = _i32()
    _check(lib().kq_read_device_status(ctypes.byref(v), int(clear)), "kq_read_device_status")
    return v.value


def set_wait_limit(ns: int = 0) -> None:
    """Time limit (ns) of the staged decode kernel's pipeline waits; 0 restores
    the default (2 s).  For fault-handling tests."""
    _check(lib().kq_set_wait_limit(int(ns)), "kq_set_wait_limit")


def _bf16_bits(x: torch.Tensor) -> torch.Tensor:
    if x.dtype == torch.bfloat16:
        return x
    if x.dtype in (torch.uint16, torch.int16):
        return x
    raise TypeError("activations must be bfloat16")


def dequantize(w: torch.Tensor, qtype: int, k: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [..., N, K] decode of wire bytes [..., N, row_bytes] (bit-exact)."""
    rows = w.numel() // max(1, w.shape[-1]) if w.dim() else 0
    _need(w, "w", 1)
    if w.dim() and _whole_blocks(qtype, k) and w.shape[-1] != row_bytes(qtype, k):
        raise ValueError(f"w: rows of {row_bytes(qtype, k)} bytes expected for k = {k}, got {w.shape[-1]}")
    if out is None:
        out = torch.empty(*w.shape[:-1], k, dtype=torch.float32, device=w.device)
    _need(out, "out", 4, rows * k)
    _need_cuda(w, out)
    _check(lib().kq_dequantize(qtype, _ptr(w), rows, k, _ptr(out), _stream(stream)), "kq_dequantize")
    return out


def quantize(w: torch.Tensor, qtype: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Wire bytes uint8 [..., row_bytes] of fp32 weights [..., K]."""
    if w.dtype != torch.float32:
        raise TypeError("weights must be float32")
    k = w.shape[-1]
    rows = w.numel() // max(1, k)
    if out is None:
        out = torch.empty(*w.shape[:-1], row_bytes(qtype, k), dtype=torch.uint8, device=w.device)
    if _whole_blocks(qtype, k):
        _need(out, "out", 1, rows * row_bytes(qtype, k))
    _need_cuda(w, out)
    _check(lib().kq_quantize(qtype, _ptr(w), rows, k, _ptr(out), _stream(stream)), "kq_quantize")
    return out


def qmv(x: torch.Tensor, w: torch.Tensor, qtype: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ dequant(w[N, :]).T for 1 <= M <= 16."""
    x = _bf16_bits(x)
    m, k = x.shape
    n = w.shape[0]
    _need_bank(w, "w", qtype, k, 2)
    if out is None:
        out = torch.empty(m, n, dtype=torch.float32, device=x.device)
    _need(out, "out", 4, m * n)
    _need_cuda(x, w, out)
    _check(lib().kq_qmv(qtype, _ptr(w), n, k, _ptr(x), m, _ptr(out), _stream(stream)), "kq_qmv")
    return out


def qmm(x: torch.Tensor, w: torch.Tensor, qtype: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ dequant(w[N, :]).T on the tcgen05 tensor cores."""
    x = _bf16_bits(x)
    m, k = x.shape
    n = w.shape[0]
    _need_bank(w, "w", qtype, k, 2)
    if out is None:
        out = torch.empty(m, n, dtype=torch.float32, device=x.device)
    _need(out, "out", 4, m * n)
    _need_cuda(x, w, out)
    _check(lib().kq_qmm(qtype, _ptr(w), n, k, _ptr(x), m, _ptr(out), _stream(stream)), "kq_qmm")
    return out


def map_capacity(rows: int, n_experts: int) -> int:
    return -(-rows // TILE_ROWS) + n_experts


def moe_sort(topk_ids: torch.Tensor, n_experts: int, x: torch.Tensor | None = None, err: torch.Tensor | None = None,
             stream=None, with_inverse: bool = False):
    """Stable sort of routed pairs by expert: (sorted_ids, sorted_pair, x_sorted),
    plus inv_order (the sorted row of every pair) when with_inverse is set."""
    t, top_k = topk_ids.shape
    rows = t * top_k
    _need(topk_ids, "topk_ids", 4)
    _need(err, "err", 4, 1)
    dev = topk_ids.device
    sids = torch.empty(rows, dtype=torch.int32, device=dev)
    pair = torch.empty(rows, dtype=torch.int32, device=dev)
    inv = torch.empty(rows, dtype=torch.int32, device=dev) if with_inverse else None
    xs = None
    k = 0
    if x is not None:
        x = _bf16_bits(x)
        k = x.shape[1]
        _need(x, "x", 2, t * k)
        xs = torch.empty(rows, k, dtype=x.dtype, device=dev)
    _need_cuda(topk_ids, x, xs, err)
    _check(lib().kq_moe_sort(_ptr(topk_ids), t, top_k, n_experts, _ptr(x), k, _ptr(sids), _ptr(pair), _ptr(inv),
                             _ptr(xs), _ptr(err), _stream(stream)), "kq_moe_sort")
    return (sids, pair, xs, inv) if with_inverse else (sids, pair, xs)


def expert_tile_map(sorted_ids: torch.Tensor, n_experts: int, cap: int | None = None,
                    err: torch.Tensor | None = None, stream=None):
    """(map int32 [cap, 3] of (expert, row_start, num_rows), count int32 [1])."""
    rows = sorted_ids.numel()
    cap = map_capacity(rows, n_experts) if cap is None else cap
    _need(sorted_ids, "sorted_ids", 4)
    _need(err, "err", 4, 1)
    m = torch.empty(cap, 3, dtype=torch.int32, device=sorted_ids.device)
    c = torch.empty(1, dtype=torch.int32, device=sorted_ids.device)
    _need_cuda(sorted_ids, err)
    _check(lib().kq_expert_tile_map(_ptr(sorted_ids), rows, n_experts, _ptr(m), cap, _ptr(c), _ptr(err),
                                    _stream(stream)), "kq_expert_tile_map")
    return m, c


def gather_qmm(x_sorted: torch.Tensor, w_bank: torch.Tensor, qtype: int, tile_map: torch.Tensor,
               count: torch.Tensor, out: torch.Tensor | None = None, err: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y[r] = x_sorted[r] @ dequant(w_bank[e(r)]).T for every row covered by a tile."""
    x_sorted = _bf16_bits(x_sorted)
    rows, k = x_sorted.shape
    e, n = w_bank.shape[0], w_bank.shape[1]
    _need_bank(w_bank, "w_bank", qtype, k, 3)
    _need(tile_map, "tile_map", 4)
    if tile_map.dim() != 2 or tile_map.shape[1] != 3:
        raise ValueError(f"tile_map: [cap, 3] expected, got {tuple(tile_map.shape)}")
    _need(count, "count", 4, 1)
    _need(err, "err", 4, 1)
    if out is None:
        out = torch.empty(rows, n, dtype=torch.float32, device=x_sorted.device)
    _need(out, "out", 4, rows * n)
    _need_cuda(x_sorted, w_bank, tile_map, count, out, err)
    _check(lib().kq_gather_qmm(qtype, _ptr(w_bank), e, n, k, _ptr(x_sorted), rows, _ptr(tile_map), _ptr(count),
                               tile_map.shape[0], _ptr(out), _ptr(err), _stream(stream)), "kq_gather_qmm")
    return out


def gather_qmv(x: torch.Tensor, w_bank: torch.Tensor, qtype: int, ids: torch.Tensor, x_per_token: bool = False,
               out: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode MoE product, one row per (token, slot) pair p = t * top_k + s:
    y[p] = x[p] @ dequant(w_bank[ids[t, s]]).T (x [T*top_k, K]), or
    x[t] @ ... with x_per_token (x [T, K]).  ids int32 [T, top_k]."""
    x = _bf16_bits(x)
    t, top_k = ids.shape
    k = x.shape[-1]
    e, n = w_bank.shape[0], w_bank.shape[1]
    _need_bank(w_bank, "w_bank", qtype, k, 3)
    _need(ids, "ids", 4)
    _need(err, "err", 4, 1)
    _need(x, "x", 2, (t if x_per_token else t * top_k) * k)
    if out is None:
        out = torch.empty(t * top_k, n, dtype=torch.float32, device=x.device)
    _need(out, "out", 4, t * top_k * n)
    _need_cuda(x, w_bank, ids, out, err)
    _check(lib().kq_gather_qmv(qtype, _ptr(w_bank), e, n, k, _ptr(x), int(bool(x_per_token)), _ptr(ids), t, top_k,
                               _ptr(out), _ptr(err), _stream(stream)), "kq_gather_qmv")
    return out


def gather_mix(y: torch.Tensor, inv_order: torch.Tensor, scores: torch.Tensor, out: torch.Tensor | None = None,
               err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum_s scores[t, s] * y[inv_order[t * top_k + s]] (fp32, slots in order)."""
    rows, n = y.shape
    t, top_k = scores.shape
    _need(y, "y", 4)
    _need(inv_order, "inv_order", 4, t * top_k)
    _need(scores, "scores", 4)
    _need(err, "err", 4, 1)
    if out is None:
        out = torch.empty(t, n, dtype=torch.float32, device=y.device)
    _need(out, "out", 4, t * n)
    _need_cuda(y, inv_order, scores, out, err)
    _check(lib().kq_gather_mix(_ptr(y), rows, n, _ptr(inv_order), _ptr(scores), t, top_k, _ptr(out), _ptr(err),
                               _stream(stream)), "kq_gather_mix")
    return out


def moe_glu_gather(x: torch.Tensor, gate_bank: torch.Tensor, up_bank: torch.Tensor, qtype: int, ids: torch.Tensor,
                   act: int = ACT_SILU, limit: float = 0.0, out: torch.Tensor | None = None,
                   err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t * top_k + s] = act(x[t] @ dequant(gate[e]).T, x[t] @ dequant(up[e]).T), e = ids[t, s]."""
    x = _bf16_bits(x)
    t, top_k = ids.shape
    k = x.shape[-1]
    e, n = gate_bank.shape[0], gate_bank.shape[1]
    _need_bank(gate_bank, "gate_bank", qtype, k, 3)
    _need_bank(up_bank, "up_bank", qtype, k, 3)
    if up_bank.shape != gate_bank.shape:
        raise ValueError(f"up_bank: shape {tuple(gate_bank.shape)} expected, got {tuple(up_bank.shape)}")
    _need(ids, "ids", 4)
    _need(err, "err", 4, 1)
    _need(x, "x", 2, t * k)
    if out is None:
        out = torch.empty(t * top_k, n, dtype=torch.float32, device=x.device)
    _need(out, "out", 4, t * top_k * n)
    _need_cuda(x, gate_bank, up_bank, ids, out, err)
    _check(lib().kq_moe_glu_gather(qtype, _ptr(gate_bank), _ptr(up_bank), e, n, k, _ptr(x), _ptr(ids), t, top_k,
                                   act, limit, _ptr(out), _ptr(err), _stream(stream)), "kq_moe_glu_gather")
    return out


# --------------------------------------------------- KV cache in q4_0 pages
# A pool is uint8 [n_pages, n_kv_heads, page_size, row_bytes(Q4_0, head_dim)],
# one for keys and one for values; a slot is page * page_size + offset.


def _place(*ts) -> int:
    """Index of the CUDA device that holds all of the tensors (None: absent),
    which are contiguous."""
    dev = None
    for t in ts:
        if t is not None:
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
            d = t.get_device()
            if dev is None:
                dev = d
            elif d != dev:
                raise ValueError("all tensors must be on one device")
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    return dev


def _call(dev: int, stream, what: str, *args) -> None:
    """The library call ``what`` on device ``dev`` and its current stream (or ``stream``)."""
    f = getattr(lib(), what)
    if dev == torch.cuda.current_device():
        rc = f(*args, _stream(stream))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _stream(stream))
    if rc:
        raise KQError(rc, what)


def _scratch(like: torch.Tensor, stream, size, dtype=torch.int32) -> torch.Tensor:
    """Memory on the device of ``like``, of the stream that the call runs on (the
    caching allocator gives freed memory to later work of the stream it was
    allocated on only)."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=like.device)


def _need_pools(k_pool: torch.Tensor, v_pool: torch.Tensor, qtype: int, heads: int | None, dim: int) -> torch.Size:
    """Shape of the two pools (heads None: whatever the pools have)."""
    shape = k_pool.shape
    if (qtype == Q4_0 and len(shape) == 4 and shape[3] * 16 == dim * 9 and (heads is None or shape[1] == heads)
            and v_pool.shape == shape and k_pool.dtype is torch.uint8 and v_pool.dtype is torch.uint8):
        return shape
    if heads is None:
        heads = shape[1] if len(shape) == 4 else 0
    _need_pool(k_pool, "k_pool", qtype, heads, dim)
    _need_pool(v_pool, "v_pool", qtype, heads, dim)
    if v_pool.shape != shape:
        raise ValueError(f"v_pool: shape {tuple(shape)} expected, got {tuple(v_pool.shape)}")
    return shape


def _need_pool(pool: torch.Tensor, what: str, qtype: int, heads: int, dim: int) -> None:
    _need(pool, what, 1)
    if pool.dim() != 4 or pool.shape[1] != heads:
        raise ValueError(f"{what}: [pages, {heads}, page_size, row_bytes] expected, got {tuple(pool.shape)}")
    if _whole_blocks(qtype, dim) and pool.shape[3] != row_bytes(qtype, dim):
        raise ValueError(f"{what}: rows of {row_bytes(qtype, dim)} bytes expected for head_dim = {dim}, got {pool.shape[3]}")


def _token_rows(x: torch.Tensor, what: str) -> int:
    """Elements between the tokens of x [tokens, heads, head_dim], whose heads
    and values are packed (a slice of a fused product's columns is such a view)."""
    if x.dim() != 3:
        raise ValueError(f"{what}: [tokens, heads, head_dim] expected, got {tuple(x.shape)}")
    t, h, d = x.shape
    st, sh, sd = x.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{what}: heads and values of a token must be contiguous")
    return st if t > 1 else h * d


def kv_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
            taken: torch.Tensor, page_size: int, cap: int, taken_out: torch.Tensor | None = None,
            err: torch.Tensor | None = None, stream=None):
    """Plan of a step from the requests' lengths (all int32, on the device):
    (seq_lens [B], cu_new [B + 1], slot_map [cap], positions [cap]).  Takes the
    pages that the new tokens need from free_pages (from place taken[0] on),
    writes them into block_table [B, max_blocks] and the new count to taken_out
    (default: taken itself).  Slots and positions behind the last token are -1.
    What does not fit gets slot -1 and sets DEV_TOO_MANY in err."""
    n = cached_lens.numel()
    table = block_table.shape
    if len(table) != 2 or table[0] != n:
        raise ValueError(f"block_table: [{n}, max_blocks] expected, got {tuple(table)}")
    if taken_out is None:
        taken_out = taken
    i32 = torch.int32
    if not (cached_lens.dtype is i32 and new_lens.dtype is i32 and block_table.dtype is i32 and free_pages.dtype is i32
            and taken.dtype is i32 and taken_out.dtype is i32 and new_lens.numel() >= n and taken.numel() and taken_out.numel()
            and err is None):
        for t, what, count in ((cached_lens, "cached_lens", n), (new_lens, "new_lens", n), (block_table, "block_table", None),
                               (free_pages, "free_pages", None), (taken, "taken", 1), (taken_out, "taken_out", 1), (err, "err", 1)):
            _need(t, what, 4, count)
    dev = _place(cached_lens, new_lens, block_table, free_pages, taken, taken_out, err)
    cap = int(cap)
    if cap < 0:
        raise ValueError(f"cap must not be negative, got {cap}")
    buf = _scratch(cached_lens, stream, 3 * n + 1 + 2 * cap)
    seq, cu, slots, pos, _ = buf.split([n, n + 1, cap, cap, n])
    at = buf.data_ptr()
    _call(dev, stream, "kq_kv_plan", cached_lens.data_ptr(), new_lens.data_ptr(), n, page_size, block_table.data_ptr(),
          table[1], free_pages.data_ptr(), free_pages.numel(), taken.data_ptr(), taken_out.data_ptr(),
          at, at + 4 * n, at + 4 * (2 * n + 1 + 2 * cap), at + 4 * (2 * n + 1), at + 4 * (2 * n + 1 + cap), cap, _ptr(err))
    return seq, cu, slots, pos


_PLAIN = {torch.float32: 0, torch.bfloat16: 30}  # ggml type ids of plain values


def kv_append(k: torch.Tensor, v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, qtype: int,
              slot_map: torch.Tensor, err: torch.Tensor | None = None, stream=None) -> None:
    """Encode k, v [tokens, kv_heads, head_dim] (float32 or bfloat16; views of a
    fused product's columns are fine) into the pools' slots; slot -1: left out.
    A slot named by several tokens holds a mixture of their bytes."""
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError(f"k and v must have one shape and type, got {tuple(k.shape)} {k.dtype}, {tuple(v.shape)} {v.dtype}")
    kind = _PLAIN.get(k.dtype)
    if kind is None:
        raise TypeError("keys and values must be float32 or bfloat16")
    ks, vs = _token_rows(k, "k"), _token_rows(v, "v")
    t, h, d = k.shape
    pool = _need_pools(k_pool, v_pool, qtype, h, d)
    _need(slot_map, "slot_map", 4, t)
    _need(err, "err", 4, 1)
    dev = _place(k_pool, v_pool, slot_map, err)
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    _call(dev, stream, "kq_kv_append", qtype, k.data_ptr(), v.data_ptr(), kind, t, ks, vs, h, d, slot_map.data_ptr(),
          k_pool.data_ptr(), v_pool.data_ptr(), pool[0], pool[2], _ptr(err))


def kv_attention_workspace(n_heads: int, n_kv_heads: int, head_dim: int, max_new: int) -> int:
    """Bytes of work space that kv_attention needs on the current device."""
    b = _i64()
    _check(lib().kq_kv_attention_workspace(n_heads, n_kv_heads, head_dim, max_new, ctypes.byref(b)),
           "kq_kv_attention_workspace")
    return b.value


@functools.lru_cache(maxsize=256)
def _workspace_bytes(dev: int, n_heads: int, n_kv_heads: int, head_dim: int, max_new: int) -> int:
    with torch.cuda.device(dev):
        return kv_attention_workspace(n_heads, n_kv_heads, head_dim, max_new)


def kv_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, qtype: int, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int, scale: float | None = None,
                 causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the new tokens q [tokens, heads, head_dim] (bfloat16) over the
    cached keys and values of their sequences, bfloat16 of q's shape.  seq_lens,
    cu_new as kv_plan gives them; max_new: the largest number of new tokens of a
    sequence; scale defaults to head_dim ** -0.5; window 0: no window.  A token
    that sees no key gets zeros; rows of no sequence are left as they are.  A
    sequence longer than its table row keeps its positions, what is past the row
    is hidden and err gets DEV_TOO_MANY.  A block scale past 8188 or not finite
    makes the rows that see it NaN."""
    q = _bf16_bits(q)
    qs = _token_rows(q, "q")
    t, hq, d = q.shape
    pages, h, page_size, _ = _need_pools(k_pool, v_pool, qtype, None, d)
    n = seq_lens.numel()
    table = block_table.shape
    if len(table) != 2 or table[0] != n:
        raise ValueError(f"block_table: [{n}, max_blocks] expected, got {tuple(table)}")
    i32 = torch.int32
    if not (block_table.dtype is i32 and seq_lens.dtype is i32 and cu_new.dtype is i32 and cu_new.numel() > n and err is None):
        _need(block_table, "block_table", 4)
        _need(seq_lens, "seq_lens", 4)
        _need(cu_new, "cu_new", 4, n + 1)
        _need(err, "err", 4, 1)
    if out is not None:
        _need(out, "out", 2, t * hq * d)
    dev = _place(k_pool, v_pool, block_table, seq_lens, cu_new, out, workspace, err)
    if q.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    if out is None:
        out = _scratch(q, stream, (t, hq, d), q.dtype)
    if workspace is None:
        workspace = _scratch(k_pool, stream, _workspace_bytes(dev, hq, h, d, max(1, max_new)), torch.uint8)
    _call(dev, stream, "kq_kv_attention", qtype, q.data_ptr(), t, qs, hq, h, d, cu_new.data_ptr(), seq_lens.data_ptr(), n,
          max_new, k_pool.data_ptr(), v_pool.data_ptr(), pages, page_size, block_table.data_ptr(), table[1],
          d ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), _ptr(err))
    return out
