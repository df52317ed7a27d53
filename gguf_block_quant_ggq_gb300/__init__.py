"""Python binding of libggq: keep-quant GEMV and MoE routed-expert GEMM over
GGUF block-quantized weights on one GB300 (sm_103a).

Argument marshalling only.  Every step of every call runs in the CUDA kernels
of ``libggq.so`` (built in-tree by ``_build.build()``); there is no CPU path.
Loading fails loudly when the library is missing.  Functions keep the C names
of ``include/ggq.h`` and take device pointers as Python ints; ``Context`` wraps
them for torch tensors (torch supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libggq.so")

TYPE = {"Q4_0": 2, "Q8_0": 8, "Q8_1": 9, "Q2_K": 10, "Q3_K": 11, "Q4_K": 12, "Q5_K": 13, "Q6_K": 14, "Q8_K": 15,
        "MXFP4": 39}
OP = {"quantize_act": 0, "dequant": 1, "mul_mat_vec": 2, "moe": 3, "kv_cache": 4}
DTYPE = {"float32": 0, "float16": 1, "bfloat16": 30}  # ggq_dtype of activations
SCORING = {"softmax": 0, "sigmoid": 1}
STATUS = {0: "GGQ_OK", 1: "GGQ_ERR_INVALID_ARG", 2: "GGQ_ERR_SHAPE", 3: "GGQ_ERR_UNSUPPORTED", 4: "GGQ_ERR_ARCH",
          5: "GGQ_ERR_CUDA", 6: "GGQ_ERR_CAPACITY", 7: "GGQ_ERR_CAPTURE_ALLOC", 8: "GGQ_ERR_DEVICE"}
BLOCK_ELEMS = {"Q4_0": 32, "Q8_0": 32, "MXFP4": 32, "Q8_1": 32, "Q4_K": 256, "Q5_K": 256, "Q6_K": 256, "Q8_K": 256,
               "Q2_K": 256, "Q3_K": 256}
BLOCK_BYTES = {"Q4_0": 18, "Q8_0": 34, "MXFP4": 17, "Q8_1": 36, "Q4_K": 144, "Q5_K": 176, "Q6_K": 210, "Q8_K": 292,
               "Q2_K": 84, "Q3_K": 110}

# Every entry point the header declares, with its ctypes signature.
_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "ggq_create": (_I32, [ctypes.POINTER(ctypes.c_void_p), _I32]),
    "ggq_destroy": (_I32, [_P]),
    "ggq_last_error": (ctypes.c_char_p, [_P]),
    "ggq_reserve": (_I32, [_P, _P, _P]),
    "ggq_scratch_bytes": (ctypes.c_size_t, [_P]),
    "ggq_set_static_weights": (_I32, [_P, _I32]),
    "ggq_set_direct_route_max_tokens": (_I32, [_P, _I32]),
    "ggq_supported": (_I32, [_I32, _I32, _I32]),
    "ggq_quantize_act": (_I32, [_P, _I32, _P, _I64, _I64, _P, _P]),
    "ggq_dequant": (_I32, [_P, _I32, _P, _I64, _I64, _P, _P]),
    "ggq_mul_mat_vec": (_I32, [_P, _I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "ggq_mul_mat_vec_q": (_I32, [_P, _I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "ggq_block_dots": (_I32, [_P, _I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "ggq_moe_experts": (_I32, [_P, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _P, _P]),
    "ggq_moe_experts_routed": (_I32, [_P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _I64, _P, _P, _P]),
    "ggq_sync_status": (_I32, [_P, _P]),
    "ggq_mul_mat_vec_noalloc": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "ggq_set_moe_counters": (_I32, [_P, _P, _I64, _P]),
    "ggq_moe_experts_q": (_I32, [_P, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _P, _P]),
    "ggq_mul_mat_vec_qa": (_I32, [_P, _I32, _I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "ggq_kv_page_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, _I32]),
    "ggq_kv_store": (_I32, [_P, _P, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P]),
    "ggq_kv_load": (_I32, [_P, _P, _I32, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P]),
    "ggq_attention": (_I32, [_P, _P, _P, _P]),
    "ggq_reserve_attention": (_I32, [_P, _P]),
    "ggq_moe_route": (_I32, [_P, _P, _I32, _P, _I64, _I64, _P, _P, _P]),
    "ggq_block_dots_qa": (_I32, [_P, _I32, _I32, _P, _I64, _I64, _P, _I64, _P, _P]),
}


class ggq_plan(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int64), ("max_k", ctypes.c_int64), ("n_experts", ctypes.c_int64),
                ("hidden", ctypes.c_int64), ("inter", ctypes.c_int64), ("top_k", ctypes.c_int64)]


class ggq_moe_weights(ctypes.Structure):
    _fields_ = [("gate_type", ctypes.c_int32), ("up_type", ctypes.c_int32), ("down_type", ctypes.c_int32),
                ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class ggq_moe_dump(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("ids", "weights", "xq", "g", "u", "h", "hq", "o", "coefs_gate",
                                               "coefs_up", "coefs_down")]


class ggq_kv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("k_type", "v_type", "n_kv_heads", "head_dim", "page_size")] + [
        ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class ggq_attn(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_tokens", ctypes.c_int64),
                ("n_seqs", ctypes.c_int64), ("q", ctypes.c_void_p), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_token", ctypes.c_int64),
                ("out_head", ctypes.c_int64), ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("max_q", ctypes.c_int64),
                ("max_len", ctypes.c_int64), ("scale", ctypes.c_float), ("cap", ctypes.c_float),
                ("window", ctypes.c_int64), ("slopes", ctypes.c_void_p)]


class ggq_router(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("scoring", "n_groups", "top_groups", "group_best", "top_k",
                                              "normalize")] + [("scale", ctypes.c_float), ("bias", ctypes.c_void_p)]


# ggq_attn and ggq_router as packed fields: filled in place for every call
_ATTN = struct.Struct("@iiqqPqqPqqPqPPqqffqP")
_ROUTER = struct.Struct("@iiiiiifP")
assert _ATTN.size == ctypes.sizeof(ggq_attn) and _ROUTER.size == ctypes.sizeof(ggq_router)


class GGQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libggq.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libggq is not built ({path} missing): run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _bind(name):
    def call(*args):
        return getattr(load(), name)(*args)
    call.__name__ = name
    return call


for _name in SIGNATURES:
    globals()[_name] = _bind(_name)


def row_bytes(fmt: str, K: int) -> int:
    return K // BLOCK_ELEMS[fmt] * BLOCK_BYTES[fmt]


def act_type(wfmt: str) -> str:
    return "Q8_1" if wfmt == "Q4_0" else "Q8_K"


def _ptr(t, dtype: str | None = None):
    """Device address of a torch CUDA tensor (None passes NULL).  The C calls
    read and write dense rows from that address, so the tensor must be on a
    CUDA device and contiguous; `dtype` (a torch dtype name) is checked where
    the call has a fixed element type.  Packed weight blocks may have any dtype."""
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"libggq takes CUDA tensors (device memory), got one on {getattr(t, 'device', type(t))}")
    if not t.is_contiguous():
        raise ValueError("libggq reads and writes dense rows: pass a contiguous tensor")
    if dtype is not None and str(t.dtype) != "torch." + dtype:
        raise ValueError(f"expected a {dtype} tensor, got {t.dtype}")
    return t.data_ptr()


class KVCache:
    """A paged key/value cache in Q8_0 or Q4_0 blocks: two uint8 pools on the
    context's device (given, or made here), and the C structure that names them."""

    def __init__(self, ctx, k_type, v_type, n_pages, page_size, n_kv_heads, head_dim, k=None, v=None):
        torch = ctx._torch
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = n_pages, page_size, n_kv_heads, head_dim
        pools = []
        for fmt, pool in ((k_type, k), (v_type, v)):
            size = load().ggq_kv_page_bytes(TYPE[fmt], n_kv_heads, head_dim, page_size)
            if not size:
                raise ValueError(f"a cache of {fmt} blocks with {n_kv_heads} heads of {head_dim} channels and pages of "
                                 f"{page_size} tokens is not supported: Q8_0 or Q4_0, head_dim 64, 128 or 256, pages of "
                                 "a multiple of 16 tokens")
            if pool is None:
                pool = torch.zeros(n_pages * size, dtype=torch.uint8, device=f"cuda:{ctx.device}")
            _ptr(pool, "uint8")
            if pool.get_device() != ctx.device:
                raise ValueError(f"expected a pool on cuda:{ctx.device}, got one on {pool.device}")
            if pool.numel() != n_pages * size:
                raise ValueError(f"{n_pages} pages of {size} bytes need a pool of {n_pages * size}, got {pool.numel()}")
            pools.append(pool)
        self.k, self.v = pools
        self.device = ctx.device
        self.struct = ggq_kv_cache(TYPE[k_type], TYPE[v_type], n_kv_heads, head_dim, page_size, n_pages,
                                   pools[0].data_ptr(), pools[1].data_ptr())
        self.ref = ctypes.addressof(self.struct)


class Context:
    """A libggq context on one CUDA device; methods take torch CUDA tensors and
    enqueue on torch's current stream (or the given one)."""

    def __init__(self, device: int = 0):
        import torch  # device memory and streams only

        self._torch = torch
        self.device = device
        self._dev = torch.device("cuda", device)
        self._f32, self._i32, self._i64 = torch.float32, torch.int32, torch.int64
        self._codes = {getattr(torch, k): v for k, v in DTYPE.items()}
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._attn_args = ctypes.create_string_buffer(_ATTN.size)
        self._router_args = ctypes.create_string_buffer(_ROUTER.size)
        self._attn_at, self._router_at = ctypes.addressof(self._attn_args), ctypes.addressof(self._router_args)
        self._attn_ready = False
        h = ctypes.c_void_p()
        st = load().ggq_create(ctypes.byref(h), device)
        if st != 0:
            raise GGQError(st, f"ggq_create(device={device}) failed")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            load().ggq_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self, stream):
        if stream is None:
            if self._raw_stream is not None:
                return self._raw_stream(self.device)
            stream = self._torch.cuda.current_stream(self.device)
        return stream.cuda_stream

    def _empty(self, shape, dtype, stream):
        """A new tensor on the context's device, of the memory of the stream that will write it: a block freed on
        another stream may still be in use there."""
        if stream is None:
            return self._torch.empty(shape, dtype=dtype, device=self._dev)
        with self._torch.cuda.stream(stream):
            return self._torch.empty(shape, dtype=dtype, device=self._dev)

    def _vec(self, t, dtype):
        """Address of a contiguous tensor of `dtype` on the context's device (None passes NULL)."""
        if t is None:
            return 0
        if t.dtype is dtype and t.get_device() == self.device and t.is_contiguous():
            return t.data_ptr()
        _ptr(t, str(dtype)[6:])
        raise ValueError(f"expected a tensor on cuda:{self.device}, got one on {t.device}")

    def _rows(self, t, heads, dim):
        """(address, ggq_dtype, token stride, head stride) of a [tokens][heads][dim] tensor on the
        context's device whose last axis is dense; the other strides are free."""
        code = self._codes.get(t.dtype)
        if code is None:
            raise ValueError(f"expected a float32, float16 or bfloat16 tensor, got {t.dtype}")
        if t.get_device() != self.device:
            raise ValueError(f"libggq takes CUDA tensors on cuda:{self.device} (device memory), got one on {t.device}")
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
            raise ValueError(f"expected a [tokens, {heads}, {dim}] tensor, got {tuple(shape)}")
        token, head, one = t.stride()
        if one != 1:
            raise ValueError("the channels of a head have to be dense")
        return t.data_ptr(), code, token, head

    def _own(self, cache):
        if cache.device != self.device:
            raise ValueError(f"the cache lies on cuda:{cache.device}, this context works on cuda:{self.device}")

    def _check(self, st):
        if st != 0:
            raise GGQError(st, load().ggq_last_error(self.handle).decode())

    def reserve(self, max_tokens=0, max_k=0, n_experts=0, hidden=0, inter=0, top_k=0, stream=None):
        plan = ggq_plan(max_tokens, max_k, n_experts, hidden, inter, top_k)
        self._check(load().ggq_reserve(self.handle, ctypes.byref(plan), self._stream(stream)))

    def set_static_weights(self, on: bool = True):
        self._check(load().ggq_set_static_weights(self.handle, 1 if on else 0))

    def set_direct_route_max_tokens(self, max_tokens: int = 32):
        self._check(load().ggq_set_direct_route_max_tokens(self.handle, int(max_tokens)))

    def scratch_bytes(self) -> int:
        return load().ggq_scratch_bytes(self.handle)

    def set_moe_counters(self, pairs=None, calls=None):
        """Expert-load telemetry: int64 CUDA tensors pairs [E] and calls [2], or None to stop."""
        n = 0 if pairs is None else pairs.numel()
        self._check(load().ggq_set_moe_counters(self.handle, _ptr(pairs, "int64"), n, _ptr(calls, "int64")))

    def sync_status(self, stream=None):
        self._check(load().ggq_sync_status(self.handle, self._stream(stream)))

    def quantize_act(self, act: str, x, out=None, stream=None):
        T, K = x.shape
        if out is None:
            out = self._empty((T, row_bytes(act, K)), self._torch.uint8, stream)
        self._check(load().ggq_quantize_act(self.handle, TYPE[act], _ptr(x, "float32"), T, K, _ptr(out, "uint8"),
                                            self._stream(stream)))
        return out

    def dequant(self, fmt: str, blocks, rows: int, K: int, out=None, stream=None):
        if out is None:
            out = self._empty((rows, K), self._torch.float32, stream)
        self._check(load().ggq_dequant(self.handle, TYPE[fmt], _ptr(blocks), rows, K, _ptr(out, "float32"),
                                       self._stream(stream)))
        return out

    def mul_mat_vec(self, fmt: str, W, N: int, K: int, X, Y=None, stream=None, reserve=True):
        T = X.shape[0]
        if Y is None:
            Y = self._empty((T, N), self._torch.float32, stream)
        if reserve:
            self.reserve(max_tokens=T, max_k=K, stream=stream)
        self._check(load().ggq_mul_mat_vec(self.handle, TYPE[fmt], _ptr(W), N, K, _ptr(X, "float32"), T,
                                           _ptr(Y, "float32"), self._stream(stream)))
        return Y

    def mul_mat_vec_q(self, fmt: str, W, N: int, K: int, Xq, T: int, Y=None, stream=None):
        if Y is None:
            Y = self._empty((T, N), self._torch.float32, stream)
        self._check(load().ggq_mul_mat_vec_q(self.handle, TYPE[fmt], _ptr(W), N, K, _ptr(Xq), T, _ptr(Y, "float32"),
                                             self._stream(stream)))
        return Y

    def mul_mat_vec_qa(self, fmt: str, act: str, W, N: int, K: int, Xq, T: int, Y=None, stream=None):
        if Y is None:
            Y = self._empty((T, N), self._torch.float32, stream)
        self._check(load().ggq_mul_mat_vec_qa(self.handle, TYPE[fmt], TYPE[act], _ptr(W), N, K, _ptr(Xq), T,
                                              _ptr(Y, "float32"), self._stream(stream)))
        return Y

    def block_dots_qa(self, fmt: str, act: str, W, N: int, K: int, Xq, T: int, stream=None):
        nc = K // BLOCK_ELEMS[fmt] * (2 if fmt in ("Q4_K", "Q5_K", "Q2_K") else 1)
        out = self._empty((T, N, nc), self._torch.int32, stream)
        self._check(load().ggq_block_dots_qa(self.handle, TYPE[fmt], TYPE[act], _ptr(W), N, K, _ptr(Xq), T,
                                             _ptr(out), self._stream(stream)))
        return out

    def block_dots(self, fmt: str, W, N: int, K: int, Xq, T: int, stream=None):
        nc = K // BLOCK_ELEMS[fmt] * (2 if fmt in ("Q4_K", "Q5_K", "Q2_K") else 1)
        out = self._empty((T, N, nc), self._torch.int32, stream)
        self._check(load().ggq_block_dots(self.handle, TYPE[fmt], _ptr(W), N, K, _ptr(Xq), T, _ptr(out),
                                          self._stream(stream)))
        return out

    def kv_cache(self, k_type: str, v_type: str, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 k=None, v=None) -> KVCache:
        """A paged cache of Q8_0 or Q4_0 blocks (zeroed pools are made where none are given)."""
        return KVCache(self, k_type, v_type, n_pages, page_size, n_kv_heads, head_dim, k, v)

    def kv_store(self, cache: KVCache, k, v, slots, stream=None):
        """Quantize k and v [tokens][kv heads][D] into the cache's slots (int64 [tokens], negative: skipped)."""
        self._own(cache)
        kp, code, kt, kh = self._rows(k, cache.n_kv_heads, cache.head_dim)
        vp, vcode, vt, vh = self._rows(v, cache.n_kv_heads, cache.head_dim)
        n = slots.numel()
        if code != vcode or k.shape[0] != n or v.shape[0] != n:
            raise ValueError("k, v and slots have to agree in type and tokens")
        st = _lib.ggq_kv_store(self.handle, cache.ref, code, kp, kt, kh, vp, vt, vh, self._vec(slots, self._i64), n,
                               self._stream(stream))
        if st:
            self._check(st)

    def kv_load(self, cache: KVCache, slots, dtype=None, k=None, v=None, stream=None):
        """Values of the cache's slots, [tokens][kv heads][D] each of K and V (float32 unless dtype or a given
        buffer says otherwise)."""
        self._own(cache)
        n, heads, dim = slots.numel(), cache.n_kv_heads, cache.head_dim
        if dtype is None:
            dtype = k.dtype if k is not None else v.dtype if v is not None else self._f32
        if k is None:
            k = self._empty((n, heads, dim), dtype, stream)
        if v is None:
            v = self._empty((n, heads, dim), dtype, stream)
        kp, code, kt, kh = self._rows(k, heads, dim)
        vp, vcode, vt, vh = self._rows(v, heads, dim)
        if code != vcode or k.shape[0] != n or v.shape[0] != n:
            raise ValueError("k, v and slots have to agree in type and tokens")
        st = _lib.ggq_kv_load(self.handle, cache.ref, code, self._vec(slots, self._i64), n, kp, kt, kh, vp, vt, vh,
                              self._stream(stream))
        if st:
            self._check(st)
        return k, v

    def attention(self, cache: KVCache, q, lens, table, q_start=None, max_q=None, max_len=0, scale=None, cap=0.0,
                  window=0, slopes=None, out=None, stream=None, reserve=True):
        """Attention of q [tokens][heads][D] over the cache: lens int32 [sequences] (new tokens included), table
        int32 [sequences][pages], q_start int32 [sequences + 1] unless every sequence has one token; max_q and
        max_len bound a sequence's rows and length (default: all rows, the table's capacity)."""
        self._own(cache)
        if q.dim() != 3:
            raise ValueError(f"expected a [tokens, heads, {cache.head_dim}] tensor, got {tuple(q.shape)}")
        n, heads, dim = q.shape
        if out is None:
            out = self._empty((n, heads, dim), q.dtype, stream)
        qp, code, qt, qh = self._rows(q, heads, cache.head_dim)
        op, ocode, ot, oh = self._rows(out, heads, cache.head_dim)
        seqs = lens.numel()
        if ocode != code or out.shape[0] != n:
            raise ValueError("out has to have q's type and tokens")
        if table.dim() != 2 or table.shape[0] != seqs or (q_start is not None and q_start.numel() != seqs + 1):
            raise ValueError(f"{seqs} sequences need a table row each and {seqs + 1} row starts")
        if q_start is None and n != seqs:
            raise ValueError(f"{n} rows for {seqs} sequences: q_start is needed")
        if slopes is not None and slopes.numel() != heads:
            raise ValueError(f"expected {heads} slopes, got {slopes.numel()}")
        raw = self._stream(stream)
        if reserve and not self._attn_ready:
            self._check(_lib.ggq_reserve_attention(self.handle, raw))
            self._attn_ready = True
        _ATTN.pack_into(self._attn_args, 0, code, heads, n, seqs, qp, qt, qh, op, ot, oh, self._vec(table, self._i32),
                        table.shape[1], self._vec(lens, self._i32), self._vec(q_start, self._i32),
                        n if max_q is None else max_q, max_len, dim ** -0.5 if scale is None else scale, cap, window,
                        self._vec(slopes, self._f32))
        st = _lib.ggq_attention(self.handle, cache.ref, self._attn_at, raw)
        if st:
            self._check(st)
        return out

    def moe_route(self, logits, top_k: int, scoring: str = "softmax", bias=None, n_groups: int = 1,
                  top_groups: int = 1, group_best: int = 1, normalize: bool = True, scale: float = 1.0, ids=None,
                  weights=None, stream=None):
        """Expert ids [tokens][top_k] int32 and weights fp32 for moe_experts, of logits [tokens][experts]."""
        T, E = logits.shape
        code = self._codes.get(logits.dtype)
        if code is None:
            raise ValueError(f"expected float32, float16 or bfloat16 logits, got {logits.dtype}")
        if bias is not None and bias.numel() != E:
            raise ValueError(f"expected a bias of {E} experts, got {bias.numel()}")
        if ids is None:
            ids = self._empty((T, max(top_k, 0)), self._i32, stream)
        elif tuple(ids.shape) != (T, top_k):
            raise ValueError(f"expected a [{T}, {top_k}] output, got {tuple(ids.shape)}")
        if weights is None:
            weights = self._empty((T, max(top_k, 0)), self._f32, stream)
        elif tuple(weights.shape) != (T, top_k):
            raise ValueError(f"expected a [{T}, {top_k}] output, got {tuple(weights.shape)}")
        _ROUTER.pack_into(self._router_args, 0, SCORING[scoring], n_groups, top_groups, group_best, top_k,
                          1 if normalize else 0, scale, self._vec(bias, self._f32))
        st = _lib.ggq_moe_route(self.handle, self._router_at, code, self._vec(logits, logits.dtype), T, E,
                                self._vec(ids, self._i32), self._vec(weights, self._f32), self._stream(stream))
        if st:
            self._check(st)
        return ids, weights

    def moe_weights(self, gate_fmt, gate, up_fmt, up, down_fmt, down):
        return ggq_moe_weights(TYPE[gate_fmt], TYPE[up_fmt], TYPE[down_fmt], _ptr(gate), _ptr(up), _ptr(down))

    def moe_experts(self, weights: ggq_moe_weights, E, H, I, top_k, X, logits=None, ids=None, route_w=None,
                    Y=None, dump: dict | None = None, stream=None, reserve=True):
        T = X.shape[0]
        if Y is None:
            Y = self._empty((T, H), self._torch.float32, stream)
        if reserve:
            self.reserve(max_tokens=T, n_experts=E, hidden=H, inter=I, top_k=top_k, stream=stream)
        d = None
        if dump is not None:
            d = ggq_moe_dump(**{k: _ptr(v) for k, v in dump.items()})
        dp = ctypes.byref(d) if d is not None else None
        if logits is not None:
            st = load().ggq_moe_experts(self.handle, ctypes.byref(weights), E, H, I, top_k, _ptr(X, "float32"),
                                        _ptr(logits, "float32"), T, _ptr(Y, "float32"), dp, self._stream(stream))
        else:
            st = load().ggq_moe_experts_routed(self.handle, ctypes.byref(weights), E, H, I, top_k, _ptr(X, "float32"),
                                               _ptr(ids, "int32"), _ptr(route_w, "float32"), T, _ptr(Y, "float32"),
                                               dp, self._stream(stream))
        self._check(st)
        return Y


def _moe_q(ctx, weights, E, H, I, top_k, Xq, logits, Y=None, dump=None, stream=None, reserve=True):
    """ggq_moe_experts_q: the layer on pre-quantized Q8_K activations Xq [T][H/256*292] (uint8)."""
    T = Xq.shape[0]
    if Y is None:
        Y = ctx._empty((T, H), ctx._torch.float32, stream)
    if reserve:
        ctx.reserve(max_tokens=T, n_experts=E, hidden=H, inter=I, top_k=top_k, stream=stream)
    d = ggq_moe_dump(**{k: _ptr(v) for k, v in dump.items()}) if dump is not None else None
    ctx._check(load().ggq_moe_experts_q(ctx.handle, ctypes.byref(weights), E, H, I, top_k, _ptr(Xq, "uint8"),
                                        _ptr(logits, "float32"), T, _ptr(Y, "float32"),
                                        ctypes.byref(d) if d is not None else None, ctx._stream(stream)))
    return Y


Context.moe_experts_q = _moe_q


def supported(w: str, act: str, op: str) -> bool:
    return bool(load().ggq_supported(TYPE.get(w, -1), TYPE.get(act, -1), OP[op]))
