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
GATE_ACT = {"none": 0, "sigmoid": 1}
ROTARY_LAYOUT = {"half": 0, "pairs": 1}
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
    "ggq_norm": (_I32, [_P, _P, _P]),
    "ggq_rotary_table": (_I32, [_P, _P, _I64, _I64, _P, _P]),
    "ggq_rotate": (_I32, [_P, _P, _P, _P]),
    "ggq_kv_append": (_I32, [_P, _P, _P, _P, _P]),
    "ggq_adapt": (_I32, [_P, _P, _P, _P]),
    "ggq_logprobs": (_I32, [_P, _P, _P]),
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


class ggq_norm_args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("gate_act", ctypes.c_int32), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("x_token", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("residual_token", ctypes.c_int64), ("gate", ctypes.c_void_p), ("gate_token", ctypes.c_int64),
                ("gate_channel", ctypes.c_int64), ("total", ctypes.c_void_p), ("total_token", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_token", ctypes.c_int64), ("packed", ctypes.c_void_p),
                ("packed_type", ctypes.c_int32), ("norms", ctypes.c_int32), ("after", ctypes.c_void_p),
                ("before", ctypes.c_void_p), ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("offset", ctypes.c_float)]


class ggq_rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_positions", ctypes.c_int64), ("turn", ctypes.c_int32),
                ("first", ctypes.c_int32), ("layout", ctypes.c_int32)]


class ggq_rotate_args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("D", ctypes.c_int32), ("T", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("x_token", ctypes.c_int64), ("x_head", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64), ("positions", ctypes.c_void_p)]


class ggq_append_args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("T", ctypes.c_int64)] + [
        f for n in ("q", "q_out", "k", "v")
        for f in ((n, ctypes.c_void_p), (n + "_token", ctypes.c_int64), (n + "_head", ctypes.c_int64))] + [
        ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class ggq_rotary_spec(ctypes.Structure):
    _fields_ = [("turn", ctypes.c_int32), ("base", ctypes.c_double), ("factors", ctypes.c_void_p), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_int64), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


class ggq_adapters(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("max_rank", ctypes.c_int32), ("n", ctypes.c_int64), ("K", ctypes.c_int64),
                ("N", ctypes.c_int64), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class ggq_adapt_args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("T", ctypes.c_int64), ("n_seqs", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("x_token", ctypes.c_int64), ("y", ctypes.c_void_p), ("y_token", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_token", ctypes.c_int64), ("ids", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


class ggq_logprobs_args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("top_k", ctypes.c_int32), ("T", ctypes.c_int64), ("V", ctypes.c_int64),
                ("logits", ctypes.c_void_p), ("row", ctypes.c_int64), ("tokens", ctypes.c_void_p), ("given", ctypes.c_int64),
                ("logprobs", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("top", ctypes.c_void_p),
                ("scale", ctypes.c_float)]


# the calls' argument structures as packed fields: filled in place for every call
_ATTN = struct.Struct("@iiqqPqqPqqPqPPqqffqP")
_ROUTER = struct.Struct("@iiiiiifP")
_NORM = struct.Struct("@iiqqPqPqPqqPqPqPiiPPfff4x")
_ROTATE = struct.Struct("@Pqiii4xiiiqPqqPqqP")  # ggq_rotary, then ggq_rotate_args
_APPEND = struct.Struct("@Pqiii4xiiqPqqPqqPqqPqqPP")  # ggq_rotary, then ggq_append_args
_ADAPT = struct.Struct("@iqqPqPqPqPP")
_LOGPROBS = struct.Struct("@iiqqPqPqPPPPf4x")
assert _ATTN.size == ctypes.sizeof(ggq_attn) and _ROUTER.size == ctypes.sizeof(ggq_router)
_ARGS_AT = ctypes.sizeof(ggq_rotary)
assert _NORM.size == ctypes.sizeof(ggq_norm_args) and _ROTATE.size == _ARGS_AT + ctypes.sizeof(ggq_rotate_args)
assert _APPEND.size == _ARGS_AT + ctypes.sizeof(ggq_append_args)
assert _ADAPT.size == ctypes.sizeof(ggq_adapt_args) and _LOGPROBS.size == ctypes.sizeof(ggq_logprobs_args)


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


class Adapters:
    """Low-rank adapters of one projection: a [n][rank][K] and b [n][N][rank] of one 16-bit type on the context's
    device, ranks int32 [n] (default: all), scales float32 [n] (default: 1).  Ranks that are no multiple of 8 are
    laid out anew with the next one, once, on `stream` (default: torch's current one) and in its memory; the object is
    made when that is done, so that any stream may use it (inside a capture, the captured stream alone).  Other
    tensors are used as they are."""

    def __init__(self, ctx, a, b, ranks=None, scales=None, stream=None):
        torch = ctx._torch
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2] or a.dtype is not b.dtype:
            raise ValueError(f"expected banks [n, rank, K] and [n, N, rank] of one type, got {tuple(a.shape)} {a.dtype} and "
                             f"{tuple(b.shape)} {b.dtype}")
        if a.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"expected float16 or bfloat16 adapters, got {a.dtype}")
        n, rank, K = a.shape
        for t in (a, b):
            ctx._vec(t, t.dtype)
        if rank % 8:
            wide = (rank + 7) // 8 * 8
            if stream is None:
                stream = torch.cuda.current_stream(ctx._dev)
            with torch.cuda.stream(stream):
                na, nb = a.new_zeros((n, wide, K)), b.new_zeros((n, b.shape[1], wide))
                na[:, :rank], nb[:, :, :rank] = a, b
                a, b = na, nb
                if ranks is None:
                    ranks = torch.full((n,), rank, dtype=torch.int32, device=a.device)
                if not torch.cuda.is_current_stream_capturing():
                    stream.synchronize()
        for t, name in ((ranks, "ranks"), (scales, "scales")):
            if t is not None and t.numel() != n:
                raise ValueError(f"expected {n} {name}, got {t.numel()}")
        self.a, self.b, self.ranks, self.scales = a, b, ranks, scales
        self.K, self.N, self.device = K, b.shape[1], ctx.device
        self.struct = ggq_adapters(ctx._codes[a.dtype], a.shape[1], n, K, self.N, a.data_ptr(), b.data_ptr(),
                                   ctx._vec(ranks, ctx._i32), ctx._vec(scales, ctx._f32))
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
        self._step_args = ctypes.create_string_buffer(max(_NORM.size, _ROTATE.size, _APPEND.size, _ADAPT.size, _LOGPROBS.size))
        self._step_at = ctypes.addressof(self._step_args)
        self._step_more = self._step_at + _ARGS_AT
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

    def _mat(self, t, shape, dtype):
        """(address, row stride) of a tensor of a two-dimensional `shape` and `dtype` on the context's device whose rows are
        dense."""
        if t.dtype is not dtype or t.get_device() != self.device:
            raise ValueError(f"expected a {dtype} tensor on cuda:{self.device}, got {t.dtype} on {t.device}")
        if t.shape != shape:
            raise ValueError(f"expected a {list(shape)} tensor, got {tuple(t.shape)}")
        row, one = t.stride()
        if one != 1 and shape[1] > 1:
            raise ValueError("the channels of a row have to be dense")
        return t.data_ptr(), row

    def _code(self, dtype):
        code = self._codes.get(dtype)
        if code is None:
            raise ValueError(f"expected a float32, float16 or bfloat16 tensor, got {dtype}")
        return code

    def _own(self, cache, what="cache is"):
        if cache.device != self.device:
            raise ValueError(f"the {what} of cuda:{cache.device}, this context works on cuda:{self.device}")

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

    def norm(self, x, before=None, after=None, gate=None, gate_act: str = "none", scale: float = 1.0, residual=None,
             eps: float = 1e-6, offset: float = 0.0, act: str | None = None, out=None, total=None, packed=None, stream=None):
        """(out, total): total = residual + scale * act(gate) * norm(x; after), out = norm(total; before), of x [tokens][H].

        before, after: float32 weights [H] (offset is added to them), True for a norm without weights (nor offset), None
        for no norm.  gate: of x's type, [tokens][H], [H], or [tokens][1].  total is made where there is a residual, or
        nothing else to return; given buffers are always written.  act: out is packed Q8_K, Q8_1 or Q8_0 rows
        (uint8, into `packed` where given) that the products take; a given `out` then gets the float rows too."""
        if x.dim() != 2:
            raise ValueError(f"expected a [tokens, channels] tensor, got {tuple(x.shape)}")
        shape = x.shape
        n, H = shape
        dtype = x.dtype
        code = self._code(dtype)
        norms = (after is not None) + 2 * (before is not None)
        if before is None and (out is not None or act is not None):
            raise ValueError("out and packed rows are the norm of the total: `before` is needed")
        if packed is not None and act is None:
            raise ValueError("packed rows of which format? `act` is needed")
        if before is not None and out is None and act is None:
            out = self._empty((n, H), dtype, stream)
        if total is None and (residual is not None or before is None):
            total = self._empty((n, H), dtype, stream)
        pp = 0
        if act is not None:
            width = row_bytes(act, H)
            if packed is None:
                packed = self._empty((n, width), self._torch.uint8, stream)
            elif tuple(packed.shape) != (n, width):
                raise ValueError(f"expected a [{n}, {width}] output, got {tuple(packed.shape)}")
            pp = self._vec(packed, self._torch.uint8)
        xp, xt = self._mat(x, shape, dtype)
        rp, rt = self._mat(residual, shape, dtype) if residual is not None else (0, 0)
        tp, tt = self._mat(total, shape, dtype) if total is not None else (0, 0)
        op, ot = self._mat(out, shape, dtype) if out is not None else (0, 0)
        gp = gt = gc = 0
        if gate is not None:
            if gate.dim() == 1 and gate.shape[0] == H:
                gp, gc = self._vec(gate, dtype), 1
            elif gate.dim() == 2 and gate.shape[1] == 1 and H != 1:
                gp, gt = self._mat(gate, (n, 1), dtype)
            else:
                gp, gt = self._mat(gate, shape, dtype)
                gc = 1
        ap = bp = 0
        if after is not None and after is not True:
            ap = self._weights(after, H)
        if before is not None and before is not True:
            bp = self._weights(before, H)
        _NORM.pack_into(self._step_args, 0, code, GATE_ACT[gate_act], n, H, xp, xt, rp, rt, gp, gt, gc, tp, tt, op, ot, pp,
                        TYPE[act] if act else 0, norms, ap, bp, scale, eps, offset)
        st = _lib.ggq_norm(self.handle, self._step_at, self._stream(stream))
        if st:
            self._check(st)
        return (packed if act is not None else out), total

    def _weights(self, w, n):
        if w.numel() != n:
            raise ValueError(f"expected {n} weights, got {w.numel()}")
        return self._vec(w, self._f32)

    def rotary_table(self, n: int, turn: int, base: float = 10000.0, factor: float = 1.0, factors=None, original_len: int = 0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, magnitude: float = 1.0, first: int = 0, out=None,
                     stream=None):
        """float32 [n][turn / 2][2]: cosine and sine of positions first .. first + n - 1.  factors: the frequencies'
        divisors (a sequence of numbers, or a CPU tensor), e.g. a model file's rope_freqs; factor and original_len slow
        positions down for long contexts (see ggq_rotary_table)."""
        if out is None:
            out = self._empty((n, turn // 2, 2), self._f32, stream)
        elif tuple(out.shape) != (n, turn // 2, 2):
            raise ValueError(f"expected a [{n}, {turn // 2}, 2] output, got {tuple(out.shape)}")
        host = None
        if factors is not None:
            host = (ctypes.c_float * len(factors))(*[float(f) for f in factors])
            if 2 * len(host) != turn:
                raise ValueError(f"expected {turn // 2} factors, got {len(host)}")
        spec = ggq_rotary_spec(turn, base, ctypes.cast(host, ctypes.c_void_p) if host is not None else None, factor,
                               original_len, beta_fast, beta_slow, magnitude)
        self._check(load().ggq_rotary_table(self.handle, ctypes.byref(spec), first, n, self._vec(out, self._f32),
                                            self._stream(stream)))
        return out

    def _rotary(self, table, positions, n):
        """(address of the table, its positions, turned channels, address of the positions) of a rotation of n tokens."""
        shape = table.shape
        if len(shape) != 3 or shape[2] != 2:
            raise ValueError(f"expected a [positions, turn / 2, 2] table, got {tuple(shape)}")
        if positions.numel() != n:
            raise ValueError(f"expected {n} positions, got {positions.numel()}")
        return self._vec(table, self._f32), shape[0], 2 * shape[1], self._vec(positions, self._i32)

    def rotate(self, x, table, positions, layout: str = "half", first: int = 0, out=None, stream=None):
        """x [tokens][heads][D] with the channels from `first` on turned by the table's rows at positions (int32
        [tokens]); out may be x."""
        if x.dim() != 3:
            raise ValueError(f"expected a [tokens, heads, channels] tensor, got {tuple(x.shape)}")
        n, heads, dim = x.shape
        if out is None:
            out = self._empty((n, heads, dim), x.dtype, stream)
        xp, code, xt, xh = self._rows(x, heads, dim)
        op, ocode, ot, oh = self._rows(out, heads, dim)
        if ocode != code or out.shape[0] != n:
            raise ValueError("out has to have x's type and tokens")
        tp, rows, turn, pos = self._rotary(table, positions, n)
        _ROTATE.pack_into(self._step_args, 0, tp, rows, turn, first, ROTARY_LAYOUT[layout], code, heads, dim, n, xp, xt, xh, op, ot,
                          oh, pos)
        st = _lib.ggq_rotate(self.handle, self._step_at, self._step_more, self._stream(stream))
        if st:
            self._check(st)
        return out

    def kv_append(self, cache: KVCache, k, v, slots, table, positions, layout: str = "half", first: int = 0, q=None, q_out=None,
                  stream=None):
        """kv_store of k turned by positions, and of v; q [tokens][heads][D], where given, is turned into q_out (which
        may be q) and returned."""
        self._own(cache)
        n, dim = slots.numel(), cache.head_dim
        kp, code, kt, kh = self._rows(k, cache.n_kv_heads, dim)
        vp, vcode, vt, vh = self._rows(v, cache.n_kv_heads, dim)
        if code != vcode or k.shape[0] != n or v.shape[0] != n:
            raise ValueError("k, v and slots have to agree in type and tokens")
        heads = qp = qt = qh = op = ot = oh = 0
        if q is not None:
            if q.dim() != 3:
                raise ValueError(f"expected a [tokens, heads, {dim}] tensor, got {tuple(q.shape)}")
            heads = q.shape[1]
            if q_out is None:
                q_out = self._empty((n, heads, dim), q.dtype, stream)
            qp, qcode, qt, qh = self._rows(q, heads, dim)
            op, ocode, ot, oh = self._rows(q_out, heads, dim)
            if qcode != code or ocode != code or q.shape[0] != n or q_out.shape[0] != n:
                raise ValueError("q and q_out have to agree with k in type and tokens")
        elif q_out is not None:
            raise ValueError("q_out without q")
        tp, rows, turn, pos = self._rotary(table, positions, n)
        _APPEND.pack_into(self._step_args, 0, tp, rows, turn, first, ROTARY_LAYOUT[layout], code, heads, n, qp, qt, qh, op, ot, oh,
                          kp, kt, kh, vp, vt, vh, self._vec(slots, self._i64), pos)
        st = _lib.ggq_kv_append(self.handle, cache.ref, self._step_at, self._step_more, self._stream(stream))
        if st:
            self._check(st)
        return q_out

    def adapters(self, a, b, ranks=None, scales=None, stream=None) -> Adapters:
        """Low-rank adapters of one projection (see Adapters)."""
        return Adapters(self, a, b, ranks, scales, stream)

    def adapt(self, adapters: Adapters, x, y, ids, q_start=None, out=None, stream=None):
        """y + scale * B (A x) with each sequence's adapter: x [tokens][K], y [tokens][N] (the projection's output), ids
        int32 [sequences] (negative: none), q_start int32 [sequences + 1] unless every sequence has one token; out may
        be y.  Rows of no sequence (behind the last one, say) are not written: of an out that is not given they hold
        anything."""
        self._own(adapters, "adapters are")
        n, seqs = x.shape[0], ids.numel()
        dtype = x.dtype
        code = self._code(dtype)
        if out is None:
            out = self._empty((n, adapters.N), dtype, stream)
        if q_start is None and n != seqs:
            raise ValueError(f"{n} rows for {seqs} sequences: q_start is needed")
        if q_start is not None and q_start.numel() != seqs + 1:
            raise ValueError(f"{seqs} sequences need {seqs + 1} row starts")
        rows = (n, adapters.N)
        xp, xt = self._mat(x, (n, adapters.K), dtype)
        yp, yt = self._mat(y, rows, dtype)
        op, ot = self._mat(out, rows, dtype)
        _ADAPT.pack_into(self._step_args, 0, code, n, seqs, xp, xt, yp, yt, op, ot, self._vec(ids, self._i32),
                         self._vec(q_start, self._i32))
        st = _lib.ggq_adapt(self.handle, adapters.ref, self._step_at, self._stream(stream))
        if st:
            self._check(st)
        return out

    def logprobs(self, logits, tokens=None, top_k: int = 0, scale: float = 1.0, logprobs=None, entropy=None, ids=None, top=None,
                 stream=None):
        """(logprobs [tokens][given] of the given ids, entropy [tokens], ids [tokens][top_k], top [tokens][top_k]) of
        softmax(scale * logits), logits [tokens][V]; tokens int32 [tokens][given] or [tokens].  What is not asked for
        is None."""
        if logits.dim() != 2:
            raise ValueError(f"expected [tokens, vocabulary] logits, got {tuple(logits.shape)}")
        shape = logits.shape
        n, V = shape
        code = self._code(logits.dtype)
        given = 0
        if tokens is not None:
            if tokens.dim() not in (1, 2) or tokens.shape[0] != n:
                raise ValueError(f"expected [{n}, given] tokens, got {tuple(tokens.shape)}")
            given = 1 if tokens.dim() == 1 else tokens.shape[1]
            if logprobs is None:
                logprobs = self._empty(tuple(tokens.shape), self._f32, stream)
            elif logprobs.numel() != n * given:
                raise ValueError(f"expected {n * given} log probabilities, got {logprobs.numel()}")
        elif logprobs is not None:
            raise ValueError("log probabilities of which tokens?")
        if entropy is None:
            entropy = self._empty((n,), self._f32, stream)
        elif entropy.numel() != n:
            raise ValueError(f"expected {n} entropies, got {entropy.numel()}")
        if top_k:
            if ids is None:
                ids = self._empty((n, top_k), self._i32, stream)
            if top is None:
                top = self._empty((n, top_k), self._f32, stream)
            if ids.numel() != n * top_k or top.numel() != n * top_k:
                raise ValueError(f"expected [{n}, {top_k}] alternatives, got {tuple(ids.shape)} and {tuple(top.shape)}")
        elif ids is not None or top is not None:
            raise ValueError("alternatives without top_k")
        lp, row = self._mat(logits, shape, logits.dtype)
        _LOGPROBS.pack_into(self._step_args, 0, code, top_k, n, V, lp, row, self._vec(tokens, self._i32), given,
                            self._vec(logprobs, self._f32), self._vec(entropy, self._f32), self._vec(ids, self._i32),
                            self._vec(top, self._f32), scale)
        st = _lib.ggq_logprobs(self.handle, self._step_at, self._stream(stream))
        if st:
            self._check(st)
        return logprobs, entropy, ids, top

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
