"""ctypes binding of libtq (include/tq.h).  Argument marshalling only.

Every computation runs in libtq's CUDA kernels; PyTorch provides device memory
and the current stream.  There is no fallback: if libtq.so is missing or fails
to load, every call raises.
"""

import ctypes
import math
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq.so")

# ---------------------------------------------------------------- constants
TQ_FORMAT_VERSION = 1
TQ_BLOCK_SIZE = 16
TQ_HEAD_DIM = 128
TQ_MAX_GROUP = 8

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_WORKSPACE, TQ_ERR_CUDA, TQ_ERR_DEVICE, TQ_ERR_VERSION = range(7)
TQ_F32, TQ_BF16 = 0, 1
TQ_ROT_HADAMARD, TQ_ROT_DENSE, TQ_RNG_QJL = 1, 2, 3
TQ_KV_PACKED, TQ_KV_BF16, TQ_KV_K8V4, TQ_KV_POLAR, TQ_KV_INT8 = 0, 1, 2, 3, 4
TQ_NORM_CORRECTED, TQ_NORM_RAW = 0, 1
TQ_ROPE_HALF, TQ_ROPE_INTERLEAVED = 0, 1
TQ_ROPE_SCALE_NONE, TQ_ROPE_SCALE_LINEAR, TQ_ROPE_SCALE_NTK, TQ_ROPE_SCALE_BANDED, TQ_ROPE_SCALE_YARN = range(5)
TQ_DEV_BAD_SLOT, TQ_DEV_BAD_BLOCK, TQ_DEV_BAD_CONTEXT, TQ_DEV_WAIT_TIMEOUT = 1, 2, 4, 8
TQ_DEV_BAD_ROW, TQ_DEV_NO_BLOCK = 32, 64

STATUS_NAMES = {
    TQ_OK: "TQ_OK", TQ_ERR_INVALID_ARG: "TQ_ERR_INVALID_ARG", TQ_ERR_UNSUPPORTED: "TQ_ERR_UNSUPPORTED",
    TQ_ERR_WORKSPACE: "TQ_ERR_WORKSPACE", TQ_ERR_CUDA: "TQ_ERR_CUDA", TQ_ERR_DEVICE: "TQ_ERR_DEVICE",
    TQ_ERR_VERSION: "TQ_ERR_VERSION",
}


class TQError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), message))
        self.status = status


class LayerFormat(ctypes.Structure):
    _fields_ = [("kv_format", ctypes.c_int32), ("bits_k", ctypes.c_int32), ("bits_v", ctypes.c_int32),
                ("qjl_k", ctypes.c_int32), ("rot_kind", ctypes.c_int32), ("norm_mode", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("format_version", ctypes.c_uint32), ("head_dim", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int64),
                ("fmt", LayerFormat), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("rotation", ctypes.c_void_p), ("qjl_proj", ctypes.c_void_p),
                ("centroids_k", ctypes.c_float * 16), ("boundaries_k", ctypes.c_float * 15),
                ("centroids_v", ctypes.c_float * 16), ("boundaries_v", ctypes.c_float * 15)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("length", ctypes.c_double)]


class Heads(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("num_heads", ctypes.c_int32),
                ("in_token_stride", ctypes.c_int64), ("in_head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


class BlockPool(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("refs", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class BlockRows(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32)]


_P = ctypes.POINTER
_D = ctypes.POINTER(CacheDesc)
_R = ctypes.POINTER(RopeDesc)
_H = ctypes.POINTER(Heads)
_SIGNATURES = {
    "tq_make_codebook": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, _P(ctypes.c_float), _P(ctypes.c_float)]),
    "tq_make_rotation": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_int, _P(ctypes.c_float)]),
    "tq_page_bytes": (ctypes.c_size_t, [_D, ctypes.c_int]),
    "tq_quantize_append": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_void_p]),
    "tq_quantize_append_layers": (ctypes.c_int, [_P(_D), ctypes.c_int, _P(ctypes.c_void_p), _P(ctypes.c_void_p),
                                                 ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "tq_quantize_rotated": (ctypes.c_int, [_D, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_void_p]),
    "tq_auto_splits": (ctypes.c_int, [_D, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "tq_workspace_bytes": (ctypes.c_size_t, [_D, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "tq_decode_attention": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float,
                                           ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_int, ctypes.c_void_p]),
    "tq_append_decode": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_int, ctypes.c_void_p]),
    "tq_decode_step": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]),
    "tq_make_rope": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_double, _P(RopeScaling), _P(ctypes.c_double),
                                    _R]),
    "tq_rope_apply": (ctypes.c_int, [_R, ctypes.c_int, _H, _H, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p]),
    "tq_rope_append": (ctypes.c_int, [_D, _R, _H, _H, _H, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_void_p]),
    "tq_attend_workspace_bytes": (ctypes.c_size_t, [_D, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "tq_attend": (ctypes.c_int, [_D, _H, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                 ctypes.c_size_t, ctypes.c_void_p]),
    "tq_prefix_workspace_bytes": (ctypes.c_size_t, [_D, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int]),
    "tq_prefix_decode": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "tq_dequantize": (ctypes.c_int, [_D, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_void_p]),
    "tq_blocks_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "tq_copy_blocks": (ctypes.c_int, [_P(_D), ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
    "tq_blocks_extend": (ctypes.c_int, [_P(BlockPool), _P(BlockRows), ctypes.c_void_p, ctypes.c_void_p]),
    "tq_blocks_release": (ctypes.c_int, [_P(BlockPool), _P(BlockRows), ctypes.c_void_p, ctypes.c_void_p]),
    "tq_blocks_reorder": (ctypes.c_int, [_P(BlockPool), _P(_D), ctypes.c_int, _P(BlockRows), ctypes.c_void_p,
                                         _P(BlockRows), ctypes.c_void_p]),
    "tq_blocks_compact": (ctypes.c_int, [_P(BlockPool), _P(_D), ctypes.c_int, _P(BlockRows), ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tq_image_bytes": (ctypes.c_size_t, [_D, ctypes.c_int64]),
    "tq_offload_blocks": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "tq_restore_blocks": (ctypes.c_int, [_D, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "tq_get_device_status": (ctypes.c_int, [ctypes.c_void_p, _P(ctypes.c_int32)]),
    "tq_last_error": (ctypes.c_char_p, []),
    "tq_format_version": (ctypes.c_uint32, []),
    "tq_launch_count": (ctypes.c_uint64, []),
}

_lib = None


def lib():
    """The loaded libtq (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libtq.so is not built (%s); run turboquant_quantized_kv_gb300.build.build()" % LIB_PATH)
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if handle.tq_format_version() != TQ_FORMAT_VERSION:
            raise RuntimeError("libtq format version mismatch")
        _lib = handle
    return _lib


def last_error():
    return lib().tq_last_error().decode("utf-8", "replace")


def _check(status):
    if status != TQ_OK:
        raise TQError(status, last_error())


# ------------------------------------------------------------------ set-up

def make_codebook(bits, head_dim=TQ_HEAD_DIM):
    """(centroids fp32 [2^bits], boundaries fp32 [2^bits - 1]) from tq_make_codebook."""
    k = 1 << bits
    c = (ctypes.c_float * k)()
    b = (ctypes.c_float * max(k - 1, 1))()
    _check(lib().tq_make_codebook(head_dim, bits, c, b))
    return np.frombuffer(c, dtype=np.float32).copy(), np.frombuffer(b, dtype=np.float32)[: k - 1].copy()


def make_rotation(kind, seed, layer=0, head_dim=TQ_HEAD_DIM):
    """Host fp32 signs [d] (Hadamard) or matrix [d, d] (dense, QJL) from tq_make_rotation."""
    n = head_dim if kind == TQ_ROT_HADAMARD else head_dim * head_dim
    out = (ctypes.c_float * n)()
    _check(lib().tq_make_rotation(kind, head_dim, ctypes.c_uint64(seed), layer, out))
    arr = np.frombuffer(out, dtype=np.float32).copy()
    return arr if kind == TQ_ROT_HADAMARD else arr.reshape(head_dim, head_dim)


# ------------------------------------------------------------ tensor glue

_torch_module = None
_dtype_codes = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t):
    global _dtype_codes
    if _dtype_codes is None:
        torch = _torch()
        _dtype_codes = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16}
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)
    return code


def _ptr(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream of the current device, without building a Stream object
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _new(make, shape, dtype, device, stream):
    """make(shape) (torch.empty or torch.zeros) for a call on `stream`: the memory comes from that stream's pool, free
    of what other streams still do with it, and is filled there."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with _torch().cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _capturing(stream):
    torch = _torch()
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


_byref = ctypes.byref


def _check_rows(x, what, n):
    """Strides of rows [n, heads, d] on the device with a contiguous last dimension; raises for others."""
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    shape = x.shape
    if len(shape) != 3 or shape[2] != TQ_HEAD_DIM or shape[0] != n:
        raise ValueError("%s must be [%d, heads, %d], got %s" % (what, n, TQ_HEAD_DIM, tuple(shape)))
    strides = x.stride()
    if strides[2] != 1 and x.numel() > 0:
        raise ValueError("%s must be contiguous in its last dimension" % what)
    return strides


def _check_outputs(q, q_out, k, k_out):
    """Raises for an output that nothing would be written to."""
    if q is None and q_out is not None:
        raise ValueError("q_out is given without q")
    if k is None and k_out is not None:
        raise ValueError("k_out is given without k")


def _heads(t, out, name, n):
    """Reference to a tq_heads of t [n, heads, d] (any token and head strides) and its output rows."""
    if t is None:
        return None
    st = so = _check_rows(t, name, n)
    if out is None:
        return _byref(Heads(t.data_ptr(), None, t.shape[1], st[0], st[1], 0, 0))
    if out is not t:
        if out.shape != t.shape or out.dtype != t.dtype:
            raise ValueError("%s_out must have %s's shape and type" % (name, name))
        so = _check_rows(out, name + "_out", n)
    return _byref(Heads(t.data_ptr(), out.data_ptr(), t.shape[1], st[0], st[1], so[0], so[1]))


def _check_queries(q, out):
    """(batch, query heads) of queries [B, H_q, d]; raises for others and for an output of another size
    (d is read and written whole, whatever the tensors hold)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != TQ_HEAD_DIM:
        raise ValueError("q must be [batch, query heads, %d], got %s" % (TQ_HEAD_DIM, tuple(shape)))
    if out is not None and out.shape != shape and out.shape != (shape[0], shape[1] * shape[2]):
        raise ValueError("out must be %s, got %s" % (tuple(shape), tuple(out.shape)))
    return shape[0], shape[1]


def _index_ptr(t, name, dtype, shape):
    """Device pointer of an index tensor after checking its type and shape."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


class Rope:
    """Rotary positions: the frequencies of a rotation (tq_make_rope).

    layout: "half" (pairs i, i + rotary_dim / 2) or "interleaved" (pairs 2 i, 2 i + 1).
    scaling: None or a dict {"kind": "linear" | "ntk" | "banded" | "yarn", "factor": f},
    for banded and yarn also "low", "high" and "length".  inv_freq: rotary_dim / 2
    frequencies in radians a position that replace base.
    """

    _LAYOUTS = {"half": TQ_ROPE_HALF, "interleaved": TQ_ROPE_INTERLEAVED}
    _KINDS = {"linear": TQ_ROPE_SCALE_LINEAR, "ntk": TQ_ROPE_SCALE_NTK, "banded": TQ_ROPE_SCALE_BANDED,
              "yarn": TQ_ROPE_SCALE_YARN}

    def __init__(self, rotary_dim=TQ_HEAD_DIM, base=10000.0, layout="half", scaling=None, inv_freq=None):
        if layout not in self._LAYOUTS:
            raise ValueError("layout must be 'half' or 'interleaved'")
        s = None
        if scaling is not None:
            if scaling.get("kind") not in self._KINDS:
                raise ValueError("scaling kind must be one of %s" % sorted(self._KINDS))
            s = RopeScaling(self._KINDS[scaling["kind"]], float(scaling["factor"]), float(scaling.get("low", 0.0)),
                            float(scaling.get("high", 0.0)), float(scaling.get("length", 0.0)))
        freqs = None
        if inv_freq is not None:
            values = np.asarray(inv_freq, np.float64).reshape(-1)
            if values.size != rotary_dim // 2:
                raise ValueError("inv_freq must hold rotary_dim / 2 frequencies")
            freqs = (ctypes.c_double * values.size)(*values)
        self.desc = RopeDesc()
        self.ref = ctypes.byref(self.desc)
        _check(lib().tq_make_rope(self._LAYOUTS[layout], rotary_dim, base, _ref(s), freqs, self.ref))
        self.layout, self.rotary_dim = layout, int(rotary_dim)
        self.amplitude = float(self.desc.amplitude)

    def turns(self):
        """Turns a position of each pair (fp64 [rotary_dim / 2], modulo one turn)."""
        return np.array(self.desc.turns[: self.rotary_dim // 2], dtype=np.uint64).astype(np.float64) * 2.0 ** -64


_rope_function = None


def _differentiable_rope():
    """The rotation as a torch.autograd.Function: its gradient is the transposed rotation."""
    global _rope_function
    if _rope_function is None:
        torch = _torch()

        class RopeFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, rope, positions, transpose, q, k):
                ctx.set_materialize_grads(False)
                ctx.rope, ctx.transpose = rope, transpose
                ctx.save_for_backward(positions)
                return apply_rope(rope, positions, q, k, transpose=transpose)

            @staticmethod
            def backward(ctx, gq, gk):
                (positions,) = ctx.saved_tensors
                # (gradients may be expanded: rows are read with a contiguous last dimension)
                gq, gk = (g.contiguous() if g is not None and g.stride(2) != 1 else g for g in (gq, gk))
                if not ctx.needs_input_grad[3]:
                    gq = None
                if not ctx.needs_input_grad[4]:
                    gk = None
                if gq is not None or gk is not None:
                    gq, gk = apply_rope(ctx.rope, positions, gq, gk, transpose=not ctx.transpose)
                return None, None, None, gq, gk

        _rope_function = RopeFunction
    return _rope_function


def apply_rope(rope, positions, q, k=None, q_out=None, k_out=None, transpose=False, stream=None):
    """Rotary positions of q and k [n_tokens, heads, d] (tq_rope_apply); positions int64
    [n_tokens].  transpose: the transposed rotation (the gradient).  q_out / k_out may be
    q / k (in place).  Returns (q_out, k_out), contiguous where they were not given.  Where q or k
    requires a gradient the results are differentiable, and outputs cannot be given."""
    torch = _torch()
    if torch.is_grad_enabled() and ((q is not None and q.requires_grad) or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out take no part in differentiation: leave them out or use torch.no_grad()")
        if stream is not None:
            with torch.cuda.stream(stream):
                return _differentiable_rope().apply(rope, positions, transpose, q, k)
        return _differentiable_rope().apply(rope, positions, transpose, q, k)
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k is needed")
    _check_outputs(q, q_out, k, k_out)
    dtype, device, n = ref.dtype, ref.device, ref.shape[0]
    if k is not None and k.dtype != dtype:
        raise TypeError("q and k must have one type")
    if q is not None and q_out is None:
        q_out = _new(torch.empty, q.shape, dtype, device, stream)
    if k is not None and k_out is None:
        k_out = _new(torch.empty, k.shape, dtype, device, stream)
    pos = _index_ptr(positions, "positions", torch.int64, (n,))
    _check(lib().tq_rope_apply(rope.ref, 1 if transpose else 0, _heads(q, q_out, "q", n), _heads(k, k_out, "k", n),
                               _dtype_code(ref), pos, n, _stream(stream)))
    return q_out, k_out


class Layer:
    """One layer of the paged cache: device pools, rotation and codebooks.

    kv_format: "packed" (TurboQuant codes), "bf16" (boundary layers), "k8v4"
    (FP8 E4M3 keys with TurboQuant values of bits_v), "polar" (PolarQuant
    angle codes of bits_k / bits_v bits with an fp16 radius; Hadamard only) or
    "int8" (8-bit codes with one step for each block and head; no rotation).
    The descriptor (`desc`) points at tensors owned by this object.
    """

    def __init__(self, num_blocks, num_kv_heads, *, kv_format="packed", bits_k=4, bits_v=4, qjl=False,
                 rot_kind=TQ_ROT_HADAMARD, seed=0, layer=0, qjl_seed=None, norm_mode=TQ_NORM_CORRECTED,
                 device="cuda", rotation=None, qjl_proj=None, fill=0):
        torch = _torch()
        self.num_blocks = int(num_blocks)
        self.num_kv_heads = int(num_kv_heads)
        self.head_dim = TQ_HEAD_DIM
        if kv_format not in ("packed", "bf16", "k8v4", "polar", "int8"):
            raise ValueError("kv_format must be 'packed', 'bf16', 'k8v4', 'polar' or 'int8'")
        self.kv_format = kv_format
        self.packed = kv_format == "packed"
        self.k8v4 = kv_format == "k8v4"
        self.polar = kv_format == "polar"
        coded_v = self.packed or self.k8v4 or self.polar  # rotated, coded layers
        d = CacheDesc()
        d.format_version = TQ_FORMAT_VERSION
        d.head_dim = TQ_HEAD_DIM
        d.num_kv_heads = self.num_kv_heads
        d.block_size = TQ_BLOCK_SIZE
        d.num_blocks = self.num_blocks
        d.fmt.kv_format = {"packed": TQ_KV_PACKED, "bf16": TQ_KV_BF16, "k8v4": TQ_KV_K8V4,
                           "polar": TQ_KV_POLAR, "int8": TQ_KV_INT8}[kv_format]
        self.int8 = kv_format == "int8"
        if self.k8v4 or self.int8:
            bits_k = 8
        if self.int8:
            bits_v = 8
        d.fmt.bits_k = bits_k if coded_v or self.int8 else 0
        d.fmt.bits_v = bits_v if coded_v or self.int8 else 0
        d.fmt.qjl_k = 1 if (qjl and self.packed) else 0
        d.fmt.rot_kind = rot_kind if coded_v else 0
        d.fmt.norm_mode = norm_mode
        self.bits_k, self.bits_v, self.qjl, self.rot_kind = bits_k, bits_v, bool(qjl and self.packed), rot_kind
        self.seed, self.layer_index = seed, layer
        self.qjl_seed = seed if qjl_seed is None else qjl_seed
        self.explicit_rotation = rotation
        self.rotation_host = None
        self.qjl_host = None
        self.cb_k = self.cb_v = None
        if coded_v:
            self.cb_k = make_codebook(bits_k) if self.packed else None
            self.cb_v = make_codebook(bits_v) if not self.polar else None
            if self.packed:
                for i, v in enumerate(self.cb_k[0]):
                    d.centroids_k[i] = float(v)
                for i, v in enumerate(self.cb_k[1]):
                    d.boundaries_k[i] = float(v)
            if self.cb_v is not None:
                for i, v in enumerate(self.cb_v[0]):
                    d.centroids_v[i] = float(v)
                for i, v in enumerate(self.cb_v[1]):
                    d.boundaries_v[i] = float(v)
            rot = make_rotation(rot_kind, seed, layer) if rotation is None else np.asarray(rotation, np.float32)
            self.rotation_host = rot
            self.rotation = torch.from_numpy(np.ascontiguousarray(rot)).to(device)
            d.rotation = self.rotation.data_ptr()
            if self.qjl:
                s = make_rotation(TQ_RNG_QJL, seed if qjl_seed is None else qjl_seed) if qjl_proj is None \
                    else np.asarray(qjl_proj, np.float32)
                self.qjl_host = s
                self.qjl_proj = torch.from_numpy(np.ascontiguousarray(s)).to(device)
                d.qjl_proj = self.qjl_proj.data_ptr()
        self.desc = d
        self.desc_ptr = ctypes.pointer(d)
        self.page_bytes_k = self.page_bytes(0)
        self.page_bytes_v = self.page_bytes(1)
        nk = self.num_blocks * self.num_kv_heads * self.page_bytes_k
        nv = self.num_blocks * self.num_kv_heads * self.page_bytes_v
        self.k_cache = torch.full((nk,), fill, dtype=torch.uint8, device=device)
        self.v_cache = torch.full((nv,), fill, dtype=torch.uint8, device=device)
        d.k_cache = self.k_cache.data_ptr()
        d.v_cache = self.v_cache.data_ptr()

    def page_bytes(self, which):
        n = lib().tq_page_bytes(ctypes.byref(self.desc), which)
        if n == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid descriptor")
        return int(n)

    # -------------------------------------------------------------- calls
    def append(self, k, v, slot_mapping, stream=None):
        """Quantize-on-append of k, v [n_tokens, H_kv, d] into slot_mapping [n_tokens] (int64)."""
        ref = k if k is not None else v
        n = int(ref.shape[0])
        _check(lib().tq_quantize_append(ctypes.byref(self.desc), _ptr(k, "k"), _ptr(v, "v"), _dtype_code(ref),
                                        _ptr(slot_mapping, "slot_mapping"), n, _stream(stream)))

    def quantize_rotated(self, which, y, norms, slot_mapping, stream=None):
        """The quantizer alone on rotated unit coordinates y [n, H_kv, d] (fp32) with norms [n, H_kv]."""
        _check(lib().tq_quantize_rotated(ctypes.byref(self.desc), which, _ptr(y, "y"), _ptr(norms, "norms"),
                                         _ptr(slot_mapping, "slot_mapping"), int(y.shape[0]), _stream(stream)))

    def workspace_bytes(self, batch, num_q_heads, max_blocks_per_seq, num_splits=0):
        n = lib().tq_workspace_bytes(ctypes.byref(self.desc), batch, num_q_heads, max_blocks_per_seq, num_splits)
        if n == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid sizes")
        return int(n)

    def auto_splits(self, batch, num_q_heads, max_blocks_per_seq):
        return int(lib().tq_auto_splits(ctypes.byref(self.desc), batch, num_q_heads, max_blocks_per_seq))

    def decode(self, q, block_table, context_lens, sm_scale=None, out=None, out_dtype=None, num_splits=0,
               workspace=None, stream=None):
        """Decode attention.  q [B, H_q, d]; block_table int32 [B, max_blocks]; context_lens int32 [B]."""
        torch = _torch()
        bsz, hq = _check_queries(q, out)
        max_blocks = int(block_table.shape[1])
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.head_dim)
        if out is None:
            out = _new(torch.empty, q.shape, q.dtype if out_dtype is None else out_dtype, q.device, stream)
        if workspace is None:
            workspace = _new(torch.zeros, self.workspace_bytes(bsz, hq, max_blocks, num_splits), torch.uint8, q.device,
                             stream)
        _check(lib().tq_decode_attention(ctypes.byref(self.desc), _ptr(q, "q"), _dtype_code(q), bsz, hq,
                                         _ptr(block_table, "block_table"), max_blocks,
                                         _ptr(context_lens, "context_lens"), ctypes.c_float(sm_scale),
                                         _ptr(out, "out"), _dtype_code(out), _ptr(workspace, "workspace"),
                                         workspace.numel(), num_splits, _stream(stream)))
        return out

    def append_decode(self, k, v, slot_mapping, q, block_table, context_lens, sm_scale=None, out=None,
                      out_dtype=None, num_splits=0, workspace=None, stream=None):
        """append(k, v, slot_mapping) then decode(q, ...) in one call (tq_append_decode: the
        decode's prologue overlaps the append).  Returns out."""
        torch = _torch()
        ref = k if k is not None else v
        n = int(ref.shape[0]) if ref is not None else 0
        bsz, hq = _check_queries(q, out)
        max_blocks = int(block_table.shape[1])
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.head_dim)
        if out is None:
            out = _new(torch.empty, q.shape, q.dtype if out_dtype is None else out_dtype, q.device, stream)
        if workspace is None:
            workspace = _new(torch.zeros, self.workspace_bytes(bsz, hq, max_blocks, num_splits), torch.uint8, q.device,
                             stream)
        _check(lib().tq_append_decode(ctypes.byref(self.desc), _ptr(k, "k"), _ptr(v, "v"),
                                      _dtype_code(ref) if ref is not None else TQ_BF16,
                                      _ptr(slot_mapping, "slot_mapping"), n, _ptr(q, "q"), _dtype_code(q), bsz, hq,
                                      _ptr(block_table, "block_table"), max_blocks,
                                      _ptr(context_lens, "context_lens"), ctypes.c_float(sm_scale),
                                      _ptr(out, "out"), _dtype_code(out), _ptr(workspace, "workspace"),
                                      workspace.numel(), num_splits, _stream(stream)))
        return out

    def decode_step(self, k_new, v_new, q, block_table, context_lens, sm_scale=None, out=None, out_dtype=None,
                    num_splits=0, workspace=None, stream=None):
        """One decode step in one kernel (tq_decode_step): k_new, v_new [B, H_kv, d] are the new
        tokens, written at position context_lens[b] - 1 of each sequence (context_lens already
        counts them), then decode(q, ...).  Returns out."""
        torch = _torch()
        bsz, hq = _check_queries(q, out)
        max_blocks = int(block_table.shape[1])
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.head_dim)
        if out is None:
            out = _new(torch.empty, q.shape, q.dtype if out_dtype is None else out_dtype, q.device, stream)
        if workspace is None:
            workspace = _new(torch.zeros, self.workspace_bytes(bsz, hq, max_blocks, num_splits), torch.uint8, q.device,
                             stream)
        _check(lib().tq_decode_step(ctypes.byref(self.desc), _ptr(k_new, "k_new"), _ptr(v_new, "v_new"),
                                    _dtype_code(k_new), _ptr(q, "q"), _dtype_code(q), bsz, hq,
                                    _ptr(block_table, "block_table"), max_blocks, _ptr(context_lens, "context_lens"),
                                    ctypes.c_float(sm_scale), _ptr(out, "out"), _dtype_code(out),
                                    _ptr(workspace, "workspace"), workspace.numel(), num_splits, _stream(stream)))
        return out

    def rope_append(self, rope, k, v, positions, slot_mapping, q=None, q_out=None, k_out=None, stream=None):
        """Append with the rotation applied on the way (tq_rope_append): k [n_tokens, H_kv, d]
        rotated to positions [n_tokens] (int64), stored with v in slot_mapping [n_tokens]
        (int64).  q [n_tokens, H_q, d] is rotated to q_out (may be q); k_out, if given, takes
        the rotated keys.  Token and head strides are free.  Nothing is recorded for
        differentiation (apply_rope is differentiable).  Returns q_out."""
        torch = _torch()
        ref = k if k is not None else v
        if ref is None:
            raise ValueError("k or v is needed")
        _check_outputs(q, q_out, k, k_out)
        dtype, n = ref.dtype, ref.shape[0]
        if (q is not None and q.dtype != dtype) or (v is not None and v.dtype != dtype):
            raise TypeError("q, k and v must have one type")
        pos = _index_ptr(positions, "positions", torch.int64, (n,))
        slots = _index_ptr(slot_mapping, "slot_mapping", torch.int64, (n,))
        if q is not None and q_out is None:
            q_out = _new(torch.empty, q.shape, dtype, q.device, stream)
        _check(lib().tq_rope_append(_byref(self.desc), rope.ref, _heads(q, q_out, "q", n), _heads(k, k_out, "k", n),
                                    _heads(v, None, "v", n), _dtype_code(ref), pos, slots, n, _stream(stream)))
        return q_out

    def attend_workspace_bytes(self, n_tokens, batch, num_q_heads, max_blocks_per_seq):
        n = lib().tq_attend_workspace_bytes(ctypes.byref(self.desc), n_tokens, batch, num_q_heads, max_blocks_per_seq)
        if n == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid sizes")
        return int(n)

    def attend(self, q, query_starts, block_table, context_lens, sm_scale=None, out=None, out_dtype=None,
               workspace=None, stream=None):
        """Causal attention of the last tokens of each sequence (tq_attend; int8 layers).  q
        [n_tokens, H_q, d], any token and head strides; query_starts int32 [B + 1]: rows
        query_starts[b] .. query_starts[b + 1] - 1 are the last tokens of sequence b, whose
        context_lens[b] tokens are in the cache already; block_table int32 [B, max_blocks];
        context_lens int32 [B].  Rows from query_starts[B] on are left as they were.  Returns out."""
        torch = _torch()
        n = int(q.shape[0])
        _check_rows(q, "q", n)
        if out is None:
            out = _new(torch.empty, q.shape, q.dtype if out_dtype is None else out_dtype, q.device, stream)
        elif out.shape != q.shape:
            raise ValueError("out must be %s, got %s" % (tuple(q.shape), tuple(out.shape)))
        if block_table.dim() != 2:
            raise ValueError("block_table must be [batch, blocks]")
        bsz, max_blocks = block_table.shape
        starts = _index_ptr(query_starts, "query_starts", torch.int32, (bsz + 1,))
        table = _index_ptr(block_table, "block_table", torch.int32, block_table.shape)
        lens = _index_ptr(context_lens, "context_lens", torch.int32, (bsz,))
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.head_dim)
        if workspace is None:
            workspace = _new(torch.zeros, self.attend_workspace_bytes(n, bsz, q.shape[1], max(1, max_blocks)), torch.uint8,
                             q.device, stream)
        sq, so = q.stride(), _check_rows(out, "out", n)
        rows = Heads(q.data_ptr(), out.data_ptr(), q.shape[1], sq[0], sq[1], so[0], so[1])
        _check(lib().tq_attend(_byref(self.desc), _byref(rows), _dtype_code(q), _dtype_code(out), n, starts, bsz, table,
                               max_blocks, lens, ctypes.c_float(sm_scale), _ptr(workspace, "workspace"), workspace.numel(),
                               _stream(stream)))
        return out

    def prefix_workspace_bytes(self, batch, num_q_heads, prefix_len, max_blocks_per_seq):
        n = lib().tq_prefix_workspace_bytes(ctypes.byref(self.desc), batch, num_q_heads, prefix_len,
                                            max_blocks_per_seq)
        if n == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid sizes")
        return int(n)

    def prefix_decode(self, q, prefix_table, prefix_len, block_table=None, context_lens=None, sm_scale=None, out=None,
                      out_dtype=None, workspace=None, stream=None):
        """Decode attention of a batch with a shared prefix (tq_prefix_decode).  q [B, H_q, d];
        prefix_table int32 [>= ceil(prefix_len / 16)] blocks of the prefix; block_table int32
        [B, max_blocks] and context_lens int32 [B]: the sequences' own tokens (None: none)."""
        torch = _torch()
        bsz, hq = _check_queries(q, out)
        prefix_len = int(prefix_len)
        if prefix_len > 0 and (prefix_table is None or prefix_table.dim() != 1 or prefix_table.shape[0] * TQ_BLOCK_SIZE < prefix_len):
            raise ValueError("prefix_table must be one row of at least ceil(prefix_len / %d) blocks" % TQ_BLOCK_SIZE)
        max_blocks = 0 if block_table is None else int(block_table.shape[1])
        if max_blocks > 0 and context_lens is None:
            raise ValueError("block_table needs context_lens")
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.head_dim)
        if out is None:
            out = _new(torch.empty, q.shape, q.dtype if out_dtype is None else out_dtype, q.device, stream)
        if workspace is None and bsz > 0:
            workspace = _new(torch.zeros, self.prefix_workspace_bytes(bsz, hq, prefix_len, max_blocks), torch.uint8,
                             q.device, stream)
        table = None if prefix_len <= 0 else _index_ptr(prefix_table, "prefix_table", torch.int32, prefix_table.shape)
        rows = lens = None
        if max_blocks > 0:
            rows = _index_ptr(block_table, "block_table", torch.int32, (bsz, max_blocks))
            lens = _index_ptr(context_lens, "context_lens", torch.int32, (bsz,))
        _check(lib().tq_prefix_decode(ctypes.byref(self.desc), _ptr(q, "q"), _dtype_code(q), bsz, hq, table,
                                      prefix_len, rows, max_blocks, lens, ctypes.c_float(sm_scale), _ptr(out, "out"),
                                      _dtype_code(out), _ptr(workspace, "workspace"),
                                      0 if workspace is None else workspace.numel(), _stream(stream)))
        return out

    def image_bytes(self, n_blocks):
        n = lib().tq_image_bytes(ctypes.byref(self.desc), int(n_blocks))
        if n == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid descriptor")
        return int(n)

    def offload(self, blocks, image=None, stream=None):
        """Host image (pinned uint8 tensor) of the pages of `blocks` (block ids), see
        tq_offload_blocks.  The image is complete once the stream reaches this call."""
        torch = _torch()
        ids = np.ascontiguousarray(np.asarray(blocks, dtype=np.int32).reshape(-1))
        if image is None:
            image = torch.empty(self.image_bytes(ids.size), dtype=torch.uint8, pin_memory=True)
        if image.is_cuda:
            raise ValueError("image must be a host (pinned) tensor")
        _check(lib().tq_offload_blocks(ctypes.byref(self.desc), ids.ctypes.data_as(ctypes.c_void_p), ids.size,
                                       ctypes.c_void_p(image.data_ptr()), image.numel(), _stream(stream)))
        return image

    def restore(self, blocks, image, stream=None):
        """Copies an image's pages into `blocks` (tq_restore_blocks)."""
        ids = np.ascontiguousarray(np.asarray(blocks, dtype=np.int32).reshape(-1))
        if image.is_cuda:
            raise ValueError("image must be a host (pinned) tensor")
        _check(lib().tq_restore_blocks(ctypes.byref(self.desc), ids.ctypes.data_as(ctypes.c_void_p), ids.size,
                                       ctypes.c_void_p(image.data_ptr()), image.numel(), _stream(stream)))

    def dequantize(self, which, slots, out_dtype=None, stream=None):
        """x_hat [n, H_kv, d] of the K (which=0) or V (which=1) records at slots [n] (int64)."""
        torch = _torch()
        dt = torch.float32 if out_dtype is None else out_dtype
        out = _new(torch.empty, (int(slots.shape[0]), self.num_kv_heads, self.head_dim), dt, slots.device, stream)
        _check(lib().tq_dequantize(ctypes.byref(self.desc), which, _ptr(slots, "slots"), int(slots.shape[0]),
                                   _ptr(out, "out"), _dtype_code(out), _stream(stream)))
        return out


def append_layers(layers, ks, vs, slot_mapping, stream=None):
    """Quantize-on-append of the same tokens into several layers (tq_quantize_append_layers):
    ks[l], vs[l] [n_tokens, H_kv, d] are layer l's inputs (either list may be None)."""
    n_layers = len(layers)
    descs = _descs(layers)
    def ptrs(ts, name):
        if ts is None:
            return None
        return (ctypes.c_void_p * n_layers)(*[_ptr(t, name) for t in ts])
    ref = (ks if ks is not None else vs)[0]
    _check(lib().tq_quantize_append_layers(descs, n_layers, ptrs(ks, "k"), ptrs(vs, "v"), _dtype_code(ref),
                                           _ptr(slot_mapping, "slot_mapping"), int(ref.shape[0]), _stream(stream)))


def _descs(layers):
    return (_D * len(layers))(*[ly.desc_ptr for ly in layers])


def copy_blocks(layers, src, dst, stream=None):
    """Pages of block src[i] to block dst[i] (int32, on the device) in both pools of every layer (tq_copy_blocks)."""
    torch = _torch()
    n = int(src.shape[0])
    _check(lib().tq_copy_blocks(_descs(layers), len(layers), _index_ptr(src, "src", torch.int32, (n,)),
                                _index_ptr(dst, "dst", torch.int32, (n,)), n, _stream(stream)))


class Blocks:
    """The blocks of the layers that share block ids: how many table entries hold each (`refs`, int32
    [num_blocks], 0: free), and the calls that hand them out, share, copy and move them.

    A row of a block table [rows, max_blocks] (int32) holds the blocks of its first context_lens[row]
    tokens (int32).  All calls are enqueued and decided on the device, lowest free block first; what went
    wrong stands in get_device_status().  Calls of one object follow one another on a stream.
    `layers`: the layers whose pages go with the ids (any formats, num_blocks blocks each)."""

    def __init__(self, num_blocks, device="cuda"):
        torch = _torch()
        self.num_blocks = int(num_blocks)
        self._refs = torch.zeros(self.num_blocks, dtype=torch.int32, device=device)
        self._workspaces = []  # (earlier ones too: captured graphs may use them; eleven at most)
        self._rows, self._pool_ref = -1, None

    @property
    def refs(self):
        return self._refs

    def _pool(self, rows, stream):
        """Reference to the tq_block_pool of `refs` and a workspace for calls of so many rows.  The object's own is made for
        the next power of two; a call that is captured while there is none has memory of the graph's instead
        (torch.cuda.graph's pool, as every tensor made in a capture), which is zero when the graph runs, not before, and free
        for the graph's later calls."""
        if rows <= self._rows:
            return self._pool_ref
        most = max(1024, 1 << (rows - 1).bit_length())
        size = lib().tq_blocks_workspace_bytes(self.num_blocks, most)
        if size == 0:
            raise TQError(TQ_ERR_INVALID_ARG, last_error() or "invalid sizes")
        pool = BlockPool(self.num_blocks, _index_ptr(self.refs, "refs", _torch().int32, (self.num_blocks,)))
        pool.memory = _new(_torch().zeros, (int(size),), _torch().uint8, self.refs.device, stream)
        pool.workspace, pool.workspace_bytes = pool.memory.data_ptr(), pool.memory.numel()
        if not _capturing(stream):
            self._workspaces.append(pool.memory)
            self._rows, self._pool_ref = most, _byref(pool)
            return self._pool_ref
        return _byref(pool)

    @staticmethod
    def _table(block_table, context_lens):
        torch = _torch()
        if block_table.dim() != 2:
            raise ValueError("block_table must be [rows, blocks], got %s" % (tuple(block_table.shape),))
        rows, width = block_table.shape
        return BlockRows(_index_ptr(block_table, "block_table", torch.int32, (rows, width)),
                         _index_ptr(context_lens, "context_lens", torch.int32, (rows,)), rows, width)

    def extend(self, block_table, context_lens, new_lens, stream=None):
        """Blocks for new_lens [rows] (int32) tokens a row, written into block_table (tq_blocks_extend)."""
        rows = self._table(block_table, context_lens)
        grown = _index_ptr(new_lens, "new_lens", _torch().int32, (rows.rows,))
        _check(lib().tq_blocks_extend(self._pool(rows.rows, stream), _byref(rows), grown, _stream(stream)))

    def release(self, block_table, context_lens, which=None, stream=None):
        """The rows with which[row] (bool; None: all) give up their blocks, in place (tq_blocks_release)."""
        rows = self._table(block_table, context_lens)
        mask = None if which is None else _index_ptr(which, "which", _torch().bool, (rows.rows,))
        _check(lib().tq_blocks_release(self._pool(0, stream), _byref(rows), mask, _stream(stream)))

    def reorder(self, layers, block_table, context_lens, parents, stream=None):
        """New rows [len(parents)], each a fork of old row parents[i] (int32; -1: an empty row): full blocks
        are shared, a last block that is not full is copied for all children but the first, rows without
        children give up theirs (tq_blocks_reorder).  Returns (block_table, context_lens) of the new rows."""
        torch = _torch()
        old = self._table(block_table, context_lens)
        if parents.dim() != 1:
            raise ValueError("parents must be one row, got %s" % (tuple(parents.shape),))
        n = int(parents.shape[0])
        index = _index_ptr(parents, "parents", torch.int32, (n,))
        device, width = block_table.device, old.max_blocks
        table = _new(torch.empty, (n, width), torch.int32, device, stream)
        lens = _new(torch.empty, (n,), torch.int32, device, stream)
        new = BlockRows(table.data_ptr(), lens.data_ptr(), n, width)
        _check(lib().tq_blocks_reorder(self._pool(max(old.rows, n), stream), _descs(layers), len(layers), _byref(old), index,
                                       _byref(new), _stream(stream)))
        return table, lens

    def compact(self, layers, block_table, context_lens, *more, moved=None, stream=None):
        """The used blocks to the lowest ids, tables rewritten in place (tq_blocks_compact); `more`: further
        tables and lengths in turn; moved: int32 [num_blocks] that takes where each block is now.  Returns the
        number of used blocks (int32 [1], on the device)."""
        torch = _torch()
        if len(more) % 2 != 0:
            raise ValueError("further tables come with their lengths")
        pairs = [(block_table, context_lens)] + [(more[i], more[i + 1]) for i in range(0, len(more), 2)]
        tables = (BlockRows * len(pairs))(*[self._table(t, n) for t, n in pairs])
        live = _new(torch.empty, (1,), torch.int32, self.refs.device, stream)
        to = None if moved is None else _index_ptr(moved, "moved", torch.int32, (self.num_blocks,))
        _check(lib().tq_blocks_compact(self._pool(0, stream), _descs(layers), len(layers), tables, len(pairs), live.data_ptr(), to,
                                       _stream(stream)))
        return live


def get_device_status(stream=None):
    """Synchronizes the stream and returns (and clears) the sticky device status bits."""
    code = ctypes.c_int32(0)
    _check(lib().tq_get_device_status(_stream(stream), ctypes.byref(code)))
    return int(code.value)


def launch_count():
    """Kernels libtq has enqueued in this process (a launch captured in a graph counts once)."""
    return int(lib().tq_launch_count())
