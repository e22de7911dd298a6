"""Python binding of libqmm: GGUF block-quantized (Q4_K / Q5_K / Q6_K / Q8_0 / Q4_0 / Q3_K / IQ4_XS) x q8_1
matmul on MI355X.

Thin ctypes marshalling over the C ABI declared in include/qmm.h; every computation runs in the
library's HIP kernels.  Function names follow the C entry points without the ``qmm_`` prefix.
Tensors are torch tensors on a ROCm device; calls are enqueued on torch's current stream.
There is no CPU fallback: if libqmm.so is missing, importing this package raises.
"""
import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "qmm.h")

Q4_0 = 2
Q8_0 = 8
Q4_K = 12
Q5_K = 13
Q6_K = 14
Q3_K = 11
IQ4_XS = 23
F32, F16, BF16 = 0, 1, 30   # element types of the row operators
BLOCK_VALUES = {Q4_0: 32, Q8_0: 32, Q4_K: 256, Q5_K: 256, Q6_K: 256, Q3_K: 256, IQ4_XS: 256}
BLOCK_BYTES = {Q4_0: 18, Q8_0: 34, Q4_K: 144, Q5_K: 176, Q6_K: 210, Q3_K: 110, IQ4_XS: 136}
Q8_1_BYTES = 36

OVR_PATH, OVR_STREAMK, OVR_TILE_J, OVR_MV_STEPS, OVR_MV_KERNEL, OVR_FUSE_COLS = 1, 2, 3, 4, 5, 6
PATH_AUTO, PATH_MATVEC, PATH_TILED = 0, 1, 2

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m block_quantized_matmul_quantize_amd.build`")

# torch ships its own HIP runtime with the same soname as the system one; loading torch first
# makes libqmm bind to that already-loaded runtime, so one HIP runtime owns the device.
import torch  # noqa: E402,F401

_L = ctypes.CDLL(LIB_PATH)
_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t


class Plan(ctypes.Structure):
    _fields_ = [("regime", ctypes.c_int32), ("tile_i", ctypes.c_int32), ("tile_j", ctypes.c_int32),
                ("ntiles", ctypes.c_int64), ("efficiency_pct", ctypes.c_int32), ("stream_k", ctypes.c_int32),
                ("k_iters", ctypes.c_int64), ("units", ctypes.c_int64), ("fixup", ctypes.c_int32),
                ("ws_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


def _sig(name, res, *args):
    fn = getattr(_L, name)
    fn.restype = res
    fn.argtypes = list(args)
    return fn


_sig("qmm_last_error", ctypes.c_char_p)
_sig("qmm_version", ctypes.c_char_p)
_sig("qmm_quantize_q8_1", _i32, _vp, _i64, _i64, _vp, _vp)
_sig("qmm_matmul_workspace", _sz, _i32, _i64, _i64, _i64)
_sig("qmm_encode_f16act", _i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp)
_sig("qmm_matmul_f16act_workspace", _sz, _i64, _i64)
_sig("qmm_matmul_f16act", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_noalloc", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp)
_sig("qmm_repack_bytes", ctypes.c_uint64, _i32, _i64, _i64)
_sig("qmm_repack", _i32, _i32, _vp, _i64, _i64, _vp, ctypes.c_uint64, _vp)
_sig("qmm_matmul_packed_workspace", _sz, _i32, _i64, _i64, _i64)
_sig("qmm_matmul_packed", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_q8_1_workspace", _sz, _i32, _i64, _i64, _i64)
_sig("qmm_matmul_q8_1", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_id_workspace", _sz, _i32, _i64, _i64, _i64, _i64, _i64, _i64)
_sig("qmm_matmul_id", _i32, _i32, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_id_invalid_count", _i32, _vp, ctypes.POINTER(_i64), _vp)
_sig("qmm_matmul_glu_workspace", _sz, _i32, _i64, _i64, _i64)
_sig("qmm_matmul_glu", _i32, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_id_glu_workspace", _sz, _i32, _i64, _i64, _i64, _i64, _i64)
_sig("qmm_matmul_id_glu", _i32, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _sz, _vp)
_sig("qmm_matmul_id_grouping_layout", _i32, _i32, _i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_i64))
_sig("qmm_debug_subdots_workspace", _sz, _i32, _i64, _i64, _i64, _i32)
_sig("qmm_debug_subdots", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i32, _vp, _vp, _sz, _vp)
_sig("qmm_set_override", _i32, _i32, _i32)
_sig("qmm_plan_dense", _i32, _i32, _i64, _i64, _i64, ctypes.c_int32, ctypes.POINTER(Plan))
_sig("qmm_tile_efficiency", ctypes.c_int32, _i64, ctypes.c_int32)
_sig("qmm_select_tile_j", ctypes.c_int32, _i64)
_sig("qmm_streamk_unit_start", _i64, _i64, _i64, _i64, _i64)
_sig("qmm_sort_ids_workspace", _sz, _i64, _i64)
_sig("qmm_sort_ids", _i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("qmm_gather_sorted", _i32, _i32, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp)
_sig("qmm_combine", _i32, _i32, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp)
_sig("qmm_combine_backward", _i32, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp)
_sig("qmm_combine_ids", _i32, _i32, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp)
_sig("qmm_combine_ids_backward", _i32, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp)
_sig("qmm_embed", _i32, _i32, _vp, _i64, _i64, _vp, _i64, ctypes.c_float, _i32, _vp, _vp)
_sig("qmm_embed_backward_workspace", _sz, _i64, _i64, _i64)
_sig("qmm_embed_backward", _i32, _i32, _vp, _i64, _i64, _vp, _i64, ctypes.c_float, _i32, _vp, _vp, _sz, _vp)
_sig("qmm_lora_workspace", _sz, _i64, _i64, _i64, _i64, _i64)
_sig("qmm_lora", _i32, _i32, _i32, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("qmm_lora_backward_workspace", _sz, _i64, _i64, _i64, _i64, _i64)
_sig("qmm_lora_backward", _i32, _i32, _i32, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
     _vp, _vp, _vp, _sz, _vp)
_sig("qmm_matvec_kernel", _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i32, ctypes.POINTER(_i32))


class QmmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"qmm status {status}: {msg}")
        self.status = status


def _check(st):
    if st != 0:
        raise QmmError(st, _L.qmm_last_error().decode())


def lib():
    return _L


def header_symbols():
    """Entry points declared in include/qmm.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(qmm_[a-z0-9_]+)\s*\(", text)))


def version():
    return _L.qmm_version().decode()


# --------------------------------------------------------------------------------------------
# Host-side planner (no GPU needed)
# --------------------------------------------------------------------------------------------
def set_override(key, value):
    _check(_L.qmm_set_override(key, value))


def plan_dense(qtype, rows, k, n, nsm=256):
    p = Plan()
    _check(_L.qmm_plan_dense(qtype, rows, k, n, nsm, ctypes.byref(p)))
    return p.as_dict()


def tile_efficiency(ntiles, nsm):
    return int(_L.qmm_tile_efficiency(ntiles, nsm))


def select_tile_j(ncols):
    return int(_L.qmm_select_tile_j(ncols))


def streamk_unit_start(u, units, ntiles, k_iters):
    return int(_L.qmm_streamk_unit_start(u, units, ntiles, k_iters))


MV_KERNEL_NAMES = {1: "mmvq_kernel", 2: "mmvq_stream_kernel", 3: "mmvq_dot4_kernel"}


def matvec_kernel(qtype, w_ptr, rows, k, x_ptr, n, x_fp32=True):
    """(kernel id, fused) a dense call would launch: 0 tiled path, 1 register-streamed, 2
    LDS-staged MFMA, 3 dot4; fused = the kernel quantizes the fp32 activations itself.  Takes
    raw addresses (ints) or tensors; only their alignment matters."""
    w_ptr = w_ptr.data_ptr() if hasattr(w_ptr, "data_ptr") else int(w_ptr)
    x_ptr = x_ptr.data_ptr() if hasattr(x_ptr, "data_ptr") else int(x_ptr)
    out = _i32(0)
    _check(_L.qmm_matvec_kernel(qtype, w_ptr, rows, k, x_ptr, n, 1 if x_fp32 else 0, ctypes.byref(out)))
    return out.value & 15, bool(out.value & 16)


def matmul_workspace(qtype, rows, k, n):
    return int(_L.qmm_matmul_workspace(qtype, rows, k, n))


def matmul_q8_1_workspace(qtype, rows, k, n):
    return int(_L.qmm_matmul_q8_1_workspace(qtype, rows, k, n))


def matmul_id_workspace(qtype, n_exp, rows, k, n_tok, top_k, x_per_tok):
    return int(_L.qmm_matmul_id_workspace(qtype, n_exp, rows, k, n_tok, top_k, x_per_tok))


def matmul_glu_workspace(qtype, rows, k, n):
    return int(_L.qmm_matmul_glu_workspace(qtype, rows, k, n))


def matmul_id_glu_workspace(qtype, n_exp, rows, k, n_tok, top_k):
    return int(_L.qmm_matmul_id_glu_workspace(qtype, n_exp, rows, k, n_tok, top_k))


# --------------------------------------------------------------------------------------------
# Device entry points (torch tensors)
# --------------------------------------------------------------------------------------------
def _torch():
    return torch


# torch's own calls for the current device and its stream's handle: without the Stream object that
# torch.cuda.current_stream() makes, 3 us of a call.  They are not public, so a torch without them is
# asked through what is.
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _get_device is None or _get_raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _get_raw_stream(_get_device())


def _need(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _on_device(**tensors):
    """Last check before a pointer crosses the C ABI: every tensor lives in device memory."""
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")


def weight_bytes(qtype, rows, k):
    """Bytes of a [rows][k] weight matrix of GGUF blocks (ValueError for an unknown type or a k
    that is not a multiple of the block size)."""
    if qtype not in BLOCK_VALUES:
        raise ValueError(f"unsupported weight type {qtype}")
    if k <= 0 or k % BLOCK_VALUES[qtype]:
        raise ValueError(f"k={k} is not a positive multiple of the block size {BLOCK_VALUES[qtype]}")
    return rows * (k // BLOCK_VALUES[qtype]) * BLOCK_BYTES[qtype]


def _need_size(t, nbytes, name):
    """The C ABI receives bare pointers, so a tensor smaller than the shape it stands for would be
    read or written past its end on the device: refuse it here."""
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes, the call needs {nbytes}")


def _need_weights(t, qtype, rows, k, name, n_mat=1):
    """Size check of a weight tensor; an unknown type or a k the type cannot take is left to the
    library, which reports it as QMM_ERR_TYPE / QMM_ERR_SHAPE (QmmError)."""
    if qtype in BLOCK_VALUES and k > 0 and k % BLOCK_VALUES[qtype] == 0 and rows > 0:
        _need_size(t, n_mat * weight_bytes(qtype, rows, k), name)


def _workspace(nbytes, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def quantize_q8_1(x, out=None):
    """fp32 [n, k] -> uint8 [n, k/32*36] q8_1 blocks."""
    torch = _torch()
    px = _need(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [n, k]")
    n, k = x.shape
    if out is None:
        out = torch.empty((n, (k // 32) * Q8_1_BYTES), dtype=torch.uint8, device=x.device)
    py = _need(out, torch.uint8, "out")
    _need_size(out, n * (k // 32) * Q8_1_BYTES, "out")
    _on_device(x=x, out=out)
    _check(_L.qmm_quantize_q8_1(px, n, k, py, _stream()))
    return out


def matmul(w, qtype, rows, k, x, out=None, ws=None):
    """Y[n, rows] = W[rows, k] . X[n, k]^T with X quantized to q8_1 on the way."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [n, {k}]")
    n = x.shape[0]
    _need_weights(w, qtype, rows, k, "w")
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    nbytes = matmul_workspace(qtype, rows, k, n)
    if ws is None:
        ws = _workspace(nbytes, x.device)
    _on_device(w=w, x=x, out=out, ws=ws)
    _check(_L.qmm_matmul(qtype, pw, rows, k, px, n, py, ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out


def repack_bytes(qtype, rows, k):
    """Bytes of the panel layout of a [rows, k] matrix (0: type or shape not supported)."""
    return int(_L.qmm_repack_bytes(qtype, rows, k))


def repack(w, qtype, rows, k, out=None):
    """One-time repack of original blocks w into the panel layout (uint8 tensor on w's device)."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    _need_weights(w, qtype, rows, k, "w")
    nb = repack_bytes(qtype, rows, k)
    if out is None:
        out = torch.empty(max(nb, 16), dtype=torch.uint8, device=w.device)
    pp = _need(out, torch.uint8, "out")
    _on_device(w=w, out=out)
    _check(_L.qmm_repack(qtype, pw, rows, k, pp, out.numel(), _stream()))
    return out


def matmul_packed_workspace(qtype, rows, k, n):
    return int(_L.qmm_matmul_packed_workspace(qtype, rows, k, n))


def matmul_packed(wp, qtype, rows, k, x, out=None, ws=None):
    """matmul with the weights in the panel layout (from repack)."""
    torch = _torch()
    pw = _need(wp, torch.uint8, "wp")
    px = _need(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [n, {k}]")
    n = x.shape[0]
    need = repack_bytes(qtype, rows, k)
    if need:
        _need_size(wp, need, "wp")
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    nbytes = matmul_packed_workspace(qtype, rows, k, n)
    if ws is None:
        ws = _workspace(nbytes, x.device)
    _on_device(wp=wp, x=x, out=out, ws=ws)
    _check(_L.qmm_matmul_packed(qtype, pw, rows, k, px, n, py, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                _stream()))
    return out


def matmul_noalloc(w, qtype, rows, k, x, out=None):
    """matmul without a workspace argument: the library's own per-GPU scratch buffer holds it (the
    call allocates nothing itself, apart from `out` when it is not given)."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [n, {k}]")
    n = x.shape[0]
    _need_weights(w, qtype, rows, k, "w")
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    _on_device(w=w, x=x, out=out)
    _check(_L.qmm_matmul_noalloc(qtype, pw, rows, k, px, n, py, _stream()))
    return out


def encode_f16act(x):
    """fp16-activation mode encoder: fp32 [n, k] -> (fp16 bit patterns int16 [n, k], prescale
    exponents int32 [n, k/32], fp32 block sums [n, k/32])."""
    torch = _torch()
    px = _need(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [n, k]")
    n, k = x.shape
    y16 = torch.empty((n, k), dtype=torch.int16, device=x.device)
    e = torch.empty((n, k // 32), dtype=torch.int32, device=x.device)
    s = torch.empty((n, k // 32), dtype=torch.float32, device=x.device)
    _on_device(x=x)
    _check(_L.qmm_encode_f16act(px, n, k, ctypes.c_void_p(y16.data_ptr()), ctypes.c_void_p(e.data_ptr()),
                                ctypes.c_void_p(s.data_ptr()), _stream()))
    return y16, e, s


def matmul_f16act_workspace(k, n):
    return _L.qmm_matmul_f16act_workspace(k, n)


def matmul_f16act(w, qtype, rows, k, x, out=None, ws=None):
    """Y[n, rows] = W[rows, k] . X[n, k]^T in the fp16-activation mode (n <= 8)."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [n, {k}]")
    n = x.shape[0]
    _need_weights(w, qtype, rows, k, "w")
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    if ws is None:
        ws = _workspace(matmul_f16act_workspace(k, n), x.device)
    _on_device(w=w, x=x, out=out, ws=ws)
    _check(_L.qmm_matmul_f16act(qtype, pw, rows, k, px, n, py, ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out


def matmul_q8_1(w, qtype, rows, k, xq, n, out=None, ws=None):
    """Same product from q8_1 activations (uint8 [n, k/32*36])."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(xq, torch.uint8, "xq")
    if xq.numel() != n * (k // 32) * Q8_1_BYTES:
        raise ValueError("xq has the wrong number of bytes")
    _need_weights(w, qtype, rows, k, "w")
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=xq.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    nbytes = matmul_q8_1_workspace(qtype, rows, k, n)
    if ws is None:
        ws = _workspace(nbytes, xq.device)
    _on_device(w=w, xq=xq, out=out, ws=ws)
    _check(_L.qmm_matmul_q8_1(qtype, pw, rows, k, px, n, py, ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out


def matmul_id(w, qtype, n_exp, rows, k, x, ids, x_per_tok=1, out=None, ws=None):
    """Expert-indexed product.  x: fp32 [n_tok*x_per_tok, k]; ids: int32 [n_tok, top_k];
    returns y fp32 [n_tok, top_k, rows] (rows with an invalid id are left as they were in `out`)."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(x, torch.float32, "x")
    pi = _need(ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D [n_tok, top_k]")
    n_tok, top_k = ids.shape
    if x.shape != (n_tok * x_per_tok, k):
        raise ValueError(f"x must be [{n_tok * x_per_tok}, {k}]")
    _need_weights(w, qtype, rows, k, "w", n_exp)
    if out is None:
        out = torch.zeros((n_tok, top_k, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n_tok * top_k * rows * 4, "out")
    nbytes = matmul_id_workspace(qtype, n_exp, rows, k, n_tok, top_k, x_per_tok)
    if ws is None:
        ws = _workspace(nbytes, x.device)
    _on_device(w=w, x=x, ids=ids, out=out, ws=ws)
    _check(_L.qmm_matmul_id(qtype, pw, n_exp, rows, k, px, x_per_tok, pi, n_tok, top_k, py,
                            ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out, ws


def matmul_glu(w_gate, w_up, qtype, rows, k, x, out=None, ws=None):
    """Y[n, rows] = silu(W_gate . X^T) * (W_up . X^T), both products of X quantized to q8_1 once."""
    torch = _torch()
    pg = _need(w_gate, torch.uint8, "w_gate")
    pu = _need(w_up, torch.uint8, "w_up")
    if w_gate.numel() != w_up.numel():
        raise ValueError("w_gate and w_up must have the same size")
    _need_weights(w_gate, qtype, rows, k, "w_gate")
    px = _need(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [n, {k}]")
    n = x.shape[0]
    if out is None:
        out = torch.empty((n, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n * rows * 4, "out")
    if ws is None:
        ws = _workspace(matmul_glu_workspace(qtype, rows, k, n), x.device)
    _on_device(w_gate=w_gate, w_up=w_up, x=x, out=out, ws=ws)
    _check(_L.qmm_matmul_glu(qtype, pg, pu, rows, k, px, n, py, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                             _stream()))
    return out


def matmul_id_glu(w_gate, w_up, qtype, n_exp, rows, k, x, ids, out=None, ws=None):
    """Expert form of matmul_glu.  x: fp32 [n_tok, k]; ids: int32 [n_tok, top_k]; returns
    (y fp32 [n_tok, top_k, rows], ws) -- rows with an invalid id keep their value in `out`."""
    torch = _torch()
    pg = _need(w_gate, torch.uint8, "w_gate")
    pu = _need(w_up, torch.uint8, "w_up")
    if w_gate.numel() != w_up.numel():
        raise ValueError("w_gate and w_up must have the same size")
    _need_weights(w_gate, qtype, rows, k, "w_gate", n_exp)
    px = _need(x, torch.float32, "x")
    pi = _need(ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D [n_tok, top_k]")
    n_tok, top_k = ids.shape
    if x.shape != (n_tok, k):
        raise ValueError(f"x must be [{n_tok}, {k}]")
    if out is None:
        out = torch.zeros((n_tok, top_k, rows), dtype=torch.float32, device=x.device)
    py = _need(out, torch.float32, "out")
    _need_size(out, n_tok * top_k * rows * 4, "out")
    if ws is None:
        ws = _workspace(matmul_id_glu_workspace(qtype, n_exp, rows, k, n_tok, top_k), x.device)
    _on_device(w_gate=w_gate, w_up=w_up, x=x, ids=ids, out=out, ws=ws)
    _check(_L.qmm_matmul_id_glu(qtype, pg, pu, n_exp, rows, k, px, pi, n_tok, top_k, py,
                                ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out, ws


def matmul_id_invalid_count(ws):
    v = _i64(0)
    _check(_L.qmm_matmul_id_invalid_count(ctypes.c_void_p(ws.data_ptr()), ctypes.byref(v), _stream()))
    return int(v.value)


def matmul_id_layout(qtype, n_exp, k, n_tok, top_k, x_per_tok=1):
    """Host logic only: workspace byte offsets of the expert grouping (sorted, bounds, tile_start,
    small), the column-tile width and the small-expert limit a matmul_id of this shape uses."""
    out = (_i64 * 6)()
    _check(_L.qmm_matmul_id_grouping_layout(qtype, n_exp, k, n_tok, top_k, x_per_tok, out))
    return tuple(int(v) for v in out)


def matmul_id_grouping(ws, qtype, n_exp, k, n_tok, top_k, x_per_tok=1):
    """Expert grouping the last matmul_id with workspace `ws` built (synchronizes the stream):
    dict of int32 CPU tensors sorted, bounds, tile_start, small, plus tile_j and small_max."""
    torch = _torch()
    out = matmul_id_layout(qtype, n_exp, k, n_tok, top_k, x_per_tok)
    torch.cuda.current_stream().synchronize()
    pairs = n_tok * top_k
    raw = ws.view(torch.uint8)

    def take(off, count):
        return raw[off:off + 4 * count].view(torch.int32).cpu()

    return {"sorted": take(out[0], pairs), "bounds": take(out[1], n_exp + 1), "tile_start": take(out[2], n_exp + 1),
            "small": take(out[3], n_exp), "tile_j": int(out[4]), "small_max": int(out[5])}


def debug_subdots_workspace(qtype, rows, k, n, path):
    return int(_L.qmm_debug_subdots_workspace(qtype, rows, k, n, path))


def debug_subdots(w, qtype, rows, k, xq, n, path):
    """Integer sub-block dots from the chosen production kernel in its production plan: int32
    [n, rows, per]."""
    torch = _torch()
    pw = _need(w, torch.uint8, "w")
    px = _need(xq, torch.uint8, "xq")
    _need_weights(w, qtype, rows, k, "w")
    _need_size(xq, n * (k // 32) * Q8_1_BYTES, "xq")
    per = k // 16 if (qtype in (Q6_K, Q3_K) and path == PATH_MATVEC) else k // 32
    out = torch.zeros((n, rows, per), dtype=torch.int32, device=xq.device)
    ws = _workspace(debug_subdots_workspace(qtype, rows, k, n, path), xq.device)
    _on_device(w=w, xq=xq, out=out, ws=ws)
    _check(_L.qmm_debug_subdots(qtype, pw, rows, k, px, n, path, ctypes.c_void_p(out.data_ptr()),
                                ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream()))
    return out


# --------------------------------------------------------------------------------------------
# Row operators: embedding, expert gather / combine, low-rank adapters (and their gradients)
#
# Like the products' calls, these are not recorded by autograd: a result requires no gradient, whatever
# its inputs do.  A training step calls the *_backward functions itself.
# --------------------------------------------------------------------------------------------
_ELEM_TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_ELEM_DTYPES = {v: d for d, v in _ELEM_TYPES.items()}


def _elem(t, name):
    """Element type of a contiguous fp32, fp16 or bf16 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    e = _ELEM_TYPES.get(t.dtype)
    if e is None:
        raise TypeError(f"{name} must have dtype float32, float16 or bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return e


def _int32(t, name):
    """Address of a contiguous int32 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must have dtype torch.int32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _arg(t, dtype, shape, name):
    """Address of a contiguous tensor of this dtype and shape (None: a null pointer)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _same_device(first, *others):
    """Last check before pointers cross the C ABI: every tensor lives on the first one's device, and that is
    the current one, on whose stream the call is enqueued."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("every tensor must be a device tensor")
    current = torch.cuda.current_device() if _get_device is None else _get_device()
    if dev != current:
        raise ValueError(f"the tensors are on {first.device}, but the current device is {current}: "
                         f"call within torch.cuda.device({dev})")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on {first.device}, got {t.device}")


def _ws_args(ws, nbytes, like):
    """(address, bytes, tensor to keep until the launch) of a workspace of at least nbytes on the device
    of a tensor."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = like.new_empty(nbytes, dtype=torch.uint8)
        return ws.data_ptr(), nbytes, ws
    _need(ws, torch.uint8, "ws")
    _same_device(like, ws)
    return ws.data_ptr(), ws.numel(), ws


def sort_ids_workspace(n, n_keys):
    return int(_L.qmm_sort_ids_workspace(n, n_keys))


def sort_ids(ids, n_keys, ws=None):
    """Stable sort of int32 ids (any shape).  Returns int32 (order [n], pos of ids' shape,
    bounds [n_keys + 1]): indices by id with ids outside [0, n_keys) last, each index's place in
    order (-1 for an id outside), and the start of each id's segment."""
    pi = _int32(ids, "ids")
    if n_keys < 1:
        raise ValueError(f"n_keys must be >= 1, got {n_keys}")
    _same_device(ids)
    n = ids.numel()
    order, pos, bounds = ids.new_empty(n), torch.empty_like(ids), ids.new_empty(n_keys + 1)
    pw, nw, ws = _ws_args(ws, _L.qmm_sort_ids_workspace(n, n_keys), ids)
    st = _L.qmm_sort_ids(pi, n, n_keys, order.data_ptr(), pos.data_ptr(), bounds.data_ptr(), pw, nw, _stream())
    if st:
        _check(st)
    return order, pos, bounds


def _valid_count(bounds):
    """Address of the number of valid ids: the last entry of sort_ids' bounds."""
    p = _int32(bounds, "bounds")
    if bounds.dim() != 1 or bounds.numel() < 2:
        raise ValueError("bounds must be 1-D [n_keys + 1]")
    return p + 4 * (bounds.numel() - 1)


def _need_pos(pos, name="pos"):
    if pos.dim() != 2 or pos.shape[1] < 1:
        raise ValueError(f"{name} must be 2-D [n_tok, top_k]")
    return pos.shape


def gather_sorted(x, pos, bounds, out=None):
    """Rows to expert order: out[pos[t, j]] = x[t] for x [n_tok, k] and sort_ids' pos [n_tok, top_k];
    rows of out [n_tok * top_k, k] past the valid pairs are zeros.  Not recorded by autograd; its
    gradient: combine(d_out, pos)."""
    e = _elem(x, "x")
    pp = _int32(pos, "pos")
    n_tok, top_k = _need_pos(pos)
    if x.dim() != 2 or x.shape[0] != n_tok:
        raise ValueError(f"x must be [{n_tok}, k]")
    k = x.shape[1]
    nv = _valid_count(bounds)
    po = _arg(out, x.dtype, (n_tok * top_k, k), "out")
    _same_device(x, pos, bounds, out)
    if out is None:
        out = x.new_empty((n_tok * top_k, k))
        po = out.data_ptr()
    st = _L.qmm_gather_sorted(e, x.data_ptr(), n_tok, top_k, k, pp, nv, po, _stream())
    if st:
        _check(st)
    return out


def _pair_ids(ids, n_exp, shape):
    """Address of matmul_id's ids [n_tok, top_k] (None: a null pointer)."""
    if ids is None:
        return None
    if n_exp is None or n_exp < 1:
        raise ValueError(f"n_exp must be >= 1 beside ids, got {n_exp}")
    return _arg(ids, torch.int32, shape, "ids")


def combine(h, pos=None, weights=None, base=None, out=None, ids=None, n_exp=None):
    """out[t] = base[t] + sum over j of weights[t, j] * h[pos[t, j]].  h: [n_tok * top_k, k] in expert
    order with pos int32 [n_tok, top_k] (entries outside the rows add nothing), or, without pos, in
    (token, slot) order [n_tok, top_k, k] as matmul_id returns it.  There ids and n_exp are matmul_id's:
    pairs whose id is outside [0, n_exp), whose rows it leaves as they were, add nothing; without ids
    every row counts.  weights: fp32 [n_tok, top_k] (None: ones); base: [n_tok, k] or None; out may be
    base.  Not recorded by autograd; its gradient: combine_backward."""
    e = _elem(h, "h")
    if ids is not None and pos is not None:
        raise ValueError("ids are of h in (token, slot) order, without pos")
    if pos is None:
        if h.dim() != 3 or h.shape[1] < 1:
            raise ValueError("h must be 3-D [n_tok, top_k, k] where pos is None")
        n_tok, top_k, k = h.shape
        pp = None
    else:
        pp = _int32(pos, "pos")
        n_tok, top_k = _need_pos(pos)
        if h.dim() != 2 or h.shape[0] != n_tok * top_k:
            raise ValueError(f"h must be [{n_tok * top_k}, k]")
        k = h.shape[1]
    pi = _pair_ids(ids, n_exp, (n_tok, top_k))
    pw = _arg(weights, torch.float32, (n_tok, top_k), "weights")
    pb = _arg(base, h.dtype, (n_tok, k), "base")
    po = _arg(out, h.dtype, (n_tok, k), "out")
    _same_device(h, pos, weights, base, out, ids)
    if out is None:
        out = h.new_empty((n_tok, k))
        po = out.data_ptr()
    if ids is None:
        st = _L.qmm_combine(e, h.data_ptr(), n_tok, top_k, k, pp, pw, pb, po, _stream())
    else:
        st = _L.qmm_combine_ids(e, h.data_ptr(), n_tok, top_k, k, pi, n_exp, pw, pb, po, _stream())
    if st:
        _check(st)
    return out


def combine_backward(dy, h, pos=None, weights=None, bounds=None, ids=None, n_exp=None):
    """Gradient of combine: (dh of h's shape and dtype, fp32 dw [n_tok, top_k]); dy [n_tok, k].  With pos,
    bounds is sort_ids' (rows of dh past the valid pairs are zeros).  With ids and n_exp, dh and dw of a
    pair whose id is outside [0, n_exp) are zeros.  The gradient of base is dy."""
    e = _elem(h, "h")
    if ids is not None and pos is not None:
        raise ValueError("ids are of h in (token, slot) order, without pos")
    if pos is None:
        if h.dim() != 3 or h.shape[1] < 1:
            raise ValueError("h must be 3-D [n_tok, top_k, k] where pos is None")
        n_tok, top_k, k = h.shape
        pp = nv = None
    else:
        pp = _int32(pos, "pos")
        n_tok, top_k = _need_pos(pos)
        if h.dim() != 2 or h.shape[0] != n_tok * top_k:
            raise ValueError(f"h must be [{n_tok * top_k}, k]")
        k = h.shape[1]
        nv = _valid_count(bounds)
    pi = _pair_ids(ids, n_exp, (n_tok, top_k))
    pd = _arg(dy, h.dtype, (n_tok, k), "dy")
    pw = _arg(weights, torch.float32, (n_tok, top_k), "weights")
    _same_device(h, dy, pos, weights, bounds, ids)
    dh = torch.empty_like(h)
    dw = h.new_empty((n_tok, top_k), dtype=torch.float32)
    if ids is None:
        st = _L.qmm_combine_backward(e, pd, h.data_ptr(), n_tok, top_k, k, pp, pw, nv, dh.data_ptr(), dw.data_ptr(),
                                     _stream())
    else:
        st = _L.qmm_combine_ids_backward(e, pd, h.data_ptr(), n_tok, top_k, k, pi, n_exp, pw, dh.data_ptr(),
                                         dw.data_ptr(), _stream())
    if st:
        _check(st)
    return dh, dw


def embed(table, qtype, vocab, k, ids, scale=1.0, dtype=torch.float32, out=None):
    """out[i] = scale * table[ids[i]] (zeros for an id outside [0, vocab)).  table: fp32, fp16 or bf16
    [vocab, k] (qtype F32, F16, BF16), or uint8 rows of GGUF blocks; ids int32 of any shape; out
    ids.shape + [k] of dtype, from blocks at a 16-byte aligned address.  With ids 0 .. vocab - 1 it
    expands a block-quantized matrix.  Not recorded by autograd; its gradient with respect to a table
    of elements: embed_backward."""
    pi = _int32(ids, "ids")
    tt = _ELEM_DTYPES.get(qtype)
    pt = _need(table, torch.uint8 if tt is None else tt, "table")
    if tt is None:
        _need_weights(table, qtype, vocab, k, "table")
    else:
        _need_size(table, vocab * k * table.element_size(), "table")
    e = _ELEM_TYPES.get(dtype)
    if e is None:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    shape = (*ids.shape, k)
    po = _arg(out, dtype, shape, "out")
    _same_device(ids, table, out)
    if out is None:
        out = ids.new_empty(shape, dtype=dtype)
        po = out.data_ptr()
    st = _L.qmm_embed(qtype, pt, vocab, k, pi, ids.numel(), scale, e, po, _stream())
    if st:
        _check(st)
    return out


def embed_backward_workspace(n, k, vocab):
    return int(_L.qmm_embed_backward_workspace(n, k, vocab))


def embed_backward(dy, ids, vocab, scale=1.0, dtype=torch.float32, out=None, ws=None):
    """Gradient of embed with respect to a table of elements: [vocab, k] of dtype, every row written;
    dy: ids.shape + [k]."""
    e = _elem(dy, "dy")
    pi = _int32(ids, "ids")
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        raise ValueError(f"dy must be {list(ids.shape)} + [k]")
    g = _ELEM_TYPES.get(dtype)
    if g is None:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    if vocab < 1:
        raise ValueError(f"vocab must be >= 1, got {vocab}")
    n, k = ids.numel(), dy.shape[-1]
    po = _arg(out, dtype, (vocab, k), "out")
    _same_device(dy, ids, out)
    if out is None:
        out = dy.new_empty((vocab, k), dtype=dtype)
        po = out.data_ptr()
    pw, nw, ws = _ws_args(ws, _L.qmm_embed_backward_workspace(n, k, vocab), dy)
    st = _L.qmm_embed_backward(e, dy.data_ptr(), n, k, pi, vocab, scale, g, po, pw, nw, _stream())
    if st:
        _check(st)
    return out


def _lora_shapes(x, a, b, ids, scale):
    e, w = _elem(x, "x"), _elem(a, "a")
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [n, k], a [n_adapters, rank, k] and b [n_adapters, rows, rank]")
    n, k = x.shape
    na, rank, rows = a.shape[0], a.shape[1], b.shape[1]
    _arg(a, a.dtype, (na, rank, k), "a")
    _arg(b, a.dtype, (na, rows, rank), "b")
    _arg(ids, torch.int32, (n,), "ids")
    ps = _arg(scale, torch.float32, (na,), "scale")
    return e, w, n, k, na, rank, rows, ps


def lora_workspace(n, k, rows, rank, n_adapters):
    return int(_L.qmm_lora_workspace(n, k, rows, rank, n_adapters))


def lora(x, a, b, ids, scale=None, base=None, out=None, keep_h=False, ws=None):
    """out[i] = base[i] + scale[c] * b[c] @ (a[c] @ x[i]) with c = ids[i]; base[i] alone for a c outside
    [0, n_adapters).  x [n, k] and base, out [n, rows] of one dtype; a [n_adapters, rank, k] and
    b [n_adapters, rows, rank] of x's dtype (beside fp32 x: any); ids int32 [n]; scale fp32
    [n_adapters]; out may be base.  Rows of one adapter are fastest as neighbours.  keep_h: returns
    (out, fp32 a[c] @ x[i] [n, rank]) for lora_backward: autograd does not record the call."""
    e, w, n, k, na, rank, rows, ps = _lora_shapes(x, a, b, ids, scale)
    pb = _arg(base, x.dtype, (n, rows), "base")
    po = _arg(out, x.dtype, (n, rows), "out")
    _same_device(x, a, b, ids, scale, base, out)
    if out is None:
        out = x.new_empty((n, rows))
        po = out.data_ptr()
    h = x.new_empty((n, rank), dtype=torch.float32) if keep_h else None
    pw, nw, ws = _ws_args(ws, _L.qmm_lora_workspace(n, k, rows, rank, na), x)
    st = _L.qmm_lora(e, w, x.data_ptr(), n, k, a.data_ptr(), b.data_ptr(), rows, rank, na, ids.data_ptr(), ps, pb, po,
                     h.data_ptr() if keep_h else None, pw, nw, _stream())
    if st:
        _check(st)
    return (out, h) if keep_h else out


def lora_backward_workspace(n, k, rows, rank, n_adapters):
    return int(_L.qmm_lora_backward_workspace(n, k, rows, rank, n_adapters))


def lora_backward(x, dy, h, a, b, ids, scale=None, dx_base=None, need_dx=True, need_dw=True, ws=None):
    """Gradient of lora: (dx [n, k] of x's dtype, fp32 da and db of a's and b's shapes).  h is what lora
    kept; dx_base [n, k] or None is what the projection itself contributes to dx.  need_dx, need_dw:
    False leaves dx, or da and db, out (None)."""
    e, w, n, k, na, rank, rows, ps = _lora_shapes(x, a, b, ids, scale)
    pd = _arg(dy, x.dtype, (n, rows), "dy")
    ph = _arg(h, torch.float32, (n, rank), "h")
    px = _arg(dx_base, x.dtype, (n, k), "dx_base")
    _same_device(x, a, b, ids, scale, dy, h, dx_base)
    dx = torch.empty_like(x) if need_dx else None
    da = a.new_empty(a.shape, dtype=torch.float32) if need_dw else None
    db = b.new_empty(b.shape, dtype=torch.float32) if need_dw else None
    pw, nw, ws = _ws_args(ws, _L.qmm_lora_backward_workspace(n, k, rows, rank, na), x)
    st = _L.qmm_lora_backward(e, w, x.data_ptr(), pd, ph, n, k, a.data_ptr(), b.data_ptr(), rows, rank, na, ids.data_ptr(),
                              ps, px, dx.data_ptr() if need_dx else None, da.data_ptr() if need_dw else None,
                              db.data_ptr() if need_dw else None, pw, nw, _stream())
    if st:
        _check(st)
    return dx, da, db
