"""Python binding of libhxq, the B200 (sm_100a) HelixLinear forward.

The C ABI (include/hxq.h) is the product: this module only marshals
arguments. Every step of the forward runs in the library's CUDA kernels;
there is no Python or CPU fallback, and importing fails loudly when the
library has not been built (python vq_compressed_linear_b200/build.py).

PyTorch is used for device memory and streams only: tensors are passed by
data pointer, the current torch stream is passed as the cudaStream_t.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhxq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libhxq.so is missing at {LIB_PATH}: build it with "
        "`python vq_compressed_linear_b200/build.py` (nvcc, sm_100a)")

lib = ctypes.CDLL(LIB_PATH)

HXQ_MODE_SCALAR8 = 0
HXQ_MODE_VQ2D12 = 1
HXQ_OK = 0
HXQ_EINVAL = -1
HXQ_ENOMEM = -2
HXQ_ECUDA = -3
HXQ_EUNSUPPORTED = -4
HXQ_ETIMEOUT = -5
HXQ_KERNEL_AUTO = 0
HXQ_KERNEL_GEMV = 1
HXQ_KERNEL_TC = 2
HXQ_OUT_F32 = 0
HXQ_OUT_BF16 = 1
HXQ_MAX_GROUP = 4
HXQ_TYPE_F32 = 0
HXQ_TYPE_BF16 = 1
HXQ_FP8_MAX_EXPERTS = 1024

_vp, _i, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
lib.hxq_linear_create.argtypes = [_vp, _vp, _i, _vp, _vp, _i64, _i, _i, ctypes.POINTER(_vp)]
lib.hxq_linear_create.restype = _i
lib.hxq_linear_forward.argtypes = [_vp, _vp, _vp, _i, _vp]
lib.hxq_linear_forward.restype = _i
lib.hxq_linear_forward_ex.argtypes = [_vp, _vp, _vp, _i, _i, _i, _vp]
lib.hxq_linear_forward_ex.restype = _i
lib.hxq_linear_forward_out.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _vp]
lib.hxq_linear_forward_out.restype = _i
lib.hxq_linear_forward_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp]
lib.hxq_linear_forward_host.restype = _i
lib.hxq_linear_forward_noalloc.argtypes = [_vp, _vp, _vp, _i, _vp]
lib.hxq_linear_forward_noalloc.restype = _i
lib.hxq_decode.argtypes = [_vp, _vp, _vp]
lib.hxq_decode.restype = _i
lib.hxq_linear_check.argtypes = [_vp]
lib.hxq_linear_check.restype = _i
lib.hxq_test_forward_withheld.argtypes = [_vp, _vp, _vp, _i, _i, ctypes.c_uint, _vp]
lib.hxq_test_forward_withheld.restype = _i
lib.hxq_linear_info.argtypes = [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i),
                                ctypes.POINTER(_i64)]
lib.hxq_linear_info.restype = _i
lib.hxq_group_create.argtypes = [ctypes.POINTER(_vp), _i, ctypes.POINTER(_vp)]
lib.hxq_group_create.restype = _i
lib.hxq_group_forward.argtypes = [_vp, _vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i, _i, _vp]
lib.hxq_group_forward.restype = _i
lib.hxq_group_destroy.argtypes = [_vp]
lib.hxq_group_destroy.restype = None
lib.hxq_assign.argtypes = [_vp, _i64, _i, _vp, _i, _vp, _vp]
lib.hxq_assign.restype = _i
lib.hxq_kmeans.argtypes = [_vp, _i64, _i, _i, _i, _vp, _vp, _vp]
lib.hxq_kmeans.restype = _i
lib.hxq_encode.argtypes = [_vp, _i, _i, _i, _vp, ctypes.c_float, _vp, _vp, _vp, _i64, _vp, _vp]
lib.hxq_encode.restype = _i
lib.hxq_fp8_ld.argtypes = [_i]
lib.hxq_fp8_ld.restype = _i64
lib.hxq_fp8_quantize.argtypes = [_vp, _i, _i64, _i, _vp, _vp, _vp]
lib.hxq_fp8_quantize.restype = _i
lib.hxq_fp8_swiglu.argtypes = [_vp, _i, _i64, _i, _vp, _vp, _vp]
lib.hxq_fp8_swiglu.restype = _i
lib.hxq_fp8_encode.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp]
lib.hxq_fp8_encode.restype = _i
lib.hxq_rmsnorm.argtypes = [_vp, _i, _vp, _vp, _i, _vp, ctypes.c_float, _i64, _i, _vp, _vp, _vp, _vp]
lib.hxq_rmsnorm.restype = _i
lib.hxq_fp8_create.argtypes = [_vp, _vp, _i, _i, _i, ctypes.POINTER(_vp)]
lib.hxq_fp8_create.restype = _i
lib.hxq_fp8_forward.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp]
lib.hxq_fp8_forward.restype = _i
lib.hxq_fp8_forward_grouped.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp]
lib.hxq_fp8_forward_grouped.restype = _i
lib.hxq_fp8_info.argtypes = [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i)]
lib.hxq_fp8_info.restype = _i
lib.hxq_fp8_check.argtypes = [_vp]
lib.hxq_fp8_check.restype = _i
lib.hxq_test_fp8_forward_withheld.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_uint, _vp]
lib.hxq_test_fp8_forward_withheld.restype = _i
lib.hxq_fp8_destroy.argtypes = [_vp]
lib.hxq_fp8_destroy.restype = None
lib.hxq_linear_destroy.argtypes = [_vp]
lib.hxq_linear_destroy.restype = None
lib.hxq_strerror.argtypes = [_i]
lib.hxq_strerror.restype = ctypes.c_char_p

EXPORTED = ("hxq_linear_create", "hxq_linear_forward", "hxq_linear_forward_ex", "hxq_linear_forward_out",
            "hxq_linear_forward_host", "hxq_linear_forward_noalloc", "hxq_group_create", "hxq_group_forward", "hxq_group_destroy", "hxq_assign", "hxq_kmeans", "hxq_encode", "hxq_decode",
            "hxq_linear_check", "hxq_test_forward_withheld", "hxq_linear_info", "hxq_linear_destroy",
            "hxq_fp8_ld", "hxq_fp8_quantize", "hxq_fp8_swiglu", "hxq_fp8_encode", "hxq_rmsnorm", "hxq_fp8_create",
            "hxq_fp8_forward", "hxq_fp8_forward_grouped", "hxq_fp8_info", "hxq_fp8_check",
            "hxq_test_fp8_forward_withheld", "hxq_fp8_destroy",
            "hxq_strerror")


class HXQError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {hxq_strerror(code)} ({code})")


def _check(code: int, what: str) -> None:
    if code != HXQ_OK:
        raise HXQError(code, what)


def _ptr(t) -> int | None:
    """Data pointer of a tensor / ndarray, or None."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def _stream(stream) -> int | None:
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    import torch
    return torch.cuda.current_stream().cuda_stream


# ---- same names as the C ABI -------------------------------------------------

def hxq_strerror(code: int) -> str:
    return lib.hxq_strerror(int(code)).decode()


def hxq_linear_create(codebook, indices, mode, sidecar_pos, sidecar_val, n_sidecar, N, K) -> int:
    """Returns the handle (an integer); raises HXQError on failure."""
    h = _vp()
    _check(lib.hxq_linear_create(_ptr(codebook), _ptr(indices), int(mode), _ptr(sidecar_pos),
                                 _ptr(sidecar_val), int(n_sidecar), int(N), int(K), ctypes.byref(h)),
           "hxq_linear_create")
    return h.value


def hxq_linear_forward(h, x, y, M, stream=None) -> None:
    _check(lib.hxq_linear_forward(h, _ptr(x), _ptr(y), int(M), _stream(stream)), "hxq_linear_forward")


def hxq_linear_forward_ex(h, x, y, M, kernel, split_k, stream=None) -> None:
    _check(lib.hxq_linear_forward_ex(h, _ptr(x), _ptr(y), int(M), int(kernel), int(split_k),
                                     _stream(stream)), "hxq_linear_forward_ex")


def hxq_linear_forward_out(h, x, bias, y, out_dtype, M, stream=None) -> None:
    _check(lib.hxq_linear_forward_out(h, _ptr(x), _ptr(bias), _ptr(y), int(out_dtype), int(M), _stream(stream)),
           "hxq_linear_forward_out")


def hxq_linear_forward_host(h, x_host, x_dev, y_dev, y_host, M, stream=None) -> None:
    _check(lib.hxq_linear_forward_host(h, _ptr(x_host), _ptr(x_dev), _ptr(y_dev), _ptr(y_host), int(M),
                                       _stream(stream)), "hxq_linear_forward_host")


def hxq_linear_forward_noalloc(h, x, y, M, stream=None) -> None:
    _check(lib.hxq_linear_forward_noalloc(h, _ptr(x), _ptr(y), int(M), _stream(stream)),
           "hxq_linear_forward_noalloc")


def _ptr_array(ts):
    """A C array of data pointers (None entries stay NULL), or NULL for None."""
    if ts is None:
        return None
    return (_vp * len(ts))(*[_ptr(t) for t in ts])


def hxq_group_create(handles) -> int:
    """Returns the group (an integer); raises HXQError on failure."""
    g = _vp()
    arr = (_vp * len(handles))(*handles)
    _check(lib.hxq_group_create(arr, len(handles), ctypes.byref(g)), "hxq_group_create")
    return g.value


def hxq_group_forward(g, x, biases, ys, out_dtype, M, stream=None) -> None:
    _check(lib.hxq_group_forward(g, _ptr(x), _ptr_array(biases), _ptr_array(ys), int(out_dtype), int(M),
                                 _stream(stream)), "hxq_group_forward")


def hxq_group_destroy(g) -> None:
    lib.hxq_group_destroy(g)


def hxq_assign(points, n, dim, centroids, k, labels, stream=None) -> None:
    _check(lib.hxq_assign(_ptr(points), int(n), int(dim), _ptr(centroids), int(k), _ptr(labels), _stream(stream)),
           "hxq_assign")


def hxq_kmeans(points, n, dim, k, iters, centroids, labels, stream=None) -> None:
    _check(lib.hxq_kmeans(_ptr(points), int(n), int(dim), int(k), int(iters), _ptr(centroids), _ptr(labels),
                          _stream(stream)), "hxq_kmeans")


def hxq_encode(W, mode, N, K, codebook, threshold, indices, sidecar_pos, sidecar_val, max_sidecar, n_sidecar,
               stream=None) -> None:
    _check(lib.hxq_encode(_ptr(W), int(mode), int(N), int(K), _ptr(codebook), float(threshold), _ptr(indices),
                          _ptr(sidecar_pos), _ptr(sidecar_val), int(max_sidecar), _ptr(n_sidecar),
                          _stream(stream)), "hxq_encode")


def hxq_decode(h, W_out, stream=None) -> None:
    _check(lib.hxq_decode(h, _ptr(W_out), _stream(stream)), "hxq_decode")


def hxq_linear_check(h) -> None:
    _check(lib.hxq_linear_check(h), "hxq_linear_check")


def hxq_test_forward_withheld(h, x, y, M, withhold_item, wait_limit_us, stream=None) -> None:
    """Test hook: the tensor-core forward with one item's activations withheld
    and every pipeline wait bounded at wait_limit_us (the next
    hxq_linear_check reports HXQ_ETIMEOUT)."""
    _check(lib.hxq_test_forward_withheld(h, _ptr(x), _ptr(y), int(M), int(withhold_item), int(wait_limit_us),
                                         _stream(stream)), "hxq_test_forward_withheld")


def hxq_linear_info(h) -> tuple[int, int, int, int]:
    m, n, k, s = _i(), _i(), _i(), _i64()
    _check(lib.hxq_linear_info(h, ctypes.byref(m), ctypes.byref(n), ctypes.byref(k), ctypes.byref(s)),
           "hxq_linear_info")
    return m.value, n.value, k.value, s.value


def hxq_linear_destroy(h) -> None:
    lib.hxq_linear_destroy(h)


def hxq_fp8_ld(K) -> int:
    return lib.hxq_fp8_ld(int(K))


def hxq_fp8_quantize(x, x_type, rows, cols, q, scales, stream=None) -> None:
    _check(lib.hxq_fp8_quantize(_ptr(x), int(x_type), int(rows), int(cols), _ptr(q), _ptr(scales), _stream(stream)),
           "hxq_fp8_quantize")


def hxq_fp8_swiglu(gate_up, type, rows, cols, q, scales, stream=None) -> None:
    _check(lib.hxq_fp8_swiglu(_ptr(gate_up), int(type), int(rows), int(cols), _ptr(q), _ptr(scales),
                              _stream(stream)), "hxq_fp8_swiglu")


def hxq_fp8_encode(W, type, n_experts, N, K, q, scales, stream=None) -> None:
    _check(lib.hxq_fp8_encode(_ptr(W), int(type), int(n_experts), int(N), int(K), _ptr(q), _ptr(scales),
                              _stream(stream)), "hxq_fp8_encode")


def hxq_rmsnorm(x, x_type, residual, sum, residual_type, weight, eps, rows, cols, y_bf16, q, scales,
                stream=None) -> None:
    _check(lib.hxq_rmsnorm(_ptr(x), int(x_type), _ptr(residual), _ptr(sum), int(residual_type), _ptr(weight),
                           float(eps), int(rows), int(cols), _ptr(y_bf16), _ptr(q), _ptr(scales), _stream(stream)),
           "hxq_rmsnorm")


def hxq_fp8_create(W, scales, n_experts, N, K) -> int:
    """Returns the handle (an integer); raises HXQError on failure."""
    h = _vp()
    _check(lib.hxq_fp8_create(_ptr(W), _ptr(scales), int(n_experts), int(N), int(K), ctypes.byref(h)),
           "hxq_fp8_create")
    return h.value


def hxq_fp8_forward(h, xq, xs, bias, y, out_type, M, stream=None) -> None:
    _check(lib.hxq_fp8_forward(h, _ptr(xq), _ptr(xs), _ptr(bias), _ptr(y), int(out_type), int(M), _stream(stream)),
           "hxq_fp8_forward")


def hxq_fp8_forward_grouped(h, xq, xs, offsets, bias, y, out_type, M, stream=None) -> None:
    _check(lib.hxq_fp8_forward_grouped(h, _ptr(xq), _ptr(xs), _ptr(offsets), _ptr(bias), _ptr(y), int(out_type),
                                       int(M), _stream(stream)), "hxq_fp8_forward_grouped")


def hxq_fp8_info(h) -> tuple[int, int, int]:
    e, n, k = _i(), _i(), _i()
    _check(lib.hxq_fp8_info(h, ctypes.byref(e), ctypes.byref(n), ctypes.byref(k)), "hxq_fp8_info")
    return e.value, n.value, k.value


def hxq_fp8_check(h) -> None:
    _check(lib.hxq_fp8_check(h), "hxq_fp8_check")


def hxq_test_fp8_forward_withheld(h, xq, xs, offsets, y, M, withhold_stage, wait_limit_us, stream=None) -> None:
    """Test hook: a product with one stage's activations withheld (-1: none) and
    every pipeline wait bounded at wait_limit_us (the next hxq_fp8_check
    reports HXQ_ETIMEOUT)"""
    _check(lib.hxq_test_fp8_forward_withheld(h, _ptr(xq), _ptr(xs), _ptr(offsets), _ptr(y), int(M),
                                             int(withhold_stage), int(wait_limit_us), _stream(stream)),
           "hxq_test_fp8_forward_withheld")


def hxq_fp8_destroy(h) -> None:
    lib.hxq_fp8_destroy(h)


# ---- convenience wrapper -----------------------------------------------------

class HelixLinear:
    """A compressed nn.Linear-shaped layer owned by libhxq.

    Arguments are tensors or arrays in the C ABI's layouts (host or device);
    the handle copies them. forward() takes x as a CUDA bf16 (or raw uint16 /
    int16 bit pattern) tensor [M, K] and returns float32 y [M, N].
    """

    def __init__(self, codebook, indices, mode, sidecar_pos, sidecar_val, N, K):
        n_sidecar = 0 if sidecar_pos is None else int(len(sidecar_pos))
        if n_sidecar == 0:
            sidecar_pos = sidecar_val = None
        self.mode, self.N, self.K = int(mode), int(N), int(K)
        self.handle = hxq_linear_create(codebook, indices, mode, sidecar_pos, sidecar_val,
                                        n_sidecar, N, K)

    @classmethod
    def from_layer(cls, layer: dict) -> "HelixLinear":
        return cls(layer["codebook"], layer["indices"], layer["mode"], layer["sidecar_pos"],
                   layer["sidecar_val"], layer["N"], layer["K"])

    def forward(self, x, y=None, kernel=HXQ_KERNEL_AUTO, split_k=0, stream=None):
        import torch
        M = int(x.shape[0])
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float32, device=x.device)
        hxq_linear_forward_ex(self.handle, x, y, M, kernel, split_k, stream)
        return y

    __call__ = forward

    def forward_out(self, x, bias=None, out_dtype=HXQ_OUT_F32, y=None, stream=None):
        """y = x . W^T (+ bias) as float32, or as bfloat16 (rounded to nearest
        even) with out_dtype=HXQ_OUT_BF16."""
        import torch
        M = int(x.shape[0])
        if y is None:
            dt = torch.bfloat16 if out_dtype == HXQ_OUT_BF16 else torch.float32
            y = torch.empty((M, self.N), dtype=dt, device=x.device)
        hxq_linear_forward_out(self.handle, x, bias, y, out_dtype, M, stream)
        return y

    def forward_host(self, x_host, y_host, x_dev, y_dev, stream=None, sync=True):
        """End-to-end call on host buffers (hxq_linear_forward_host): copy x
        (pinned) in, run, copy y (pinned) out, all on `stream`. The caller
        owns the four buffers. With sync=False the call returns after
        enqueuing; synchronise the stream before reading y_host."""
        import torch
        s = stream or torch.cuda.current_stream()
        hxq_linear_forward_host(self.handle, x_host, x_dev, y_dev, y_host, int(x_dev.shape[0]), s)
        if sync:
            s.synchronize()
        return y_host

    def decode(self, stream=None):
        import torch
        W = torch.empty((self.N, self.K), dtype=torch.float32, device="cuda")
        hxq_decode(self.handle, W, stream)
        return W

    def check(self) -> None:
        hxq_linear_check(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            hxq_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HelixGroup:
    """HelixLinear layers that read the same activations (one mode, one K),
    run by one launch for M <= 4 tokens. Borrows the layers: keep them alive
    while the group is used."""

    def __init__(self, layers):
        self.layers = list(layers)
        self.handle = hxq_group_create([l.handle for l in self.layers])

    def forward(self, x, biases=None, out_dtype=HXQ_OUT_F32, ys=None, stream=None):
        """[y_i = x . W_i^T (+ bias_i)] for every layer, float32 or bfloat16."""
        import torch
        M = int(x.shape[0])
        if ys is None:
            dt = torch.bfloat16 if out_dtype == HXQ_OUT_BF16 else torch.float32
            ys = [torch.empty((M, l.N), dtype=dt, device=x.device) for l in self.layers]
        hxq_group_forward(self.handle, x, biases, ys, out_dtype, M, stream)
        return ys

    __call__ = forward

    def close(self) -> None:
        if getattr(self, "handle", None):
            hxq_group_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- encoder convenience ------------------------------------------------------

def kmeans(points, init, iters, stream=None):
    """Lloyd k-means on the GPU: points float32 CUDA [n] or [n, 2], init
    [k] or [k, 2]. Returns (centroids like init, labels int16 bits of the
    uint16 indices as an int32 tensor)."""
    import torch
    dim = 1 if points.dim() == 1 else int(points.shape[1])
    n, k = int(points.shape[0]), int(init.shape[0])
    cent = init.detach().to(device=points.device, dtype=torch.float32).contiguous().clone()
    lab = torch.empty(n, dtype=torch.int16, device=points.device)
    hxq_kmeans(points.contiguous(), n, dim, k, iters, cent, lab, stream)
    return cent, lab.to(torch.int32) & 0xFFFF


def encode(W, mode, codebook, threshold, max_sidecar=None, stream=None):
    """Indices and sidecar of W (float32 CUDA [N, K]) for a trained codebook,
    in the layout HelixLinear takes. Returns (indices uint8, sidecar_pos
    int64, sidecar_val float32), all CUDA tensors."""
    import torch
    N, K = int(W.shape[0]), int(W.shape[1])
    W = W.contiguous()
    cb = codebook.to(device=W.device, dtype=torch.float32).contiguous()
    nbytes = N * K if mode == HXQ_MODE_SCALAR8 else 3 * N * K // 4
    idx = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    count = torch.zeros(1, dtype=torch.int64, device=W.device)
    cap = max(1024, N * K // 100) if max_sidecar is None else int(max_sidecar)
    while True:
        pos = torch.empty(max(cap, 1), dtype=torch.int64, device=W.device)
        val = torch.empty(max(cap, 1), dtype=torch.float32, device=W.device)
        hxq_encode(W, mode, N, K, cb, threshold, idx, pos, val, cap, count, stream)
        n = int(count.item())
        if n <= cap or max_sidecar is not None:
            m = min(n, cap)
            return idx, pos[:m], val[:m]
        cap = n


# ---- 8-bit-float layers --------------------------------------------------------
# Tensors are checked here for what the C ABI cannot see: shape, type,
# contiguity and device. A mismatch raises HXQError with HXQ_EINVAL. A call
# runs on the current torch stream, or on `stream` as if it were that. These
# wrappers sit in the path of a decode step: they call the library directly,
# take outputs that exist already, and build no message unless they raise. None
# of these operators has a backward pass: results carry no gradient, whatever
# the inputs require.

class _Torch:
    """What the wrappers use of torch, looked up once (importing this module
    does not import torch)."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.i32 = torch.float32, torch.bfloat16, torch.int32
        self.q, self.q8 = torch.float8_e4m3fn, (torch.float8_e4m3fn, torch.uint8)
        self.code = {torch.float32: HXQ_TYPE_F32, torch.bfloat16: HXQ_TYPE_BF16}
        self.empty = torch.empty
        self.device = torch.cuda.current_device
        # the current stream's handle without building a Stream object
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)


_torch = None


def _t() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _refuse(what: str):
    raise HXQError(HXQ_EINVAL, what)


def _on(stream):
    """`stream` (a Stream, or its handle) as the current one: what a wrapper
    copies or allocates then belongs to the stream that its kernel runs on."""
    import torch
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _input(t, dims: int, what: str):
    """`t` contiguous (other layouts are copied) and its HXQ_TYPE_*: float32
    or bfloat16 on the current CUDA device."""
    code = _t().code.get(t.dtype)
    if code is None or not t.is_cuda or t.dim() != dims or t.get_device() != _torch.device():
        _refuse(f"{what}: a {dims}D float32 or bfloat16 tensor on the current CUDA device")
    return (t if t.is_contiguous() else t.contiguous()), code


def _output(t, shape, dtype, device: int, what: str):
    """`t`, checked, or a new tensor of that shape and type."""
    if t is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _refuse(f"{what}: a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {device}")
    return t


def _bytes(t, shape, device: int, what: str):
    """As _output for 8-bit values, which may also come as uint8."""
    if t is None or t.dtype is _torch.q:
        return _output(t, shape, _torch.q, device, what)
    return _output(t, shape, _torch.q8[1], device, what)


def fp8_quantize(x, q=None, scales=None, stream=None):
    """x [M, K] (float32 or bfloat16 CUDA) as an 8-bit activation. Returns
    (q float8_e4m3fn [M, K rounded up to 16], scales float32 [M, ceil(K / 128)])."""
    if stream is not None:
        with _on(stream):
            return fp8_quantize(x, q, scales)
    x, code = _input(x, 2, "fp8_quantize")
    (rows, cols), dev = x.shape, x.get_device()
    q = _bytes(q, (rows, (cols + 15) // 16 * 16), dev, "fp8_quantize: q")
    scales = _output(scales, (rows, (cols + 127) // 128), _torch.f32, dev, "fp8_quantize: scales")
    _check(lib.hxq_fp8_quantize(x.data_ptr(), code, rows, cols, q.data_ptr(), scales.data_ptr(), _torch.raw_stream(dev)),
           "hxq_fp8_quantize")
    return q, scales


def fp8_swiglu(gate_up, q=None, scales=None, stream=None):
    """silu(gate) * up of gate_up [M, 2 K] (gate first) as an 8-bit
    activation [M, K]; returns (q, scales) as fp8_quantize."""
    if stream is not None:
        with _on(stream):
            return fp8_swiglu(gate_up, q, scales)
    x, code = _input(gate_up, 2, "fp8_swiglu")
    (rows, both), dev = x.shape, x.get_device()
    if both % 2:
        _refuse("fp8_swiglu: gate_up is [M, 2 K]")
    cols = both // 2
    q = _bytes(q, (rows, (cols + 15) // 16 * 16), dev, "fp8_swiglu: q")
    scales = _output(scales, (rows, (cols + 127) // 128), _torch.f32, dev, "fp8_swiglu: scales")
    _check(lib.hxq_fp8_swiglu(x.data_ptr(), code, rows, cols, q.data_ptr(), scales.data_ptr(), _torch.raw_stream(dev)),
           "hxq_fp8_swiglu")
    return q, scales


def fp8_encode(W, q=None, scales=None, stream=None):
    """Weights [N, K] or [E, N, K] (float32 or bfloat16 CUDA) as 8-bit values
    of the same shape and scales [(E,) ceil(N / 128), ceil(K / 128)]: what
    Fp8Linear takes."""
    if stream is not None:
        with _on(stream):
            return fp8_encode(W, q, scales)
    W, code = _input(W, 3 if W.dim() == 3 else 2, "fp8_encode")
    dev, (N, K) = W.get_device(), W.shape[-2:]
    q = _bytes(q, W.shape, dev, "fp8_encode: q")
    scales = _output(scales, (*W.shape[:-2], (N + 127) // 128, (K + 127) // 128), _torch.f32, dev, "fp8_encode: scales")
    _check(lib.hxq_fp8_encode(W.data_ptr(), code, W.shape[0] if W.dim() == 3 else 1, N, K, q.data_ptr(),
                              scales.data_ptr(), _torch.raw_stream(dev)), "hxq_fp8_encode")
    return q, scales


def rmsnorm(x, weight=None, eps=1e-6, residual=None, sum_out=None, y=None, q=None, scales=None, want=None,
            stream=None):
    """t = x + residual (rounded to the residual's type), then
    h = t / sqrt(mean(t^2) + eps) * weight per row of x [M, K]; weight is
    float32 [K].

    want: "q" for h as an 8-bit activation (what Fp8Linear takes), "y" for h
    as bfloat16 (what HelixLinear takes), "qy" for both; by default what is
    given of y and q (q if neither is). sum_out receives t (it may be the
    residual itself; a new tensor if there is a residual and none is given).
    Returns (q, scales, y, sum), None for what was not asked for."""
    if stream is not None:
        with _on(stream):
            return rmsnorm(x, weight, eps, residual, sum_out, y, q, scales, want)
    x, xt = _input(x, 2, "rmsnorm")
    rt = xt
    T = _torch
    shape, dev = x.shape, x.get_device()
    rows, cols = shape
    if want is None:
        want_y, want_q = y is not None, q is not None or y is None
    else:
        want_y, want_q = "y" in want, "q" in want
        if want not in ("q", "y", "qy", "yq") or (y is not None and not want_y) or (q is not None and not want_q):
            _refuse("rmsnorm: want is 'q', 'y' or 'qy', and covers the outputs that are given")
    rp = sp = wp = yp = qp = cp = None
    if residual is not None:
        if residual.dtype is not x.dtype or residual.shape != shape or not residual.is_contiguous() or \
                residual.get_device() != dev:  # (not the common case)
            residual, rt = _input(residual, 2, "rmsnorm: residual")
            if residual.shape != shape:
                _refuse("rmsnorm: residual has the shape of x")
        sum_out = _output(sum_out, shape, residual.dtype, dev, "rmsnorm: sum_out")
        rp, sp = residual.data_ptr(), sum_out.data_ptr()
    elif sum_out is not None:
        _refuse("rmsnorm: sum_out without a residual")
    if weight is not None:
        wp = _output(weight, (cols,), T.f32, dev, "rmsnorm: weight").data_ptr()
    if want_q:
        q = _bytes(q, (rows, (cols + 15) // 16 * 16), dev, "rmsnorm: q")
        scales = _output(scales, (rows, (cols + 127) // 128), T.f32, dev, "rmsnorm: scales")
        qp, cp = q.data_ptr(), scales.data_ptr()
    elif scales is not None:
        _refuse("rmsnorm: scales without q")
    if want_y:
        y = _output(y, shape, T.bf16, dev, "rmsnorm: y")
        yp = y.data_ptr()
    rc = lib.hxq_rmsnorm(x.data_ptr(), xt, rp, sp, rt, wp, eps, rows, cols, yp, qp, cp,
                         T.raw_stream(dev))
    if rc:
        raise HXQError(rc, "hxq_rmsnorm")
    return q, scales, y, sum_out


class Fp8Linear:
    """8-bit-float weights owned by libhxq: of one layer (W [N, K], scales
    [ceil(N / 128), ceil(K / 128)]) or of the experts of one ([E, N, K] and
    [E, ...]), host or device tensors; the handle copies them. Activations
    come as the pair that fp8_quantize, fp8_swiglu and rmsnorm return.
    """

    def __init__(self, W, scales):
        T = _t()
        if W.dim() not in (2, 3) or W.numel() == 0 or W.dtype not in T.q8:
            _refuse("Fp8Linear: W is [N, K] or [E, N, K], 8 bits")
        self.grouped = W.dim() == 3
        self.E = int(W.shape[0]) if self.grouped else 1
        self.N, self.K = int(W.shape[-2]), int(W.shape[-1])
        self._ld, self._kb = (self.K + 15) // 16 * 16, (self.K + 127) // 128
        if scales.dtype is not T.f32 or scales.shape != (*W.shape[:-2], (self.N + 127) // 128, self._kb):
            _refuse("Fp8Linear: scales are float32, one per 128 x 128 block")
        self.handle = hxq_fp8_create(W.contiguous(), scales.contiguous(), self.E, self.N, self.K)
        self._dev = T.device()

    @classmethod
    def from_weight(cls, W) -> "Fp8Linear":
        """From float32 or bfloat16 CUDA weights [N, K] or [E, N, K]."""
        return cls(*fp8_encode(W))

    def _args(self, xq, xs, bias, out_dtype, y):
        T = _torch
        M, dev = xq.shape[0], xq.get_device()
        if dev != self._dev:
            _refuse(f"Fp8Linear: xq is on the weights' device, CUDA device {self._dev}")
        _bytes(xq, (M, self._ld), dev, "Fp8Linear: xq")
        _output(xs, (M, self._kb), T.f32, dev, "Fp8Linear: xs")
        bp = None
        if bias is not None:
            bp = _output(bias, (self.E, self.N) if self.grouped else (self.N,), T.f32, dev, "Fp8Linear: bias").data_ptr()
        y = _output(y, (M, self.N), T.bf16 if out_dtype == HXQ_OUT_BF16 else T.f32, dev, "Fp8Linear: y")
        return M, xq.data_ptr(), xs.data_ptr(), bp, y, T.raw_stream(dev)

    def forward(self, xq, xs, bias=None, out_dtype=HXQ_OUT_F32, y=None, stream=None):
        """y = x . W^T (+ bias [N]) as float32, or as bfloat16 with
        out_dtype=HXQ_OUT_BF16."""
        if stream is not None:
            with _on(stream):
                return self.forward(xq, xs, bias, out_dtype, y)
        if self.grouped:
            _refuse("Fp8Linear: forward_grouped runs the experts")
        M, xp, sp, bp, y, st = self._args(xq, xs, bias, out_dtype, y)
        _check(lib.hxq_fp8_forward(self.handle, xp, sp, bp, y.data_ptr(), out_dtype, M, st), "hxq_fp8_forward")
        return y

    __call__ = forward

    def forward_grouped(self, xq, xs, offsets, bias=None, out_dtype=HXQ_OUT_F32, y=None, stream=None):
        """Rows offsets[e] .. offsets[e + 1] - 1 (int32 CUDA [E + 1]) times
        expert e's weights (+ bias [E, N]). Rows outside all of them are left
        as they were in y (unwritten in a new y)."""
        if stream is not None:
            with _on(stream):
                return self.forward_grouped(xq, xs, offsets, bias, out_dtype, y)
        if not self.grouped or offsets is None:
            _refuse("Fp8Linear: forward_grouped takes weights [E, N, K] and offsets")
        M, xp, sp, bp, y, st = self._args(xq, xs, bias, out_dtype, y)
        op = _output(offsets, (self.E + 1,), _torch.i32, xq.get_device(), "Fp8Linear: offsets").data_ptr()
        _check(lib.hxq_fp8_forward_grouped(self.handle, xp, sp, op, bp, y.data_ptr(), out_dtype, M, st),
               "hxq_fp8_forward_grouped")
        return y

    def check(self) -> None:
        hxq_fp8_check(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            hxq_fp8_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
