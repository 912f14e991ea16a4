"""Python binding of libsq, the separated-quantization decode linear layer.

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libsq.so`` (include/sq.h).  PyTorch provides device memory and the stream.
There is no CPU fallback: importing works without a GPU (so the library can
be inspected), but every call needs the built library and an sm_100 device,
and fails loudly otherwise.

Method (m.lqnn.cn/news/241359, sections 2.1-2.3): W ~ alpha_r*sign(W) + W_res
with an INT8 group residual, activations split into cached fp32 outlier
channels and per-token INT8 codes, and one fused kernel summing the trunk
(bit operations), the residual (integer products) and the outliers.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libsq.so")
HEADER = os.path.join(os.path.dirname(PKG_DIR), "include", "sq.h")

SQ_LAUNCH_PDL = 1
SQ_TRUNK_ONLY = 2
SQ_ZERO_REST = 4
SQ_LAYOUT_ROWS = 0
SQ_LAYOUT_TILES = 1
SQ_LAYOUT_TILES_SPARSE = 2
SQ_LAYOUT_TILES_ASYM = 3
SQ_GATE_TOPK = 0
SQ_GATE_ALL = 1
SQ_TYPE_F32 = 0
SQ_TYPE_F16 = 1
SQ_TYPE_BF16 = 2

STATUS = {
    0: "SQ_OK", 1: "SQ_ERR_INVALID_ARG", 2: "SQ_ERR_SHAPE", 3: "SQ_ERR_ALIGN",
    4: "SQ_ERR_UNSUPPORTED_DEVICE", 5: "SQ_ERR_CUDA", 6: "SQ_ERR_NONFINITE",
    7: "SQ_ERR_TIMEOUT", 8: "SQ_ERR_WORKSPACE",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}


class SQError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.name = STATUS.get(code, f"status {code}")
        super().__init__(f"{where}: {self.name}")


class SqPackedWeight(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("sign_stride", ctypes.c_int32), ("res_stride", ctypes.c_int32),
        ("scale_stride", ctypes.c_int32),
        ("sign_bits", ctypes.c_void_p), ("mask_bits", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p), ("res_q", ctypes.c_void_p), ("res_scale", ctypes.c_void_p),
        ("keep_bits", ctypes.c_void_p), ("res_bytes", ctypes.c_void_p),
        ("res_zero", ctypes.c_void_p),
    ]


class SqNvfp4Matrix(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("K", ctypes.c_int32), ("per_row", ctypes.c_int32),
        ("rows_pad", ctypes.c_int32), ("code_stride", ctypes.c_int32), ("sf_chunks", ctypes.c_int32),
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("g", ctypes.c_void_p),
    ]


class SqLoraBank(ctypes.Structure):
    _fields_ = [
        ("S", ctypes.c_int32), ("R", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
        ("type", ctypes.c_int32), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
        ("scale", ctypes.c_void_p), ("rank", ctypes.c_void_p),
    ]


_lib = None


def lib():
    """The loaded libsq.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m decode_matvec_sq_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
    pw = ctypes.POINTER(SqPackedWeight)
    nm = ctypes.POINTER(SqNvfp4Matrix)
    lb = ctypes.POINTER(SqLoraBank)
    i64 = ctypes.c_int64
    sig = {
        "sq_nvfp4_bytes": ([i32, i32, i32], sz),
        "sq_nvfp4_view": ([vp, i32, i32, i32, nm], ctypes.c_int),
        "sq_nvfp4_quantize": ([vp, nm, vp, vp], ctypes.c_int),
        "sq_nvfp4_linear": ([nm, nm, vp, vp, vp], ctypes.c_int),
        "sq_testing_nvfp4_stalled": ([nm, nm, vp, i32, ctypes.c_uint64, vp, vp], ctypes.c_int),
        "sq_testing_mma_peak": ([i32, i32, ctypes.POINTER(ctypes.c_double), vp, vp], ctypes.c_int),
        "sq_testing_read_peak": ([vp, ctypes.c_uint64, i32, ctypes.POINTER(ctypes.c_double), vp], ctypes.c_int),
        "sq_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "sq_device_check": ([], ctypes.c_int),
        "sq_packed_bytes": ([i32, i32, i32, i32, i32], sz),
        "sq_packed_view": ([vp, i32, i32, i32, i32, i32, pw], ctypes.c_int),
        "sq_decompose_pack": ([vp, i32, i32, i32, pw, vp, vp], ctypes.c_int),
        "sq_decompose_pack_sparse": ([vp, i32, i32, i32, i32, pw, vp, vp], ctypes.c_int),
        "sq_residual_errors_scratch_bytes": ([i32], sz),
        "sq_residual_errors": ([vp, pw, vp, vp, sz, vp, vp], ctypes.c_int),
        "sq_decompose_pack_auto": ([vp, i32, i32, i32, pw, vp, sz, vp, vp, vp, vp], ctypes.c_int),
        "sq_calibrate_outliers": ([vp, i32, i32, i32, vp, vp, vp], ctypes.c_int),
        "sq_quantize_act": ([vp, i32, i32, vp, i32, vp, vp, vp, vp, u32, vp], ctypes.c_int),
        "sq_linear_workspace_bytes": ([pw, i32], sz),
        "sq_quantize_linear_workspace_bytes": ([pw, i32, i32], sz),
        "sq_quantize_linear_tokens_per_pass": ([pw, i32], i32),
        "sq_linear_tokens_per_pass": ([pw, u32], i32),
        "sq_linear": ([pw, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp, u32, vp], ctypes.c_int),
        "sq_linear_accumulators": ([pw, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp, u32, vp],
                                   ctypes.c_int),
        "sq_linear_noalloc": ([pw, vp, vp, vp, vp, i32, i32, vp, vp, u32, vp], ctypes.c_int),
        "sq_quantize_linear": ([pw, vp, i32, vp, i32, vp, vp, sz, vp, u32, vp], ctypes.c_int),
        "sq_route_workspace_bytes": ([i32, i32, i32], sz),
        "sq_route": ([vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp, u32, vp], ctypes.c_int),
        "sq_segment_workspace_bytes": ([i32, i32], sz),
        "sq_segment": ([vp, i32, i32, vp, vp, vp, vp, sz, vp, u32, vp], ctypes.c_int),
        "sq_expert_view": ([pw, i32, i32, i32, pw], ctypes.c_int),
        "sq_grouped_linear_workspace_bytes": ([pw, i32, i32, i32], sz),
        "sq_testing_grouped_stalled": ([pw, i32, i32, vp, vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, sz, i32,
                                        ctypes.c_uint64, vp, vp], ctypes.c_int),
        "sq_grouped_linear": ([pw, i32, i32, vp, vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp, u32, vp],
                              ctypes.c_int),
        "sq_lora_workspace_bytes": ([lb, i32], sz),
        "sq_lora_add": ([lb, vp, i32, vp, vp, vp, vp, i64, vp, i64, vp, sz, vp, u32, vp], ctypes.c_int),
        "sq_combine": ([vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, u32, vp], ctypes.c_int),
        "sq_testing_prefill_stalled": ([pw, vp, vp, vp, vp, i32, i32, vp, i32, ctypes.c_uint64, vp,
                                        vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _ck(rc: int, where: str) -> None:
    if rc != 0:
        raise SQError(rc, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def ceil_div(a: int, b: int) -> int:
    return -(-a // b)


def round_up(a: int, b: int) -> int:
    return ceil_div(a, b) * b


def device_check() -> None:
    _ck(lib().sq_device_check(), "sq_device_check")


# ---- packed weights ------------------------------------------------------------

def default_layout(group_size: int) -> int:
    """The tensor-core layout for group size 128, the row layout otherwise."""
    return SQ_LAYOUT_TILES if group_size == 128 else SQ_LAYOUT_ROWS


@dataclass
class PackedWeight:
    """A packed weight in one device allocation (``buf``) with its C view.
    The array accessors return the raw arrays in the weight's layout
    (include/sq.h documents both layouts)."""
    N: int
    K: int
    group_size: int
    with_mask: bool
    layout: int
    buf: object                 # torch.uint8 device tensor (of an expert: a tensor of its stack)
    view: SqPackedWeight
    arrays: dict = None         # an expert of a stack: its rows of the stack's arrays (kept alive here)

    @property
    def nbytes(self) -> int:
        if self.arrays is not None:
            return sum(t.numel() * t.element_size() for t in self.arrays.values())
        return int(self.buf.numel())

    @property
    def tiled(self) -> bool:
        return self.layout in (SQ_LAYOUT_TILES, SQ_LAYOUT_TILES_SPARSE, SQ_LAYOUT_TILES_ASYM)

    @property
    def rows(self) -> int:
        """Rows of every array: N, or N padded to 16 in the tiled layouts."""
        return round_up(self.N, 16) if self.tiled else self.N

    def _arr(self, field: str, dtype, shape):
        import torch
        if self.arrays is not None:
            return self.arrays[field].view(*shape)
        base = self.buf.data_ptr()
        off = getattr(self.view, field) - base
        count = 1
        for s in shape:
            count *= s
        itemsize = torch.empty(0, dtype=dtype).element_size()
        return self.buf[off:off + count * itemsize].view(dtype).view(*shape)

    def sign_bits(self):
        import torch
        return self._arr("sign_bits", torch.int32, (self.rows, self.view.sign_stride))

    def mask_bits(self):
        import torch
        if not self.with_mask:
            return None
        return self._arr("mask_bits", torch.int32, (self.rows, self.view.sign_stride))

    def alpha(self):
        import torch
        return self._arr("alpha", torch.float32, (self.rows,))[:self.N]

    def res_q(self):
        import torch
        return self._arr("res_q", torch.int8, (self.rows, self.view.res_stride))

    def res_scale(self):
        import torch
        return self._arr("res_scale", torch.float32, (self.rows, self.view.scale_stride))

    def res_zero(self):
        """Zero-points of the asymmetric residual, indexed like res_scale."""
        import torch
        if self.layout != SQ_LAYOUT_TILES_ASYM:
            return None
        return self._arr("res_zero", torch.int32, (self.rows, self.view.scale_stride))

    def keep_bits(self):
        import torch
        if self.layout != SQ_LAYOUT_TILES_SPARSE:
            return None
        return self._arr("keep_bits", torch.int32, (self.rows, self.view.sign_stride))

    def res_bytes(self):
        """Packed code bytes of every tile (sparse layout)."""
        import torch
        if self.layout != SQ_LAYOUT_TILES_SPARSE:
            return None
        tiles = (self.rows // 16) * (self.view.res_stride // 128)
        return self._arr("res_bytes", torch.int32, (tiles,))


def packed_bytes(N: int, K: int, group_size: int = 128, with_mask: bool = False,
                 layout: int = None) -> int:
    if layout is None:
        layout = default_layout(group_size)
    return int(lib().sq_packed_bytes(N, K, group_size, int(with_mask), layout))


def alloc_packed(N: int, K: int, group_size: int = 128, with_mask: bool = False,
                 layout: int = None, device=None) -> PackedWeight:
    import torch
    if layout is None:
        layout = default_layout(group_size)
    nbytes = packed_bytes(N, K, group_size, with_mask, layout)
    if nbytes == 0:
        raise SQError(STATUS_CODE["SQ_ERR_SHAPE"], "sq_packed_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    v = SqPackedWeight()
    _ck(lib().sq_packed_view(_ptr(buf), N, K, group_size, int(with_mask), layout,
                             ctypes.byref(v)), "sq_packed_view")
    return PackedWeight(N, K, group_size, with_mask, layout, buf, v)


def decompose_pack(W, trunk_percent: int = -1, group_size: int = 128, layout: int = None,
                   out: PackedWeight = None, status=None, stream=None) -> PackedWeight:
    """Offline split of W[N][K] (float32, device) into the packed form
    (default layout: tiles for group size 128, rows otherwise)."""
    N, K = W.shape
    if out is None:
        out = alloc_packed(N, K, group_size, trunk_percent > 0, layout, device=W.device)
    _ck(lib().sq_decompose_pack(_ptr(W), N, K, trunk_percent, ctypes.byref(out.view),
                                _ptr(status), _stream(stream)), "sq_decompose_pack")
    return out


def decompose_pack_sparse(W, residual_percent: int, trunk_percent: int = -1,
                          out: PackedWeight = None, status=None, stream=None) -> PackedWeight:
    """sq_decompose_pack with the residual entries at or below the per-row
    residual_percent-th percentile of |r| dropped, into SQ_LAYOUT_TILES_SPARSE."""
    N, K = W.shape
    if out is None:
        out = alloc_packed(N, K, 128, trunk_percent > 0, SQ_LAYOUT_TILES_SPARSE, device=W.device)
    _ck(lib().sq_decompose_pack_sparse(_ptr(W), N, K, trunk_percent, residual_percent,
                                       ctypes.byref(out.view), _ptr(status), _stream(stream)),
        "sq_decompose_pack_sparse")
    return out


def residual_errors(W, pw: PackedWeight, status=None, stream=None):
    """(err_split, err_plain): sum over the layer of (W - What)^2 for the
    packed weight and for plain symmetric INT8 groups of W (binary64, on the
    device; include/sq.h sq_residual_errors).  Reads the two numbers back."""
    import torch
    err = torch.zeros(2, dtype=torch.float64, device=W.device)
    nb = int(lib().sq_residual_errors_scratch_bytes(pw.N))
    scratch = torch.empty(nb, dtype=torch.uint8, device=W.device)
    _ck(lib().sq_residual_errors(_ptr(W), ctypes.byref(pw.view), _ptr(err), _ptr(scratch), nb,
                                 _ptr(status), _stream(stream)), "sq_residual_errors")
    e = err.cpu().tolist()
    return e[0], e[1]


def decompose_pack_auto(W, trunk_percent: int = -1, layout: int = None, status=None, stream=None):
    """The split with the per-layer fallback (include/sq.h
    sq_decompose_pack_auto): plain INT8 groups (an empty trunk) when they
    reconstruct W at least as well as the split.  Returns (packed weight,
    fell_back).  Synchronous."""
    import torch
    N, K = W.shape
    out = alloc_packed(N, K, 128, True, layout, device=W.device)
    nb = int(lib().sq_residual_errors_scratch_bytes(N)) + 256
    scratch = torch.empty(nb, dtype=torch.uint8, device=W.device)
    fell = ctypes.c_int32(0)
    _ck(lib().sq_decompose_pack_auto(_ptr(W), N, K, trunk_percent, ctypes.byref(out.view),
                                     _ptr(scratch), nb, ctypes.byref(fell), None, _ptr(status),
                                     _stream(stream)), "sq_decompose_pack_auto")
    if not out.view.mask_bits:
        out.with_mask = False
    return out, bool(fell.value)


def calibrate_outliers(X, k: int, out=None, status=None, stream=None):
    """Top-k channels of X[T][K] by max |x| (ties: lower channel), ascending int32."""
    import torch
    T, K = X.shape
    idx = out if out is not None else torch.empty(k, dtype=torch.int32, device=X.device)
    _ck(lib().sq_calibrate_outliers(_ptr(X), T, K, k, _ptr(idx), _ptr(status), _stream(stream)),
        "sq_calibrate_outliers")
    return idx


def quantize_act(x, idx, xq=None, sx=None, x_out=None, status=None, pdl: bool = False,
                 stream=None):
    """x[M][K] float32 -> (xq [M][roundup(K,128)] int8, sx [M], x_out [M][n_out])."""
    import torch
    M, K = x.shape
    n = 0 if idx is None else int(idx.numel())
    dev = x.device
    if xq is None:
        xq = torch.empty(M, round_up(K, 128), dtype=torch.int8, device=dev)
    if sx is None:
        sx = torch.empty(M, dtype=torch.float32, device=dev)
    if x_out is None:
        x_out = torch.empty(M, max(n, 1), dtype=torch.float32, device=dev)
    _ck(lib().sq_quantize_act(_ptr(x), M, K, _ptr(idx) if n else None, n, _ptr(xq), _ptr(sx),
                              _ptr(x_out) if n else None, _ptr(status),
                              SQ_LAUNCH_PDL if pdl else 0, _stream(stream)), "sq_quantize_act")
    return xq, sx, x_out


def workspace_bytes(pw: PackedWeight, M: int = 1) -> int:
    return int(lib().sq_linear_workspace_bytes(ctypes.byref(pw.view), M))


def workspace_counters(ws, pw: PackedWeight, M: int = 1):
    """The per-row arrival counters inside a workspace (they end every call at zero)."""
    base = workspace_bytes(pw, M) - round_up(4 * pw.N, 256)
    return ws[base: base + 4 * pw.N]


def new_workspace(pw: PackedWeight, M: int = 1, device=None):
    """A zero-filled workspace for sq_linear (zero once; calls keep it zeroed)."""
    import torch
    return torch.zeros(max(workspace_bytes(pw, M), 16), dtype=torch.uint8,
                       device=device or pw.buf.device)


def fused_workspace_bytes(pw: PackedWeight, M: int = 1, n_out: int = 0) -> int:
    """Workspace with which quantize_linear may run the activation split once
    and the linear layer on its codes (where that is faster)."""
    return int(lib().sq_quantize_linear_workspace_bytes(ctypes.byref(pw.view), M, n_out))


def new_fused_workspace(pw: PackedWeight, M: int = 1, n_out: int = 0, device=None):
    """A zero-filled workspace of fused_workspace_bytes."""
    import torch
    return torch.zeros(max(fused_workspace_bytes(pw, M, n_out), 16), dtype=torch.uint8,
                       device=device or pw.buf.device)


def _flags(pdl: bool, trunk_only: bool = False) -> int:
    return (SQ_LAUNCH_PDL if pdl else 0) | (SQ_TRUNK_ONLY if trunk_only else 0)


def linear(pw: PackedWeight, xq, sx, x_out, idx, y=None, workspace=None, status=None,
           pdl: bool = False, stream=None, trunk_only: bool = False):
    """y[M][N] = fused trunk + residual + outlier product (float32).
    The weight's layout picks the kernel: tiles -> tensor cores, rows -> dp4a.
    trunk_only (tiles): the residual path skipped."""
    import torch
    M = xq.shape[0]
    n = 0 if idx is None else int(idx.numel())
    if y is None:
        y = torch.empty(M, pw.N, dtype=torch.float32, device=xq.device)
    if workspace is None:
        workspace = new_workspace(pw, M)
    _ck(lib().sq_linear(ctypes.byref(pw.view), _ptr(xq), _ptr(sx), _ptr(x_out) if n else None,
                        _ptr(idx) if n else None, n, M, _ptr(y), _ptr(workspace),
                        workspace.numel(), _ptr(status), _flags(pdl, trunk_only),
                        _stream(stream)), "sq_linear")
    return y


def quantize_linear(pw: PackedWeight, x, idx, y=None, workspace=None, status=None,
                    pdl: bool = False, stream=None, trunk_only: bool = False):
    """y[M][N] from fp32 activations x[M][K]: the activation split and the
    linear layer in one kernel (tiled layout), or, for larger M * K with a
    workspace of fused_workspace_bytes, the split once and the linear layer."""
    import torch
    M = x.shape[0]
    n = 0 if idx is None else int(idx.numel())
    if y is None:
        y = torch.empty(M, pw.N, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = new_fused_workspace(pw, M, n)
    _ck(lib().sq_quantize_linear(ctypes.byref(pw.view), _ptr(x), M, _ptr(idx) if n else None, n,
                                 _ptr(y), _ptr(workspace), workspace.numel(), _ptr(status),
                                 _flags(pdl, trunk_only), _stream(stream)), "sq_quantize_linear")
    return y


# the fixed scratch size of sq_linear_noalloc (include/sq.h)
NOALLOC_SCRATCH_BYTES = 16 << 20


def linear_noalloc(pw: PackedWeight, xq, sx, x_out, idx, y, status=None, pdl: bool = False,
                   stream=None, trunk_only: bool = False):
    """sq_linear with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory at call time).  y [M][N]
    float32 is the caller's.  Calls on one device must not overlap in time."""
    M = xq.shape[0]
    n = 0 if idx is None else int(idx.numel())
    _ck(lib().sq_linear_noalloc(ctypes.byref(pw.view), _ptr(xq), _ptr(sx),
                                _ptr(x_out) if n else None, _ptr(idx) if n else None, n, M,
                                _ptr(y), _ptr(status), _flags(pdl, trunk_only), _stream(stream)),
        "sq_linear_noalloc")
    return y


def testing_prefill_stalled(pw: PackedWeight, xq, sx, x_out, idx, y, skip_group: int,
                            wait_ns: int, status=None, stream=None):
    """include/sq_testing.h: the prefill kernel with its waits limited to
    wait_ns and channel group skip_group's operands never requested (-1:
    none), so that its bounded waits run out (tests of the wind-down path)."""
    M = xq.shape[0]
    n = 0 if idx is None else int(idx.numel())
    _ck(lib().sq_testing_prefill_stalled(ctypes.byref(pw.view), _ptr(xq), _ptr(sx),
                                         _ptr(x_out) if n else None, _ptr(idx) if n else None, n,
                                         M, _ptr(y), skip_group, wait_ns, _ptr(status),
                                         _stream(stream)),
        "sq_testing_prefill_stalled")
    return y


def linear_accumulators(pw: PackedWeight, xq, sx, x_out, idx, workspace=None, status=None,
                        stream=None):
    """(y, T [M][N] int32, R [M][N][ceil(K/G)] int32) from the decode kernel."""
    import torch
    M = xq.shape[0]
    n = 0 if idx is None else int(idx.numel())
    dev = xq.device
    ng = ceil_div(pw.K, pw.group_size)
    y = torch.full((M, pw.N), float("nan"), dtype=torch.float32, device=dev)
    T = torch.empty(M, pw.N, dtype=torch.int32, device=dev)
    R = torch.empty(M, pw.N, ng, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = new_workspace(pw, M)
    _ck(lib().sq_linear_accumulators(ctypes.byref(pw.view), _ptr(xq), _ptr(sx),
                                     _ptr(x_out) if n else None, _ptr(idx) if n else None, n, M,
                                     _ptr(y), _ptr(T), _ptr(R), _ptr(workspace),
                                     workspace.numel(), _ptr(status), _flags(False),
                                     _stream(stream)), "sq_linear_accumulators")
    return y, T, R


# ---- NVFP4 prefill (format separation; include/sq.h documents the format) ----

@dataclass
class Nvfp4Matrix:
    """An NVFP4 matrix [rows][K] in one device allocation with its C view."""
    rows: int
    K: int
    per_row: bool
    buf: object                 # torch.uint8 device tensor
    view: SqNvfp4Matrix

    def _arr(self, field: str, dtype, count: int):
        import torch
        off = getattr(self.view, field) - self.buf.data_ptr()
        itemsize = torch.empty(0, dtype=dtype).element_size()
        return self.buf[off:off + count * itemsize].view(dtype)

    def codes(self):
        """[rows_pad][code_stride] uint8, two E2M1 codes a byte."""
        import torch
        v = self.view
        return self._arr("codes", torch.uint8, v.rows_pad * v.code_stride).view(v.rows_pad,
                                                                                v.code_stride)

    def scales(self):
        """The UE4M3 scale chunks, flat: [rows_pad/128 * sf_chunks * 512] uint8."""
        import torch
        v = self.view
        return self._arr("scales", torch.uint8, (v.rows_pad // 128) * v.sf_chunks * 512)

    def g(self):
        """Second-level scales: [rows] (per row) or [1] (per tensor)."""
        import torch
        return self._arr("g", torch.float32, self.view.rows_pad if self.per_row else 1)[
            :self.rows if self.per_row else 1]


def alloc_nvfp4(rows: int, K: int, per_row: bool, device=None) -> Nvfp4Matrix:
    import torch
    nbytes = lib().sq_nvfp4_bytes(rows, K, int(per_row))
    if nbytes == 0:
        raise SQError(STATUS_CODE["SQ_ERR_SHAPE"], "sq_nvfp4_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    v = SqNvfp4Matrix()
    _ck(lib().sq_nvfp4_view(_ptr(buf), rows, K, int(per_row), ctypes.byref(v)), "sq_nvfp4_view")
    return Nvfp4Matrix(rows, K, bool(per_row), buf, v)


def nvfp4_quantize(X, per_row: bool, out: Nvfp4Matrix = None, status=None,
                   stream=None) -> Nvfp4Matrix:
    """X[rows][K] (float32, device) -> NVFP4 (per tensor for a weight, per
    row for activations)."""
    rows, K = X.shape
    if out is None:
        out = alloc_nvfp4(rows, K, per_row, device=X.device)
    _ck(lib().sq_nvfp4_quantize(_ptr(X), ctypes.byref(out.view), _ptr(status), _stream(stream)),
        "sq_nvfp4_quantize")
    return out


def nvfp4_linear(w: Nvfp4Matrix, x: Nvfp4Matrix, y=None, status=None, stream=None):
    """y [x.rows][w.rows] float32 = dequantized x @ dequantized w^T on the
    block-scaled tensor cores."""
    import torch
    if y is None:
        y = torch.empty(x.rows, w.rows, dtype=torch.float32, device=x.buf.device)
    _ck(lib().sq_nvfp4_linear(ctypes.byref(w.view), ctypes.byref(x.view), _ptr(y), _ptr(status),
                              _stream(stream)), "sq_nvfp4_linear")
    return y


def testing_nvfp4_stalled(w: Nvfp4Matrix, x: Nvfp4Matrix, y, skip_stage: int, wait_ns: int,
                          status=None, stream=None):
    """include/sq_testing.h: sq_nvfp4_linear with one channel stage never
    requested and every wait limited to wait_ns (tests of the timeout path)."""
    _ck(lib().sq_testing_nvfp4_stalled(ctypes.byref(w.view), ctypes.byref(x.view), _ptr(y), skip_stage,
                                       wait_ns, _ptr(status), _stream(stream)), "sq_testing_nvfp4_stalled")


# ---- weights that depend on the token (include/sq.h documents the arrays) -----

_NO_DEVICE = -2  # no tensor's device (a CPU tensor's is -1)


def _refuse(where: str, what: str, code: str = "SQ_ERR_INVALID_ARG"):
    raise SQError(STATUS_CODE[code], f"{where}: {what}")


def _arg(t, dtype, shape, dev: int, where: str, name: str) -> int:
    """The address of a tensor argument: a contiguous CUDA tensor of this type
    and shape on the current device `dev`, else the call is refused."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous CUDA tensor of {dtype}")
    if t.shape != shape:
        _refuse(where, f"{name} must be {list(shape)}, got {list(t.shape)}", "SQ_ERR_SHAPE")
    _refuse(where, f"{name} is not on the current device")


def _opt(t, dtype, shape, dev: int, where: str, name: str):
    return None if t is None else _arg(t, dtype, shape, dev, where, name)


def _status_arg(status, dev: int, where: str):
    if status is None:
        return None
    import torch
    return _arg(status, torch.int32, (1,), dev, where, "status")


def _stream_arg(dev: int) -> int:
    """The handle of the current stream of device `dev`."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (the public call costs 3 us)
    return raw(dev) if raw else torch.cuda.current_stream().cuda_stream


def _on(stream, call, *args):
    """A call with `stream` as the current one, so that results and scratch come
    from that stream's memory: what was freed on another may still be in use
    there, and scratch is freed while the kernels of this one still use it."""
    import torch
    with torch.cuda.stream(stream):
        return call(*args)


def _workspace_arg(ws, need: int, device, dev: int, where: str):
    """(tensor, address, bytes) of a uint8 workspace of at least `need` bytes;
    allocated here when the caller keeps none."""
    import torch
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, _arg(ws, torch.uint8, (ws.numel(),), dev, where, "workspace"), ws.numel()


@dataclass
class Segments:
    """Entries sorted by id: segment s is the places offsets[s] .. offsets[s+1]."""
    offsets: object   # [S + 1] int32
    order: object     # [n] int32: the entry at each place, -1 behind the last segment
    place: object     # the place of each entry, -1 without an id


@dataclass
class Route(Segments):
    ids: object       # [T][k] int32
    gates: object     # [T][k] float32


def route(logits, k: int, gate: str = "topk", workspace=None, status=None, pdl: bool = False,
          stream=None) -> Route:
    """Top-k of logits [T][E] (float32) with softmax gates over the chosen
    ("topk") or over all experts ("all"), and the entries sorted by expert."""
    import torch
    if stream is not None:
        return _on(stream, route, logits, k, gate, workspace, status, pdl)
    if gate not in ("topk", "all"):
        _refuse("sq_route", 'gate must be "topk" or "all"')
    if logits.dim() != 2:
        _refuse("sq_route", "logits must be [T][E]", "SQ_ERR_SHAPE")
    T, E = logits.shape
    cur = torch.cuda.current_device() if logits.is_cuda else _NO_DEVICE
    lp = _arg(logits, torch.float32, (T, E), cur, "sq_route", "logits")
    if not 1 <= k <= 32 or T < 1 or T * k > 1 << 24:
        _refuse("sq_route", "T or k", "SQ_ERR_SHAPE")
    dev, i32 = logits.device, torch.int32
    if T * k % 4 == 0:  # one allocation: each array stays 16-byte aligned
        ids, gates, order, place = torch.empty(4, T, k, dtype=i32, device=dev).unbind(0)
        gates, order = gates.view(torch.float32), order.view(-1)
    else:
        ids = torch.empty(T, k, dtype=i32, device=dev)
        gates = torch.empty(T, k, dtype=torch.float32, device=dev)
        order = torch.empty(T * k, dtype=i32, device=dev)
        place = torch.empty(T, k, dtype=i32, device=dev)
    offsets = torch.empty(E + 1, dtype=i32, device=dev)
    L = lib()
    ws, wp, wn = _workspace_arg(workspace, L.sq_route_workspace_bytes(T, E, k), dev, cur, "sq_route")
    rc = L.sq_route(lp, T, E, k, SQ_GATE_ALL if gate == "all" else SQ_GATE_TOPK, ids.data_ptr(),
                    gates.data_ptr(), offsets.data_ptr(), order.data_ptr(), place.data_ptr(), wp, wn,
                    _status_arg(status, cur, "sq_route"), _flags(pdl), _stream_arg(cur))
    if rc:
        _ck(rc, "sq_route")
    return Route(offsets, order, place, ids, gates)


def segment(ids, S: int, workspace=None, status=None, pdl: bool = False, stream=None) -> Segments:
    """Entries with ids (int32, any shape, -1 = none) in [0, S) sorted by id."""
    import torch
    if stream is not None:
        return _on(stream, segment, ids, S, workspace, status, pdl)
    n = ids.numel()
    cur = torch.cuda.current_device() if ids.is_cuda else _NO_DEVICE
    ip = _arg(ids, torch.int32, ids.shape, cur, "sq_segment", "ids")
    if not 1 <= S <= 1024 or not 1 <= n <= 1 << 24:
        _refuse("sq_segment", "n or S", "SQ_ERR_SHAPE")
    dev = ids.device
    offsets = torch.empty(S + 1, dtype=torch.int32, device=dev)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    place = torch.empty(ids.shape, dtype=torch.int32, device=dev)
    L = lib()
    ws, wp, wn = _workspace_arg(workspace, L.sq_segment_workspace_bytes(n, S), dev, cur, "sq_segment")
    _ck(L.sq_segment(ip, n, S, offsets.data_ptr(), order.data_ptr(), place.data_ptr(), wp, wn,
                     _status_arg(status, cur, "sq_segment"), _flags(pdl), _stream_arg(cur)), "sq_segment")
    return Segments(offsets, order, place)


@dataclass
class PackedExperts:
    """E experts of shape [N][K] in one packed weight (include/sq.h
    sq_expert_view); ``keep`` holds the device tensors its view points into: one
    allocation, or the arrays in the order of ARRAYS (None: absent)."""
    ARRAYS = ("sign_bits", "alpha", "res_q", "res_scale", "mask_bits", "res_zero")
    E: int
    N: int
    K: int
    view: SqPackedWeight
    keep: object

    def expert(self, e: int) -> PackedWeight:
        """Expert e as a packed weight of its own: decompose into it, or use it
        with every call on one weight.  It keeps the stack's memory alive."""
        v = SqPackedWeight()
        _ck(lib().sq_expert_view(ctypes.byref(self.view), self.E, self.N, e, ctypes.byref(v)),
            "sq_expert_view")
        rows = round_up(self.N, 16)
        mine = {name: t[e * rows:(e + 1) * rows] for name, t in self._arrays().items()}
        return PackedWeight(self.N, self.K, 128, bool(v.mask_bits), v.layout, self.keep[0], v, mine)

    def _arrays(self) -> dict:
        """The stack's arrays by name, a row of the stack in each row."""
        if len(self.keep) > 1:
            return {name: t for name, t in zip(self.ARRAYS, self.keep) if t is not None}
        w = PackedWeight(self.view.N, self.K, 128, bool(self.view.mask_bits), self.view.layout, self.keep[0], self.view)
        arrays = {"sign_bits": w.sign_bits(), "alpha": w.alpha(), "res_q": w.res_q(), "res_scale": w.res_scale(),
                  "mask_bits": w.mask_bits(), "res_zero": w.res_zero()}
        return {name: t for name, t in arrays.items() if t is not None}


def alloc_experts(E: int, N: int, K: int, with_mask: bool = False, layout: int = SQ_LAYOUT_TILES,
                  device=None) -> PackedExperts:
    """An empty stack of experts: decompose each expert's weight into
    ``.expert(e)`` (all with, or all without a trunk percentile)."""
    if layout not in (SQ_LAYOUT_TILES, SQ_LAYOUT_TILES_ASYM):
        _refuse("alloc_experts", "layout must be tiles or tiles with an asymmetric residual")
    if E < 1 or E > 1024 or N < 1:
        _refuse("alloc_experts", "E or N", "SQ_ERR_SHAPE")
    pw = alloc_packed(E * round_up(N, 16), K, 128, with_mask, layout, device)
    return PackedExperts(E, N, K, pw.view, (pw.buf,))


def experts_from_arrays(E: int, N: int, K: int, sign_bits, alpha, res_q, res_scale, mask_bits=None,
                        res_zero=None) -> PackedExperts:
    """A stack over arrays that already lie in device memory in the tiled layout
    (for instance loaded from a file): int32 sign (and mask) words
    [E*rows][cols/32], float32 alpha [E*rows], int8 codes [E*rows][cols], float32
    scales (and int32 zero-points) [E*rows][cols/128], rows = roundup(N, 16),
    cols = roundup(K, 128).  The arrays are used in place."""
    import torch
    w = "experts_from_arrays"
    if E < 1 or E > 1024 or N < 1 or K < 1:
        _refuse(w, "E, N or K", "SQ_ERR_SHAPE")
    rows, cols = E * round_up(N, 16), round_up(K, 128)
    cur = torch.cuda.current_device() if torch.cuda.is_available() else _NO_DEVICE
    v = SqPackedWeight()
    v.N, v.K, v.group_size = rows, K, 128
    v.layout = SQ_LAYOUT_TILES if res_zero is None else SQ_LAYOUT_TILES_ASYM
    v.sign_stride, v.res_stride, v.scale_stride = cols // 32, cols, cols // 128
    v.sign_bits = _arg(sign_bits, torch.int32, (rows, cols // 32), cur, w, "sign_bits")
    v.mask_bits = _opt(mask_bits, torch.int32, (rows, cols // 32), cur, w, "mask_bits")
    v.alpha = _arg(alpha, torch.float32, (rows,), cur, w, "alpha")
    v.res_q = _arg(res_q, torch.int8, (rows, cols), cur, w, "res_q")
    v.res_scale = _arg(res_scale, torch.float32, (rows, cols // 128), cur, w, "res_scale")
    v.res_zero = _opt(res_zero, torch.int32, (rows, cols // 128), cur, w, "res_zero")
    e0 = SqPackedWeight()
    _ck(lib().sq_expert_view(ctypes.byref(v), E, N, 0, ctypes.byref(e0)), w)  # the library's own checks
    return PackedExperts(E, N, K, v, (sign_bits, alpha, res_q, res_scale, mask_bits, res_zero))  # (ARRAYS)


def grouped_workspace_bytes(experts: PackedExperts, n: int) -> int:
    return int(lib().sq_grouped_linear_workspace_bytes(ctypes.byref(experts.view), experts.E, experts.N, n))


def new_grouped_workspace(experts: PackedExperts, n: int, device=None):
    """A workspace for grouped_linear over up to n places (one per call that may
    overlap another)."""
    import torch
    return torch.empty(max(grouped_workspace_bytes(experts, n), 16), dtype=torch.uint8, device=device or "cuda")


def grouped_linear(experts: PackedExperts, xq, sx, x_out, idx, offsets, order=None, div: int = 1, y=None,
                   workspace=None, status=None, pdl: bool = False, stream=None):
    """y [n][N] float32: place p of segment e is expert e's weight times the
    activations (as from quantize_act) of row order[p] // div, or of row p
    without an order.  The rows from offsets[E] on (of dropped entries) are 0 in a
    result allocated here, and not written in a `y` given."""
    import torch
    if stream is not None:
        return _on(stream, grouped_linear, experts, xq, sx, x_out, idx, offsets, order, div, y, workspace, status, pdl)
    w = "sq_grouped_linear"
    E, N = experts.E, experts.N
    if xq.dim() != 2:
        _refuse(w, "xq must be [rows][roundup(K,128)]", "SQ_ERR_SHAPE")
    f32, i32, cur = torch.float32, torch.int32, torch.cuda.current_device() if xq.is_cuda else _NO_DEVICE
    rows, nout = xq.shape[0], 0 if idx is None else idx.numel()
    xp = _arg(xq, torch.int8, (rows, experts.view.res_stride), cur, w, "xq")
    if experts.keep[0].get_device() != cur:
        _refuse(w, "the experts are not on the current device")
    sp = _arg(sx, f32, (rows,), cur, w, "sx")
    op = ip = None
    if nout:
        op = _arg(x_out, f32, (rows, nout), cur, w, "x_out")
        ip = _arg(idx, i32, (nout,), cur, w, "idx")
    n = rows if order is None else order.numel()
    dp = _opt(order, i32, (n,), cur, w, "order")
    fp = _arg(offsets, i32, (E + 1,), cur, w, "offsets")
    flags = _flags(pdl)
    if y is None:
        y = torch.empty(n, N, dtype=f32, device=xq.device)
        flags |= SQ_ZERO_REST  # (a quantize_act before the next layer reads every row)
    yp = _arg(y, f32, (n, N), cur, w, "y")
    L = lib()
    need = 0 if workspace is not None else grouped_workspace_bytes(experts, n)
    workspace, wp, wn = _workspace_arg(workspace, need, xq.device, cur, w)
    rc = L.sq_grouped_linear(ctypes.byref(experts.view), E, N, xp, sp, op, ip, nout, rows, dp, div, fp, n, yp, wp,
                             wn, _status_arg(status, cur, w), flags, _stream_arg(cur))
    if rc:
        _ck(rc, w)
    return y


def testing_grouped_stalled(experts: PackedExperts, xq, sx, x_out, idx, offsets, order, div: int, y, workspace,
                            skip_group: int, wait_ns: int, status=None, stream=None):
    """include/sq_testing.h: sq_grouped_linear with one channel group never
    requested and every wait limited to wait_ns (tests of the timeout path)."""
    _ck(lib().sq_testing_grouped_stalled(
        ctypes.byref(experts.view), experts.E, experts.N, _ptr(xq), _ptr(sx), _ptr(x_out), _ptr(idx), idx.numel(),
        xq.shape[0], _ptr(order), div, _ptr(offsets), y.shape[0], _ptr(y), _ptr(workspace), workspace.numel(),
        skip_group, wait_ns, _ptr(status), _stream(stream)), "sq_testing_grouped_stalled")


def combine(z, gates, place, base=None, out=None, status=None, pdl: bool = False, stream=None):
    """out [T][N] = base + sum_j gates[t][j] * z[place[t][j]] (float32); place -1
    adds nothing.  out may be base, not z."""
    import torch
    if stream is not None:
        return _on(stream, combine, z, gates, place, base, out, status, pdl)
    w = "sq_combine"
    if z.dim() != 2 or gates.dim() != 2:
        _refuse(w, "z must be [rows][N] and gates [T][k]", "SQ_ERR_SHAPE")
    rows, N = z.shape
    T, k = gates.shape
    f32, cur = torch.float32, torch.cuda.current_device() if z.is_cuda else _NO_DEVICE
    zp = _arg(z, f32, (rows, N), cur, w, "z")
    gp = _arg(gates, f32, (T, k), cur, w, "gates")
    pp = _arg(place, torch.int32, (T, k), cur, w, "place")
    bp = _opt(base, f32, (T, N), cur, w, "base")
    if out is None:
        out = torch.empty(T, N, dtype=f32, device=z.device)
    op = _arg(out, f32, (T, N), cur, w, "out")
    rc = lib().sq_combine(zp, rows, gp, pp, T, k, N, bp, op, _status_arg(status, cur, w), _flags(pdl),
                          _stream_arg(cur))
    if rc:
        _ck(rc, w)
    return out


class LoraBank:
    """S low-rank adapters of one projection: A [S][R][K], B [S][N][R] (float32,
    float16 or bfloat16), scale [S] float32, rank [S] int32 (None: all R).  The
    tensors are used in place: write an adapter's rows to load or replace it."""

    def __init__(self, A, B, scale, rank=None):
        import torch
        w = "LoraBank"
        types = {torch.float32: SQ_TYPE_F32, torch.float16: SQ_TYPE_F16, torch.bfloat16: SQ_TYPE_BF16}
        if A.dim() != 3 or B.dim() != 3 or A.dtype not in types:
            _refuse(w, "A must be [S][R][K] and B [S][N][R], float32, float16 or bfloat16")
        self.S, self.R, self.K = A.shape
        self.N = B.shape[1]
        cur = torch.cuda.current_device() if A.is_cuda else _NO_DEVICE
        v = SqLoraBank(S=self.S, R=self.R, K=self.K, N=self.N, type=types[A.dtype])
        v.A = _arg(A, A.dtype, (self.S, self.R, self.K), cur, w, "A")
        v.B = _arg(B, A.dtype, (self.S, self.N, self.R), cur, w, "B")
        v.scale = _arg(scale, torch.float32, (self.S,), cur, w, "scale")
        v.rank = _opt(rank, torch.int32, (self.S,), cur, w, "rank")
        self.view, self.A, self.B, self.scale, self.rank = v, A, B, scale, rank


def lora_workspace_bytes(bank: LoraBank, M: int) -> int:
    return int(lib().sq_lora_workspace_bytes(ctypes.byref(bank.view), M))


def new_lora_workspace(bank: LoraBank, M: int, device=None):
    """A workspace for lora_add over M tokens (one per call that may overlap
    another)."""
    import torch
    return torch.empty(max(lora_workspace_bytes(bank, M), 16), dtype=torch.uint8, device=device or bank.A.device)


def _rows_arg(t, shape, dev: int, where: str, name: str):
    """(address, row stride) of a float32 CUDA matrix with unit column stride."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or not t.is_cuda or t.dim() != 2:
        _refuse(where, f"{name} must be a float32 CUDA matrix")
    if t.shape != shape:
        _refuse(where, f"{name} must be {list(shape)}, got {list(t.shape)}", "SQ_ERR_SHAPE")
    ld, step = t.stride()
    if (step != 1 and shape[1] > 1) or (shape[0] > 1 and ld < shape[1]):
        _refuse(where, f"{name} must have unit column stride and rows that do not overlap")
    if t.get_device() != dev:
        _refuse(where, f"{name} is not on the current device")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def lora_add(bank: LoraBank, x, ids, base=None, y=None, segments: Segments = None, workspace=None, status=None,
             pdl: bool = False, stream=None):
    """y [M][N] = base + scale_a B_a (A_a x), a = ids[t] (int32, -1: no adapter).
    base and y may be column slices of wider matrices, and the same one (in
    place).  segments: segment(ids, bank.S), kept for the projections of a step."""
    import torch
    if stream is not None:
        return _on(stream, lora_add, bank, x, ids, base, y, segments, workspace, status, pdl)
    w = "sq_lora_add"
    if x.dim() != 2:
        _refuse(w, "x must be [M][K]", "SQ_ERR_SHAPE")
    M, N = x.shape[0], bank.N
    cur = torch.cuda.current_device() if x.is_cuda else _NO_DEVICE
    xp = _arg(x, torch.float32, (M, bank.K), cur, w, "x")
    if bank.A.get_device() != cur:
        _refuse(w, "the adapters are not on the current device")
    ip = _arg(ids, torch.int32, (M,), cur, w, "ids")
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=x.device)
    yp, ldy = _rows_arg(y, (M, N), cur, w, "y")
    bp, ldb = (None, N) if base is None else _rows_arg(base, (M, N), cur, w, "base")
    fp = op = None
    if segments is not None:
        fp = _arg(segments.offsets, torch.int32, (bank.S + 1,), cur, w, "segments.offsets")
        op = _arg(segments.order, torch.int32, (M,), cur, w, "segments.order")
    need = 0 if workspace is not None else lora_workspace_bytes(bank, M)
    workspace, wp, wn = _workspace_arg(workspace, need, x.device, cur, w)
    rc = lib().sq_lora_add(ctypes.byref(bank.view), xp, M, ip, fp, op, bp, ldb, yp, ldy, wp, wn,
                           _status_arg(status, cur, w), _flags(pdl), _stream_arg(cur))
    if rc:
        _ck(rc, w)
    return y


def testing_read_peak(buf, iters: int = 20, stream=None) -> float:
    """include/sq_testing.h: bytes per second of read-only sweeps of a CUDA
    tensor `buf` (contiguous, 16-byte aligned, size a multiple of 16)."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise SQError(STATUS_CODE["SQ_ERR_INVALID_ARG"], "sq_testing_read_peak: a contiguous CUDA tensor")
    out = ctypes.c_double(0.0)
    nbytes = buf.numel() * buf.element_size()
    _ck(lib().sq_testing_read_peak(buf.data_ptr(), nbytes, iters, ctypes.byref(out), _stream(stream)),
        "sq_testing_read_peak")
    return out.value


def testing_mma_peak(kind: int, iters: int = 4000, status=None, stream=None) -> float:
    """include/sq_testing.h: the measured dense tensor-core rate in ops/s
    (kind 0: int8 MMA, 1: NVFP4 block-scaled MMA)."""
    out = ctypes.c_double(0.0)
    _ck(lib().sq_testing_mma_peak(kind, iters, ctypes.byref(out), _ptr(status), _stream(stream)),
        "sq_testing_mma_peak")
    return out.value
