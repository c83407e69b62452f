"""Python binding of the W4 C ABI (include/w4.h).

Argument marshalling only: every step of the computation runs in the HIP kernels of
``libw4.so``.  PyTorch supplies device memory and the current stream.  There is no fallback:
if the library is not built, every call raises ``RuntimeError``.

Formats are named ``"nf4_f16"``, ``"nf4_bf16"``, ``"int4_f16"`` and ``"int4_bf16"`` (weight format
x activation dtype).  Scales are fp32 ``[N, K/64]`` for NF4 and bf16 bit patterns stored in an
int16 tensor ``[N, K/128]`` for INT4.  ``"fp4_*"`` (E2M1, NF4's layout), ``"int4a_*"`` (int32 words
``[N, K/128]``) and ``"mxfp4_*"`` (E2M1, uint8 power-of-two scales ``[N, K/32]``) are the others.
"""
from __future__ import annotations

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libw4.so")

FORMATS = {"nf4_f16": 1, "nf4_bf16": 2, "int4_f16": 3, "int4_bf16": 4, "fp4_f16": 5, "fp4_bf16": 6,
           "int4a_f16": 7, "int4a_bf16": 8, "mxfp4_f16": 16, "mxfp4_bf16": 17}
PATHS = {"auto": 0, "gemv": 1, "splitk": 2, "mfma": 3, "twopass": 4, "tiled": 5, "tiled_f16": 6}
PATH_NAMES = {v: k for k, v in PATHS.items()}
STATUS = {0: "OK", -1: "NULL", -2: "SHAPE", -3: "ALIGN", -4: "FORMAT", -5: "NONFINITE",
          -6: "WORKSPACE", -7: "PATH", -8: "HIP", -9: "ALIAS"}
MAX_BATCH = 4096
TILED_FROM_BATCH = 128
TILED_FROM_ROWS = 4096
MAX_SPLIT_K = 64
NOALLOC_SCRATCH_BYTES = 8 << 20

_lib = None
_torch = None  # torch, once a call has loaded it: an import statement in each of them costs as much as their checks


class W4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class W4ValueError(W4Error, ValueError):
    pass


def lib() -> ctypes.CDLL:
    """The loaded ``libw4.so``; raises RuntimeError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"W4 HIP library not built ({LIB_PATH} missing); run "
                "`python -m bit_weight_only_w4_amd.build` on a machine with ROCm")
        try:
            import torch  # noqa: F401  (its HIP runtime first: torch sees no GPU through another one)
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, sz, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.w4_quantize_nf4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.w4_quantize_int4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.w4_quantize_fp4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.w4_quantize_int4_asym.argtypes = [vp, i64, i64, vp, vp, vp]
        L.w4_quantize_mxfp4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.w4_gptq_block_update.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, i64, i64, vp, vp,
                                           vp, vp]
        L.w4_gptq_lazy_update.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp]
        L.w4_gptq_quantize.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, i64, vp, vp, vp, vp]
        L.w4_sparse24_compress.argtypes = [vp, i64, i64, ci, vp, vp, vp]
        L.w4_sparse24_gemv.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp]
        L.w4_sparse24_gemv_grouped.argtypes = [vp, ci, vp, vp, vp, ci, i64, i64, vp, vp]
        L.w4_moe_route.argtypes = [vp, ci, i64, i64, i64, ci, vp, vp, vp]
        L.w4_moe.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, i64, i64, i64, i64, i64, vp, vp, sz, vp]
        L.w4_gated.argtypes = [vp, vp, vp, ci, ci, i64, i64, i64, vp, vp, vp, sz, vp]
        L.w4_gated_workspace_bytes.argtypes = [ci, i64, i64, i64]
        L.w4_gated_workspace_bytes.restype = sz
        L.w4_gated_grad.argtypes = [vp, vp, ci, ci, i64, i64, vp, vp]
        L.w4_gemm_grad.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp, sz, vp]
        L.w4_gemm_grad_workspace_bytes.argtypes = [ci, i64, i64, i64]
        L.w4_gemm_grad_workspace_bytes.restype = sz
        L.w4_quantize_int8.argtypes = [vp, ci, i64, i64, vp, vp, vp]
        L.w4_gemm_int8.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ci, vp, sz, vp]
        L.w4_gated_int8.argtypes = [vp, vp, vp, vp, ci, i64, i64, i64, vp, vp, ci, vp, sz, vp]
        L.w4_int8_workspace_bytes.argtypes = [i64, i64, i64, ci]
        L.w4_int8_workspace_bytes.restype = sz
        L.w4_moe_workspace_bytes.argtypes = [ci, i64, i64, i64, i64, i64]
        L.w4_moe_workspace_bytes.restype = sz
        L.w4_gemv.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp]
        L.w4_gemm_smallbatch.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp]
        L.w4_gemm_prefill.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp]
        L.w4_matmul_ex.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, ci, ci, vp, sz, vp]
        L.w4_workspace_bytes.argtypes = [ci, i64, i64, i64, ci, ci]
        L.w4_workspace_bytes.restype = sz
        L.w4_auto_path.argtypes = [ci, i64, i64, i64, sz, ctypes.POINTER(ci)]
        ip = ctypes.POINTER(ci)
        L.w4_gemv_plan.argtypes = [ci, i64, i64, i64, ci, ip, ip, ip, ip, ip]
        L.w4_moe_plan.argtypes = [ci, i64, i64, i64, i64, i64, ip, ip, ip, ip, ip]
        L.w4_nf4_codebook.restype = ctypes.POINTER(ctypes.c_float)
        L.w4_status_string.argtypes = [ci]
        L.w4_status_string.restype = ctypes.c_char_p
        vpp = ctypes.POINTER(vp)
        L.w4_gemv_grouped.argtypes = [vp, ci, vpp, vpp, ctypes.POINTER(i64), vpp, ci, i64, i64, vp]
        L.w4_gemm_smallbatch_grouped.argtypes = [vp, ci, vpp, vpp, ctypes.POINTER(i64), vpp, ci, i64,
                                                 i64, vp]
        L.w4_gemv_grouped_plan.argtypes = [ci, ci, ctypes.POINTER(i64), i64, i64, ip, ip, ip, ip, ip]
        L.w4_probe_read.argtypes = [vp, sz, vp, vp]
        L.w4_probe_copy.argtypes = [vp, vp, sz, vp]
        L.w4_matmul_splitk_noalloc.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, ci, vp]
        L.w4_set_path.argtypes = [ci]
        L.w4_get_path.argtypes = []
        L.w4_set_workspace.argtypes = [vp, sz]
        for name in ("w4_quantize_nf4", "w4_quantize_int4", "w4_quantize_fp4", "w4_quantize_int4_asym",
                     "w4_quantize_mxfp4", "w4_gemv", "w4_gemm_smallbatch", "w4_matmul_ex", "w4_auto_path",
                     "w4_gemv_plan", "w4_version", "w4_probe_read", "w4_probe_copy",
                     "w4_gemv_grouped", "w4_gemv_grouped_plan", "w4_gemm_smallbatch_grouped",
                     "w4_gemm_prefill", "w4_gptq_block_update", "w4_gptq_lazy_update",
                     "w4_gptq_quantize", "w4_sparse24_compress", "w4_sparse24_gemv",
                     "w4_sparse24_gemv_grouped", "w4_set_path", "w4_get_path",
                     "w4_matmul_splitk_noalloc",
                     "w4_set_workspace", "w4_moe_route", "w4_moe", "w4_moe_plan",
                     "w4_gated", "w4_gated_grad", "w4_gemm_grad", "w4_quantize_int8", "w4_gemm_int8",
                     "w4_gated_int8"):
            getattr(L, name).restype = ci
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().w4_status_string(int(status)).decode()


def check(status: int, what: str = "w4") -> None:
    if status == 0:
        return
    msg = f"{what}: {STATUS.get(status, status)} ({status_string(status)})"
    if status == -8:
        raise W4Error(status, msg)
    raise W4ValueError(status, msg)


def nf4_codebook():
    """The 16 fp32 NF4 code points the kernels decode with (host copy from the library)."""
    p = lib().w4_nf4_codebook()
    return [p[i] for i in range(16)]


def _fmt(fmt) -> int:
    if isinstance(fmt, int):
        return fmt
    try:
        return FORMATS[fmt]
    except KeyError:
        raise ValueError(f"unknown format {fmt!r}; expected one of {sorted(FORMATS)}") from None


def _stream(stream=None) -> int:
    if stream is None:
        import torch

        # the current stream's handle without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the GPU")


def quantize_nf4(w, stream=None):
    """fp32 [N, K] device weights -> (packed uint8 [N, K/2], absmax fp32 [N, K/64])."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    absmax = torch.empty((n, max(k // 64, 1)), dtype=torch.float32, device=w.device)
    check(lib().w4_quantize_nf4(_ptr(w), n, k, _ptr(packed), _ptr(absmax), _stream(stream)),
          "w4_quantize_nf4")
    return packed, absmax


def quantize_fp4(w, stream=None):
    """fp32 [N, K] device weights -> (packed uint8 [N, K/2], scale fp32 [N, K/64]) in FP4 (E2M1)."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((n, max(k // 64, 1)), dtype=torch.float32, device=w.device)
    check(lib().w4_quantize_fp4(_ptr(w), n, k, _ptr(packed), _ptr(scale), _stream(stream)),
          "w4_quantize_fp4")
    return packed, scale


def quantize_int4(w, stream=None):
    """fp32 [N, K] device weights -> (packed uint8 [N, K/2], bf16 scale bits int16 [N, K/128])."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((n, max(k // 128, 1)), dtype=torch.int16, device=w.device)
    check(lib().w4_quantize_int4(_ptr(w), n, k, _ptr(packed), _ptr(scale), _stream(stream)),
          "w4_quantize_int4")
    return packed, scale


def quantize_int4_asym(w, stream=None):
    """fp32 [N, K] device weights -> (packed uint8 [N, K/2], words int32 [N, K/128]) in asymmetric
    INT4: each word holds the group's bf16 scale bits (bits 0-15) and zero point (bits 16-19)."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    words = torch.empty((n, max(k // 128, 1)), dtype=torch.int32, device=w.device)
    check(lib().w4_quantize_int4_asym(_ptr(w), n, k, _ptr(packed), _ptr(words), _stream(stream)),
          "w4_quantize_int4_asym")
    return packed, words


def quantize_mxfp4(w, stream=None):
    """fp32 [N, K] device weights -> (packed uint8 [N, K/2], scale uint8 [N, K/32]) in MXFP4: E2M1
    codes, scale 2^(byte - 127) per block of 32."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((n, max(k // 32, 1)), dtype=torch.uint8, device=w.device)
    check(lib().w4_quantize_mxfp4(_ptr(w), n, k, _ptr(packed), _ptr(scale), _stream(stream)),
          "w4_quantize_mxfp4")
    return packed, scale


def weight_format(fmt: str) -> str:
    """"nf4", "int4", "int4a", "fp4" or "mxfp4": the weight encoding of a format name such as "fp4_bf16"."""
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    return fmt.split("_")[0]


def quantize(fmt: str, w, stream=None):
    """Quantize fp32 [N, K] device weights in the weight encoding of `fmt` (activation type aside):
    the packed nibbles and the scales that the matmul entry points take for that format."""
    q = {"nf4": quantize_nf4, "int4": quantize_int4, "int4a": quantize_int4_asym,
         "fp4": quantize_fp4, "mxfp4": quantize_mxfp4}[weight_format(fmt)]
    return q(w, stream)


def _mm_shapes(x, packed):
    if x.dim() == 1:
        x = x.unsqueeze(0)
    b, k = x.shape
    n = packed.shape[0]
    return x, n, k, b


def gemv(x, packed, scales, fmt, y=None, stream=None):
    """y[B, N] = x[B, K] . W_hat^T via the fused single-pass GEMV (B <= 8)."""
    import torch

    x, n, k, b = _mm_shapes(x, packed)
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _need_cuda(x, packed, scales, y)
    check(lib().w4_gemv(_ptr(x), _ptr(packed), _ptr(scales), _fmt(fmt), n, k, b, _ptr(y),
                        _stream(stream)), "w4_gemv")
    return y


def grouped_args(x, packed, scales, ys):
    """ctypes arrays for w4_gemv_grouped: (packed**, scales**, N*, y**) over the members."""
    g = len(packed)
    vp = ctypes.c_void_p
    return ((vp * g)(*[p.data_ptr() for p in packed]), (vp * g)(*[s.data_ptr() for s in scales]),
            (ctypes.c_int64 * g)(*[p.shape[0] for p in packed]),
            (vp * g)(*[y.data_ptr() for y in ys]))


def _grouped_call(entry, x, packed, scales, fmt, ys, stream):
    import torch

    if len(packed) != len(scales) or (ys is not None and len(ys) != len(packed)):
        raise ValueError("packed, scales and ys must have one entry per member")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    b, k = x.shape
    if ys is None:
        ys = [torch.empty((b, p.shape[0]), dtype=torch.float32, device=x.device) for p in packed]
    _need_cuda(x, *packed, *scales, *ys)
    pp, sp, n, yp = grouped_args(x, packed, scales, ys)
    check(getattr(lib(), entry)(_ptr(x), len(packed), pp, sp, n, yp, _fmt(fmt), k, b,
                                _stream(stream)), entry)
    return ys


def gemv_grouped(x, packed, scales, fmt, ys=None, stream=None):
    """[y_g] = [x . W_hat_g^T] for weight matrices that share x, in one fused-GEMV launch.
    packed / scales are equal-length lists (at most 4 members); returns the list of y_g [B, N_g]."""
    return _grouped_call("w4_gemv_grouped", x, packed, scales, fmt, ys, stream)


def gemm_smallbatch_grouped(x, packed, scales, fmt, ys=None, stream=None):
    """gemv_grouped for batches up to W4_MAX_BATCH: one launch of the kernel the automatic path
    picks for the members' summed rows (the fused GEMV, or the MFMA kernel for larger batches);
    from W4_TILED_FROM_BATCH rows one tiled launch over the members of TILED_FROM_ROWS rows and
    more, one MFMA launch over the others."""
    return _grouped_call("w4_gemm_smallbatch_grouped", x, packed, scales, fmt, ys, stream)


def gemm_smallbatch(x, packed, scales, fmt, y=None, stream=None):
    """y[B, N] = x[B, K] . W_hat^T for B <= MAX_BATCH, GEMV, MFMA or tiled path chosen by the
    library."""
    import torch

    x, n, k, b = _mm_shapes(x, packed)
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _need_cuda(x, packed, scales, y)
    check(lib().w4_gemm_smallbatch(_ptr(x), _ptr(packed), _ptr(scales), _fmt(fmt), n, k, b,
                                   _ptr(y), _stream(stream)), "w4_gemm_smallbatch")
    return y


def gemm_prefill(x, packed, scales, fmt, y=None, stream=None):
    """y[B, N] = x[B, K] . W_hat^T through the tiled GEMM (prefill: B = prompt tokens)."""
    import torch

    x, n, k, b = _mm_shapes(x, packed)
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _need_cuda(x, packed, scales, y)
    check(lib().w4_gemm_prefill(_ptr(x), _ptr(packed), _ptr(scales), _fmt(fmt), n, k, b,
                                _ptr(y), _stream(stream)), "w4_gemm_prefill")
    return y


def workspace_bytes(fmt, n, k, b, path="auto", split_k=0) -> int:
    return int(lib().w4_workspace_bytes(_fmt(fmt), n, k, b, PATHS[path], split_k))


def auto_path(fmt, n, k, b, workspace_bytes=0):
    """(path name, split count) that the automatic choice would run."""
    sk = ctypes.c_int(0)
    r = lib().w4_auto_path(_fmt(fmt), n, k, b, workspace_bytes, ctypes.byref(sk))
    if r < 0:
        check(r, "w4_auto_path")
    return PATH_NAMES[r], sk.value


def gemv_plan(fmt, n, k, b, split_k=1):
    """dict(threads, team, iters, chunks_per_split, grid_x) of the fused GEMV launch."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    r = lib().w4_gemv_plan(_fmt(fmt), n, k, b, split_k, *[ctypes.byref(v) for v in vals])
    check(r, "w4_gemv_plan")
    return dict(zip(("threads", "team", "iters", "chunks_per_split", "grid_x"),
                    (v.value for v in vals)))


def gemv_grouped_plan(fmt, ns, k, b):
    """dict(threads, team, iters, grid_x, grid_z) of the grouped fused-GEMV launch over members
    of ns rows."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    arr = (ctypes.c_int64 * len(ns))(*ns)
    r = lib().w4_gemv_grouped_plan(_fmt(fmt), len(ns), arr, k, b, *[ctypes.byref(v) for v in vals])
    check(r, "w4_gemv_grouped_plan")
    return dict(zip(("threads", "team", "iters", "grid_x", "grid_z"), (v.value for v in vals)))


def matmul_ex(x, packed, scales, fmt, path="auto", split_k=0, workspace=None, y=None,
              stream=None):
    """The same product with an explicit path, split count and workspace (a uint8 tensor)."""
    import torch

    x, n, k, b = _mm_shapes(x, packed)
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _need_cuda(x, packed, scales, y, workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().w4_matmul_ex(_ptr(x), _ptr(packed), _ptr(scales), _fmt(fmt), n, k, b, _ptr(y),
                             PATHS[path], int(split_k), _ptr(workspace), wbytes, _stream(stream)),
          f"w4_matmul_ex[{path}]")
    return y


def set_path(path) -> None:
    """Override the automatic path of w4_gemv / w4_gemm_smallbatch ("auto" removes it)."""
    check(lib().w4_set_path(PATHS[path] if isinstance(path, str) else int(path)), "w4_set_path")


def get_path() -> str:
    """The current override's name; raises if W4_FORCE_PATH held an unknown value."""
    r = lib().w4_get_path()
    if r < 0:
        check(r, "w4_get_path")
    return PATH_NAMES[r]


def set_workspace(ws=None) -> None:
    """Register a device tensor (or None to unregister) as the current device's workspace for
    w4_gemv / w4_gemm_smallbatch.  The caller keeps the tensor alive while it is registered."""
    if ws is None:
        check(lib().w4_set_workspace(None, 0), "w4_set_workspace")
    else:
        _need_cuda(ws)
        check(lib().w4_set_workspace(_ptr(ws), ws.numel() * ws.element_size()), "w4_set_workspace")


def probe_read(src, sink, stream=None):
    _need_cuda(src, sink)
    check(lib().w4_probe_read(_ptr(src), src.numel() * src.element_size(), _ptr(sink),
                              _stream(stream)), "w4_probe_read")


def probe_copy(src, dst, stream=None):
    _need_cuda(src, dst)
    check(lib().w4_probe_copy(_ptr(src), _ptr(dst), src.numel() * src.element_size(),
                              _stream(stream)), "w4_probe_copy")


def _gptq_args(w, u, scale, zero, group):
    import torch

    _need_cuda(w, u, scale, zero)
    for t in (w, u, scale, zero):
        if t.dtype != torch.float32 or t.dim() != 2:
            raise ValueError("w, u, scale and zero must be 2-D float32 tensors")
    rows, cols = w.shape
    if tuple(u.shape) != (cols, cols):
        raise ValueError("u must be [cols, cols]")
    group = cols if group is None else int(group)
    if group < 1 or cols % group or tuple(scale.shape) != (rows, cols // group) or \
            tuple(zero.shape) != (rows, cols // group):
        raise ValueError("scale and zero must be [rows, cols // group]")
    return rows, cols, group


def gptq_outputs(w):
    """Empty (q_hat fp32, codes uint8, err fp32) buffers shaped like w."""
    import torch

    return (torch.empty_like(w), torch.empty(w.shape, dtype=torch.uint8, device=w.device),
            torch.empty_like(w))


def gptq_quantize(w, u, scale, zero, qmin, qmax, group=None, block=128, stream=None):
    """GPTQ's column loop on w [rows, cols] (fp32, updated in place) with U the upper Cholesky
    factor of the dampened inverse Hessian [cols, cols], grid scale/zero [rows, cols // group],
    codes in [qmin, qmax], lazy blocks of `block` columns.  Returns (q_hat, codes, err)."""
    rows, cols, group = _gptq_args(w, u, scale, zero, group)
    q_hat, codes, err = gptq_outputs(w)
    check(lib().w4_gptq_quantize(_ptr(w), _ptr(u), _ptr(scale), _ptr(zero), rows, cols, group,
                                 int(qmin), int(qmax), int(block), _ptr(q_hat), _ptr(codes),
                                 _ptr(err), _stream(stream)), "w4_gptq_quantize")
    return q_hat, codes, err


def gptq_block_update(w, u, scale, zero, qmin, qmax, col0, bcols, q_hat, codes, err, group=None,
                      stream=None):
    """One lazy block [col0, col0 + bcols) of the column loop (outputs written in place)."""
    rows, cols, group = _gptq_args(w, u, scale, zero, group)
    _need_cuda(q_hat, codes, err)
    check(lib().w4_gptq_block_update(_ptr(w), _ptr(u), _ptr(scale), _ptr(zero), rows, cols, group,
                                     int(qmin), int(qmax), int(col0), int(bcols), _ptr(q_hat),
                                     _ptr(codes), _ptr(err), _stream(stream)),
          "w4_gptq_block_update")


def gptq_lazy_update(w, u, err, col0, bcols, stream=None):
    """W[:, col0 + bcols:] -= E[:, col0:col0 + bcols] U[col0:col0 + bcols, col0 + bcols:]."""
    _need_cuda(w, u, err)
    rows, cols = w.shape
    check(lib().w4_gptq_lazy_update(_ptr(w), _ptr(u), _ptr(err), rows, cols, int(col0), int(bcols),
                                    _stream(stream)), "w4_gptq_lazy_update")


S24_TYPES = {"f16": 0, "bf16": 1}


def sparse24_compress(w, xtype="f16", stream=None):
    """fp32 [N, K] device weights -> (values int16 [N, K/2] (16-bit bits of `xtype`), codes uint8
    [N, K/8]) in the 2:4 format: the two largest magnitudes of every group of four kept."""
    import torch

    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    values = torch.empty((n, k // 2), dtype=torch.int16, device=w.device)
    meta = torch.empty((n, max(k // 8, 1)), dtype=torch.uint8, device=w.device)
    check(lib().w4_sparse24_compress(_ptr(w), n, k, S24_TYPES[xtype], _ptr(values), _ptr(meta),
                                     _stream(stream)), "w4_sparse24_compress")
    return values, meta


def sparse24_gemv(x, values, meta, y=None, stream=None):
    """y [B, N] fp32 = x [B, K] (fp16 or bf16) times the 2:4 matrix (values of x's type)."""
    import torch

    _need_cuda(x, values, meta)
    x2 = x if x.dim() == 2 else x.view(1, -1)
    xtype = {torch.float16: "f16", torch.bfloat16: "bf16"}[x2.dtype]
    b, k = x2.shape
    n = values.shape[0]
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    check(lib().w4_sparse24_gemv(_ptr(x2), _ptr(values), _ptr(meta), S24_TYPES[xtype], n, k, b,
                                 _ptr(y), _stream(stream)), "w4_sparse24_gemv")
    return y


def sparse24_gemv_grouped(x, values, meta, ys=None, stream=None):
    """Several 2:4 matrices sharing x in one launch: returns [y_g] (fp32 [B, N_g])."""
    import torch

    x2 = x if x.dim() == 2 else x.view(1, -1)
    _need_cuda(x2, *values, *meta)
    xtype = {torch.float16: "f16", torch.bfloat16: "bf16"}[x2.dtype]
    b, k = x2.shape
    ns = [v.shape[0] for v in values]
    if ys is None:
        ys = [torch.empty((b, n), dtype=torch.float32, device=x.device) for n in ns]
    g = len(values)
    arr = ctypes.c_void_p * g
    check(lib().w4_sparse24_gemv_grouped(
        _ptr(x2), g, arr(*[v.data_ptr() for v in values]), arr(*[m.data_ptr() for m in meta]),
        (ctypes.c_int64 * g)(*ns), S24_TYPES[xtype], k, b, arr(*[y.data_ptr() for y in ys]),
        _stream(stream)), "w4_sparse24_gemv_grouped")
    return ys


MOE_MAX_EXPERTS = 1024
MOE_MAX_TOPK = 16
_MOE_SCALES = {"nf4": ("float32", 64), "fp4": ("float32", 64), "int4": ("int16", 128),
               "int4a": ("int32", 128), "mxfp4": ("uint8", 32)}


def _expect(name, t, shape, dtype, index):
    """Refuse a tensor that is not contiguous, of this shape and type, on GPU `index`."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the first tensor's GPU")


def _on_device(index, stream):
    """None where the call can go ahead on the current device and stream, else a context to make it in:
    allocations and launches go to `stream`, or to the current stream of the tensors' device."""
    import torch

    if stream is not None:
        if stream.device.index != index:
            raise ValueError("stream and tensors must be on one device")
        return torch.cuda.stream(stream)
    # (torch.cuda.current_device() without its check that CUDA is initialized: a tensor on the GPU is)
    return None if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def moe_route(logits, top_k, renormalize=True, ids=None, weights=None, stream=None):
    """The top_k experts of each token and their softmax weights from router logits [T, E] (fp32, fp16
    or bf16): (ids int32 [T, top_k], weights fp32 [T, top_k]).  Descending, ties to the lowest expert; the
    weights are normalized over the chosen experts, or over all of them (renormalize=False).  NaN
    and -inf logits are never chosen: slots left over get id -1 and weight 0."""
    import torch

    kind = 0 if logits.dtype is torch.float32 else 1 if logits.dtype is torch.float16 else \
        2 if logits.dtype is torch.bfloat16 else None
    index = logits.get_device()
    if kind is None or logits.dim() != 2 or index < 0 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous 2-D float32, float16 or bfloat16 tensor on the GPU")
    t, e = logits.shape
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return moe_route(logits, top_k, renormalize, ids, weights)
    if ids is None:
        ids = torch.empty((t, top_k), dtype=torch.int32, device=logits.device)
    else:
        _expect("ids", ids, (t, top_k), torch.int32, index)
    if weights is None:
        weights = torch.empty((t, top_k), dtype=torch.float32, device=logits.device)
    else:
        _expect("weights", weights, (t, top_k), torch.float32, index)
    status = lib().w4_moe_route(logits.data_ptr(), kind, t, e, top_k, 1 if renormalize else 0, ids.data_ptr(),
                                weights.data_ptr(), torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_moe_route")
    return ids, weights


def moe_workspace_bytes(fmt, tokens, hidden, inter, experts, top_k) -> int:
    return int(lib().w4_moe_workspace_bytes(_fmt(fmt), tokens, hidden, inter, experts, top_k))


def moe_plan(fmt, tokens, hidden, inter, experts, top_k):
    """dict(kind, up_groups, down_groups, up_window, down_window) of a layer's launches: kind 0 a wave per
    (token, slot) pair, 1 products that an expert's pairs share, 2 the same with the pairs sorted first."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    check(lib().w4_moe_plan(_fmt(fmt), tokens, hidden, inter, experts, top_k, *[ctypes.byref(v) for v in vals]),
          "w4_moe_plan")
    return dict(zip(("kind", "up_groups", "down_groups", "up_window", "down_window"), (v.value for v in vals)))


def moe(x, ids, weights, gate_up, gate_up_scales, down, down_scales, fmt, y=None, workspace=None,
        stream=None):
    """A mixture-of-experts layer over 4-bit experts: y [T, H] fp32 with
    y[t] = sum_j weights[t, j] * Down_e(silu(Gate_e x[t]) * (Up_e x[t])), e = ids[t, j].

    x [T, H] of the format's activation type; ids int32 and weights fp32 [T, top_k] (as moe_route gives
    them; ids outside [0, E) are absent slots); gate_up uint8 [E, 2 I, H/2] (gate rows, then up
    rows) and down uint8 [E, H, I/2] with the format's scales [E, 2 I, H/g] and [E, H, I/g].
    `workspace` is a uint8 tensor of moe_workspace_bytes(...), allocated by the call if not given."""
    import torch

    code = FORMATS.get(fmt)
    if code is None:
        raise ValueError(f"unknown format {fmt!r}; expected one of {sorted(FORMATS)}")
    weight, xtype = fmt.split("_")
    index = x.get_device()
    if x.dim() != 2 or index < 0 or not x.is_contiguous() or \
            x.dtype is not (torch.float16 if xtype == "f16" else torch.bfloat16):
        raise ValueError(f"x must be a contiguous 2-D GPU tensor of the activation type of {fmt!r}")
    if ids.dim() != 2 or gate_up.dim() != 3 or down.dim() != 3:
        raise ValueError("ids must be [T, top_k], gate_up [E, 2 I, H/2] and down [E, H, I/2]")
    t, h = x.shape
    k = ids.shape[1]
    e, i = gate_up.shape[0], down.shape[2] * 2
    dtype, group = _MOE_SCALES[weight]
    dtype = getattr(torch, dtype)
    _expect("ids", ids, (t, k), torch.int32, index)
    _expect("weights", weights, (t, k), torch.float32, index)
    _expect("gate_up", gate_up, (e, 2 * i, h // 2), torch.uint8, index)
    _expect("gate_up_scales", gate_up_scales, (e, 2 * i, h // group), dtype, index)
    _expect("down", down, (e, h, i // 2), torch.uint8, index)
    _expect("down_scales", down_scales, (e, h, i // group), dtype, index)
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return moe(x, ids, weights, gate_up, gate_up_scales, down, down_scales, fmt, y, workspace)
    L = lib()
    if y is None:
        y = torch.empty((t, h), dtype=torch.float32, device=x.device)
    else:
        _expect("y", y, (t, h), torch.float32, index)
    if workspace is None:
        size = L.w4_moe_workspace_bytes(code, t, h, i, e, k)
        workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on x's GPU")
        size = workspace.numel() * workspace.element_size()
    status = L.w4_moe(x.data_ptr(), ids.data_ptr(), weights.data_ptr(), gate_up.data_ptr(),
                      gate_up_scales.data_ptr(), down.data_ptr(), down_scales.data_ptr(), code, t, h, i, e,
                      k, y.data_ptr(), workspace.data_ptr(), size, torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_moe")
    return y


ACTS = {"silu": 0, "gelu_tanh": 1}


def _load_torch():
    global _torch
    import torch

    _torch = torch
    return torch


def _act(act) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}; expected one of {sorted(ACTS)}")
    return code


def _type16(name, dtype) -> int:
    torch = _torch or _load_torch()
    if dtype is torch.float16:
        return 1
    if dtype is torch.bfloat16:
        return 2
    raise ValueError(f"{name} must be float16 or bfloat16")


def _rows(name, x, what):
    """The GPU index of a contiguous 2-D GPU tensor."""
    index = x.get_device()
    if x.dim() != 2 or index < 0 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D GPU tensor {what}")
    return index


@functools.lru_cache(maxsize=4096)
def _scratch_bytes(index, entry, *sizes):
    """A workspace size of the library (a function of the sizes and of the current device, `index`)."""
    return int(getattr(lib(), entry)(*sizes))


def _scratch(workspace, size, like, index):
    """(address, bytes, tensor) of a call's workspace: the one given, else `size` bytes allocated on `like`'s GPU."""
    torch = _torch or _load_torch()
    if workspace is None:
        if not size:
            return None, 0, None
        workspace = like.new_empty(size, dtype=torch.uint8)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the first tensor's GPU")
    else:
        size = workspace.numel() * workspace.element_size()
    return workspace.data_ptr(), size, workspace


def _block_outputs(t, i, dtype, like, index, h, products, save):
    """h [t, i] and, where wanted, products [t, 2 i], allocated like `like` if not given."""
    if h is None:
        h = like.new_empty((t, i), dtype=dtype)
    else:
        _expect("h", h, (t, i), dtype, index)
    if products is not None:
        _expect("products", products, (t, 2 * i), dtype, index)
    elif save:
        products = like.new_empty((t, 2 * i), dtype=dtype)
    return h, products


_FORMAT_SPECS = {}


def _format_spec(fmt):
    """(code, activation type, scale type, weights a scale) of a format name, kept in _FORMAT_SPECS."""
    torch = _torch or _load_torch()
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}; expected one of {sorted(FORMATS)}")
    weight, xtype = fmt.split("_")
    stype, group = _MOE_SCALES[weight]
    spec = (FORMATS[fmt], torch.float16 if xtype == "f16" else torch.bfloat16, getattr(torch, stype), group)
    _FORMAT_SPECS[fmt] = spec
    return spec


def gated_workspace_bytes(fmt, tokens, hidden, inter) -> int:
    return int(lib().w4_gated_workspace_bytes(_fmt(fmt), tokens, hidden, inter))


def gated(x, gate_up, gate_up_scales, fmt, act="silu", save=False, h=None, products=None, workspace=None,
          stream=None):
    """The first half of a gated feed-forward block over 4-bit weights, in one call: h [T, I] of x's type with
    h = act(g) * u, g = x . Wg^T, u = x . Wu^T ("silu" or "gelu_tanh").

    x [T, H] of the format's activation type; gate_up uint8 [2 I, H/2] (gate rows, then up rows) with the
    format's scales [2 I, H/g].  With save=True (or `products` given) it returns (h, products), products [T, 2 I] of x's type
    holding g | u, which gated_grad takes; results carry no autograd graph.  `workspace` is a uint8 tensor of
    gated_workspace_bytes(...), allocated by the call if not given and needed."""
    torch = _torch or _load_torch()
    a = ACTS.get(act)
    spec = _FORMAT_SPECS.get(fmt) or _format_spec(fmt)
    index = x.get_device()
    if a is None:
        raise ValueError(f"unknown activation {act!r}; expected one of {sorted(ACTS)}")
    if x.dim() != 2 or gate_up.dim() != 2 or index < 0:
        raise ValueError("x must be [T, H] and gate_up [2 I, H/2], on the GPU")
    code, dtype, stype, group = spec
    t, k = x.shape
    n = gate_up.shape[0]
    if not (x.dtype is dtype and gate_up.dtype is torch.uint8 and gate_up_scales.dtype is stype and n % 2 == 0
            and gate_up.shape[1] * 2 == k and gate_up_scales.shape == (n, k // group)
            and gate_up.get_device() == index and gate_up_scales.get_device() == index
            and x.is_contiguous() and gate_up.is_contiguous() and gate_up_scales.is_contiguous()):
        raise ValueError(f"{fmt!r} takes contiguous x [T, H] {dtype}, gate_up [2 I, H/2] uint8 and its scales "
                         f"[2 I, H/{group}] {stype}, on one GPU")
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return gated(x, gate_up, gate_up_scales, fmt, act, save, h, products, workspace)
    L = lib()
    h, products = _block_outputs(t, n // 2, dtype, x, index, h, products, save)
    address, size, workspace = _scratch(workspace, _scratch_bytes(index, "w4_gated_workspace_bytes", code, t, k, n // 2),
                                        x, index)
    status = L.w4_gated(x.data_ptr(), gate_up.data_ptr(), gate_up_scales.data_ptr(), code, a, t, k, n // 2, h.data_ptr(),
                        None if products is None else products.data_ptr(), address, size,
                        torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_gated")
    return h if products is None else (h, products)


def gated_grad(dh, products, act="silu", d_products=None, stream=None):
    """The gradients of a gated block's products from that of its output: d_products [T, 2 I] = dg | du with
    dg = dh * u * act'(g), du = dh * act(g), from dh [T, I] and products [T, 2 I] = g | u (fp16 or bf16)."""
    torch = _torch or _load_torch()
    kind, a = _type16("dh", dh.dtype), ACTS.get(act)
    index = dh.get_device()
    if a is None:
        raise ValueError(f"unknown activation {act!r}; expected one of {sorted(ACTS)}")
    if dh.dim() != 2 or index < 0:
        raise ValueError("dh must be [T, I], on the GPU")
    t, i = dh.shape
    if not (products.dtype is dh.dtype and products.shape == (t, 2 * i) and products.get_device() == index
            and dh.is_contiguous() and products.is_contiguous()):
        raise ValueError("dh [T, I] and products [T, 2 I] must be contiguous and of one type, on one GPU")
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return gated_grad(dh, products, act, d_products)
    if d_products is None:
        d_products = torch.empty_like(products)
    else:
        _expect("d_products", d_products, (t, 2 * i), dh.dtype, index)
    status = lib().w4_gated_grad(dh.data_ptr(), products.data_ptr(), kind, a, t, i, d_products.data_ptr(),
                                 torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_gated_grad")
    return d_products


def gemm_grad_workspace_bytes(fmt, n, k, b) -> int:
    return int(lib().w4_gemm_grad_workspace_bytes(_fmt(fmt), n, k, b))


def gemm_grad(d, packed, scales, fmt, dx=None, workspace=None, stream=None):
    """The input gradient of a product with frozen 4-bit weights: dx [B, K] = d [B, N] . W_hat, of d's type (the
    format's activation type).  The backward pass of gated is gemm_grad(gated_grad(dh, products), gate_up, ...), to be
    called by the user's autograd function: none of these calls is recorded.  `workspace` is a uint8 tensor of gemm_grad_workspace_bytes(...), allocated by the
    call if not given and needed."""
    torch = _torch or _load_torch()
    code, dtype, stype, group = _FORMAT_SPECS.get(fmt) or _format_spec(fmt)
    index = d.get_device()
    if d.dim() != 2 or packed.dim() != 2 or index < 0:
        raise ValueError("d must be [B, N] and packed [N, K/2], on the GPU")
    b, n = d.shape
    k = packed.shape[1] * 2
    if not (d.dtype is dtype and packed.dtype is torch.uint8 and scales.dtype is stype and packed.shape[0] == n
            and scales.shape == (n, k // group) and packed.get_device() == index and scales.get_device() == index
            and d.is_contiguous() and packed.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{fmt!r} takes contiguous d [B, N] {dtype}, packed [N, K/2] uint8 and its scales "
                         f"[N, K/{group}] {stype}, on one GPU")
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return gemm_grad(d, packed, scales, fmt, dx, workspace)
    L = lib()
    if dx is None:
        dx = d.new_empty((b, k))
    else:
        _expect("dx", dx, (b, k), dtype, index)
    address, size, workspace = _scratch(workspace, _scratch_bytes(index, "w4_gemm_grad_workspace_bytes", code, n, k, b),
                                        d, index)
    status = L.w4_gemm_grad(d.data_ptr(), packed.data_ptr(), scales.data_ptr(), code, n, k, b, dx.data_ptr(), address,
                            size, torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_gemm_grad")
    return dx


INT8_MAX_K = 131008


def _type(dtype) -> int:
    torch = _torch or _load_torch()
    return 0 if dtype is torch.float32 else _type16("the type", dtype)


def quantize_int8(x, codes=None, scales=None, stream=None):
    """Rows to 8 bits (tokens, or the channels of a weight matrix): x [R, K] fp32, fp16 or bf16 -> (codes int8
    [R, K], scales fp32 [R]), scale max|x| / 127, code the integer nearest to x / scale (ties to even).  A row
    that holds an infinity or NaN gets scale NaN."""
    torch = _torch or _load_torch()
    index = _rows("x", x, "[R, K]")
    kind = _type(x.dtype)
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return quantize_int8(x, codes, scales)
    r, k = x.shape
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.int8)
    else:
        _expect("codes", codes, (r, k), torch.int8, index)
    if scales is None:
        scales = x.new_empty(r, dtype=torch.float32)
    else:
        _expect("scales", scales, (r,), torch.float32, index)
    status = lib().w4_quantize_int8(x.data_ptr(), kind, r, k, codes.data_ptr(), scales.data_ptr(),
                                    torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_quantize_int8")
    return codes, scales


def _int8_operands(xq, xs, wq, ws):
    """(GPU index, tokens, K, weight rows) of the operands of an 8-bit product."""
    torch = _torch or _load_torch()
    index = xq.get_device()
    if xq.dim() != 2 or wq.dim() != 2 or index < 0:
        raise ValueError("xq must be [B, K] and wq [N, K], on the GPU")
    b, k = xq.shape
    n = wq.shape[0]
    i8, f32 = torch.int8, torch.float32
    if not (xq.dtype is i8 and wq.dtype is i8 and xs.dtype is f32 and ws.dtype is f32 and wq.shape[1] == k
            and xs.shape == (b,) and ws.shape == (n,) and wq.get_device() == index and xs.get_device() == index
            and ws.get_device() == index and xq.is_contiguous() and wq.is_contiguous() and xs.is_contiguous()
            and ws.is_contiguous()):
        raise ValueError("xq int8 [B, K], xs float32 [B], wq int8 [N, K] and ws float32 [N] must be contiguous, on one GPU")
    return index, b, k, n


def int8_workspace_bytes(n, k, b, gated=False) -> int:
    return int(lib().w4_int8_workspace_bytes(n, k, b, 1 if gated else 0))


def gemm_int8(xq, xs, wq, ws, dtype=None, y=None, workspace=None, stream=None):
    """y [B, N] = (xq . wq^T) * xs * ws: 8-bit codes xq int8 [B, K] and wq int8 [N, K] with a scale for each token
    and each channel (as quantize_int8 gives them), exact int32 sums.  dtype: float32 (default), float16 or bfloat16.
    `workspace` is a uint8 tensor of int8_workspace_bytes(...), allocated by the call if not given and needed."""
    torch = _torch or _load_torch()
    index, b, k, n = _int8_operands(xq, xs, wq, ws)
    if dtype is None:
        dtype = torch.float32 if y is None else y.dtype
    kind = _type(dtype)
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return gemm_int8(xq, xs, wq, ws, dtype, y, workspace)
    L = lib()
    if y is None:
        y = xs.new_empty((b, n), dtype=dtype)
    else:
        _expect("y", y, (b, n), dtype, index)
    address, size, workspace = _scratch(workspace, _scratch_bytes(index, "w4_int8_workspace_bytes", n, k, b, 0), xq, index)
    status = L.w4_gemm_int8(xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), n, k, b, y.data_ptr(), kind,
                            address, size, torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_gemm_int8")
    return y


def gated_int8(xq, xs, wq, ws, act="silu", dtype=None, save=False, h=None, products=None, workspace=None,
               stream=None):
    """gated over 8-bit tokens and weights: wq int8 [2 I, K] (gate rows, then up rows), ws [2 I]; h and products are
    of `dtype` (bfloat16, the default, or float16); `workspace` of int8_workspace_bytes(I, K, T, gated=True)."""
    torch = _torch or _load_torch()
    index, t, k, n = _int8_operands(xq, xs, wq, ws)
    if n % 2:
        raise ValueError("wq must hold as many gate rows as up rows")
    if dtype is None:
        dtype = torch.bfloat16 if h is None else h.dtype
    kind, a = _type16("the type", dtype), _act(act)
    context = _on_device(index, stream)
    if context is not None:
        with context:
            return gated_int8(xq, xs, wq, ws, act, dtype, save, h, products, workspace)
    L = lib()
    h, products = _block_outputs(t, n // 2, dtype, xq, index, h, products, save)
    address, size, workspace = _scratch(workspace, _scratch_bytes(index, "w4_int8_workspace_bytes", n // 2, k, t, 1), xq,
                                        index)
    status = L.w4_gated_int8(xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), a, t, k, n // 2, h.data_ptr(),
                             _ptr(products), kind, address, size, torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status, "w4_gated_int8")
    return h if products is None else (h, products)
