"""Python binding of libspfuse: argument marshalling only.

Every function named like a C entry point (``sp_rs_dropout_residual_norm_fwd``,
``sp_rs_bwd_workspace_bytes``, ``sp_rs_dropout_residual_norm_bwd``, ``sp2hp``,
``hp2sp``, ``sp_quantize_q8``, ``sp_matmul_q8``) passes tensor pointers, sizes and the current CUDA stream to the
function of the same name in ``libspfuse.so`` and raises ``RuntimeError`` with
the library's status string when it reports an error.  All arithmetic runs in
the library's CUDA kernels; there is no other implementation to fall back to:
if the library is missing, the first call raises.

``forward`` / ``backward`` / ``sp2hp_out`` / ``hp2sp_out`` are conveniences
that allocate the outputs with torch (device memory only) and call the above;
so are ``forward_q8``, ``quantize_q8``, ``matmul_q8`` and
``linear_q8_backward``, the 8-bit operators behind the norm.

An 8-bit tensor is a pair: values ([R, C], ``torch.float8_e4m3fn`` or
``torch.float8_e5m2``) and scale bytes ([R, ceil(C/128)] ``torch.uint8``, or
[ceil(R/128), ceil(C/128)] for 128 x 128 blocks; a byte b stands for
2^(b - 127), as ``torch.float8_e8m0fnu`` reads it).  Both have row strides of
a multiple of 16 bytes (``q8_empty`` allocates such a matrix).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from .build import LIB_PATH, source_hash

SP_F32, SP_BF16 = 0, 1
SP_RMSNORM, SP_LAYERNORM = 0, 1
DTYPE_CODE = {torch.float32: SP_F32, torch.bfloat16: SP_BF16}
NAME_CODE = {"f32": SP_F32, "bf16": SP_BF16}
NORM_CODE = {"rms": SP_RMSNORM, "ln": SP_LAYERNORM}
ELEM_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.float8_e5m2: 3}
Q8_DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
Q8_GROUP = 128


class SpRsDesc(ctypes.Structure):
    """Mirror of sp_rs_desc_t (include/spfuse.h)."""
    _fields_ = [("T", ctypes.c_int32), ("j", ctypes.c_int32), ("S", ctypes.c_int64),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("p", ctypes.c_float), ("eps", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("nshards", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("status", ctypes.c_void_p)]

    @property
    def R(self) -> int:
        return (self.S // self.T) * self.B

    @property
    def rows(self) -> int:
        return self.R * max(1, self.nshards)


class SpKernelPlan(ctypes.Structure):
    """Mirror of sp_kernel_plan_t (include/spfuse.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("tma", "block", "nthr", "tpr", "vpt", "row_groups",
                                              "rows_per_stage", "stages", "chunked", "noalloc_fits")] + \
               [(n, ctypes.c_int64) for n in ("stage_bytes", "smem_bytes", "rows_per_cta", "ctas",
                                              "workspace_bytes")]


class SpPlanInfo(ctypes.Structure):
    """Mirror of sp_plan_info_t (include/spfuse.h)."""
    _fields_ = [("fwd", SpKernelPlan), ("bwd", SpKernelPlan)]


class SpQuantizeQ8Desc(ctypes.Structure):
    """Mirror of sp_quantize_q8_desc_t (include/spfuse.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("M", "K", "ldx", "ldx_scale", "ldq", "ldq_scale", "ldqt",
                                              "ldqt_scale")] + \
               [(n, ctypes.c_int32) for n in ("x_dtype", "q_dtype", "x_scale_rows", "block")] + \
               [("reserved", ctypes.c_int64)]


class SpMatmulQ8Desc(ctypes.Structure):
    """Mirror of sp_matmul_q8_desc_t (include/spfuse.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("M", "N", "K", "lda", "ldb", "lda_scale", "ldb_scale", "ldc")] + \
               [(n, ctypes.c_int32) for n in ("a_dtype", "b_dtype", "c_dtype", "a_scale_rows", "b_scale_rows",
                                              "accumulate")] + [("status", ctypes.c_void_p)]


class SpMatmulQ8Plan(ctypes.Structure):
    """Mirror of sp_matmul_q8_plan_t (include/spfuse.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("pair", "swapped", "bn", "split_k", "stages", "block", "tmem_cols",
                                              "acc1_col", "scale_col", "ctas_per_sm")] + \
               [(n, ctypes.c_int64) for n in ("stage_bytes", "smem_bytes", "tiles", "ctas")]


def make_desc(T, j, S, B, H, dtype="bf16", norm="rms", p=0.0, eps=1e-6, seed=0, nshards=1,
              status=None):
    """status: an int32/uint32 CUDA tensor of one element (the device status
    word, see include/spfuse.h) or None."""
    return SpRsDesc(T=T, j=j, S=S, B=B, H=H, dtype=NAME_CODE.get(dtype, dtype),
                    norm=NORM_CODE.get(norm, norm), p=p, eps=eps, seed=int(seed) & (2**64 - 1),
                    nshards=nshards, reserved=0, status=_ptr(status))


_lib = None


def lib() -> ctypes.CDLL:
    """Load libspfuse.so (built by ``residual_sp_rs_gb300.build.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libspfuse.so is not built ({LIB_PATH}); run residual_sp_rs_gb300.build.build() "
                "with the CUDA toolkit installed. There is no fallback implementation.")
        L = ctypes.CDLL(LIB_PATH)
        L.sp_build_hash.restype = ctypes.c_char_p
        L.sp_build_hash.argtypes = []
        _verify_hash(L, source_hash())
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(SpRsDesc)
        L.sp_rs_dropout_residual_norm_fwd.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_fwd.argtypes = [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sp_rs_dropout_residual_norm_fwd_rows.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_fwd_rows.argtypes = [D, i64, i64, vp, vp, vp, vp, vp, vp, vp,
                                                           vp, vp, vp]
        L.sp_rs_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.sp_rs_bwd_workspace_bytes.argtypes = [D]
        L.sp_rs_dropout_residual_norm_bwd.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_bwd.argtypes = [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                      vp, vp, ctypes.c_size_t, vp]
        L.sp_rs_dropout_residual_norm_bwd_rows.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_bwd_rows.argtypes = [D, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp,
                                                           vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.sp_rs_dropout_residual_norm_fwd_q8.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_fwd_q8.argtypes = [D, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp]
        L.sp_rs_dropout_residual_norm_fwd_q8_rows.restype = ctypes.c_int
        L.sp_rs_dropout_residual_norm_fwd_q8_rows.argtypes = [D, i64, i64, vp, vp, vp, vp, vp, vp, i64, vp, i64,
                                                              vp, vp, vp, vp]
        L.sp_quantize_q8.restype = ctypes.c_int
        L.sp_quantize_q8.argtypes = [ctypes.POINTER(SpQuantizeQ8Desc), vp, vp, vp, vp, vp, vp, vp]
        L.sp_matmul_q8.restype = ctypes.c_int
        L.sp_matmul_q8.argtypes = [ctypes.POINTER(SpMatmulQ8Desc), vp, vp, vp, vp, vp, vp]
        L.sp_matmul_q8_plan.restype = ctypes.c_int
        L.sp_matmul_q8_plan.argtypes = [ctypes.POINTER(SpMatmulQ8Desc), i32, i32, ctypes.POINTER(SpMatmulQ8Plan)]
        for name in ("sp2hp", "hp2sp"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [vp, vp, i64, i64, i32, i32, vp]
        L.sp_status_string.restype = ctypes.c_char_p
        L.sp_status_string.argtypes = [ctypes.c_int]
        L.sp_version.restype = ctypes.c_int32
        L.sp_version.argtypes = []
        L.sp_last_cuda_error.restype = ctypes.c_char_p
        L.sp_last_cuda_error.argtypes = []
        L.sp_plan_describe.restype = ctypes.c_int
        L.sp_plan_describe.argtypes = [D, i32, i32, i32, i32, ctypes.POINTER(SpPlanInfo)]
        _lib = L
    return _lib


def _verify_hash(L: ctypes.CDLL, expected: str) -> None:
    """Refuse a library built from other sources than these."""
    got = L.sp_build_hash().decode()
    if got != expected:
        raise RuntimeError(f"libspfuse.so is stale: built from sources {got[:12]}, the tree is "
                           f"{expected[:12]}; rebuild it with residual_sp_rs_gb300.build.build()")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("libspfuse takes dense row-major tensors")
    return t.data_ptr()


def _addr(t):
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _rows2d(t):
    """Address and row stride (elements) of a matrix with dense rows."""
    if t is None:
        return None, 0
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("libspfuse takes matrices with dense rows")
    return t.data_ptr(), stride[0] if shape[0] > 1 else max(stride[0], shape[1])


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(code: int):
    if code != 0:
        msg = lib().sp_status_string(code).decode()
        if code == 6:  # SP_ERR_CUDA
            msg += f" ({lib().sp_last_cuda_error().decode()})"
        raise RuntimeError(msg)


def sp_plan_describe(desc: SpRsDesc, sms: int, smem_optin: int, has_dh: bool = True,
                     has_mask: bool = True) -> dict:
    """The launch configurations the forward and backward would use on a device
    with `sms` multiprocessors and `smem_optin` bytes of opt-in shared memory
    per block; host arithmetic only (no GPU needed).  Returns
    {"fwd": {...}, "bwd": {...}} with the fields of sp_kernel_plan_t."""
    info = SpPlanInfo()
    _check(lib().sp_plan_describe(ctypes.byref(desc), int(sms), int(smem_optin), int(bool(has_dh)),
                                  int(bool(has_mask)), ctypes.byref(info)))
    out = {}
    for k in ("fwd", "bwd"):
        kp = getattr(info, k)
        out[k] = {n: getattr(kp, n) for n, _ in SpKernelPlan._fields_}
    return out


def status_string(code: int) -> str:
    return lib().sp_status_string(code).decode()


# ---- C entry points, same names ---------------------------------------------------

def sp_rs_dropout_residual_norm_fwd(desc: SpRsDesc, partials, residual, gamma, beta, h_out, y_out,
                                    mask_out, rstd_out, mean_out, stream=None) -> None:
    arr = (ctypes.c_void_p * max(1, len(partials)))(*[_ptr(p) for p in partials])
    _check(lib().sp_rs_dropout_residual_norm_fwd(
        ctypes.byref(desc), arr, _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(h_out),
        _ptr(y_out), _ptr(mask_out), _ptr(rstd_out), _ptr(mean_out), _stream(stream)))


def sp_rs_dropout_residual_norm_fwd_rows(desc: SpRsDesc, row_begin: int, row_count: int, partials,
                                         residual, gamma, beta, h_out, y_out, mask_out, rstd_out,
                                         mean_out, stream=None) -> None:
    arr = (ctypes.c_void_p * max(1, len(partials)))(*[_ptr(p) for p in partials])
    _check(lib().sp_rs_dropout_residual_norm_fwd_rows(
        ctypes.byref(desc), int(row_begin), int(row_count), arr, _ptr(residual), _ptr(gamma),
        _ptr(beta), _ptr(h_out), _ptr(y_out), _ptr(mask_out), _ptr(rstd_out), _ptr(mean_out),
        _stream(stream)))


def sp_rs_bwd_workspace_bytes(desc: SpRsDesc) -> int:
    return int(lib().sp_rs_bwd_workspace_bytes(ctypes.byref(desc)))


def sp_rs_dropout_residual_norm_bwd(desc: SpRsDesc, dy, dh_out, h_saved, gamma, mask, rstd, mean,
                                    d_residual, d_sum, dgamma, dbeta, workspace,
                                    workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().sp_rs_dropout_residual_norm_bwd(
        ctypes.byref(desc), _ptr(dy), _ptr(dh_out), _ptr(h_saved), _ptr(gamma), _ptr(mask),
        _ptr(rstd), _ptr(mean), _ptr(d_residual), _ptr(d_sum), _ptr(dgamma), _ptr(dbeta),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def sp_rs_dropout_residual_norm_bwd_rows(desc: SpRsDesc, row_begin: int, row_count: int, accumulate: bool,
                                         dy, dh_out, h_saved, gamma, mask, rstd, mean, d_residual, d_sum,
                                         dgamma, dbeta, workspace, stream=None) -> None:
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().sp_rs_dropout_residual_norm_bwd_rows(
        ctypes.byref(desc), int(row_begin), int(row_count), int(bool(accumulate)), _ptr(dy), _ptr(dh_out),
        _ptr(h_saved), _ptr(gamma), _ptr(mask), _ptr(rstd), _ptr(mean), _ptr(d_residual), _ptr(d_sum),
        _ptr(dgamma), _ptr(dbeta), _ptr(workspace), nbytes, _stream(stream)))


def sp2hp(inp, out, N, H, T, dtype, stream=None) -> None:
    _check(lib().sp2hp(_ptr(inp), _ptr(out), N, H, T, NAME_CODE.get(dtype, dtype), _stream(stream)))


def hp2sp(inp, out, N, H, T, dtype, stream=None) -> None:
    _check(lib().hp2sp(_ptr(inp), _ptr(out), N, H, T, NAME_CODE.get(dtype, dtype), _stream(stream)))


def sp_rs_dropout_residual_norm_fwd_q8(desc: SpRsDesc, partials, residual, gamma, beta, h_out, q_out, scale_out,
                                       mask_out, rstd_out, mean_out, stream=None) -> None:
    arr = (ctypes.c_void_p * max(1, len(partials)))(*[_ptr(p) for p in partials])
    q, ldq = _rows2d(q_out)
    s, lds = _rows2d(scale_out)
    _check(lib().sp_rs_dropout_residual_norm_fwd_q8(
        ctypes.byref(desc), arr, _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(h_out), q, ldq, s, lds,
        _ptr(mask_out), _ptr(rstd_out), _ptr(mean_out), _stream(stream)))


def sp_rs_dropout_residual_norm_fwd_q8_rows(desc: SpRsDesc, row_begin: int, row_count: int, partials, residual,
                                            gamma, beta, h_out, q_out, scale_out, mask_out, rstd_out, mean_out,
                                            stream=None) -> None:
    arr = (ctypes.c_void_p * max(1, len(partials)))(*[_ptr(p) for p in partials])
    q, ldq = _rows2d(q_out)
    s, lds = _rows2d(scale_out)
    _check(lib().sp_rs_dropout_residual_norm_fwd_q8_rows(
        ctypes.byref(desc), int(row_begin), int(row_count), arr, _ptr(residual), _ptr(gamma), _ptr(beta),
        _ptr(h_out), q, ldq, s, lds, _ptr(mask_out), _ptr(rstd_out), _ptr(mean_out), _stream(stream)))


def sp_quantize_q8(desc: SpQuantizeQ8Desc, x, x_scale, q, q_scale, qt, qt_scale, stream=None) -> None:
    """Pointers or tensors; the strides are the descriptor's."""
    _check(lib().sp_quantize_q8(ctypes.byref(desc), _addr(x), _addr(x_scale), _addr(q), _addr(q_scale), _addr(qt),
                                _addr(qt_scale), _stream(stream)))


def sp_matmul_q8(desc: SpMatmulQ8Desc, a, a_scale, b, b_scale, c, stream=None) -> None:
    """Pointers or tensors; the strides are the descriptor's."""
    _check(lib().sp_matmul_q8(ctypes.byref(desc), _addr(a), _addr(a_scale), _addr(b), _addr(b_scale), _addr(c),
                              _stream(stream)))


def sp_matmul_q8_plan(desc: SpMatmulQ8Desc, sms: int, smem_optin: int) -> dict:
    """The launch configuration of the product `desc` on a device with `sms`
    multiprocessors and `smem_optin` bytes of opt-in shared memory per block;
    host arithmetic only (no GPU needed)."""
    info = SpMatmulQ8Plan()
    _check(lib().sp_matmul_q8_plan(ctypes.byref(desc), int(sms), int(smem_optin), ctypes.byref(info)))
    return {n: getattr(info, n) for n, _ in SpMatmulQ8Plan._fields_}


# ---- conveniences that allocate outputs ------------------------------------------

def forward(desc: SpRsDesc, partials, residual, gamma, beta=None, stream=None,
            store_mask: bool = True) -> dict:
    """store_mask=False: the mask is not stored (the backward regenerates it)."""
    rows, H = desc.rows, desc.H
    dev, dt = residual.device, residual.dtype
    out = dict(h=torch.empty((rows, H), device=dev, dtype=dt),
               y=torch.empty((rows, H), device=dev, dtype=dt),
               mask=torch.empty((rows, H), device=dev, dtype=torch.uint8)
               if desc.p > 0 and store_mask else None,
               rstd=torch.empty(rows, device=dev, dtype=torch.float32),
               mean=torch.empty(rows, device=dev, dtype=torch.float32)
               if desc.norm == SP_LAYERNORM else None)
    sp_rs_dropout_residual_norm_fwd(desc, partials, residual, gamma, beta, out["h"], out["y"],
                                    out["mask"], out["rstd"], out["mean"], stream)
    return out


def workspace_for(desc: SpRsDesc, device) -> torch.Tensor:
    n = sp_rs_bwd_workspace_bytes(desc)
    return torch.empty(max(16, n), device=device, dtype=torch.uint8)


def backward(desc: SpRsDesc, dy, dh_out, h_saved, gamma, mask, rstd, mean=None, workspace=None,
             stream=None) -> dict:
    rows, H = desc.rows, desc.H
    dev, dt = dy.device, dy.dtype
    if workspace is None:
        workspace = workspace_for(desc, dev)
    out = dict(d_res=torch.empty((rows, H), device=dev, dtype=dt),
               d_sum=torch.empty((rows, H), device=dev, dtype=dt),
               dgamma=torch.empty(H, device=dev, dtype=torch.float32),
               dbeta=torch.empty(H, device=dev, dtype=torch.float32)
               if desc.norm == SP_LAYERNORM else None)
    sp_rs_dropout_residual_norm_bwd(desc, dy, dh_out, h_saved, gamma, mask, rstd, mean,
                                    out["d_res"], out["d_sum"], out["dgamma"], out["dbeta"],
                                    workspace, stream=stream)
    return out


def sp2hp_out(x: torch.Tensor, T: int, stream=None) -> torch.Tensor:
    N, H = x.shape
    out = torch.empty((T, N, H // T), device=x.device, dtype=x.dtype)
    sp2hp(x, out, N, H, T, DTYPE_CODE[x.dtype], stream)
    return out


def hp2sp_out(x: torch.Tensor, stream=None) -> torch.Tensor:
    T, N, Hc = x.shape
    out = torch.empty((N, Hc * T), device=x.device, dtype=x.dtype)
    hp2sp(x, out, N, Hc * T, T, DTYPE_CODE[x.dtype], stream)
    return out


# ---- the 8-bit operators -----------------------------------------------------------

def q8_empty(rows: int, cols: int, device, dtype=torch.uint8) -> torch.Tensor:
    """An uninitialised [rows, cols] matrix of one-byte values whose rows start
    a multiple of 16 bytes apart, as the 8-bit operators take them (of 128 for
    longer rows, which then begin at cache lines: the gradients of 8177 tokens
    took 14% longer over rows that straddle lines)."""
    return torch.empty_strided((rows, cols), (_q8_ld(cols), 1), dtype=dtype, device=device)


def _q8_ld(n: int) -> int:
    return (n + 127) // 128 * 128 if n >= 512 else (n + 15) // 16 * 16 or 16


def _groups(n: int) -> int:
    return (n + Q8_GROUP - 1) // Q8_GROUP


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device and the caller's stream as the current ones, so that
    outputs and intermediates are allocated for the stream that uses them."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _elsewhere(dev, stream) -> bool:
    """Whether a call for tensors on device `dev` (an index) has to go through _on."""
    return stream is not None or dev != torch.cuda.current_device()


def _same_device(*tensors):
    """The index of the CUDA device that every tensor (or None) is on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}: all must be on one device")
    if dev < 0:
        raise ValueError("libspfuse takes CUDA tensors")
    return dev


_Q8_CODE = {torch.float8_e4m3fn: 2, torch.float8_e5m2: 3}
_SCALE_DTYPES = {torch.uint8, torch.float8_e8m0fnu}


def _q8_operand(name, t, scale):
    """(address, row stride, scales' address, their row stride, rows per scale) of an 8-bit tensor."""
    if t.dtype not in _Q8_CODE:
        raise ValueError(f"{name}: float8_e4m3fn or float8_e5m2 expected, got {t.dtype}")
    if scale is None or scale.dtype not in _SCALE_DTYPES:
        raise ValueError(f"{name}: a matrix of scale bytes expected")
    shape, sshape = t.shape, scale.shape
    if len(shape) != 2 or len(sshape) != 2:
        raise ValueError(f"{name}: a matrix and its matrix of scale bytes expected")
    rows, cols = shape
    srows, groups = sshape
    if groups != (cols + 127) // 128 or (srows != rows and srows != (rows + 127) // 128):
        raise ValueError(f"{name}: values {tuple(shape)} do not go with scales {tuple(sshape)}")
    ld, step = t.stride()
    lds, sstep = scale.stride()
    if (step != 1 and cols > 1) or (sstep != 1 and groups > 1):
        raise ValueError(f"{name}: libspfuse takes matrices with dense rows")
    if rows <= 1 or groups == 0:  # the stride is not used, and a view may carry any
        ld, lds = _q8_ld(cols), _q8_ld(groups)
    elif srows == 1:
        lds = _q8_ld(groups)
    return t.data_ptr(), ld, scale.data_ptr(), lds, 1 if srows == rows else Q8_GROUP


def forward_q8(desc: SpRsDesc, partials, residual, gamma, beta=None, stream=None, store_mask: bool = True) -> dict:
    """`forward` with the norm's output in e4m3: `q` [rows, H] and `scale`
    [rows, ceil(H/128)] in the place of `y`.  `backward` takes the rest."""
    dev = _same_device(residual, gamma, beta, *partials)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return forward_q8(desc, partials, residual, gamma, beta, store_mask=store_mask)
    rows, H, T, ln = desc.rows, desc.H, desc.T, desc.norm == SP_LAYERNORM
    dt = residual.dtype
    if DTYPE_CODE.get(dt) != desc.dtype or gamma.dtype != dt:
        raise ValueError("the tensors' types do not match the descriptor")
    if len(partials) != T or residual.numel() != rows * H or gamma.numel() != H:
        raise ValueError("the tensors' sizes do not match the descriptor")
    n = desc.S * desc.B * H
    for t in partials:
        if t.dtype != dt or t.numel() != n:
            raise ValueError("the partials' types or sizes do not match the descriptor")
    if ln and (beta is None or beta.dtype != dt or beta.numel() != H):
        raise ValueError("LayerNorm needs beta, as gamma")
    cuda, groups = residual.device, _groups(H)
    h = torch.empty((rows, H), device=cuda, dtype=dt)
    q = q8_empty(rows, H, cuda, torch.float8_e4m3fn)
    s = q8_empty(rows, groups, cuda)
    mask = torch.empty((rows, H), device=cuda, dtype=torch.uint8) if store_mask and desc.p > 0 else None
    rstd = torch.empty(rows, device=cuda, dtype=torch.float32)
    mean = torch.empty(rows, device=cuda, dtype=torch.float32) if ln else None
    _check(lib().sp_rs_dropout_residual_norm_fwd_q8(
        ctypes.byref(desc), (ctypes.c_void_p * T)(*[_ptr(p) for p in partials]), _ptr(residual), _ptr(gamma),
        _ptr(beta), h.data_ptr(), q.data_ptr(), _q8_ld(H), s.data_ptr(), _q8_ld(groups), _ptr(mask),
        rstd.data_ptr(), _ptr(mean), _stream(None)))
    return dict(h=h, q=q, scale=s, mask=mask, rstd=rstd, mean=mean)


def quantize_q8(x: torch.Tensor, fmt: str = "e4m3", block: bool = False, rowwise: bool = True, colwise: bool = False,
                scale: torch.Tensor | None = None, stream=None) -> dict:
    """x [M, K] (float32, bfloat16, or 8-bit values with their `scale` bytes) to
    8 bits: `q`, `scale` along its rows and/or `qt` [K, M], `scale_t` along its
    columns (the transposed tensor); with `block` one scale per 128 x 128 block.
    Outputs not asked for are None."""
    xcode, out8 = ELEM_CODE.get(x.dtype, -1), Q8_DTYPE.get(fmt)
    if len(x.shape) != 2 or xcode < 0 or out8 is None:
        raise ValueError("a matrix of float32, bfloat16 or 8-bit values and a format e4m3 or e5m2 expected")
    if not rowwise and not colwise:
        raise ValueError("neither rowwise nor colwise: nothing to do")
    dev = _same_device(x, scale)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return quantize_q8(x, fmt, block, rowwise, colwise, scale)
    M, K = x.shape
    ps, ldxs, srows = None, 0, 0
    if xcode >= 2:
        px, ldx, ps, ldxs, srows = _q8_operand("x", x, scale)
    else:
        if scale is not None:
            raise ValueError("only an 8-bit x has scales")
        px, ldx = _rows2d(x)
    mg, kg = _groups(M), _groups(K)
    q = s = qt = st = pq = pqs = pqt = pqts = None
    ldq, ldqt = _q8_ld(K), _q8_ld(M)
    cuda = x.device
    if rowwise:
        q, s = q8_empty(M, K, cuda, out8), q8_empty(mg if block else M, kg, cuda)
        pq, pqs = q.data_ptr(), s.data_ptr()
    if colwise:
        qt, st = q8_empty(K, M, cuda, out8), q8_empty(kg if block else K, mg, cuda)
        pqt, pqts = qt.data_ptr(), st.data_ptr()
    if M > 0 and K > 0:
        d = SpQuantizeQ8Desc(M, K, ldx, ldxs, ldq, _q8_ld(kg), ldqt, _q8_ld(mg), xcode, ELEM_CODE[out8], srows,
                             1 if block else 0, 0)
        _check(lib().sp_quantize_q8(ctypes.byref(d), px, ps, pq, pqs, pqt, pqts, _stream(None)))
    return dict(q=q, scale=s, qt=qt, scale_t=st)


def matmul_q8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
              out: torch.Tensor | None = None, out_dtype=torch.bfloat16, accumulate: bool = False,
              stream=None, status=None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed, both 8-bit tensors, to [M, N] of
    `out_dtype` (bfloat16 or float32); into `out` when given (its type then
    counts), added to what a float32 `out` holds with `accumulate`.  `status`:
    the device status word (as in `make_desc`) that a wait that ran out is
    reported in; the tiles that it left unfinished are NaN."""
    if accumulate and out is None:
        raise ValueError("accumulate needs the out to add to")
    dev = _same_device(a, a_scale, b, b_scale, out, status)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return matmul_q8(a, a_scale, b, b_scale, out, out_dtype, accumulate, status=status)
    pa, lda, psa, ldas, asr = _q8_operand("a", a, a_scale)
    pb, ldb, psb, ldbs, bsr = _q8_operand("b", b, b_scale)
    (M, K), (N, Kb) = a.shape, b.shape
    if K != Kb:
        raise ValueError(f"a [M, K] and b [N, K] expected, got {tuple(a.shape)} and {tuple(b.shape)}")
    if out is None:
        out = torch.empty((M, N), device=a.device, dtype=out_dtype)
        pc, ldc = out.data_ptr(), N
    else:
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out is {tuple(out.shape)}, the product {(M, N)}")
        pc, ldc = _rows2d(out)
    code = DTYPE_CODE.get(out.dtype)
    if code is None:
        raise ValueError("out: bfloat16 or float32 expected")
    if M > 0 and N > 0:
        d = SpMatmulQ8Desc(M, N, K, lda, ldb, ldas, ldbs, ldc, _Q8_CODE[a.dtype], _Q8_CODE[b.dtype], code, asr, bsr,
                           1 if accumulate else 0, _ptr(status))
        _check(lib().sp_matmul_q8(ctypes.byref(d), pa, psa, pb, psb, pc, _stream(None)))
    return out


def linear_q8_backward(dy: torch.Tensor, x_q: torch.Tensor, x_scale: torch.Tensor, wt_q: torch.Tensor,
                       wt_scale: torch.Tensor, fmt: str = "e4m3", dw: torch.Tensor | None = None,
                       dx_dtype=torch.bfloat16, stream=None, status=None) -> dict:
    """Gradients of y = x W^T from dy [M, N] (float32 or bfloat16): `dx` [M, K]
    = dy W and `dw` [N, K] = dy^T x (float32; added to the given `dw`).  x_q
    [M, K] is the forward's 8-bit input, wt_q [K, N] the transposed weight
    (quantize_q8's qt).  dy goes to 8 bits (`fmt`) along N for dx and along its
    tokens for dw, where x is requantised along its tokens too.  A product whose
    wait runs out reports it in the `status` word, as `matmul_q8` does."""
    dev = _same_device(dy, x_q, x_scale, wt_q, wt_scale, dw, status)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return linear_q8_backward(dy, x_q, x_scale, wt_q, wt_scale, fmt, dw, dx_dtype, status=status)
    q8, code = _Q8_CODE.get(Q8_DTYPE.get(fmt)), DTYPE_CODE.get(dy.dtype)
    if len(dy.shape) != 2 or code is None or q8 is None:
        raise ValueError("dy: a matrix of float32 or bfloat16 and a format e4m3 or e5m2 expected")
    px, ldx, pxs, ldxs, xsr = _q8_operand("x_q", x_q, x_scale)
    pw, ldw, pws, ldws, wsr = _q8_operand("wt_q", wt_q, wt_scale)
    (M, N), K = dy.shape, x_q.shape[1]
    if x_q.shape[0] != M or tuple(wt_q.shape) != (K, N):
        raise ValueError(f"dy [M, N], x_q [M, K] and wt_q [K, N] expected, got {tuple(dy.shape)}, {tuple(x_q.shape)} "
                         f"and {tuple(wt_q.shape)}")
    if dx_dtype not in DTYPE_CODE:
        raise ValueError("dx: bfloat16 or float32 expected")
    accumulate, cuda = 0 if dw is None else 1, dy.device
    if accumulate and (dw.dtype != torch.float32 or tuple(dw.shape) != (N, K)):
        raise ValueError(f"dw: float32 of {(N, K)} expected, got {dw.dtype} of {tuple(dw.shape)}")
    if M == 0 or N == 0 or K == 0:  # sums of nothing
        return dict(dx=torch.zeros((M, K), device=cuda, dtype=dx_dtype),
                    dw=torch.zeros((N, K), device=cuda, dtype=torch.float32) if dw is None else dw)
    dx = torch.empty((M, K), device=cuda, dtype=dx_dtype)
    if dw is None:
        dw = torch.empty((N, K), device=cuda, dtype=torch.float32)
    pdy, ldy = _rows2d(dy)
    pdw, lddw = _rows2d(dw)
    # dY in both directions and x^T, values and scales, in one buffer of the
    # current stream, each part at a cache line
    ldm, ldmg, ldn, ldng = _q8_ld(M), _q8_ld(_groups(M)), _q8_ld(N), _q8_ld(_groups(N))
    at, total = [], 0
    for n in (M * ldn, M * ldng, N * ldm, N * ldmg, K * ldm, K * ldmg):
        at.append(total)
        total += (n + 127) // 128 * 128
    buf = torch.empty(total, device=cuda, dtype=torch.uint8)
    q, qs, qt, qts, xt, xts = [buf.data_ptr() + n for n in at]
    L, st, ref, xcode, word = lib(), _stream(None), ctypes.byref, _Q8_CODE[x_q.dtype], _ptr(status)
    _check(L.sp_quantize_q8(ref(SpQuantizeQ8Desc(M, N, ldy, 0, ldn, ldng, ldm, ldmg, code, q8, 0, 0, 0)),
                            pdy, None, q, qs, qt, qts, st))
    _check(L.sp_quantize_q8(ref(SpQuantizeQ8Desc(M, K, ldx, ldxs, 0, 0, ldm, ldmg, xcode, xcode, xsr, 0, 0)),
                            px, pxs, None, None, xt, xts, st))
    _check(L.sp_matmul_q8(ref(SpMatmulQ8Desc(M, K, N, ldn, ldw, ldng, ldws, K, q8, _Q8_CODE[wt_q.dtype],
                                             DTYPE_CODE[dx_dtype], 1, wsr, 0, word)), q, qs, pw, pws, dx.data_ptr(), st))
    _check(L.sp_matmul_q8(ref(SpMatmulQ8Desc(N, K, M, ldm, ldm, ldmg, ldmg, lddw, q8, xcode, 0, 1, 1, accumulate, word)),
                          qt, qts, xt, xts, pdw, st))
    return dict(dx=dx, dw=dw)
