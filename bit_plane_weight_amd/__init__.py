"""bit_plane_weight_amd - ternary bit-plane (.trit v1) GEMV on AMD Instinct MI355X (gfx950).

A thin binding over libbpw's C ABI (include/bpw.h) with the same entry-point names. Every step
of the computation runs in libbpw's HIP kernels; this module only marshals arguments. PyTorch
is used for device memory (tensors passed by data_ptr()) and streams. Host buffers are numpy
arrays.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

from . import _lib
from ._lib import (BpwDevMat, BpwError, BpwGemvJob, BpwQuantJob, KERNEL_AUTO, KERNEL_BITSERIAL,  # noqa: F401
                   KERNEL_BYTELANE, KERNEL_MFMA)

__all__ = [
    "BpwError", "KERNEL_AUTO", "KERNEL_BITSERIAL", "KERNEL_BYTELANE", "KERNEL_MFMA",
    "bpw_abi_version", "bpw_status_string", "bpw_last_error", "bpw_device_check",
    "bpw_pack_i8", "bpw_validate", "bpw_load", "HostMat", "bpw_upload", "DevMat",
    "gemv_job", "bpw_gemv_workspace_bytes", "bpw_gemv", "bpw_gemv_noalloc", "GemvPlan",
    "intmlp_job", "bpw_gemv_intmlp_workspace_bytes",
    "bpw_gemm_small_batch", "sb_job", "bpw_gemm_small_batch_workspace_bytes", "SmallBatchPlan", "quant_job", "bpw_quantize_workspace_bytes", "bpw_quantize", "QuantPlan",
    "bpw_dense_head_gemv", "bpw_stream_read_probe", "PROBE_SHAPES", "bpw_cache_flush",
    "TritFile", "TritFormatError", "TritTensor", "bpw_fnv1a64", "trit_write", "TRIT_F32", "TRIT_TERNARY", "TRIT_BF16",
    "BitcosHost", "bpw_bitcos_pack_i8", "bpw_bitcos_from_planes", "DevBitcos", "bpw_bitcos_upload", "bitcos_job",
    "bpw_bitcos_workspace_bytes", "BitcosPlan",
    "PagedKv", "QkNormRopePlan", "bpw_qk_norm_rope", "KvAppendPlan", "bpw_kv_append",
    "bpw_attn_shared_prefix_workspace_bytes", "SharedPrefixAttnPlan", "bpw_attn_shared_prefix",
    "bpw_verify_draft_workspace_bytes", "DraftVerifyPlan", "bpw_verify_draft",
]


def _np(a: np.ndarray, dtype) -> np.ndarray:
    a = np.ascontiguousarray(a)
    if a.dtype != dtype:
        raise TypeError(f"expected {np.dtype(dtype)}, got {a.dtype}")
    return a


def _dptr(t) -> int | None:
    """Device address of a torch tensor (None stays NULL)."""
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise TypeError("expected a GPU tensor")
    if not t.is_contiguous():
        raise ValueError("GPU tensor must be contiguous")
    return t.data_ptr()


def _checked(t, dtype: str, n: int, what: str) -> int | None:
    """Device address of a tensor the kernels read or write, after checking its element type and
    that it holds at least n elements (None stays NULL). The C ABI carries no lengths for outputs,
    so this is where an undersized or mistyped buffer is refused, before anything is launched."""
    if t is None:
        return None
    import torch
    want = getattr(torch, dtype)
    if t.dtype != want:
        raise TypeError(f"{what} must be {want}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, needs at least {n}")
    return _dptr(t)


def _bytes_of(t, what: str) -> int:
    """Byte length of a one-byte-element tensor (int8 codes, uint8 planes)."""
    if t.element_size() != 1:
        raise TypeError(f"{what} must have one-byte elements (int8 or uint8), got {t.dtype}")
    return t.numel()


class _Job:
    """One job of a grouped call: the ctypes record the C ABI reads (``c``) plus every object whose
    device memory that record names (the matrix and its plane buffer, activations, scales, outputs).
    Plans hold their jobs, so those buffers live as long as the plan that launches on them."""

    def __init__(self, c, keep):
        object.__setattr__(self, "c", c)
        object.__setattr__(self, "_keep", keep)

    # the record's fields read and write through the job (job.d_x, job.m.rows, ...)
    def __getattr__(self, name):
        return getattr(self.c, name)

    def __setattr__(self, name, value):
        setattr(self.c, name, value)


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------------------ library


def bpw_abi_version() -> int:
    return _lib.lib().bpw_abi_version()


def bpw_status_string(status: int) -> str:
    return _lib.lib().bpw_status_string(status).decode()


def bpw_last_error() -> str:
    return _lib.lib().bpw_last_error().decode()


def bpw_device_check() -> None:
    _lib.check(_lib.lib().bpw_device_check())


# ------------------------------------------------------------------------------ host side


def bpw_pack_i8(w: np.ndarray) -> np.ndarray:
    """int8 [rows, cols] in {-1, 0, +1} -> .trit v1 plane bytes (uint8 [rows * bpr * 16])."""
    w = _np(w, np.int8)
    rows, cols = w.shape
    out = np.empty(rows * ((cols + 63) // 64) * 16, dtype=np.uint8)
    err = _lib.BpwErr()
    _lib.check(_lib.lib().bpw_pack_i8(w.ctypes.data, rows, cols, out.ctypes.data, out.size, ctypes.byref(err)),
               err)
    return out


def bpw_validate(planes: np.ndarray, rows: int, cols: int) -> None:
    planes = _np(planes, np.uint8)
    err = _lib.BpwErr()
    _lib.check(_lib.lib().bpw_validate(planes.ctypes.data, planes.size, rows, cols, ctypes.byref(err)), err)


class HostMat:
    """A validated, library-owned host copy of one matrix's planes (bpw_host_mat)."""

    def __init__(self, handle: int, rows: int, cols: int, w_scale: float):
        self._h = ctypes.c_void_p(handle)
        self.rows, self.cols, self.w_scale = rows, cols, w_scale

    @property
    def nbytes(self) -> int:
        return _lib.lib().bpw_host_mat_bytes(self._h)

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_host_mat_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def bpw_load(planes: np.ndarray, rows: int, cols: int, w_scale: float) -> HostMat:
    planes = _np(planes, np.uint8)
    h = ctypes.c_void_p()
    err = _lib.BpwErr()
    _lib.check(_lib.lib().bpw_load(planes.ctypes.data, planes.size, rows, cols, float(w_scale), ctypes.byref(h),
                                   ctypes.byref(err)), err)
    return HostMat(h.value, rows, cols, w_scale)


class DevMat:
    """A matrix resident on the GPU (bpw_dev_mat) plus the tensor that holds its planes."""

    def __init__(self, desc: BpwDevMat, buf):
        self.desc, self.buf = desc, buf

    @property
    def rows(self) -> int:
        return self.desc.rows

    @property
    def cols(self) -> int:
        return self.desc.cols

    @property
    def bpr(self) -> int:
        return self.desc.bpr


def bpw_upload(m: HostMat, d_buf, stream=None) -> DevMat:
    """Copy m's planes into the uint8 GPU tensor d_buf (>= m.nbytes, 256-byte aligned)."""
    desc = BpwDevMat()
    nbytes = d_buf.numel() * d_buf.element_size()
    _lib.check(_lib.lib().bpw_upload(m._h, _dptr(d_buf), nbytes, _stream(stream), ctypes.byref(desc)))
    return DevMat(desc, d_buf)


# ------------------------------------------------------------------------------ batch-1 GEMV


def gemv_job(m: DevMat, x, x_scale: float, out_i32, out_f32=None, x_scale_dev=None) -> _Job:
    """One bpw_gemv_job: x int8 GPU tensor (>= bpr * 64 bytes), outputs int32 / float32 [rows].
    x_scale_dev (a float32 GPU tensor of one element) makes the kernel read the scale there. The
    returned job keeps m, x, the outputs and x_scale_dev alive."""
    j = BpwGemvJob()
    j.m = m.desc
    j.x_len = _bytes_of(x, "x")
    j.d_x = _dptr(x)
    j.x_scale = float(x_scale)
    if out_i32 is None:
        raise ValueError("out_i32 is required")
    j.d_out_i32 = _checked(out_i32, "int32", m.rows, "out_i32")
    j.d_out_f32 = _checked(out_f32, "float32", m.rows, "out_f32")
    j.d_x_scale = _checked(x_scale_dev, "float32", 1, "x_scale_dev")
    return _Job(j, (m, x, out_i32, out_f32, x_scale_dev))


def _records(jobs, ctype):
    """ctypes array of the jobs' records (a _Job's ``c``, or a bare record)."""
    recs = [j.c if isinstance(j, _Job) else j for j in jobs]
    return (ctype * max(1, len(recs)))(*recs), len(recs)


def _jobs_array(jobs):
    return _records(jobs, BpwGemvJob)


def bpw_gemv_workspace_bytes(jobs) -> int:
    arr, n = _jobs_array(jobs)
    return _lib.lib().bpw_gemv_workspace_bytes(arr, n)


def intmlp_job(gate: DevMat, up: DevMat, x, x_scale: float, t_out, k_out, gate_i32=None, up_i32=None,
               x_scale_dev=None) -> _Job:
    """One bpw_intmlp_job: gate and up (same shape) read the int8 GPU tensor x; t_out int64 [rows]
    receives relu(a_g)^2 * a_u, k_out float64 [1] receives K; gate_i32 / up_i32 optional int32 [rows]."""
    j = _lib.BpwIntMlpJob()
    j.gate = gate.desc
    j.up = up.desc
    j.x_len = _bytes_of(x, "x")
    j.d_x = _dptr(x)
    j.x_scale = float(x_scale)
    j.d_x_scale = _checked(x_scale_dev, "float32", 1, "x_scale_dev")
    if t_out is None or k_out is None:
        raise ValueError("t_out and k_out are required")
    j.d_t = _checked(t_out, "int64", gate.rows, "t_out")
    j.d_k = _checked(k_out, "float64", 1, "k_out")
    j.d_gate_i32 = _checked(gate_i32, "int32", gate.rows, "gate_i32")
    j.d_up_i32 = _checked(up_i32, "int32", gate.rows, "up_i32")
    return _Job(j, (gate, up, x, x_scale_dev, t_out, k_out, gate_i32, up_i32))


def _mlp_array(mlp):
    return _records(list(mlp or []), _lib.BpwIntMlpJob)


def bpw_gemv_intmlp_workspace_bytes(jobs, mlp) -> int:
    arr, n = _jobs_array(jobs)
    marr, nm = _mlp_array(mlp)
    return _lib.lib().bpw_gemv_intmlp_workspace_bytes(arr, n, marr, nm)


def bpw_gemv(jobs, d_ws, kernel: int = KERNEL_AUTO, stream=None) -> None:
    arr, n = _jobs_array(jobs)
    ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
    _lib.check(_lib.lib().bpw_gemv(arr, n, kernel, _dptr(d_ws), ws_len, _stream(stream)))


def bpw_gemv_noalloc(jobs, kernel: int = KERNEL_AUTO, stream=None) -> None:
    """bpw_gemv with the library's fixed device scratch in place of a workspace (allocates nothing)."""
    arr, n = _jobs_array(jobs)
    _lib.check(_lib.lib().bpw_gemv_noalloc(arr, n, kernel, _stream(stream)))


class GemvPlan:
    """bpw_gemv_plan: the job table written once into d_ws; run() queues the one launch. With mlp
    (a list of intmlp_job) the plan is made by bpw_gemv_intmlp_plan_create."""

    def __init__(self, jobs, d_ws, kernel: int = KERNEL_AUTO, stream=None, mlp=None):
        arr, n = _jobs_array(jobs)
        ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
        h = ctypes.c_void_p()
        if mlp is None:
            _lib.check(_lib.lib().bpw_gemv_plan_create(arr, n, kernel, _dptr(d_ws), ws_len, _stream(stream),
                                                       ctypes.byref(h)))
        else:
            marr, nm = _mlp_array(mlp)
            _lib.check(_lib.lib().bpw_gemv_intmlp_plan_create(arr, n, marr, nm, kernel, _dptr(d_ws), ws_len,
                                                              _stream(stream), ctypes.byref(h)))
        self._h, self._keep = h, (jobs, mlp, d_ws)

    def run(self, stream=None) -> None:
        _lib.check(_lib.lib().bpw_gemv_plan_run(self._h, _stream(stream)))

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_gemv_plan_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------------------------------------------ quantiser


def quant_job(h, g, q, scale, eps: float) -> _Job:
    """One bpw_quant_job: h, g float32 GPU tensors [n]; q int8 GPU tensor (>= n); scale float32 [1]."""
    j = BpwQuantJob()
    j.n = h.numel()
    if g.numel() != j.n:
        raise ValueError("h and g must have the same length")
    j.d_h, j.d_g = _checked(h, "float32", j.n, "h"), _checked(g, "float32", j.n, "g")
    j.q_len = _bytes_of(q, "q")
    j.d_q = _dptr(q)
    if scale is None:
        raise ValueError("scale is required")
    j.d_scale = _checked(scale, "float32", 1, "scale")
    j.eps = float(eps)
    return _Job(j, (h, g, q, scale))


def _quant_array(jobs):
    return _records(jobs, BpwQuantJob)


def bpw_quantize_workspace_bytes(n_jobs: int) -> int:
    return _lib.lib().bpw_quantize_workspace_bytes(n_jobs)


def bpw_quantize(jobs, d_ws, stream=None) -> None:
    arr, n = _quant_array(jobs)
    ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
    _lib.check(_lib.lib().bpw_quantize(arr, n, _dptr(d_ws), ws_len, _stream(stream)))


class QuantPlan:
    """bpw_quant_plan: the quantiser's job table written once into d_ws; run() queues one launch."""

    def __init__(self, jobs, d_ws, stream=None):
        arr, n = _quant_array(jobs)
        ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
        h = ctypes.c_void_p()
        _lib.check(_lib.lib().bpw_quant_plan_create(arr, n, _dptr(d_ws), ws_len, _stream(stream), ctypes.byref(h)))
        self._h, self._keep = h, (jobs, d_ws)

    def run(self, stream=None) -> None:
        _lib.check(_lib.lib().bpw_quant_plan_run(self._h, _stream(stream)))

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_quant_plan_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------------------------------------------ small batch


def bpw_gemm_small_batch(m: DevMat, X, x_scales, out_i32, out_f32, kernel: int = KERNEL_AUTO, stream=None) -> None:
    """X int8 GPU tensor [batch, ldx]; x_scales host float32 [batch]; outputs [batch, rows]."""
    batch, ldx = X.shape
    _bytes_of(X, "X")
    xs = np.ascontiguousarray(np.asarray(x_scales, dtype=np.float32))
    if xs.shape != (batch,):
        raise ValueError(f"x_scales must hold {batch} values")
    if out_i32 is None:
        raise ValueError("out_i32 is required")
    oi = _checked(out_i32, "int32", batch * m.rows, "out_i32")
    of = _checked(out_f32, "float32", batch * m.rows, "out_f32")
    _lib.check(_lib.lib().bpw_gemm_small_batch(ctypes.byref(m.desc), _dptr(X), batch, ldx, xs.ctypes.data,
                                               oi, of, kernel, _stream(stream)))


class _SbJob:
    """One grouped small-batch job; keeps its host scales alive until the plan has copied them, and
    its device tensors as long as the job (the plan reads X and writes the outputs at every run)."""

    def __init__(self, m: DevMat, X, x_scales, out_i32, out_f32=None):
        batch, ldx = X.shape
        self.batch = batch
        self.scales = np.ascontiguousarray(np.asarray(x_scales, dtype=np.float32))
        if self.scales.shape != (batch,):
            raise ValueError(f"x_scales must hold {batch} values")
        _bytes_of(X, "X")
        if out_i32 is None:
            raise ValueError("out_i32 is required")
        j = _lib.BpwSbJob()
        j.m = m.desc
        j.d_X = _dptr(X)
        j.ldx = ldx
        j.x_scales = self.scales.ctypes.data
        j.d_out_i32 = _checked(out_i32, "int32", batch * m.rows, "out_i32")
        j.d_out_f32 = _checked(out_f32, "float32", batch * m.rows, "out_f32")
        self.c = j
        self._keep = (m, X, out_i32, out_f32)


def sb_job(m: DevMat, X, x_scales, out_i32, out_f32=None) -> _SbJob:
    """One job of a grouped small-batch plan: X int8 GPU tensor [batch, ldx], x_scales host [batch],
    outputs [batch, rows]."""
    return _SbJob(m, X, x_scales, out_i32, out_f32)


def _sb_array(jobs):
    arr = (_lib.BpwSbJob * max(1, len(jobs)))(*[j.c for j in jobs])
    return arr, len(jobs)


def bpw_gemm_small_batch_workspace_bytes(jobs, batch: int) -> int:
    arr, n = _sb_array(jobs)
    return _lib.lib().bpw_gemm_small_batch_workspace_bytes(arr, n, batch)


class SmallBatchPlan:
    """bpw_sb_plan: several small-batch calls with one batch size, one launch per run()."""

    def __init__(self, jobs, batch: int, d_ws, kernel: int = KERNEL_AUTO, stream=None):
        if any(j.batch != batch for j in jobs):
            raise ValueError(f"every job's X must hold batch = {batch} rows")
        arr, n = _sb_array(jobs)
        ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
        h = ctypes.c_void_p()
        _lib.check(_lib.lib().bpw_gemm_small_batch_plan_create(arr, n, batch, kernel, _dptr(d_ws), ws_len,
                                                               _stream(stream), ctypes.byref(h)))
        self._h, self._keep = h, (jobs, d_ws)

    def run(self, stream=None) -> None:
        _lib.check(_lib.lib().bpw_gemm_small_batch_plan_run(self._h, _stream(stream)))

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_gemm_small_batch_plan_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------------------------------------------ .trit v1 container

TRIT_F32, TRIT_TERNARY, TRIT_BF16 = 0, 1, 2


class TritFormatError(BpwError):
    """A failed container check: check is its number in the format page's section 4 (1..19)."""

    def __init__(self, status: int, reason: str, e):
        super().__init__(status, reason, e.row, e.beat, e.col)
        self.check, self.offset, self.tensor = e.check, e.offset, e.tensor


class TritTensor:
    def __init__(self, t, index: int):
        self.index = index
        self.name = ctypes.string_at(t.name, t.name_len).decode("utf-8")
        self.dtype, self.dims = t.dtype, list(t.dims[: t.ndim])
        self.scale, self.offset, self.byte_len = t.scale, t.offset, t.byte_len
        self._data = t.data

    def bytes(self) -> bytes:
        return ctypes.string_at(self._data, self.byte_len) if self.byte_len else b""


def bpw_fnv1a64(data) -> int:
    buf = np.frombuffer(memoryview(data), dtype=np.uint8)
    return _lib.lib().bpw_fnv1a64(buf.ctypes.data if buf.size else None, buf.size)


def trit_write(tensors, config: bytes = b"", with_hash: bool = True) -> bytes:
    """bpw_trit_write: a .trit v1 container from [(name, dtype, dims, scale, data)] (name str, dtype one of
    TRIT_F32 / TRIT_TERNARY / TRIT_BF16, dims a sequence of 1..4 ints, data a bytes-like payload: .trit
    planes for a ternary tensor, little-endian elements otherwise). Records come out sorted by name;
    the same tensors in any order give the same bytes. Raises TritFormatError naming the check a reader
    would fail."""
    arr = (_lib.BpwTritTensorIn * max(1, len(tensors)))()
    keep = []
    for k, (name, dtype, dims, scale, data) in enumerate(tensors):
        nb = name.encode("utf-8") if isinstance(name, str) else bytes(name)
        buf = np.frombuffer(memoryview(data), dtype=np.uint8)
        keep += [nb, buf]
        e = arr[k]
        e.name, e.name_len, e.dtype, e.ndim = nb, len(nb), int(dtype), len(dims)
        if len(dims) > 4:
            raise ValueError(f"tensor {k}: {len(dims)} dims (at most 4)")
        for j, d in enumerate(dims):
            e.dims[j] = int(d)
        e.scale = float(scale)
        e.data = buf.ctypes.data if buf.size else None
        e.byte_len = buf.size
    cfg = bytes(config)
    err = _lib.BpwTritErr()
    need = ctypes.c_uint64()
    st = _lib.lib().bpw_trit_write_size(arr, len(tensors), len(cfg), ctypes.byref(need), ctypes.byref(err))
    if st != _lib.OK:
        raise TritFormatError(st, _lib.lib().bpw_last_error().decode(), err)
    out = np.empty(max(1, need.value), dtype=np.uint8)
    written = ctypes.c_uint64()
    st = _lib.lib().bpw_trit_write(arr, len(tensors), cfg, len(cfg), int(bool(with_hash)), out.ctypes.data,
                                   need.value, ctypes.byref(written), ctypes.byref(err))
    if st != _lib.OK:
        raise TritFormatError(st, _lib.lib().bpw_last_error().decode(), err)
    return out[: written.value].tobytes()


class TritFile:
    """bpw_trit_file: a .trit v1 container in host memory (bytes, bytearray, mmap, numpy uint8), opened
    with checks 1-16; verify() runs checks 17-19. The object keeps the buffer alive."""

    def __init__(self, data):
        self._buf = np.frombuffer(memoryview(data), dtype=np.uint8)
        self._h = ctypes.c_void_p()
        err = _lib.BpwTritErr()
        st = _lib.lib().bpw_trit_open(self._buf.ctypes.data if self._buf.size else None, self._buf.size,
                                      ctypes.byref(self._h), ctypes.byref(err))
        if st != _lib.OK:
            raise TritFormatError(st, _lib.lib().bpw_last_error().decode(), err)

    def verify(self, check_hash: bool = True) -> None:
        err = _lib.BpwTritErr()
        st = _lib.lib().bpw_trit_verify(self._h, int(bool(check_hash)), ctypes.byref(err))
        if st != _lib.OK:
            raise TritFormatError(st, _lib.lib().bpw_last_error().decode(), err)

    def __len__(self) -> int:
        return _lib.lib().bpw_trit_tensor_count(self._h)

    def tensor(self, index: int) -> TritTensor:
        t = _lib.BpwTritTensor()
        _lib.check(_lib.lib().bpw_trit_tensor_info(self._h, index, ctypes.byref(t)))
        return TritTensor(t, index)

    @property
    def tensors(self) -> list:
        return [self.tensor(i) for i in range(len(self))]

    def find(self, name: str) -> int:
        nb = name.encode("utf-8")
        return _lib.lib().bpw_trit_find(self._h, nb, len(nb))

    @property
    def config(self) -> bytes:
        p, n = ctypes.c_void_p(), ctypes.c_size_t()
        _lib.check(_lib.lib().bpw_trit_config(self._h, ctypes.byref(p), ctypes.byref(n)))
        return ctypes.string_at(p, n.value) if n.value else b""

    @property
    def stored_hash(self) -> int:
        return _lib.lib().bpw_trit_stored_hash(self._h)

    def load(self, index: int) -> HostMat:
        """A ternary tensor as a validated host matrix (for bpw_upload)."""
        t = self.tensor(index)
        h = ctypes.c_void_p()
        err = _lib.BpwErr()
        _lib.check(_lib.lib().bpw_trit_load(self._h, index, ctypes.byref(h), ctypes.byref(err)), err)
        return HostMat(h.value, t.dims[0], t.dims[1], t.scale)

    def close(self) -> None:
        if self._h:
            _lib.lib().bpw_trit_close(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------------------ dense head


def bpw_dense_head_gemv(w_bf16, x_bf16, y, stream=None) -> None:
    """w_bf16 [rows, cols] and x_bf16 [cols] GPU tensors of bf16 bits (int16/uint16/bfloat16); y float32."""
    rows, cols = w_bf16.shape
    for t, what in ((w_bf16, "w_bf16"), (x_bf16, "x_bf16")):
        if t.element_size() != 2:
            raise TypeError(f"{what} must hold 16-bit elements (bf16 bit patterns), got {t.dtype}")
    if x_bf16.numel() < cols:
        raise ValueError(f"x_bf16 holds {x_bf16.numel()} elements, needs at least {cols}")
    _lib.check(_lib.lib().bpw_dense_head_gemv(_dptr(w_bf16), rows, cols, _dptr(x_bf16),
                                              _checked(y, "float32", rows, "y"), _stream(stream)))


# ------------------------------------------------------------------------------ decode step: heads, cache, attention, drafts


def _dtype_code(t, what: str, cache: bool = False) -> int:
    import torch
    code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}.get(t.dtype)
    if code is None or (cache and code == _lib.F32):
        raise TypeError(f"{what} must be {'' if cache else 'float32, '}bfloat16 or float16, got {t.dtype}")
    return code


def _shaped(t, dtype: str, shape: tuple, what: str) -> int | None:
    """As _checked, and refuses a larger tensor of several dimensions whose rows have another length than those of `shape`: the
    kernels would take them from other places."""
    n = math.prod(shape)
    if t is not None and t.dim() > 1 and t.numel() > n and math.prod(t.shape[1:]) != math.prod(shape[1:]):
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    return _checked(t, dtype, n, what)


def _gpu(t, what: str) -> int:
    """Device address of a strided GPU tensor."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: expected a GPU tensor")
    return t.data_ptr()


def _heads(t, tokens: int, head_dim: int, what: str) -> "_lib.BpwHeads":
    """A [tokens, heads, head_dim] GPU tensor, any strides with contiguous elements (None: no heads)."""
    h = _lib.BpwHeads()
    if t is None:
        return h
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != head_dim:
        raise ValueError(f"{what} must be [{tokens}, heads, {head_dim}], got {list(t.shape)}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{what}: a head's elements must be contiguous")
    h.dtype = _dtype_code(t, what)
    h.d, h.heads = _gpu(t, what), t.shape[1]
    # the stride of a dimension of one is free: 0, as nothing is reached by it
    h.token_stride = t.stride(0) if t.shape[0] > 1 else 0
    h.head_stride = t.stride(1) if t.shape[1] > 1 else 0
    return h


def _written(h, t, what: str) -> None:
    """Refuses an output whose rows repeat (an expanded view)."""
    if t is not None and (t.shape[0] > 1 and t.stride(0) == 0 or t.shape[1] > 1 and t.stride(1) == 0):
        raise ValueError(f"{what} is an expanded view: its rows share memory")


def _rotation(positions, inv_freq, tokens: int, interleaved: bool) -> "_lib.BpwRotation":
    r = _lib.BpwRotation()
    if inv_freq is None:
        return r
    r.rot_dim = 2 * inv_freq.numel()
    r.d_inv_freq = _checked(inv_freq, "float64", 1, "inv_freq") if r.rot_dim else None
    if r.rot_dim and positions is None:
        raise ValueError("positions are required with inv_freq")
    r.d_positions = _checked(positions, "int32", tokens, "positions")
    r.interleaved = int(bool(interleaved))
    return r


class PagedKv:
    """A paged key/value cache (bpw_paged_kv): k_pages and v_pages are GPU tensors [pages, kv_heads, page_size,
    head_dim] of bfloat16 or float16, any strides with contiguous elements (``x.transpose(1, 2)`` of a
    [pages, page_size, kv_heads, head_dim] cache too)."""

    def __init__(self, k_pages, v_pages):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must both be [pages, kv_heads, page_size, head_dim]")
        if k_pages.dtype != v_pages.dtype:
            raise TypeError("k_pages and v_pages have different types")
        for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError(f"{what}: a head's elements must be contiguous")
            if any(n > 1 and st == 0 for n, st in zip(t.shape, t.stride())):
                raise ValueError(f"{what} is an expanded view: its rows share memory")
        c = _lib.BpwPagedKv()
        c.dtype = _dtype_code(k_pages, "a cache", cache=True)
        c.n_pages, c.kv_heads, c.page_size, c.head_dim = k_pages.shape
        c.d_k, c.d_v = _gpu(k_pages, "k_pages"), _gpu(v_pages, "v_pages")
        # the stride of a dimension of one is free: 0, as nothing is reached by it
        st = [[x if n > 1 else 0 for n, x in zip(t.shape, t.stride())] for t in (k_pages, v_pages)]
        c.k_page_stride, c.k_head_stride, c.k_row_stride = st[0][:3]
        c.v_page_stride, c.v_head_stride, c.v_row_stride = st[1][:3]
        self.c, self.k_pages, self.v_pages = c, k_pages, v_pages

    @property
    def page_size(self) -> int:
        return self.c.page_size


_raw_stream = None  # torch's current stream of a device as an address, where this torch has that call


def _current_stream(device: int) -> int:
    """The address of torch's current stream: 0.1 us by torch's own accessor, 2.7 us through a Stream object, in
    calls whose launch takes 4."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


class _Bound:
    """Arguments checked and bound once; run() queues the launches on a stream. The tensors named stay
    alive with the plan and are read and written as they are when the work runs, so a plan may be run
    again after their contents change, and its runs captured into a graph."""

    def _bind(self, fn: str, args, keep, d_ws=None):
        t = next(x for x in keep if hasattr(x, "device"))
        self._device = t.device.index or 0
        self._fn, self._args, self._ref, self._keep = getattr(_lib.lib(), fn), args, ctypes.byref(args), (keep, d_ws)
        self._ws = None if d_ws is None else (_dptr(d_ws), d_ws.numel() * d_ws.element_size())

    def run(self, stream=None) -> None:
        stream = _current_stream(self._device) if stream is None else _stream(stream)
        if self._ws is None:
            status = self._fn(self._ref, stream)
        else:
            status = self._fn(self._ref, self._ws[0], self._ws[1], stream)
        if status:
            _lib.check(status)


class QkNormRopePlan(_Bound):
    """bpw_qk_norm_rope: q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] normed (where a gain, float32
    [head_dim], is given) and rotated into q_out and k_out. positions int32 [tokens], inv_freq float64
    [rot_dim / 2] (None: no rotation). q and q_out, or k and k_out, may be None; an output may be its input."""

    def __init__(self, q, k, q_out, k_out, positions, inv_freq, q_gain=None, k_gain=None, eps: float = 1e-6,
                 interleaved: bool = False):
        first = q if q is not None else k
        if first is None or first.dim() != 3:
            raise ValueError("q or k must be [tokens, heads, head_dim]")
        T, D = first.shape[0], first.shape[2]
        a = _lib.BpwQkNormRopeArgs()
        a.n_tokens, a.head_dim = T, D
        a.q, a.k = _heads(q, T, D, "q"), _heads(k, T, D, "k")
        a.q_out, a.k_out = _heads(q_out, T, D, "q_out"), _heads(k_out, T, D, "k_out")
        _written(a.q_out, q_out, "q_out")
        _written(a.k_out, k_out, "k_out")
        a.d_q_gain, a.d_k_gain = _checked(q_gain, "float32", D, "q_gain"), _checked(k_gain, "float32", D, "k_gain")
        a.eps = float(eps)
        a.rot = _rotation(positions, inv_freq, T, interleaved)
        self._bind("bpw_qk_norm_rope", a, (q, k, q_out, k_out, positions, inv_freq, q_gain, k_gain))


def bpw_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, q_gain=None, k_gain=None, eps: float = 1e-6,
                     interleaved: bool = False, stream=None) -> None:
    """One run of a QkNormRopePlan."""
    QkNormRopePlan(q, k, q_out, k_out, positions, inv_freq, q_gain, k_gain, eps, interleaved).run(stream)


class KvAppendPlan(_Bound):
    """bpw_kv_append: k and v [tokens, kv_heads, head_dim] written to the cache at slots (int64 [tokens]: page * page_size
    + offset; outside the cache: not written), k normed and rotated on the way; q, if given, normed and rotated
    into q_out in the same launch."""

    def __init__(self, kv: PagedKv, k, v, slots, positions=None, inv_freq=None, k_gain=None, q=None, q_out=None,
                 q_gain=None, eps: float = 1e-6, interleaved: bool = False):
        if k.dim() != 3:
            raise ValueError("k must be [tokens, kv_heads, head_dim]")
        T, D = k.shape[0], kv.c.head_dim
        a = _lib.BpwKvAppendArgs()
        a.n_tokens, a.kv = T, kv.c
        a.k, a.v, a.q, a.q_out = (_heads(k, T, D, "k"), _heads(v, T, D, "v"), _heads(q, T, D, "q"),
                                  _heads(q_out, T, D, "q_out"))
        _written(a.q_out, q_out, "q_out")
        if slots is None:
            raise ValueError("slots are required")
        a.d_slots = _checked(slots, "int64", T, "slots")
        a.d_q_gain, a.d_k_gain = _checked(q_gain, "float32", D, "q_gain"), _checked(k_gain, "float32", D, "k_gain")
        a.eps = float(eps)
        a.rot = _rotation(positions, inv_freq, T, interleaved)
        self._bind("bpw_kv_append", a, (kv, k, v, slots, positions, inv_freq, k_gain, q, q_out, q_gain))


def bpw_kv_append(kv: PagedKv, k, v, slots, positions=None, inv_freq=None, k_gain=None, q=None, q_out=None, q_gain=None,
                  eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """One run of a KvAppendPlan."""
    KvAppendPlan(kv, k, v, slots, positions, inv_freq, k_gain, q, q_out, q_gain, eps, interleaved).run(stream)


def _attn_args(kv: PagedKv, q, prefix_len: int, n_seqs: int, max_q: int, max_pages: int):
    a = _lib.BpwAttnArgs()
    a.kv = kv.c
    a.n_tokens, a.n_seqs, a.max_q = q.shape[0], int(n_seqs), int(max_q)
    a.q = _heads(q, q.shape[0], kv.c.head_dim, "q")
    a.prefix_len, a.max_pages = int(prefix_len), int(max_pages)
    return a


def bpw_attn_shared_prefix_workspace_bytes(kv: PagedKv, q, prefix_len: int, n_seqs: int, max_q: int,
                                           max_pages: int | None = None) -> int:
    """Workspace bytes of a SharedPrefixAttnPlan over this cache and q [tokens, q_heads, head_dim]. max_pages: columns of
    the page table (None: the cache's pages, which covers every table)."""
    a = _attn_args(kv, q, prefix_len, n_seqs, max_q, kv.c.n_pages if max_pages is None else max_pages)
    return _lib.lib().bpw_attn_shared_prefix_workspace_bytes(ctypes.byref(a))


class SharedPrefixAttnPlan(_Bound):
    """bpw_attn_shared_prefix: decode attention of sequences that share a prefix. q and out [tokens, q_heads,
    head_dim] of the cache's type; prefix_pages int32 holds the prefix_len shared positions (None if 0); table
    int32 [sequences, max_pages], lens int32 [sequences] each sequence's own positions; q_starts int32 [sequences + 1]
    the first token of each; max_q the most tokens of one; d_ws a uint8 workspace; lse float32 [tokens, q_heads]
    or None; scale None: 1 / sqrt(head_dim)."""

    def __init__(self, kv: PagedKv, q, out, prefix_pages, prefix_len: int, table, lens, q_starts, max_q: int, d_ws,
                 scale: float | None = None, lse=None):
        if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be [sequences, max_pages] with contiguous rows")
        if q.dim() != 3:
            raise ValueError("q must be [tokens, q_heads, head_dim]")
        n_seqs = table.shape[0]
        a = _attn_args(kv, q, prefix_len, n_seqs, max_q, table.shape[1])
        a.out = _heads(out, q.shape[0], kv.c.head_dim, "out")
        _written(a.out, out, "out")
        import torch
        if table.dtype != torch.int32:
            raise TypeError(f"table must be torch.int32, got {table.dtype}")
        a.d_lens = _checked(lens, "int32", n_seqs, "lens")
        a.d_q_starts = _checked(q_starts, "int32", n_seqs + 1, "q_starts")
        need = -(-a.prefix_len // kv.c.page_size) if a.prefix_len > 0 else 0
        a.d_prefix_pages = _checked(prefix_pages, "int32", need, "prefix_pages") if need else None
        if need and prefix_pages is None:
            raise ValueError("prefix_pages are required with a prefix")
        a.d_table = _gpu(table, "table")
        a.table_stride = max(table.stride(0), table.shape[1]) if n_seqs == 1 else table.stride(0)
        a.scale = kv.c.head_dim ** -0.5 if scale is None else float(scale)
        a.d_lse = _shaped(lse, "float32", (q.shape[0], q.shape[1]), "lse")
        if d_ws is None:
            raise ValueError("a workspace is required")
        self._bind("bpw_attn_shared_prefix", a, (kv, q, out, prefix_pages, table, lens, q_starts, lse), d_ws)


def bpw_attn_shared_prefix(kv: PagedKv, q, out, prefix_pages, prefix_len: int, table, lens, q_starts, max_q: int, d_ws,
                           scale: float | None = None, lse=None, stream=None) -> None:
    """One run of a SharedPrefixAttnPlan."""
    SharedPrefixAttnPlan(kv, q, out, prefix_pages, prefix_len, table, lens, q_starts, max_q, d_ws, scale, lse).run(stream)


def bpw_verify_draft_workspace_bytes(n_seqs: int, vocab: int) -> int:
    return _lib.lib().bpw_verify_draft_workspace_bytes(int(n_seqs), int(vocab))


class DraftVerifyPlan(_Bound):
    """bpw_verify_draft: target [sequences, drafts + 1, vocab] and draft [sequences, drafts, vocab] probabilities
    (draft None: the drafted tokens were certain), tokens int32 [sequences, drafts], accept_u float32
    [sequences, drafts], sample_u float32 [sequences], n_draft int32 [sequences] or None (all). out_tokens int32 [sequences,
    drafts + 1] gets the accepted tokens, the drawn one, then -1; accepted int32 [sequences] their count."""

    def __init__(self, target, draft, tokens, accept_u, sample_u, out_tokens, accepted, d_ws, n_draft=None):
        if target.dim() != 3:
            raise ValueError("target must be [sequences, drafts + 1, vocab]")
        B, K, V = target.shape[0], target.shape[1] - 1, target.shape[2]
        if draft is not None and tuple(draft.shape) != (B, K, V):
            raise ValueError(f"draft must be [{B}, {K}, {V}], got {list(draft.shape)}")
        if draft is not None and draft.dtype != target.dtype:
            raise TypeError("target and draft have different types")
        for t, what in ((target, "target"), (draft, "draft")):
            if t is not None and V > 1 and t.stride(2) != 1:
                raise ValueError(f"{what}: a row must be contiguous")
        a = _lib.BpwVerifyArgs()
        a.n_seqs, a.max_drafts, a.vocab, a.dtype = B, K, V, _dtype_code(target, "target")
        a.d_target, a.target_seq_stride, a.target_step_stride = _gpu(target, "target"), target.stride(0), target.stride(1)
        if draft is not None:
            a.d_draft, a.draft_seq_stride, a.draft_step_stride = _gpu(draft, "draft"), draft.stride(0), draft.stride(1)
        for t, what in ((tokens, "tokens"), (accept_u, "accept_u"), (sample_u, "sample_u"), (out_tokens, "out_tokens"),
                        (accepted, "accepted")):
            if t is None:
                raise ValueError(f"{what} is required")
        a.d_tokens = _shaped(tokens, "int32", (B, K), "tokens")
        a.d_n_draft = _checked(n_draft, "int32", B, "n_draft")
        a.d_accept_u = _shaped(accept_u, "float32", (B, K), "accept_u")
        a.d_sample_u = _checked(sample_u, "float32", B, "sample_u")
        a.d_out_tokens = _shaped(out_tokens, "int32", (B, K + 1), "out_tokens")
        a.d_accepted = _checked(accepted, "int32", B, "accepted")
        if d_ws is None:
            raise ValueError("a workspace is required")
        self._bind("bpw_verify_draft", a, (target, draft, tokens, accept_u, sample_u, out_tokens, accepted, n_draft), d_ws)


def bpw_verify_draft(target, draft, tokens, accept_u, sample_u, out_tokens, accepted, d_ws, n_draft=None,
                     stream=None) -> None:
    """One run of a DraftVerifyPlan."""
    DraftVerifyPlan(target, draft, tokens, accept_u, sample_u, out_tokens, accepted, d_ws, n_draft).run(stream)


# ------------------------------------------------------------------------------ measurement


PROBE_SHAPES = 5


def bpw_stream_read_probe(d_buf, d_sink, stream=None, shape: int = 0) -> None:
    if d_sink is None or d_sink.element_size() != 4 or d_sink.numel() < 1:
        raise ValueError("d_sink must be a 4-byte-element tensor of at least one element")
    _lib.check(_lib.lib().bpw_stream_read_probe_shape(_dptr(d_buf), d_buf.numel() * d_buf.element_size(),
                                                      _dptr(d_sink), int(shape), _stream(stream)))


def bpw_cache_flush(d_buf, stream=None) -> None:
    _lib.check(_lib.lib().bpw_cache_flush(_dptr(d_buf), d_buf.numel() * d_buf.element_size(), _stream(stream)))


# ------------------------------------------------------------------------------ BITCOS


class BitcosHost:
    """A library-owned BITCOS matrix on the host (bpw_bitcos_host)."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)

    def arrays(self):
        """(presence uint64 [rows * bpr], signs uint32 [sign_words], row_start uint32 [rows + 1], nnz),
        copied out of the library's arrays."""
        p, s, r = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        nw, nnz = ctypes.c_int64(), ctypes.c_int64()
        _lib.check(_lib.lib().bpw_bitcos_arrays(self._h, ctypes.byref(p), ctypes.byref(s), ctypes.byref(r),
                                                ctypes.byref(nw), ctypes.byref(nnz)))
        rows = self.rows

        def view(ptr, n, ct, dt):
            if n == 0:
                return np.zeros(0, dt)
            return np.ctypeslib.as_array(ctypes.cast(ptr, ctypes.POINTER(ct)), shape=(n,)).copy()

        return (view(p, rows * self.bpr, ctypes.c_uint64, np.uint64), view(s, nw.value, ctypes.c_uint32, np.uint32),
                view(r, rows + 1, ctypes.c_uint32, np.uint32), nnz.value)

    @property
    def device_bytes(self) -> int:
        return _lib.lib().bpw_bitcos_device_bytes(self._h)

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_bitcos_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def bpw_bitcos_pack_i8(w: np.ndarray, w_scale: float) -> BitcosHost:
    """int8 [rows, cols] in {-1, 0, +1} -> a BITCOS matrix."""
    w = _np(w, np.int8)
    rows, cols = w.shape
    h = ctypes.c_void_p()
    err = _lib.BpwErr()
    _lib.check(_lib.lib().bpw_bitcos_pack_i8(w.ctypes.data, rows, cols, float(w_scale), ctypes.byref(h),
                                             ctypes.byref(err)), err)
    out = BitcosHost(h.value)
    out.rows, out.cols, out.bpr, out.w_scale = rows, cols, (cols + 63) // 64, w_scale
    return out


def bpw_bitcos_from_planes(m: HostMat) -> BitcosHost:
    """The same matrix as a validated .trit host matrix, re-encoded."""
    h = ctypes.c_void_p()
    _lib.check(_lib.lib().bpw_bitcos_from_planes(m._h, ctypes.byref(h)))
    out = BitcosHost(h.value)
    out.rows, out.cols, out.bpr, out.w_scale = m.rows, m.cols, (m.cols + 63) // 64, m.w_scale
    return out


class DevBitcos:
    """A BITCOS matrix resident on the GPU (bpw_dev_bitcos) plus the tensor that holds it."""

    def __init__(self, desc: _lib.BpwDevBitcos, buf):
        self.desc, self.buf = desc, buf

    @property
    def rows(self) -> int:
        return self.desc.rows

    @property
    def cols(self) -> int:
        return self.desc.cols

    @property
    def bpr(self) -> int:
        return self.desc.bpr


def bpw_bitcos_upload(h: BitcosHost, d_buf, stream=None) -> DevBitcos:
    """Copy h into the uint8 GPU tensor d_buf (>= h.device_bytes, 256-byte aligned)."""
    desc = _lib.BpwDevBitcos()
    nbytes = d_buf.numel() * d_buf.element_size()
    _lib.check(_lib.lib().bpw_bitcos_upload(h._h, _dptr(d_buf), nbytes, _stream(stream), ctypes.byref(desc)))
    return DevBitcos(desc, d_buf)


def bitcos_job(m: DevBitcos, x, x_scale: float, out_i32, out_f32=None) -> _Job:
    """One bpw_bitcos_job (outputs int32 / float32 [rows]); the job keeps m, x and the outputs alive."""
    j = _lib.BpwBitcosJob()
    j.m = m.desc
    j.x_len = _bytes_of(x, "x")
    j.d_x = _dptr(x)
    j.x_scale = float(x_scale)
    if out_i32 is None:
        raise ValueError("out_i32 is required")
    j.d_out_i32 = _checked(out_i32, "int32", m.rows, "out_i32")
    j.d_out_f32 = _checked(out_f32, "float32", m.rows, "out_f32")
    return _Job(j, (m, x, out_i32, out_f32))


def _bitcos_array(jobs):
    return _records(list(jobs), _lib.BpwBitcosJob)


def bpw_bitcos_workspace_bytes(jobs) -> int:
    arr, n = _bitcos_array(jobs)
    return _lib.lib().bpw_bitcos_workspace_bytes(arr, n)


class BitcosPlan:
    """bpw_bitcos_plan: job and tile tables written once into d_ws; run() queues the one launch."""

    def __init__(self, jobs, d_ws, stream=None):
        arr, n = _bitcos_array(jobs)
        ws_len = 0 if d_ws is None else d_ws.numel() * d_ws.element_size()
        h = ctypes.c_void_p()
        _lib.check(_lib.lib().bpw_bitcos_plan_create(arr, n, _dptr(d_ws), ws_len, _stream(stream), ctypes.byref(h)))
        self._h, self._keep = h, (jobs, d_ws)

    def run(self, stream=None) -> None:
        _lib.check(_lib.lib().bpw_bitcos_plan_run(self._h, _stream(stream)))

    def free(self) -> None:
        if self._h:
            _lib.lib().bpw_bitcos_plan_free(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
