"""B200 (sm_100a) QLoRA NF4 + LoRA quantized linear: Python binding.

This module only marshals arguments to the C ABI declared in
``include/qlora.h`` (``libqlora.so``, built in-tree by ``build.py``). Every
step of the computation runs in the library's CUDA kernels; PyTorch supplies
device memory and streams. If the shared library is missing the import
fails: there is no fallback of any kind.

Functions carry the C names:

    qlora_nf4_bytes, qlora_nf4_codebook, qlora_quantize_nf4, qlora_dequantize,
    qlora_workspace_bytes, qlora_fwd_workspace_bytes, qlora_linear_fwd, qlora_linear_fwd_ex,
    qlora_linear_fwd_noalloc, qlora_linear_bwd, qlora_device_status, qlora_status_string, qlora_version,
    qlora_launch_count, qlora_selftest_wait_timeout, qlora_selftest_ring_timeout, qlora_merge_lora, qlora_adamw_step, qlora_adamw_host,
    qlora_adamw_paged, qlora_adamw_staged, qlora_set_gemm_schedule, qlora_get_gemm_schedule,
    qlora_quantize_fp8, qlora_dequantize_fp8, qlora_quantize_fp8_rows, qlora_fp8_workspace_bytes,
    qlora_fp8_linear_fwd, qlora_fp8_linear_bwd, qlora_rmsnorm_fwd, qlora_rmsnorm_workspace_bytes,
    qlora_rmsnorm_bwd, qlora_adamw_multi
"""

import array
import ctypes
import operator
import os

__all__ = [
    "LIB_PATH", "lib", "QloraError", "NF4Weight", "Nf4Struct",
    "qlora_nf4_bytes", "qlora_nf4_codebook", "DQ_U8_256", "DQ_U8_255", "DQ_S8_MID", "qlora_quantize_nf4", "qlora_dequantize",
    "qlora_workspace_bytes", "qlora_fwd_workspace_bytes", "qlora_linear_fwd", "qlora_linear_fwd_ex", "qlora_linear_fwd_noalloc",
    "qlora_linear_bwd",
    "qlora_device_status", "qlora_status_string", "qlora_version", "qlora_launch_count",
    "qlora_selftest_wait_timeout", "qlora_selftest_ring_timeout", "SELFTEST_RING_NEVER", "SELFTEST_RING_LATE",
    "SELFTEST_RING_ONE", "qlora_merge_lora", "qlora_adamw_step", "qlora_adamw_host", "qlora_adamw_paged",
    "qlora_adamw_staged", "qlora_set_gemm_schedule", "qlora_get_gemm_schedule",
    "AdamwParams",
    "FP8_E4M3", "FP8_E5M2", "FP8Weight", "FP8Rows", "Fp8Struct", "Fp8RowsStruct", "qlora_quantize_fp8",
    "qlora_dequantize_fp8", "qlora_quantize_fp8_rows", "qlora_fp8_workspace_bytes", "qlora_fp8_linear_fwd",
    "qlora_fp8_linear_bwd", "qlora_rmsnorm_fwd", "qlora_rmsnorm_workspace_bytes", "qlora_rmsnorm_bwd",
    "AdamWGroup", "qlora_adamw_multi",
    "FWD_AUTO", "FWD_GEMM", "FWD_GEMV", "SCHED_AUTO", "SCHED_DATA_PARALLEL", "SCHED_STREAM_K",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlora.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python bit_nf4_quantized_06_b200/build.py` "
        "(there is no CPU or Python fallback)")

lib = ctypes.CDLL(LIB_PATH)

FWD_AUTO, FWD_GEMM, FWD_GEMV = 0, 1, 2
SCHED_AUTO, SCHED_DATA_PARALLEL, SCHED_STREAM_K = 0, 1, 2
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "SHAPE", 3: "ALIGNMENT", 4: "WORKSPACE",
                5: "UNSUPPORTED_DEVICE", 6: "CUDA", 7: "TIMEOUT"}


class Nf4Struct(ctypes.Structure):
    """Mirror of ``qlora_nf4_t``."""
    _fields_ = [
        ("n_out", ctypes.c_int64),
        ("k_in", ctypes.c_int64),
        ("block", ctypes.c_int32),
        ("dq_group", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scale_codes", ctypes.c_void_p),
        ("absmax", ctypes.c_void_p),
        ("dq_code", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_P = ctypes.POINTER
lib.qlora_nf4_bytes.argtypes = [_i64, _i64, _i32, _P(_sz)]
lib.qlora_nf4_bytes.restype = _sz
lib.qlora_nf4_bytes_ex.argtypes = [_i64, _i64, _i32, _i32, _P(_sz)]
lib.qlora_nf4_bytes_ex.restype = _sz
lib.qlora_nf4_codebook.argtypes = [_P(ctypes.c_float)]
lib.qlora_nf4_codebook.restype = ctypes.c_int
lib.qlora_quantize_nf4.argtypes = [_vp, _P(Nf4Struct), _vp]
lib.qlora_quantize_nf4.restype = ctypes.c_int
lib.qlora_dequantize.argtypes = [_P(Nf4Struct), _vp, _vp]
lib.qlora_dequantize.restype = ctypes.c_int
lib.qlora_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32]
lib.qlora_workspace_bytes.restype = _sz
lib.qlora_fwd_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32]
lib.qlora_fwd_workspace_bytes.restype = _sz
lib.qlora_linear_fwd.argtypes = [_P(Nf4Struct), _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _sz, _vp]
lib.qlora_linear_fwd.restype = ctypes.c_int
lib.qlora_linear_fwd_ex.argtypes = [_P(Nf4Struct), _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _sz, _i32,
                                    _vp]
lib.qlora_linear_fwd_ex.restype = ctypes.c_int
lib.qlora_linear_fwd_noalloc.argtypes = [_P(Nf4Struct), _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp]
lib.qlora_linear_fwd_noalloc.restype = ctypes.c_int
lib.qlora_linear_bwd.argtypes = [_P(Nf4Struct), _vp, _vp, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _vp,
                                 _sz, _vp]
lib.qlora_linear_bwd.restype = ctypes.c_int
lib.qlora_device_status.argtypes = [_vp, _P(ctypes.c_uint32)]
lib.qlora_device_status.restype = ctypes.c_int
lib.qlora_status_string.argtypes = [ctypes.c_int]
lib.qlora_status_string.restype = ctypes.c_char_p
lib.qlora_version.argtypes = []
lib.qlora_version.restype = _i32
class AdamwParams(ctypes.Structure):
    """qlora_adamw_t: lr, beta1, beta2, eps, weight_decay, step (1-based)."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int32)]


lib.qlora_adamw_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, ctypes.POINTER(AdamwParams), _vp]
lib.qlora_adamw_step.restype = ctypes.c_int
lib.qlora_adamw_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, ctypes.POINTER(AdamwParams)]
lib.qlora_adamw_host.restype = ctypes.c_int
lib.qlora_adamw_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.POINTER(AdamwParams), _vp]
lib.qlora_adamw_paged.restype = ctypes.c_int
lib.qlora_adamw_staged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.POINTER(AdamwParams), _vp]
lib.qlora_adamw_staged.restype = ctypes.c_int
lib.qlora_merge_lora.argtypes = [_P(Nf4Struct), _vp, _vp, _i32, _f32, _vp, _vp]
lib.qlora_merge_lora.restype = ctypes.c_int
lib.qlora_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _vp]
lib.qlora_selftest_wait_timeout.restype = ctypes.c_int
lib.qlora_selftest_ring_timeout.argtypes = [ctypes.c_uint32, _i32, _vp, _vp]
lib.qlora_selftest_ring_timeout.restype = ctypes.c_int
lib.qlora_launch_count.argtypes = []
lib.qlora_launch_count.restype = ctypes.c_uint64
lib.qlora_set_gemm_schedule.argtypes = [ctypes.c_int32]
lib.qlora_set_gemm_schedule.restype = ctypes.c_int
lib.qlora_get_gemm_schedule.argtypes = []
lib.qlora_get_gemm_schedule.restype = ctypes.c_int32


class QloraError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        msg = lib.qlora_status_string(status).decode()
        super().__init__(f"{where}: QLORA_ERR_{STATUS_NAMES.get(status, status)} ({msg})")


def _check(status, where):
    if status != 0:
        raise QloraError(status, where)


_torch_module = None


def _torch():
    # imported on first use, kept: an import statement costs as much as a launch's arguments
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_ptr(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def qlora_version():
    return int(lib.qlora_version())


def qlora_launch_count():
    """Kernels launched by the library in this process so far."""
    return int(lib.qlora_launch_count())


def qlora_set_gemm_schedule(mode):
    """Process-wide schedule of the pair GEMMs: SCHED_AUTO, SCHED_DATA_PARALLEL or SCHED_STREAM_K."""
    _check(lib.qlora_set_gemm_schedule(int(mode)), "qlora_set_gemm_schedule")


def qlora_get_gemm_schedule():
    return int(lib.qlora_get_gemm_schedule())


def qlora_status_string(status):
    return lib.qlora_status_string(int(status)).decode()


# scale codes of the double quantization (qlora_dq_code_t)
DQ_U8_256, DQ_U8_255, DQ_S8_MID = 0, 1, 2


def qlora_nf4_bytes(n_out, k_in, dq_group=256, dq_code=DQ_U8_256):
    """(codes, scale codes, group constants) byte sizes of the stored format."""
    out = (ctypes.c_size_t * 3)()
    total = lib.qlora_nf4_bytes_ex(int(n_out), int(k_in), int(dq_group), int(dq_code), out)
    if total == 0:
        raise QloraError(2, "qlora_nf4_bytes")
    return int(out[0]), int(out[1]), int(out[2])


def qlora_nf4_codebook():
    """The library's 16 fp32 NF4 levels (a list of Python floats)."""
    buf = (ctypes.c_float * 16)()
    _check(lib.qlora_nf4_codebook(buf), "qlora_nf4_codebook")
    return [float(v) for v in buf]


class NF4Weight:
    """Device buffers of one packed NF4 weight. dq=True: codes, 8-bit scale
    codes and the group constants of `dq_code` per 256 blocks (double
    quantization); dq=False: codes and one fp32 scale per 64-weight block (no
    scale codes)."""

    def __init__(self, n_out, k_in, device="cuda", dq=True, dq_code=DQ_U8_256):
        torch = _torch()
        self.dq = bool(dq)
        self.dq_code = int(dq_code) if self.dq else DQ_U8_256
        b_codes, b_q2, b_smax = qlora_nf4_bytes(n_out, k_in, 256 if self.dq else 0, self.dq_code)
        self.n_out, self.k_in = int(n_out), int(k_in)
        self.codes = torch.empty(b_codes, dtype=torch.uint8, device=device)
        self.scale_codes = torch.empty(b_q2, dtype=torch.uint8, device=device)
        self.absmax = torch.empty(b_smax // 4, dtype=torch.float32, device=device)

    def struct(self):
        q2 = self.scale_codes.data_ptr() if self.dq else 0
        return Nf4Struct(self.n_out, self.k_in, 64, 256 if self.dq else 0, self.codes.data_ptr(), q2,
                         self.absmax.data_ptr(), self.dq_code, 0)

    def nbytes(self):
        return self.codes.numel() + self.scale_codes.numel() + 4 * self.absmax.numel()


def qlora_quantize_nf4(w, out=None, stream=None, dq=True, dq_code=DQ_U8_256):
    """Quantize a bf16 CUDA weight [N, K] into an :class:`NF4Weight` (with
    double quantization in scale code `dq_code` unless dq=False, or as `out`
    says)."""
    assert w.is_cuda and w.dim() == 2 and w.is_contiguous()
    q = out if out is not None else NF4Weight(w.shape[0], w.shape[1], device=w.device, dq=dq, dq_code=dq_code)
    s = q.struct()
    _check(lib.qlora_quantize_nf4(_ptr(w), ctypes.byref(s), _stream_ptr(stream)), "qlora_quantize_nf4")
    return q


def qlora_dequantize(q, out=None, stream=None):
    """Restore W_hat [N, K] bf16 from an :class:`NF4Weight`."""
    torch = _torch()
    if out is None:
        out = torch.empty((q.n_out, q.k_in), dtype=torch.bfloat16, device=q.codes.device)
    s = q.struct()
    _check(lib.qlora_dequantize(ctypes.byref(s), _ptr(out), _stream_ptr(stream)), "qlora_dequantize")
    return out


def qlora_workspace_bytes(m, n_out, k_in, r):
    return int(lib.qlora_workspace_bytes(int(m), int(n_out), int(k_in), int(r)))


def qlora_fwd_workspace_bytes(m, n_out, k_in, r):
    return int(lib.qlora_fwd_workspace_bytes(int(m), int(n_out), int(k_in), int(r)))


def _workspace(ws, m, q, r, device):
    torch = _torch()
    need = qlora_workspace_bytes(m, q.n_out, q.k_in, r)
    if ws is None:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    return ws


def qlora_linear_fwd_ex(q, x, a, b, alpha, path=FWD_AUTO, y=None, u=None, ws=None, stream=None,
                        want_u=True):
    """Forward; returns (y [m, N] bf16, u' [m, r] bf16 or None)."""
    torch = _torch()
    m = x.shape[0]
    r = a.shape[0]
    if y is None:
        y = torch.empty((m, q.n_out), dtype=torch.bfloat16, device=x.device)
    if u is None and want_u:
        u = torch.empty((m, r), dtype=torch.bfloat16, device=x.device)
    ws = _workspace(ws, m, q, r, x.device)
    s = q.struct()
    st = lib.qlora_linear_fwd_ex(ctypes.byref(s), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(y), _ptr(u),
                                 _ptr(ws), ws.numel(), int(path), _stream_ptr(stream))
    _check(st, "qlora_linear_fwd_ex")
    return y, u


def qlora_linear_fwd(q, x, a, b, alpha, y=None, u=None, ws=None, stream=None, want_u=True):
    """Forward with the library's own path choice; returns (y, u')."""
    torch = _torch()
    m = x.shape[0]
    r = a.shape[0]
    if y is None:
        y = torch.empty((m, q.n_out), dtype=torch.bfloat16, device=x.device)
    if u is None and want_u:
        u = torch.empty((m, r), dtype=torch.bfloat16, device=x.device)
    ws = _workspace(ws, m, q, r, x.device)
    s = q.struct()
    st = lib.qlora_linear_fwd(ctypes.byref(s), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(y), _ptr(u),
                              _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(st, "qlora_linear_fwd")
    return y, u


def qlora_linear_fwd_noalloc(q, x, a, b, alpha, y=None, u=None, stream=None, want_u=True):
    """Forward without a caller workspace (library-owned fixed scratch); returns (y, u')."""
    torch = _torch()
    m = x.shape[0]
    r = a.shape[0]
    if y is None:
        y = torch.empty((m, q.n_out), dtype=torch.bfloat16, device=x.device)
    if u is None and want_u:
        u = torch.empty((m, r), dtype=torch.bfloat16, device=x.device)
    s = q.struct()
    st = lib.qlora_linear_fwd_noalloc(ctypes.byref(s), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(y),
                                      _ptr(u), _stream_ptr(stream))
    _check(st, "qlora_linear_fwd_noalloc")
    return y, u


def qlora_linear_bwd(q, x, u, dy, a, b, alpha, dx=None, da=None, db=None, ws=None, stream=None, want_dx=True):
    """Backward; returns (dX bf16 or None, dA fp32 [r, K], dB fp32 [N, r])."""
    torch = _torch()
    m = x.shape[0]
    r = a.shape[0]
    if dx is None and want_dx:
        dx = torch.empty((m, q.k_in), dtype=torch.bfloat16, device=x.device)
    if da is None:
        da = torch.empty((r, q.k_in), dtype=torch.float32, device=x.device)
    if db is None:
        db = torch.empty((q.n_out, r), dtype=torch.float32, device=x.device)
    ws = _workspace(ws, m, q, r, x.device)
    s = q.struct()
    st = lib.qlora_linear_bwd(ctypes.byref(s), _ptr(x), _ptr(u), _ptr(dy), m, _ptr(a), _ptr(b), r, float(alpha),
                              _ptr(dx), _ptr(da), _ptr(db), _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(st, "qlora_linear_bwd")
    return dx, da, db


def qlora_device_status(stream=None):
    """(status, bits): synchronises the stream and reads/clears the device status word."""
    bits = ctypes.c_uint32(0)
    st = lib.qlora_device_status(_stream_ptr(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


def qlora_selftest_wait_timeout(limit_us, stream=None):
    """Launch the bounded-wait self test (a wait that nothing completes); the
    timeout shows up in the next qlora_device_status()."""
    _check(lib.qlora_selftest_wait_timeout(int(limit_us), _stream_ptr(stream)), "qlora_selftest_wait_timeout")


SELFTEST_RING_NEVER, SELFTEST_RING_LATE, SELFTEST_RING_ONE = 0, 1, 2


def qlora_selftest_ring_timeout(limit_us, mode, out, stream=None):
    """Launch the self test of a ring of bulk copies whose wait gives up; `out`
    (int32 CUDA tensor of 129) gets the landings each thread saw and whether
    every copy landed before the kernel ended."""
    torch = _torch()
    if out.dtype is not torch.int32 or out.shape != (129,) or not out.is_cuda or not out.is_contiguous():
        raise ValueError("qlora_selftest_ring_timeout: out must be a contiguous int32 CUDA tensor of 129")
    _check(lib.qlora_selftest_ring_timeout(int(limit_us), int(mode), out.data_ptr(), _stream_ptr(stream)),
           "qlora_selftest_ring_timeout")


def qlora_merge_lora(q, a, b, alpha, out=None, stream=None):
    """bf16(W_hat + (alpha/r) B A) as a new [N, K] bf16 tensor (or into `out`)."""
    torch = _torch()
    r = a.shape[0]
    if out is None:
        out = torch.empty((q.n_out, q.k_in), dtype=torch.bfloat16, device=q.codes.device)
    s = q.struct()
    _check(lib.qlora_merge_lora(ctypes.byref(s), _ptr(a), _ptr(b), r, float(alpha), _ptr(out),
                                _stream_ptr(stream)), "qlora_merge_lora")
    return out


def qlora_adamw_step(master, grad, m, v, step, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                     param=None, stream=None):
    """One AdamW step in place on fp32 `master`, `m`, `v` (device tensors or
    pinned host tensors the GPU can address); `param` (bf16, optional)
    receives the bf16 copy. All arguments hold the same number of elements."""
    n = master.numel()
    for t in (grad, m, v) + ((param,) if param is not None else ()):
        if t.numel() != n:
            raise ValueError("qlora_adamw_step: element counts differ")
    hp = AdamwParams(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step))
    _check(lib.qlora_adamw_step(_ptr(master), _ptr(param) if param is not None else None, _ptr(grad), _ptr(m),
                                _ptr(v), n, ctypes.byref(hp), _stream_ptr(stream)), "qlora_adamw_step")


def qlora_adamw_staged(master, grad, m_host, v_host, m_stage, v_stage, step, lr=1e-4, betas=(0.9, 0.999),
                       eps=1e-8, weight_decay=0.0, param=None, stream=None):
    """One AdamW step with m, v in pinned host memory, staged through the
    device buffers m_stage, v_stage by copies on `stream` (H2D, update, D2H)."""
    n = master.numel()
    for t in (grad, m_host, v_host, m_stage, v_stage) + ((param,) if param is not None else ()):
        if t.numel() != n:
            raise ValueError("qlora_adamw_staged: element counts differ")
    hp = AdamwParams(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step))
    _check(lib.qlora_adamw_staged(_ptr(master), _ptr(param) if param is not None else None, _ptr(grad),
                                  _ptr(m_host), _ptr(v_host), _ptr(m_stage), _ptr(v_stage), n, ctypes.byref(hp),
                                  _stream_ptr(stream)), "qlora_adamw_staged")


def qlora_adamw_host(master, grad, m, v, step, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                     param=None):
    """AdamW on the host CPU, in place on CPU fp32 tensors; `param` (CPU
    bf16 tensor, optional) receives the bf16 copy."""
    n = master.numel()
    hp = AdamwParams(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step))
    _check(lib.qlora_adamw_host(_ptr(master), _ptr(param) if param is not None else None, _ptr(grad), _ptr(m),
                                _ptr(v), n, ctypes.byref(hp)), "qlora_adamw_host")


def qlora_adamw_paged(grad_dev, master_host, m_host, v_host, grad_host, step, param_dev=None, param_host=None,
                      lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, stream=None):
    """Enqueue one paged optimizer step on `stream` (D2H grad, CPU AdamW as a
    stream host function, H2D bf16 adapter). Host tensors must be pinned."""
    n = master_host.numel()
    hp = AdamwParams(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step))
    _check(lib.qlora_adamw_paged(_ptr(grad_dev), _ptr(param_dev), _ptr(master_host), _ptr(m_host), _ptr(v_host),
                                 _ptr(grad_host), _ptr(param_host), n, ctypes.byref(hp), _stream_ptr(stream)),
           "qlora_adamw_paged")


# ---------------------------------------------------------------- 8-bit linear, RMS norm, AdamW over many tensors
# Tensors are checked here (type, shape, device, contiguity), the rest by the
# library. A call works on the device of its tensors; `stream` (a
# torch.cuda.Stream of that device) replaces the current stream, and what the
# call allocates then belongs to that stream.
FP8_E4M3, FP8_E5M2 = 0, 1
_STATE_BLOCK = 256
_dtype_of = operator.attrgetter("dtype")


class Fp8Struct(ctypes.Structure):
    """Mirror of ``qlora_fp8_t``."""
    _fields_ = [("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class Fp8RowsStruct(ctypes.Structure):
    """Mirror of ``qlora_fp8_rows_t``."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


lib.qlora_quantize_fp8.argtypes = [_vp, _P(Fp8Struct), _vp]
lib.qlora_quantize_fp8.restype = ctypes.c_int
lib.qlora_dequantize_fp8.argtypes = [_P(Fp8Struct), _vp, _vp]
lib.qlora_dequantize_fp8.restype = ctypes.c_int
lib.qlora_quantize_fp8_rows.argtypes = [_vp, _P(Fp8RowsStruct), _vp]
lib.qlora_quantize_fp8_rows.restype = ctypes.c_int
lib.qlora_fp8_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.qlora_fp8_workspace_bytes.restype = _sz
lib.qlora_fp8_linear_fwd.argtypes = [_P(Fp8Struct), _vp, _P(Fp8RowsStruct), _i64, _vp, _vp, _sz, _vp]
lib.qlora_fp8_linear_fwd.restype = ctypes.c_int
lib.qlora_fp8_linear_bwd.argtypes = [_P(Fp8Struct), _vp, _P(Fp8RowsStruct), _i32, _i64, _vp, _vp, _sz, _vp]
lib.qlora_fp8_linear_bwd.restype = ctypes.c_int
lib.qlora_rmsnorm_fwd.argtypes = [_vp, _vp, _vp, _i64, _i64, _f32, _vp, _vp, _P(Fp8RowsStruct), _vp, _vp]
lib.qlora_rmsnorm_fwd.restype = ctypes.c_int
lib.qlora_rmsnorm_workspace_bytes.argtypes = [_i64, _i64]
lib.qlora_rmsnorm_workspace_bytes.restype = _sz
lib.qlora_rmsnorm_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]
lib.qlora_rmsnorm_bwd.restype = ctypes.c_int
lib.qlora_adamw_multi.argtypes = [_vp, _i64, _i32, _P(AdamwParams), _vp]
lib.qlora_adamw_multi.restype = ctypes.c_int


def _elsewhere(dev, stream, where):
    """None if the call can go ahead on the current device and stream, else a
    context that makes the tensors' device and the asked-for stream current."""
    torch = _torch()
    if dev < 0:
        raise ValueError(f"{where}: CUDA tensors are needed")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{where}: the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _raw_stream(dev):
    return _torch_module._C._cuda_getCurrentRawStream(dev)


def _is(t, dtype, shape, dev):
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _matrix(rows, cols, dtype, device):
    # the cheapest of torch's allocating calls for a shape of two
    return _torch_module.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _want(ok, where, what):
    if not ok:
        raise ValueError(f"{where}: {what}")


def _fp8_dtype(fmt):
    torch = _torch()
    if fmt == FP8_E4M3:
        return torch.float8_e4m3fn
    if fmt == FP8_E5M2:
        return torch.float8_e5m2
    raise ValueError("fmt must be FP8_E4M3 or FP8_E5M2")


class FP8Weight:
    """A weight [N, K] in e4m3 (`codes`, contiguous, K % 16 == 0) with one fp32
    scale per 128 x 128 block (`scales` [ceil(N/128), ceil(K/128)]): the
    weight is codes * scales block by block."""

    def __init__(self, codes, scales):
        torch = _torch()
        _want(codes.dim() == 2 and codes.dtype is torch.float8_e4m3fn and codes.is_contiguous(), "FP8Weight",
              "codes must be a contiguous float8_e4m3fn matrix")
        n, k = codes.shape
        _want(_is(scales, torch.float32, (-(-n // 128), -(-k // 128)), codes.get_device()), "FP8Weight",
              "scales must be contiguous fp32 [ceil(N/128), ceil(K/128)] on the codes' device")
        self.codes, self.scales, self.n_out, self.k_in = codes, scales, n, k

    @classmethod
    def empty(cls, n_out, k_in, device="cuda"):
        torch = _torch()
        return cls(torch.empty((n_out, k_in), dtype=torch.float8_e4m3fn, device=device),
                   torch.empty((-(-n_out // 128), -(-k_in // 128)), dtype=torch.float32, device=device))

    def struct(self):
        return Fp8Struct(self.n_out, self.k_in, self.codes.data_ptr(), self.scales.data_ptr())


class FP8Rows:
    """Rows in 8 bits: `codes` [rows, cols] float8_e4m3fn or float8_e5m2, each
    row contiguous and rows a multiple of 16 bytes apart, and one fp32 scale
    per 128 columns (`scales` [rows, ceil(cols/128)])."""

    def __init__(self, codes, scales):
        torch = _torch()
        _want(codes.dim() == 2 and codes.dtype in (torch.float8_e4m3fn, torch.float8_e5m2), "FP8Rows",
              "codes must be a float8_e4m3fn or float8_e5m2 matrix")
        rows, cols = codes.shape
        ld = codes.stride(0) if rows > 1 else -(-cols // 16) * 16
        _want((codes.stride(1) == 1 or cols == 1) and ld % 16 == 0 and ld >= cols, "FP8Rows",
              "rows must be contiguous and a multiple of 16 bytes apart")
        _want(_is(scales, torch.float32, (rows, -(-cols // 128)), codes.get_device()), "FP8Rows",
              "scales must be contiguous fp32 [rows, ceil(cols/128)] on the codes' device")
        self.codes, self.scales, self.ld = codes, scales, ld
        self.fmt = FP8_E4M3 if codes.dtype is torch.float8_e4m3fn else FP8_E5M2

    @classmethod
    def empty(cls, rows, cols, fmt=FP8_E4M3, device="cuda"):
        torch = _torch()
        dtype, ld = _fp8_dtype(fmt), (cols + 15) & ~15
        codes = _matrix(rows, ld, dtype, device)
        self = cls.__new__(cls)      # right by construction: no checks
        self.codes = codes if ld == cols else codes[:, :cols]
        self.scales = _matrix(rows, (cols + 127) >> 7, torch.float32, device)
        self.ld, self.fmt = ld, fmt
        return self

    def struct(self):
        rows, cols = self.codes.shape
        return Fp8RowsStruct(rows, cols, self.ld, self.codes.data_ptr(), self.scales.data_ptr(), self.fmt, 0)

    def dequantize(self):
        """The values the rows stand for, fp32."""
        cols = self.codes.shape[1]
        return self.codes.float() * self.scales.repeat_interleave(128, 1)[:, :cols]


def qlora_quantize_fp8(w, out=None, stream=None):
    """A bf16 CUDA weight [N, K] as an :class:`FP8Weight`."""
    torch = _torch()
    dev = w.get_device()
    if (at := _elsewhere(dev, stream, "qlora_quantize_fp8")) is not None:
        with at:
            return qlora_quantize_fp8(w, out)
    _want(w.dim() == 2 and _is(w, torch.bfloat16, w.shape, dev), "qlora_quantize_fp8", "w must be a contiguous bf16 matrix")
    if out is None:
        out = FP8Weight.empty(*w.shape, device=w.device)
    _want(out.codes.shape == w.shape and out.codes.get_device() == dev, "qlora_quantize_fp8", "out has another shape or device")
    _check(lib.qlora_quantize_fp8(w.data_ptr(), out.struct(), _raw_stream(dev)), "qlora_quantize_fp8")
    return out


def qlora_dequantize_fp8(q, out=None, stream=None):
    """bf16 [N, K] from an :class:`FP8Weight`."""
    torch = _torch()
    dev = q.codes.get_device()
    if (at := _elsewhere(dev, stream, "qlora_dequantize_fp8")) is not None:
        with at:
            return qlora_dequantize_fp8(q, out)
    if out is None:
        out = torch.empty((q.n_out, q.k_in), dtype=torch.bfloat16, device=q.codes.device)
    _want(_is(out, torch.bfloat16, (q.n_out, q.k_in), dev), "qlora_dequantize_fp8", "out must be contiguous bf16 [N, K]")
    _check(lib.qlora_dequantize_fp8(q.struct(), out.data_ptr(), _raw_stream(dev)), "qlora_dequantize_fp8")
    return out


def qlora_quantize_fp8_rows(x, fmt=FP8_E4M3, out=None, stream=None):
    """bf16 rows [rows, cols] as :class:`FP8Rows`."""
    torch = _torch()
    dev = x.get_device()
    if (at := _elsewhere(dev, stream, "qlora_quantize_fp8_rows")) is not None:
        with at:
            return qlora_quantize_fp8_rows(x, fmt, out)
    _want(x.dim() == 2 and _is(x, torch.bfloat16, x.shape, dev), "qlora_quantize_fp8_rows",
          "x must be a contiguous bf16 matrix")
    if out is None:
        out = FP8Rows.empty(*x.shape, fmt=fmt, device=x.device)
    _want(out.codes.shape == x.shape and out.codes.get_device() == dev, "qlora_quantize_fp8_rows",
          "out has another shape or device")
    _check(lib.qlora_quantize_fp8_rows(x.data_ptr(), out.struct(), _raw_stream(dev)), "qlora_quantize_fp8_rows")
    return out


def qlora_fp8_workspace_bytes(m, n_out, k_in):
    return int(lib.qlora_fp8_workspace_bytes(int(m), int(n_out), int(k_in)))


def _fp8_product(call, where, q, x, fmt, cols_in, cols_out, out, ws):
    torch = _torch_module
    dev = q.codes.get_device()
    rows = x.struct() if type(x) is FP8Rows else None
    src = x if rows is None else x.codes
    if not (src.dim() == 2 and src.shape[1] == cols_in and src.get_device() == dev and
            (rows is not None or (src.dtype is torch.bfloat16 and src.is_contiguous()))):
        raise ValueError(f"{where}: rows must be FP8Rows or contiguous bf16 [m, {cols_in}] on the weight's device")
    m = src.shape[0]
    if out is None:
        out = _matrix(m, cols_out, torch.bfloat16, src.device)
    elif not _is(out, torch.bfloat16, (m, cols_out), dev):
        raise ValueError(f"{where}: the output must be contiguous bf16 [m, {cols_out}]")
    at = size = 0
    if ws is not None:
        _want(ws.get_device() == dev and ws.is_contiguous(), where, "the workspace must be contiguous, on the weight's device")
        at, size = ws.data_ptr(), ws.numel() * ws.element_size()
    elif rows is None:           # rows already in 8 bits need none, nor do a few
        size = lib.qlora_fp8_workspace_bytes(m, q.n_out, q.k_in)
        if size:
            ws = torch.empty(size, dtype=torch.uint8, device=src.device)
            at = ws.data_ptr()
    x16, stream = x.data_ptr() if rows is None else None, _raw_stream(dev)
    st = (call(q.struct(), x16, rows, m, out.data_ptr(), at, size, stream) if fmt is None else
          call(q.struct(), x16, rows, int(fmt), m, out.data_ptr(), at, size, stream))
    if st:
        raise QloraError(st, where)
    return out


def qlora_fp8_linear_fwd(q, x, y=None, ws=None, stream=None):
    """y [m, N] bf16 = x W^T; x is bf16 [m, K] (quantized to e4m3 rows within
    the call) or :class:`FP8Rows`."""
    if (at := _elsewhere(q.codes.get_device(), stream, "qlora_fp8_linear_fwd")) is not None:
        with at:
            return qlora_fp8_linear_fwd(q, x, y, ws)
    return _fp8_product(lib.qlora_fp8_linear_fwd, "qlora_fp8_linear_fwd", q, x, None, q.k_in, q.n_out, y, ws)


def qlora_fp8_linear_bwd(q, dy, fmt=FP8_E4M3, dx=None, ws=None, stream=None):
    """dX [m, K] bf16 = dY W; dY is bf16 [m, N] (quantized to rows of `fmt`
    within the call) or :class:`FP8Rows`."""
    if (at := _elsewhere(q.codes.get_device(), stream, "qlora_fp8_linear_bwd")) is not None:
        with at:
            return qlora_fp8_linear_bwd(q, dy, fmt, dx, ws)
    return _fp8_product(lib.qlora_fp8_linear_bwd, "qlora_fp8_linear_bwd", q, dy, fmt, q.n_out, q.k_in, dx, ws)


def qlora_rmsnorm_fwd(x, gamma, eps=1e-6, residual=None, fp8=False, fmt=FP8_E4M3, y=None, h=None, rstd=None,
                      stream=None):
    """(y, h, rstd): h = bf16(x + residual) (x itself without a residual),
    rstd fp32 per row, y = h rstd gamma as bf16 or, with fp8=True, as
    :class:`FP8Rows`. x, residual [rows, d], gamma [d] bf16."""
    torch = _torch()
    dev = x.get_device()
    if (at := _elsewhere(dev, stream, "qlora_rmsnorm_fwd")) is not None:
        with at:
            return qlora_rmsnorm_fwd(x, gamma, eps, residual, fp8, fmt, y, h, rstd)
    bf16, shape, device = torch.bfloat16, x.shape, x.device
    if not (len(shape) == 2 and x.dtype is bf16 and x.is_contiguous() and _is(gamma, bf16, shape[1:], dev) and
            (residual is None or _is(residual, bf16, shape, dev))):
        raise ValueError("qlora_rmsnorm_fwd: x, residual [rows, d] and gamma [d] must be contiguous bf16 on one device")
    rows, d = shape
    if y is None:
        y = FP8Rows.empty(rows, d, fmt, device) if fp8 else torch.empty_like(x)
    else:
        _want((isinstance(y, FP8Rows) and y.codes.shape == shape and y.codes.get_device() == dev) if fp8
              else _is(y, bf16, shape, dev), "qlora_rmsnorm_fwd", "y has another type, shape or device")
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
    else:
        _want(_is(rstd, torch.float32, (rows,), dev), "qlora_rmsnorm_fwd", "rstd must be fp32 [rows]")
    at_res = at_h = None
    if residual is not None:
        if h is None:
            h = torch.empty_like(x)
        else:
            _want(_is(h, bf16, shape, dev), "qlora_rmsnorm_fwd", "h must be contiguous bf16 [rows, d]")
        at_res, at_h = residual.data_ptr(), h.data_ptr()
    else:
        _want(h is None, "qlora_rmsnorm_fwd", "h is written only with a residual")
        h = x
    y16, y8 = (None, y.struct()) if fp8 else (y.data_ptr(), None)
    st = lib.qlora_rmsnorm_fwd(x.data_ptr(), at_res, gamma.data_ptr(), rows, d, eps, at_h, y16, y8, rstd.data_ptr(),
                               _raw_stream(dev))
    if st:
        raise QloraError(st, "qlora_rmsnorm_fwd")
    return y, h, rstd


def qlora_rmsnorm_workspace_bytes(rows, d):
    return int(lib.qlora_rmsnorm_workspace_bytes(int(rows), int(d)))


def qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=None, dx=None, dgamma=None, ws=None, want_dgamma=True, stream=None):
    """(dx bf16 [rows, d], dgamma fp32 [d] or None) from dy, the forward's h
    and rstd, and `dres`, the gradient that reaches h past the norm. dx is the
    gradient of x and of the residual alike."""
    torch = _torch()
    dev = dy.get_device()
    if (at := _elsewhere(dev, stream, "qlora_rmsnorm_bwd")) is not None:
        with at:
            return qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres, dx, dgamma, ws, want_dgamma)
    _want(dy.dim() == 2, "qlora_rmsnorm_bwd", "dy must be a matrix")
    rows, d = dy.shape
    bf16, f32 = torch.bfloat16, torch.float32
    _want(_is(dy, bf16, dy.shape, dev) and _is(h, bf16, dy.shape, dev) and _is(gamma, bf16, (d,), dev) and
          _is(rstd, f32, (rows,), dev) and (dres is None or _is(dres, bf16, dy.shape, dev)), "qlora_rmsnorm_bwd",
          "dy, h, dres [rows, d] and gamma [d] must be contiguous bf16, rstd [rows] fp32, on one device")
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _want(_is(dx, bf16, dy.shape, dev), "qlora_rmsnorm_bwd", "dx must be contiguous bf16 [rows, d]")
    if dgamma is not None:
        _want(_is(dgamma, f32, (d,), dev), "qlora_rmsnorm_bwd", "dgamma must be fp32 [d]")
    elif want_dgamma:
        dgamma = torch.empty(d, dtype=f32, device=dy.device)
    if ws is None and dgamma is not None:
        ws = torch.empty(lib.qlora_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device=dy.device)
    elif ws is not None:
        _want(ws.get_device() == dev and ws.is_contiguous(), "qlora_rmsnorm_bwd", "the workspace must be contiguous, on dy's device")
    st = lib.qlora_rmsnorm_bwd(dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(),
                               None if dres is None else dres.data_ptr(), rows, d, dx.data_ptr(),
                               None if dgamma is None else dgamma.data_ptr(), None if ws is None else ws.data_ptr(),
                               0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(dev))
    _check(st, "qlora_rmsnorm_bwd")
    return dx, dgamma


class AdamWGroup:
    """Tensors that qlora_adamw_multi updates together: fp32 `masters`, their
    bf16 copies `params` (optional) and the Adam states, in flat buffers where
    every tensor starts at a multiple of 256 values. bits=32: `m`, `v` fp32.
    bits=8: `m` holds e4m3 codes of m and `v` e4m3 codes of sqrt(v), with one
    fp32 scale per 256 values (`m_scales`, `v_scales`). States that are not
    given start at zero. The group keeps the tensors; their storage must stay
    where it is."""

    def __init__(self, masters, params=None, bits=32, m=None, v=None, m_scales=None, v_scales=None):
        import numpy as np
        torch = _torch()
        self.masters = list(masters)
        self.params = None if params is None else list(params)
        _want(self.masters, "AdamWGroup", "no tensors")
        _want(bits in (8, 32), "AdamWGroup", "bits must be 8 or 32")
        dev = self.masters[0].get_device()
        _want(dev >= 0, "AdamWGroup", "CUDA tensors are needed")
        _want(all(_is(t, torch.float32, t.shape, dev) for t in self.masters), "AdamWGroup",
              "masters must be contiguous fp32 on one device")
        self.sizes = [t.numel() for t in self.masters]
        if self.params is not None:
            _want(len(self.params) == len(self.sizes) and all(
                _is(t, torch.bfloat16, t.shape, dev) and t.numel() == n for t, n in zip(self.params, self.sizes)),
                "AdamWGroup", "params must be contiguous bf16, as many and as long as the masters, on their device")
        starts = np.concatenate([[0], np.cumsum([-(-n // _STATE_BLOCK) * _STATE_BLOCK for n in self.sizes])])
        total = int(starts[-1])
        self.bits, self.device = bits, self.masters[0].device
        dtype, width = (torch.float32, 4) if bits == 32 else (torch.float8_e4m3fn, 1)
        names = (("m", m, dtype, total), ("v", v, dtype, total))
        if bits == 8:
            names += (("m_scales", m_scales, torch.float32, total // _STATE_BLOCK),
                      ("v_scales", v_scales, torch.float32, total // _STATE_BLOCK))
        else:
            _want(m_scales is None and v_scales is None, "AdamWGroup", "32-bit states have no scales")
        self.m_scales = self.v_scales = None
        for name, t, ty, n in names:
            if t is None:
                t = torch.zeros(n, dtype=torch.float32 if ty is torch.float32 else torch.uint8, device=self.device).view(ty)
            _want(_is(t, ty, (n,), dev), "AdamWGroup", f"{name} must be contiguous {ty} of {n} values on the masters' device")
            setattr(self, name, t)
        self._at = [t.data_ptr() for t in self.masters], [t.data_ptr() for t in self.params or []]
        self._states_at = self._states()
        desc = np.zeros((len(self.sizes), 8), dtype=np.uint64)     # rows of qlora_adamw_tensor_t
        desc[:, 0] = self._at[0]
        if self.params is not None:
            desc[:, 1] = self._at[1]
        at = starts[:-1].astype(np.uint64)
        desc[:, 3] = self.m.data_ptr() + at * np.uint64(width)
        desc[:, 4] = self.v.data_ptr() + at * np.uint64(width)
        if bits == 8:
            blocks = at // np.uint64(_STATE_BLOCK) * np.uint64(4)
            desc[:, 5] = self.m_scales.data_ptr() + blocks
            desc[:, 6] = self.v_scales.data_ptr() + blocks
        desc[:, 7] = self.sizes
        self._desc = desc

    def _states(self):
        # scales None: 32-bit states
        return [None if t is None else t.data_ptr() for t in (self.m, self.v, self.m_scales, self.v_scales)]


def qlora_adamw_multi(group, grads, step, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, stream=None):
    """One AdamW step over all tensors of an :class:`AdamWGroup` (in place on
    its masters, params and states) with fp32 `grads` in the group's order."""
    torch = _torch()
    T = torch.Tensor
    dev = group.masters[0].get_device()
    if (at := _elsewhere(dev, stream, "qlora_adamw_multi")) is not None:
        with at:
            return qlora_adamw_multi(group, grads, step, lr, betas, eps, weight_decay)
    # a few C-level passes over the lists: with hundreds of tensors this is most of the call's host time
    _want(list(map(T.numel, grads)) == group.sizes, "qlora_adamw_multi", "grads must match the masters in number and length")
    _want(set(map(_dtype_of, grads)) == {torch.float32} and all(map(T.is_contiguous, grads)) and
          set(map(T.get_device, grads)) == {dev}, "qlora_adamw_multi", "grads must be contiguous fp32 on the group's device")
    _want(list(map(T.data_ptr, group.masters)) == group._at[0] and
          list(map(T.data_ptr, group.params or ())) == group._at[1] and group._states() == group._states_at,
          "qlora_adamw_multi", "a master's, param's or state's storage has moved since the group was made")
    desc = group._desc.copy()
    desc[:, 2] = array.array("Q", map(T.data_ptr, grads))      # numpy takes its memory as it is
    hp = AdamwParams(lr, betas[0], betas[1], eps, weight_decay, step)
    _check(lib.qlora_adamw_multi(desc.ctypes.data, len(grads), group.bits, hp, _raw_stream(dev)), "qlora_adamw_multi")
