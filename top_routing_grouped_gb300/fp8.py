"""Binding of the 8-bit operators in libmoe.so (the C ABI in include/moe_fp8.h).

Argument marshalling only, as in ``moe``: outputs and workspaces are the caller's tensors, and
every call enqueues its kernels on the current stream (or ``stream``) and returns.  The checks of
the calls that run once a layer or more are compiled (``_fp8``, csrc/binding.cpp).  8-bit tensors
are torch.float8_e4m3fn, their block factors torch.float8_e8m0fnu (or the bytes as uint8); a row
of c values has ``scale_cols(c)`` factors.  A wrong type, shape or layout, a tensor outside GPU memory and
tensors (or a stream) of more than one device raise ValueError before the library is called; the library's
own checks raise ``moe.MoEError``.  The tensors' device is made current for the call.
"""
import ctypes

import torch

from .moe import MOE_BF16, MOE_F32, MOE_OK, MoEError, MoeExpertConfig, MoEPlan, _lib, _PATHS

try:
    from . import _fp8  # after torch and libmoe.so, which it is linked with
except ImportError as e:
    raise ImportError("the binding of the 8-bit operators (_fp8.so) is missing or does not load: build it with "
                      "__graft_entry__.build(), where g++ and the headers of Python and torch are") from e

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
E4M3 = torch.float8_e4m3fn


class MoeFp8MatmulConfig(ctypes.Structure):
    _fields_ = [("max_rows", _I64), ("k", _I32), ("n", _I32), ("n_experts", _I32), ("n_sources", _I32),
                ("out_dtype", _I32), ("path", _I32), ("wait_timeout_ns", _I64)]


def _declare(name, *argtypes, restype=ctypes.c_int):
    f = getattr(_lib, name)
    f.argtypes, f.restype = list(argtypes), restype
    return f


_declare("moe_fp8_scale_cols", _I64, restype=_I64)
_declare("moe_fp8_quantize", _P, _I32, _I64, _I64, _I64, _I32, _I64, _P, _P, _P)
_declare("moe_rmsnorm", _P, _P, _P, _I32, _I64, _I32, _I64, _I64, _F, _P, _P, _P, _P, _P, _P)
_rmsnorm_ws = _declare("moe_rmsnorm_backward_workspace", _I64, _I32, restype=ctypes.c_size_t)
_declare("moe_rmsnorm_backward", _P, _I32, _P, _P, _P, _P, _I32, _I64, _I32, _I64, _P, _P, _P, ctypes.c_size_t, _P)
_matmul_plan = _declare("moe_fp8_matmul_plan", ctypes.POINTER(MoeFp8MatmulConfig), ctypes.POINTER(_P),
                        ctypes.POINTER(ctypes.c_size_t))
_declare("moe_fp8_matmul", *[_P] * 8, ctypes.c_size_t, _P)
_expert_plan = _declare("moe_fp8_expert_plan", ctypes.POINTER(MoeExpertConfig), ctypes.POINTER(_P),
                        ctypes.POINTER(ctypes.c_size_t))
_declare("moe_fp8_expert_forward", *[_P] * 13, ctypes.c_size_t, _P)
_plan_destroy = _declare("moe_fp8_plan_destroy", _P, restype=None)
_device_status = _declare("moe_fp8_get_device_status", _P, _P, _P)
_declare("moe_fp8_forward", *[_P] * 14, ctypes.c_size_t, _P)
_declare("moe_checkpoint_restore_rows", *[_P] * 4, _I64, _I32, _P, _P, _P, _P)
_layer_ckpt_bytes = _declare("moe_checkpoint_bytes", _P, restype=ctypes.c_size_t)
_layer_ckpt_save = _declare("moe_checkpoint_save", _P, _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P)
_layer_ckpt_restore = _declare("moe_checkpoint_restore", _P, _P, _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P)
_declare("moe_checkpoint_save_rows", _P, _P, _I64, _I32, _P, _P, _P, _P, _P)
_declare("moe_checkpoint_backward_rows", *[_P] * 5, _I64, _I32, _P, _P, _P, _P)


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def _want(cond, what):
    if not cond:
        raise ValueError(what)


_raw_stream = torch._C._cuda_getCurrentRawStream  # an order cheaper than building a torch.cuda.Stream


def _bytes(t):
    """The address of a workspace or checkpoint."""
    if t.dtype is not torch.uint8 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspaces and checkpoints must be contiguous uint8 tensors in GPU memory")
    return t.data_ptr()


def _one_device(*ts, stream=None):
    """The one device of these tensors and of the stream, made current for the call."""
    d = ts[0].get_device()
    if any(t.get_device() != d for t in ts) or (stream is not None and stream.device_index != d):
        raise ValueError("all tensors and the stream must be on one device")
    return torch.cuda.device(d)


def _stream(stream, t):
    """The given stream, or the current one of t's device."""
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def scale_cols(cols):
    """Factors of a row of `cols` values: one for every 128, in whole words of four."""
    return (int(cols) + 511) // 512 * 4 if cols > 0 else 0


def quantize(x, q, scales, stream=None):
    """Rows x [n, c] (fp32 or bf16; any row pitch) into q [n, c] with scales [n, scale_cols(c)]."""
    _check(_fp8.quantize(x, q, scales, stream), "moe_fp8_quantize")


def quantize_weights(w, q, scales, stream=None):
    """Weights w [E, n, c] (fp32 or bf16) into q [E, n, c] with scales [E, ceil(n/128), scale_cols(c)]."""
    _check(_fp8.quantize_weights(w, q, scales, stream), "moe_fp8_quantize")


def rmsnorm(x, weight, residual=None, residual_out=None, out=None, q=None, scales=None, rstd=None, eps=1e-6, stream=None):
    """r = x + residual, n = r * rstd * weight into whichever outputs are given (moe_rmsnorm):
    residual_out and out [T, d] in x's type, q e4m3 with scales, rstd [T] fp32.  x and residual may
    have any row pitch; weight fp32 [d] or None for ones."""
    _check(_fp8.rmsnorm(x, weight, residual, residual_out, out, q, scales, rstd, eps, stream), "moe_rmsnorm")


def rmsnorm_backward_workspace(T, d, device="cuda"):
    """The workspace of rmsnorm_backward for [T, d] (when dweight is wanted)."""
    return torch.empty(max(1, int(_rmsnorm_ws(int(T), int(d)))), dtype=torch.uint8, device=device)


def rmsnorm_backward(dout, r, weight, rstd, dx, dweight=None, workspace=None, dresidual=None, stream=None):
    """dx and dweight from dout = dL/dn (fp32 or bf16) and what the forward kept: r (its
    residual_out, or x without a residual; any row pitch) and rstd; dresidual is the gradient that
    reaches r on its other way.  dx may be dresidual, dout or r itself."""
    _check(_fp8.rmsnorm_backward(dout, r, weight, rstd, dx, dweight, workspace, dresidual, stream), "moe_rmsnorm_backward")


class _Fp8Plan:
    def _make(self, make, cfg, where):
        self._h = ctypes.c_void_p()
        wsb = ctypes.c_size_t(0)
        _check(make(ctypes.byref(cfg), ctypes.byref(self._h), ctypes.byref(wsb)), where)
        self.workspace_bytes = wsb.value

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            _plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    @property
    def handle(self):
        return self._h

    def new_workspace(self, device="cuda"):
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)

    def device_status(self, workspace, stream=None):
        """Synchronises the stream; returns the status code (MOE_OK == 0)."""
        p = _bytes(workspace)
        with _one_device(workspace, stream=stream):
            return _device_status(self._h, p, _stream(stream, workspace))


class Fp8MatmulPlan(_Fp8Plan):
    """out[p] = A[p] . W_e^T for rows grouped by expert (moe_fp8_matmul): K columns in, n out."""

    def __init__(self, max_rows, K, n, n_experts=1, n_sources=1, out_dtype="bf16", path="auto", wait_timeout_ns=0):
        self.out_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        self.cfg = MoeFp8MatmulConfig(int(max_rows), int(K), int(n), int(n_experts), int(n_sources), _DTYPES[self.out_dtype],
                                      _PATHS[path], int(wait_timeout_ns))
        self._make(_matmul_plan, self.cfg, "moe_fp8_matmul_plan")
        c = self.cfg
        self._args = (self._h.value, c.max_rows, c.k, c.n, c.n_experts, c.n_experts * c.n_sources, int(out_dtype == "bf16"))

    def forward(self, seg_counts, a, a_scales, w, w_scales, out, workspace, stream=None):
        """seg_counts: int32 rows of each (source, expert) segment, or None for one segment of
        max_rows rows."""
        _check(_fp8.matmul(*self._args, seg_counts, a, a_scales, w, w_scales, out, workspace, stream), "moe_fp8_matmul")


class Fp8ExpertPlan(_Fp8Plan):
    """The expert stage in 8 bits (moe_fp8_expert_forward); the arguments are moe.ExpertPlan's."""

    def __init__(self, max_rows, d, E_local, n_sources, F, path="auto", wait_timeout_ns=0):
        R, d, E, W, F = int(max_rows), int(d), int(E_local), int(n_sources), int(F)
        self.cfg = MoeExpertConfig(R, d, E, W, F, MOE_BF16, _PATHS[path], int(wait_timeout_ns))
        self._make(_expert_plan, self.cfg, "moe_fp8_expert_plan")
        self.max_rows, self.d, self.E_local, self.n_sources, self.F = R, d, E, W, F
        self._args = (self._h.value, R, d, E, E * W, F)

    def forward(self, seg_counts, x_rows, x_scales, gates, w1, s1, w3, s3, w2, s2, y_rows, workspace, stream=None):
        _check(_fp8.experts(*self._args, seg_counts, x_rows, x_scales, gates, w1, s1, w3, s3, w2, s2, y_rows, workspace, stream),
               "moe_fp8_expert_forward")


class Fp8MoEPlan(MoEPlan):
    """The whole layer with its experts in 8 bits (moe_fp8_forward): the arguments are MoEPlan's."""

    def __init__(self, T, d, E, k, F, out_dtype="bf16", tau=1.0, has_bias=False, keep_logits=False, wait_timeout_ns=0,
                 renorm_gates=False):
        super().__init__(T, d, E, k, F, dtype="bf16", out_dtype=out_dtype, tau=tau, has_bias=has_bias, keep_logits=keep_logits,
                         wait_timeout_ns=wait_timeout_ns, renorm_gates=renorm_gates, fp8_experts=True)
        self._args = (self.handle.value, self.T, self.d, self.E, self.F, int(self.out_dtype is torch.bfloat16))

    def forward(self, x, x_q, x_scales, w_router, bias, w1, s1, w3, s3, w2, s2, y, workspace, stream=None):
        """x (bf16) for the router, x_q with x_scales for the experts: both as rmsnorm writes them."""
        _check(_fp8.layer(*self._args, x, x_q, x_scales, w_router, bias, w1, s1, w3, s3, w2, s2, y, workspace, stream),
               "moe_fp8_forward")


class LayerCheckpoint:
    """What one training forward of `plan` (a MoEPlan with training=True) has to leave for its backward,
    with the pre-activations in 8 bits, so that the layers of a stack can share a workspace:
    save(workspace) after plan.forward, restore(x, workspace) before plan.backward."""

    def __init__(self, plan, device="cuda"):
        self.plan = plan
        n = int(_layer_ckpt_bytes(plan.handle))
        _want(n > 0, "checkpoints need a plan with training=True")
        self.data = torch.empty(n, dtype=torch.uint8, device=device)

    def _rows(self, x):
        p = self.plan
        if x.is_cuda and x.dtype is p.act_dtype and x.shape == (p.T, p.d) and x.is_contiguous():
            return x.data_ptr()
        raise ValueError("x must be in GPU memory" if not x.is_cuda else
                         f"x must be a contiguous {(p.T, p.d)} tensor of {p.act_dtype}")

    def save(self, workspace, stream=None):
        ws, data = _bytes(workspace), _bytes(self.data)
        with _one_device(workspace, self.data, stream=stream):
            _check(_layer_ckpt_save(self.plan.handle, ws, workspace.numel(), data, self.data.numel(),
                                    _stream(stream, workspace)), "moe_checkpoint_save")

    def restore(self, x, workspace, stream=None):
        px, ws, data = self._rows(x), _bytes(workspace), _bytes(self.data)
        with _one_device(x, workspace, self.data, stream=stream):
            _check(_layer_ckpt_restore(self.plan.handle, px, data, self.data.numel(), ws, workspace.numel(),
                                       _stream(stream, x)), "moe_checkpoint_restore")


def checkpoint_save(a, b, qa, sa, qb, sb, stream=None):
    """The pre-activations a, b [n, F] (bf16) into 8 bits (moe_checkpoint_save_rows)."""
    _check(_fp8.checkpoint_save(a, b, qa, sa, qb, sb, stream), "moe_checkpoint_save_rows")


def checkpoint_restore(qa, sa, qb, sb, a=None, b=None, h=None, stream=None):
    """The values of a checkpoint and h = silu(a) * b into whichever of a, b, h are given, [n, F] bf16
    (moe_checkpoint_restore_rows)."""
    _check(_fp8.checkpoint_restore(qa, sa, qb, sb, a, b, h, stream), "moe_checkpoint_restore_rows")


def checkpoint_backward(qa, sa, qb, sb, dh, da, db, h=None, stream=None):
    """The SwiGLU's backward out of the checkpoint (moe_checkpoint_backward_rows): da, db and, if
    given, the hidden rows h, all [n, F] bf16, from dh."""
    _check(_fp8.checkpoint_backward(qa, sa, qb, sb, dh, da, db, h, stream), "moe_checkpoint_backward_rows")
