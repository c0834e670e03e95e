"""ctypes binding of the 8-bit operators in libmoe.so (the C ABI in include/moe_fp8.h).

Argument marshalling only, as in ``moe``: outputs and workspaces are the caller's tensors, and
every call enqueues its kernels on the current stream (or ``stream``) and returns.  8-bit tensors
are torch.float8_e4m3fn, their block factors torch.float8_e8m0fnu (or the bytes as uint8); a row
of c values has ``scale_cols(c)`` factors.  A wrong type, shape or layout raises ValueError before
the library is called; the library's own checks raise ``moe.MoEError``.
"""
import ctypes

import torch

from .moe import MOE_BF16, MOE_F32, MOE_OK, MoEError, MoeExpertConfig, MoEPlan, _lib, _PATHS

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
_SCALES = (torch.float8_e8m0fnu, torch.uint8)
E4M3 = torch.float8_e4m3fn
_FLOATS, _E4, _F32, _BF16 = tuple(_DTYPES), (E4M3,), (torch.float32,), (torch.bfloat16,)


class MoeFp8MatmulConfig(ctypes.Structure):
    _fields_ = [("max_rows", _I64), ("k", _I32), ("n", _I32), ("n_experts", _I32), ("n_sources", _I32),
                ("out_dtype", _I32), ("path", _I32), ("wait_timeout_ns", _I64)]


def _declare(name, *argtypes, restype=ctypes.c_int):
    f = getattr(_lib, name)
    f.argtypes, f.restype = list(argtypes), restype
    return f


_declare("moe_fp8_scale_cols", _I64, restype=_I64)
_quantize = _declare("moe_fp8_quantize", _P, _I32, _I64, _I64, _I64, _I32, _I64, _P, _P, _P)
_rmsnorm = _declare("moe_rmsnorm", _P, _P, _P, _I32, _I64, _I32, _I64, _I64, _F, _P, _P, _P, _P, _P, _P)
_rmsnorm_ws = _declare("moe_rmsnorm_backward_workspace", _I64, _I32, restype=ctypes.c_size_t)
_rmsnorm_bwd = _declare("moe_rmsnorm_backward", _P, _I32, _P, _P, _P, _P, _I32, _I64, _I32, _I64, _P, _P, _P,
                        ctypes.c_size_t, _P)
_matmul_plan = _declare("moe_fp8_matmul_plan", ctypes.POINTER(MoeFp8MatmulConfig), ctypes.POINTER(_P),
                        ctypes.POINTER(ctypes.c_size_t))
_matmul = _declare("moe_fp8_matmul", *[_P] * 8, ctypes.c_size_t, _P)
_expert_plan = _declare("moe_fp8_expert_plan", ctypes.POINTER(MoeExpertConfig), ctypes.POINTER(_P),
                        ctypes.POINTER(ctypes.c_size_t))
_expert_forward = _declare("moe_fp8_expert_forward", *[_P] * 13, ctypes.c_size_t, _P)
_plan_destroy = _declare("moe_fp8_plan_destroy", _P, restype=None)
_device_status = _declare("moe_fp8_get_device_status", _P, _P, _P)
_layer_forward = _declare("moe_fp8_forward", *[_P] * 14, ctypes.c_size_t, _P)
_ckpt_restore_rows = _declare("moe_checkpoint_restore_rows", *[_P] * 4, _I64, _I32, _P, _P, _P, _P)
_layer_ckpt_bytes = _declare("moe_checkpoint_bytes", _P, restype=ctypes.c_size_t)
_layer_ckpt_save = _declare("moe_checkpoint_save", _P, _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P)
_layer_ckpt_restore = _declare("moe_checkpoint_restore", _P, _P, _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P)
_ckpt_save = _declare("moe_checkpoint_save_rows", _P, _P, _I64, _I32, _P, _P, _P, _P, _P)
_ckpt_backward = _declare("moe_checkpoint_backward_rows", *[_P] * 5, _I64, _I32, _P, _P, _P, _P)


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def _want(cond, what):
    if not cond:
        raise ValueError(what)


_raw_stream = torch._C._cuda_getCurrentRawStream  # an order cheaper than building a torch.cuda.Stream


# The checks below run on every call, and a call of a few rows takes the GPU two or three
# microseconds: messages are put together only when a check has failed.

def _refuse(t, shape, dtypes, name, how):
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must be in GPU memory")
    raise ValueError(f"{name} must be a {how} {tuple(shape)} tensor of {' or '.join(str(d) for d in dtypes)}")


def _rows(t, shape, dtypes, name):
    """The address of a row-major contiguous GPU tensor of this shape and type."""
    if t is not None and t.dtype in dtypes and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, shape, dtypes, name, "contiguous")


def _maybe(t, shape, dtypes, name):
    return None if t is None else _rows(t, shape, dtypes, name)


def _pitched(t, shape, dtypes, name):
    """(address, row pitch) of a 2-D GPU tensor whose rows are contiguous and separate."""
    if t.dtype in dtypes and t.shape == shape and t.is_cuda:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        pitch, step = t.stride()
        if (step == 1 or shape[1] == 1) and (pitch >= shape[1] or shape[0] == 1):
            return t.data_ptr(), max(pitch, shape[1])
    _refuse(t, shape, dtypes, name, "row-contiguous")


def _bytes(t):
    """The address of a workspace or checkpoint."""
    if t.dtype is not torch.uint8 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspaces and checkpoints must be contiguous uint8 tensors in GPU memory")
    return t.data_ptr()


def _stream(stream, t):
    """The given stream, or the current one of t's device."""
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def scale_cols(cols):
    """Factors of a row of `cols` values: one for every 128, in whole words of four."""
    return (int(cols) + 511) // 512 * 4 if cols > 0 else 0


def quantize(x, q, scales, stream=None):
    """Rows x [n, c] (fp32 or bf16; any row pitch) into q [n, c] with scales [n, scale_cols(c)]."""
    n, c = x.shape
    px, ldx = _pitched(x, (n, c), _FLOATS, "x")
    _check(_quantize(px, _DTYPES[x.dtype], n, c, ldx, 1, 0, _rows(q, (n, c), _E4, "q"),
                     _rows(scales, (n, scale_cols(c)), _SCALES, "scales"), _stream(stream, x)), "moe_fp8_quantize")


def quantize_weights(w, q, scales, stream=None):
    """Weights w [E, n, c] (fp32 or bf16) into q [E, n, c] with scales [E, ceil(n/128), scale_cols(c)]."""
    E, n, c = w.shape
    _check(_quantize(_rows(w, (E, n, c), _FLOATS, "w"), _DTYPES[w.dtype], E * n, c, c, 128, n,
                     _rows(q, (E, n, c), _E4, "q"),
                     _rows(scales, (E, (n + 127) // 128, scale_cols(c)), _SCALES, "scales"), _stream(stream, w)),
           "moe_fp8_quantize")


def rmsnorm(x, weight, residual=None, residual_out=None, out=None, q=None, scales=None, rstd=None, eps=1e-6, stream=None):
    """r = x + residual, n = r * rstd * weight into whichever outputs are given (moe_rmsnorm):
    residual_out and out [T, d] in x's type, q e4m3 with scales, rstd [T] fp32.  x and residual may
    have any row pitch; weight fp32 [d] or None for ones."""
    _want(x.dim() == 2 and x.dtype in _DTYPES, "x must be a 2-D fp32 or bf16 tensor")
    T, d = x.shape
    t = (x.dtype,)
    px, ldx = _pitched(x, (T, d), t, "x")
    pr, ldr = (None, d) if residual is None else _pitched(residual, (T, d), t, "residual")
    _check(_rmsnorm(px, pr, _maybe(weight, (d,), _F32, "weight"), _DTYPES[x.dtype], T, d, ldx, ldr, eps,
                    _maybe(residual_out, (T, d), t, "residual_out"), _maybe(out, (T, d), t, "out"),
                    _maybe(q, (T, d), _E4, "q"),
                    _maybe(scales, (T, scale_cols(d)), _SCALES, "scales"),
                    _maybe(rstd, (T,), _F32, "rstd"), _stream(stream, x)), "moe_rmsnorm")


def rmsnorm_backward_workspace(T, d, device="cuda"):
    """The workspace of rmsnorm_backward for [T, d] (when dweight is wanted)."""
    return torch.empty(max(1, int(_rmsnorm_ws(int(T), int(d)))), dtype=torch.uint8, device=device)


def rmsnorm_backward(dout, r, weight, rstd, dx, dweight=None, workspace=None, dresidual=None, stream=None):
    """dx and dweight from dout = dL/dn (fp32 or bf16) and what the forward kept: r (its
    residual_out, or x without a residual; any row pitch) and rstd; dresidual is the gradient that
    reaches r on its other way."""
    _want(r.dim() == 2 and r.dtype in _DTYPES, "r must be a 2-D fp32 or bf16 tensor")
    T, d = r.shape
    t, f32 = (r.dtype,), _F32
    pr, ldr = _pitched(r, (T, d), t, "r")
    pd = _rows(dout, (T, d), _FLOATS, "dout")
    _check(_rmsnorm_bwd(pd, _DTYPES[dout.dtype], pr, _maybe(weight, (d,), f32, "weight"), _rows(rstd, (T,), f32, "rstd"),
                        _maybe(dresidual, (T, d), t, "dresidual"), _DTYPES[r.dtype], T, d, ldr, _rows(dx, (T, d), t, "dx"),
                        _maybe(dweight, (d,), f32, "dweight"), None if workspace is None else _bytes(workspace),
                        0 if workspace is None else workspace.numel(), _stream(stream, dout)), "moe_rmsnorm_backward")


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
        return _device_status(self._h, _bytes(workspace), _stream(stream, workspace))


class Fp8MatmulPlan(_Fp8Plan):
    """out[p] = A[p] . W_e^T for rows grouped by expert (moe_fp8_matmul): K columns in, n out."""

    def __init__(self, max_rows, K, n, n_experts=1, n_sources=1, out_dtype="bf16", path="auto", wait_timeout_ns=0):
        self.out_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        self.cfg = MoeFp8MatmulConfig(int(max_rows), int(K), int(n), int(n_experts), int(n_sources), _DTYPES[self.out_dtype],
                                      _PATHS[path], int(wait_timeout_ns))
        R, E = int(max_rows), int(n_experts)
        self._make(_matmul_plan, self.cfg, "moe_fp8_matmul_plan")
        self._a, self._sa = (R, int(K)), (R, scale_cols(K))
        self._w, self._sw = (E, int(n), int(K)), (E, (int(n) + 127) // 128, scale_cols(K))
        self._out, self._seg = (R, int(n)), (E * int(n_sources),)

    def forward(self, seg_counts, a, a_scales, w, w_scales, out, workspace, stream=None):
        """seg_counts: int32 rows of each (source, expert) segment, or None for one segment of
        max_rows rows."""
        _check(_matmul(self._h, _maybe(seg_counts, self._seg, (torch.int32,), "seg_counts"),
                       _rows(a, self._a, _E4, "a"), _rows(a_scales, self._sa, _SCALES, "a_scales"),
                       _rows(w, self._w, _E4, "w"), _rows(w_scales, self._sw, _SCALES, "w_scales"),
                       _rows(out, self._out, (self.out_dtype,), "out"), _bytes(workspace), workspace.numel(),
                       _stream(stream, a)), "moe_fp8_matmul")


class Fp8ExpertPlan(_Fp8Plan):
    """The expert stage in 8 bits (moe_fp8_expert_forward); the arguments are moe.ExpertPlan's."""

    def __init__(self, max_rows, d, E_local, n_sources, F, path="auto", wait_timeout_ns=0):
        R, d, E, W, F = int(max_rows), int(d), int(E_local), int(n_sources), int(F)
        self.cfg = MoeExpertConfig(R, d, E, W, F, MOE_BF16, _PATHS[path], int(wait_timeout_ns))
        self._make(_expert_plan, self.cfg, "moe_fp8_expert_plan")
        self.max_rows, self.d, self.E_local, self.n_sources, self.F = R, d, E, W, F
        self._x, self._sx = (R, d), (R, scale_cols(d))
        self._w13, self._s13 = (E, F, d), (E, (F + 127) // 128, scale_cols(d))
        self._w2, self._s2 = (E, d, F), (E, (d + 127) // 128, scale_cols(F))
        self._seg = (E * W,)

    def forward(self, seg_counts, x_rows, x_scales, gates, w1, s1, w3, s3, w2, s2, y_rows, workspace, stream=None):
        _check(_expert_forward(self._h, _maybe(seg_counts, self._seg, (torch.int32,), "seg_counts"),
                               _rows(x_rows, self._x, _E4, "x_rows"), _rows(x_scales, self._sx, _SCALES, "x_scales"),
                               _rows(gates, (self.max_rows,), _F32, "gates"),
                               _rows(w1, self._w13, _E4, "w1"), _rows(s1, self._s13, _SCALES, "s1"),
                               _rows(w3, self._w13, _E4, "w3"), _rows(s3, self._s13, _SCALES, "s3"),
                               _rows(w2, self._w2, _E4, "w2"), _rows(s2, self._s2, _SCALES, "s2"),
                               _rows(y_rows, self._x, _BF16, "y_rows"), _bytes(workspace), workspace.numel(),
                               _stream(stream, x_rows)), "moe_fp8_expert_forward")


class Fp8MoEPlan(MoEPlan):
    """The whole layer with its experts in 8 bits (moe_fp8_forward): the arguments are MoEPlan's."""

    def __init__(self, T, d, E, k, F, out_dtype="bf16", tau=1.0, has_bias=False, keep_logits=False, wait_timeout_ns=0,
                 renorm_gates=False):
        super().__init__(T, d, E, k, F, dtype="bf16", out_dtype=out_dtype, tau=tau, has_bias=has_bias, keep_logits=keep_logits,
                         wait_timeout_ns=wait_timeout_ns, renorm_gates=renorm_gates, fp8_experts=True)
        T, d, E, F = self.T, self.d, self.E, self.F
        self._x, self._sx, self._wr = (T, d), (T, scale_cols(d)), (E, d)
        self._w13, self._s13 = (E, F, d), (E, (F + 127) // 128, scale_cols(d))
        self._w2, self._s2 = (E, d, F), (E, (d + 127) // 128, scale_cols(F))

    def forward(self, x, x_q, x_scales, w_router, bias, w1, s1, w3, s3, w2, s2, y, workspace, stream=None):
        """x (bf16) for the router, x_q with x_scales for the experts: both as rmsnorm writes them."""
        _check(_layer_forward(self._h, _rows(x, self._x, _BF16, "x"), _rows(x_q, self._x, _E4, "x_q"),
                              _rows(x_scales, self._sx, _SCALES, "x_scales"), _rows(w_router, self._wr, _BF16, "w_router"),
                              _maybe(bias, (self.E,), _F32, "bias"),
                              _rows(w1, self._w13, _E4, "w1"), _rows(s1, self._s13, _SCALES, "s1"),
                              _rows(w3, self._w13, _E4, "w3"), _rows(s3, self._s13, _SCALES, "s3"),
                              _rows(w2, self._w2, _E4, "w2"), _rows(s2, self._s2, _SCALES, "s2"),
                              _rows(y, self._x, (self.out_dtype,), "y"), _bytes(workspace), workspace.numel(),
                              _stream(stream, x)),
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

    def save(self, workspace, stream=None):
        _check(_layer_ckpt_save(self.plan.handle, _bytes(workspace), workspace.numel(), _bytes(self.data),
                                self.data.numel(), _stream(stream, workspace)), "moe_checkpoint_save")

    def restore(self, x, workspace, stream=None):
        p = self.plan
        _check(_layer_ckpt_restore(p.handle, _rows(x, (p.T, p.d), (p.act_dtype,), "x"), _bytes(self.data), self.data.numel(),
                                   _bytes(workspace), workspace.numel(), _stream(stream, x)),
               "moe_checkpoint_restore")


def checkpoint_save(a, b, qa, sa, qb, sb, stream=None):
    """The pre-activations a, b [n, F] (bf16) into 8 bits (moe_checkpoint_save_rows)."""
    _want(a.dim() == 2, "a must be 2-D")
    n, F = a.shape
    s = (n, scale_cols(F))
    _check(_ckpt_save(_rows(a, (n, F), _BF16, "a"), _rows(b, (n, F), _BF16, "b"), n, F, _rows(qa, (n, F), _E4, "qa"),
                      _rows(sa, s, _SCALES, "sa"), _rows(qb, (n, F), _E4, "qb"), _rows(sb, s, _SCALES, "sb"),
                      _stream(stream, a)), "moe_checkpoint_save_rows")


def checkpoint_restore(qa, sa, qb, sb, a=None, b=None, h=None, stream=None):
    """The values of a checkpoint and h = silu(a) * b into whichever of a, b, h are given, [n, F] bf16
    (moe_checkpoint_restore_rows)."""
    _want(qa.dim() == 2, "qa must be 2-D")
    n, F = qa.shape
    s = (n, scale_cols(F))
    _check(_ckpt_restore_rows(_rows(qa, (n, F), _E4, "qa"), _rows(sa, s, _SCALES, "sa"), _rows(qb, (n, F), _E4, "qb"),
                              _rows(sb, s, _SCALES, "sb"), n, F, _maybe(a, (n, F), _BF16, "a"), _maybe(b, (n, F), _BF16, "b"),
                              _maybe(h, (n, F), _BF16, "h"), _stream(stream, qa)),
           "moe_checkpoint_restore_rows")


def checkpoint_backward(qa, sa, qb, sb, dh, da, db, h=None, stream=None):
    """The SwiGLU's backward out of the checkpoint (moe_checkpoint_backward_rows): da, db and, if
    given, the hidden rows h, all [n, F] bf16, from dh."""
    _want(qa.dim() == 2, "qa must be 2-D")
    n, F = qa.shape
    s = (n, scale_cols(F))
    _check(_ckpt_backward(_rows(qa, (n, F), _E4, "qa"), _rows(sa, s, _SCALES, "sa"), _rows(qb, (n, F), _E4, "qb"),
                          _rows(sb, s, _SCALES, "sb"), _rows(dh, (n, F), _BF16, "dh"), n, F, _rows(da, (n, F), _BF16, "da"),
                          _rows(db, (n, F), _BF16, "db"), _maybe(h, (n, F), _BF16, "h"), _stream(stream, qa)),
           "moe_checkpoint_backward_rows")
