"""The optimiser's step over many tensors (the C ABI in include/moe_optim.h): the gradients' norm with the
factor that clips it, and AdamW with moments in fp32 or in 8 bits.

As in ``fp8``: a call enqueues its kernels on the current stream (or ``stream``) and returns, and a
wrong type, shape, layout or device raises ValueError before the library is called; the library's own
checks raise ``moe.MoEError``.
"""
import ctypes

import torch

from .fp8 import E4M3, _check, _declare, _fp8, _want

_P, _I32 = ctypes.c_void_p, ctypes.c_int32
_norm_workspace = _declare("moe_grad_norm_workspace", _I32, restype=ctypes.c_size_t)
_declare("moe_grad_norm", _P, _I32, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P)
_declare("moe_adamw", _P, _I32, _P, _P, _P, _P, _P)
E8M0 = torch.float8_e8m0fnu


class AdamwTensor(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("param", "master", "grad", "m", "v", "m_scales", "v_scales")] + [
        ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("param_dtype", _I32), ("grad_dtype", _I32)]


class AdamwConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("lr_device", _P), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("seed", ctypes.c_uint64)]


class GradTensor(ctypes.Structure):
    _fields_ = [("grad", _P), ("n", ctypes.c_int64), ("dtype", _I32)]


def grad_norm_workspace(grads):
    """The workspace of grad_norm for this list of tensors (zeros before the first call; the calls leave it ready)."""
    return torch.zeros(int(_norm_workspace(len(grads))), dtype=torch.uint8, device=grads[0].device if grads else "cuda")


def grad_norm(grads, norm, workspace, max_norm=1.0, factor=None, stream=None):
    """norm [1] (fp32) = the 2-norm of all values of the tensors (fp32 or bf16) together; factor [1] (fp32) =
    min(1, max_norm / norm), NaN where the norm is infinite or NaN (moe_grad_norm)."""
    _check(_fp8.grad_norm(grads, norm, factor, max_norm, workspace, stream), "moe_grad_norm")


def new_state(param, bits=32):
    """Moments of a parameter before the first step: (m, v) in fp32, or (m, m_scales, r, r_scales) in 8 bits: m and
    r = sqrt(v) as e4m3 with an e8m0 factor for every 128 consecutive values."""
    _want(bits in (8, 32), "moments have 8 or 32 bits")
    if bits == 32:
        return tuple(torch.zeros(param.shape, dtype=torch.float32, device=param.device) for _ in range(2))
    blocks = (param.numel() + 127) // 128
    return tuple(t for _ in range(2) for t in (torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(E4M3),
                                               torch.zeros(blocks, dtype=torch.uint8, device=param.device).view(E8M0)))


def moments(state):
    """The values (m, v) that a tensor's state stands for, in fp32."""
    if len(state) == 2:
        return tuple(state)
    m, r = ((q.float().view(-1) * s.float().repeat_interleave(128)[:q.numel()]).view(q.shape) for q, s in (state[:2], state[2:]))
    return m, r.square()


class AdamW:
    """AdamW over a list of parameters, in place (moe_adamw).  All that a step changes are tensors that the
    caller may keep and save: the parameters, ``masters``, ``state`` and ``steps``.

    params: fp32 or bf16, contiguous, on one GPU; no two of them share memory.  masters: None, or a list with an fp32 tensor or None for each:
    a bf16 parameter with a master is rounded from it, one without is rounded stochastically.  weight_decay:
    one for all, or a list.  bits: 32 or 8, of the moments, one for all or a list; ignored with state, a list
    of what new_state makes.  steps: the steps taken so far, a number or an int64 tensor of shape (1,) on
    the GPU, which each step raises.  A captured step replays with the steps as they then are; lr as a
    tensor of shape (1,) is read at each replay too."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, masters=None, state=None, steps=0, seed=0):
        self.params = tuple(params)
        n = len(self.params)
        _want(n > 0, "AdamW needs parameters")

        def each(v):
            v = tuple(v) if isinstance(v, (list, tuple)) else (v,) * n
            _want(len(v) == n, f"a list for {n} parameters must have as many entries")
            return v

        self.masters = each(masters)
        self.weight_decay = tuple(float(v) for v in each(weight_decay))
        self.state = tuple(new_state(p, b) for p, b in zip(self.params, each(bits))) if state is None else each(tuple(map(tuple, state)))
        _want(all(len(s) in (2, 4) for s in self.state), "a state is (m, v) or (m, m_scales, r, r_scales)")
        written = sorted((t.data_ptr(), t.numel() * t.element_size()) for t in (*self.params, *(w for w in self.masters if w is not None),
                                                                                *(t for s in self.state for t in s)) if t.numel())
        _want(all(a + n <= b for (a, n), (b, _) in zip(written, written[1:])), "two of the tensors that a step writes overlap")
        self.lr, self.betas, self.eps, self.seed = lr, (float(betas[0]), float(betas[1])), float(eps), int(seed)
        device = self.params[0].device
        self.steps = steps if isinstance(steps, torch.Tensor) else torch.full((1,), int(steps), dtype=torch.int64, device=device)
        self._ticket = torch.zeros(1, dtype=torch.int32, device=device)
        small = [len(s) == 4 for s in self.state]
        self._lists = ([s[0] for s in self.state], [s[2 if q else 1] for s, q in zip(self.state, small)],
                       [s[1] if q else None for s, q in zip(self.state, small)], [s[3] if q else None for s, q in zip(self.state, small)])

    def step(self, grads, lr=None, grad_factor=None, stream=None):
        """One step with these gradients (fp32 or bf16, contiguous, shaped as the parameters).  grad_factor: a tensor of shape (1,)
        that every gradient is multiplied with (grad_norm's factor); where it is infinite or NaN nothing changes."""
        lr = self.lr if lr is None else lr
        host, device = (0.0, lr) if isinstance(lr, torch.Tensor) else (lr, None)
        _check(_fp8.adamw(self.params, self.masters, grads, *self._lists, self.weight_decay, host, device, *self.betas, self.eps,
                          self.seed, grad_factor, self.steps, self._ticket, stream), "moe_adamw")
