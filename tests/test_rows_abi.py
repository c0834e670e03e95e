"""Refusals and host logic of the sorted rows and the optimiser's step, without a GPU: every bad argument is
turned down on the host before any CUDA call (the fake addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
A = [P((1 << 40) * (i + 1)) for i in range(16)]  # a terabyte apart
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from top_routing_grouped_gb300 import build as b
    if not b.up_to_date():
        b.build()
    from top_routing_grouped_gb300 import moe, optim, rows  # noqa: F401  (they declare the calls)
    return moe.lib()


def off(p, n):
    return P(p.value + n)


def refused(call, ok, bad, status=INVALID):
    for kw in bad:
        assert set(kw) <= set(ok), kw
        assert call(**{**ok, **kw}) == status, kw


def test_workspace(lib):
    from top_routing_grouped_gb300 import rows
    assert rows._workspace(4, 4, 64) == 0  # one launch
    for T, k, E in ((32768, 4, 64), (70000, 1, 3), (1 << 20, 64, 1024)):
        assert rows._workspace(T, k, E) >= 64 * E * 4 and rows._workspace(T, k, E) % 256 == 0
    for bad in ((-1, 4, 64), (1, 0, 64), (1, 65, 64), (1, 4, 0), (1, 4, 1025), (1 << 31, 1, 4), (1 << 30, 2, 4)):
        assert rows._workspace(*bad) == 0


def dispatch(lib):
    ok = dict(idx=A[0], ib=4, T=100, k=4, E=8, counts=A[1], pos=A[2], row_slot=A[3], x=A[4], eb=2, d=64, ldx=64, R=400, xr=A[5], xs=None, rs=None,
              sb=0, gates=A[6], rg=A[7], ws=None, wsb=0)

    def call(**a):
        return lib.moe_rows_dispatch(a["idx"], a["ib"], a["T"], a["k"], a["E"], a["counts"], a["pos"], a["row_slot"], a["x"], a["eb"], a["d"],
                                     a["ldx"], a["R"], a["xr"], a["xs"], a["rs"], a["sb"], a["gates"], a["rg"], a["ws"], a["wsb"], None)
    return call, ok


def test_dispatch_refusals(lib):
    call, ok = dispatch(lib)
    refused(call, ok, [dict(idx=None), dict(counts=None), dict(pos=None), dict(x=None), dict(xr=None), dict(ib=2), dict(T=-1), dict(k=0),
                       dict(k=65), dict(E=0), dict(E=1025), dict(eb=3), dict(eb=8), dict(d=0), dict(ldx=63), dict(R=-1), dict(gates=None),
                       dict(rg=None), dict(xs=A[8], rs=None, sb=4), dict(xs=A[8], rs=A[9], sb=0), dict(xs=A[8], rs=A[9], sb=6),
                       dict(idx=off(A[0], 2)), dict(ib=8, idx=off(A[0], 4)), dict(counts=off(A[1], 2)), dict(pos=off(A[2], 1)), dict(row_slot=off(A[3], 2)),
                       dict(x=off(A[4], 1)), dict(xr=off(A[5], 1)), dict(xs=off(A[8], 2), rs=A[9], sb=4), dict(gates=off(A[6], 2)),
                       # written arrays that overlap
                       dict(xr=A[4]), dict(xr=off(A[4], 100 * 64 * 2 - 2)), dict(pos=A[0]), dict(counts=A[2]), dict(counts=off(A[2], 1596)),
                       dict(row_slot=A[2]), dict(rg=A[6]), dict(rg=off(A[5], 400)), dict(counts=A[6])])
    refused(call, ok, [dict(T=1 << 30), dict(d=1 << 40, ldx=1 << 40)], UNSUPPORTED)
    big = dict(T=10000, R=1)  # a workspace is needed
    refused(call, ok, [dict(big), dict(big, ws=A[8], wsb=2047), dict(big, ws=off(A[8], 128), wsb=4096), dict(big, ws=A[4], wsb=4096)])


def test_gather_and_sort_refusals(lib):
    def gather(T=100, k=4, pos=A[0], x=A[1], xr=A[2], R=400):
        return lib.moe_rows_gather(pos, T, k, x, 4, 8, 8, R, xr, None, None, 0, None, None, None)
    for kw in (dict(pos=None), dict(xr=A[0]), dict(x=None), dict(xr=None), dict(k=65), dict(xr=A[1])):
        assert gather(**kw) == INVALID, kw
    assert gather(T=0, pos=None, x=None, xr=None) == 0  # nothing to do
    assert lib.moe_rows_sort(A[0], 4, 100, 4, 8, A[1], None, None, None, 0, None) == INVALID
    assert lib.moe_rows_sort(A[0], 4, 100, 4, 8, A[1], A[1], None, None, 0, None) == INVALID


def test_combine_refusals(lib):
    ok = dict(y=A[0], yt=1, R=400, pos=A[1], g=A[2], T=100, k=4, d=64, res=A[3], out=A[4], ot=1)

    def call(**a):
        return lib.moe_rows_combine(a["y"], a["yt"], a["R"], a["pos"], a["g"], a["T"], a["k"], a["d"], a["res"], a["out"], a["ot"], None)
    refused(call, ok, [dict(y=None), dict(pos=None), dict(out=None), dict(yt=2), dict(ot=7), dict(R=-1), dict(T=-1), dict(k=0), dict(d=0),
                       dict(y=off(A[0], 1)), dict(out=off(A[4], 1)), dict(pos=off(A[1], 2)), dict(g=off(A[2], 1)), dict(res=off(A[3], 1)),
                       dict(out=A[0]), dict(out=A[1]), dict(out=A[2]), dict(out=off(A[3], 2)), dict(out=off(A[3], 64 * 2))])
    assert call(**{**ok, "T": 0, "pos": None, "out": None}) == 0


def test_combine_backward_refusals(lib):
    ok = dict(do=A[0], dt=0, pos=A[1], g=A[2], T=100, k=4, d=64, R=400, y=A[3], dy=A[4], yt=1, dg=A[5])

    def call(**a):
        return lib.moe_rows_combine_backward(a["do"], a["dt"], a["pos"], a["g"], a["T"], a["k"], a["d"], a["R"], a["y"], a["dy"], a["yt"], a["dg"], None)
    refused(call, ok, [dict(do=None), dict(pos=None), dict(y=None), dict(dy=None, dg=None), dict(dt=3), dict(yt=-1), dict(T=-1), dict(k=65), dict(d=0),
                       dict(R=-1), dict(do=off(A[0], 2)), dict(y=off(A[3], 1)), dict(dy=off(A[4], 1)), dict(dg=off(A[5], 2)), dict(dy=A[0]),
                       dict(dy=off(A[3], 2)), dict(dg=A[2]), dict(dg=A[1]), dict(dg=A[4]), dict(dg=A[3])])
    assert call(**{**ok, "T": 0, "do": None, "pos": None}) == 0


# ------------------------------------------------------------------ the optimiser's step

def step(lib, tensor=None, n=1, cfg=None, factor=None, steps=A[10], ticket=A[11], no_cfg=False):
    from top_routing_grouped_gb300 import optim
    t = dict(param=A[0].value, master=A[1].value, grad=A[2].value, m=A[3].value, v=A[4].value, m_scales=None, v_scales=None, n=1000, weight_decay=0.1,
             param_dtype=1, grad_dtype=0, **{}) | (tensor or {})
    c = dict(lr=1e-3, lr_device=None, beta1=0.9, beta2=0.999, eps=1e-8, seed=0) | (cfg or {})
    arr = (optim.AdamwTensor * 1)(optim.AdamwTensor(**t))
    return lib.moe_adamw(None if n < 0 else arr, abs(n), None if no_cfg else ctypes.byref(optim.AdamwConfig(**c)), factor, steps, ticket, None)


def test_adamw_refusals(lib):
    a = [p.value for p in A]
    nan, inf = float("nan"), float("inf")
    for t in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param_dtype=2), dict(grad_dtype=9), dict(n=-1), dict(n=(1 << 35) + 1),
              dict(weight_decay=-0.1), dict(weight_decay=nan), dict(weight_decay=inf), dict(param_dtype=0), dict(m_scales=a[5]), dict(v_scales=a[5]),
              dict(param=a[0] + 1), dict(master=a[1] + 2), dict(grad=a[2] + 2), dict(m=a[3] + 2), dict(v=a[4] + 1), dict(grad=a[0]),
              dict(master=a[0] + 1996), dict(m=a[4] + 3996), dict(v=a[2]), dict(m_scales=a[5], v_scales=a[5] + 7), dict(m_scales=a[3] + 999, v_scales=a[5])):
        assert step(lib, t) == INVALID, t
    for c in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(lr=1e39), dict(lr_device=a[6] + 2), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan),
              dict(beta2=1.5), dict(eps=0.0), dict(eps=1e-60), dict(eps=1e-39), dict(eps=inf), dict(eps=-1e-8)):
        assert step(lib, cfg=c) == INVALID, c
    for kw in (dict(factor=off(A[6], 1)), dict(steps=None), dict(steps=off(A[10], 4)), dict(ticket=None), dict(ticket=off(A[11], 2)), dict(n=-1), dict(no_cfg=True)):
        assert step(lib, **kw) == INVALID, kw


def test_grad_norm_refusals(lib):
    from top_routing_grouped_gb300 import optim
    ok = dict(grad=A[0].value, n=100, dtype=0, max_norm=1.0, norm=A[1], factor=A[2], ws=A[3], wsb=1 << 20, count=1)

    def call(**a):
        arr = (optim.GradTensor * 1)(optim.GradTensor(a["grad"], a["n"], a["dtype"]))
        return lib.moe_grad_norm(None if a["count"] < 0 else arr, abs(a["count"]), a["max_norm"], a["norm"], a["factor"], a["ws"], a["wsb"], None)
    refused(call, ok, [dict(grad=None), dict(grad=A[0].value + 2), dict(n=-1), dict(n=(1 << 35) + 1), dict(dtype=2), dict(max_norm=0.0), dict(max_norm=float("nan")),
                       dict(max_norm=float("inf")), dict(norm=None), dict(norm=off(A[1], 2)), dict(factor=off(A[2], 1)), dict(factor=A[1]), dict(ws=None),
                       dict(ws=off(A[3], 64)), dict(wsb=100), dict(count=-1), dict(count=-2)])
    assert [lib.moe_grad_norm_workspace(n) for n in (-1, (1 << 20) + 1)] == [0, 0]
    assert lib.moe_grad_norm_workspace(0) == lib.moe_grad_norm_workspace(420) < lib.moe_grad_norm_workspace(421) <= 2 * lib.moe_grad_norm_workspace(420)


def test_python_refusals(lib):
    """Types, shapes and places, before the library is called."""
    from top_routing_grouped_gb300 import optim, rows
    i32, f8 = torch.int32, torch.float8_e4m3fn
    idx, x, counts, pos, xr = torch.zeros(4, 2, dtype=i32), torch.zeros(4, 8), torch.zeros(3, dtype=i32), torch.zeros(4, 2, dtype=i32), torch.zeros(8, 8)
    for bad in (dict(idx=idx.short()), dict(idx=idx[0]), dict(idx=idx.T), dict(x=x.double()), dict(x=x[:3]), dict(x=x.T), dict(counts=counts.long()), dict(pos=pos[:3]),
                dict(xr=xr.bfloat16()), dict(xr=torch.zeros(8, 9)), dict(gates=torch.zeros(4, 2)), dict(row_gates=torch.zeros(8)),
                dict(x_scales=torch.zeros(4, 4, dtype=torch.uint8), row_scales=torch.zeros(8, 4, dtype=torch.uint8)), dict(row_slot=torch.zeros(7, dtype=i32)), {}):
        a = {**dict(idx=idx, x=x, counts=counts, pos=pos, xr=xr), **bad}
        with pytest.raises(ValueError):
            rows.dispatch(a["idx"], a["x"], a["counts"], a["pos"], a["xr"], **{k: v for k, v in bad.items() if k not in ("idx", "x", "counts", "pos", "xr")})
    with pytest.raises(ValueError, match="GPU memory"):
        rows.dispatch(idx, x, counts, pos, xr)
    with pytest.raises(ValueError, match="x_scales"):
        rows.gather(pos, x.to(f8), xr.to(f8), x_scales=torch.zeros(4, 4, dtype=torch.uint8))
    for bad in (dict(out=torch.zeros(3, 8)), dict(y_rows=xr.half()), dict(gates=torch.zeros(4, 2).bfloat16()), dict(residual=x.bfloat16()), {}):
        with pytest.raises(ValueError):
            rows.combine(**{**dict(y_rows=xr, slot_pos=pos, out=x), **bad})
    for bad in (dict(dgates=torch.zeros(4, 3)), dict(dy_rows=xr.bfloat16()), dict(y_rows=None), dict(dout=x.half()), {}):
        with pytest.raises(ValueError):
            rows.combine_backward(**{**dict(dout=x, slot_pos=pos, gates=None, y_rows=xr), **bad})
    p = [torch.zeros(3, 5), torch.zeros(7).bfloat16()]
    for bad in (dict(weight_decay=[0.1]), dict(masters=[None]), dict(bits=16), dict(state=[(p[0],)] * 2), dict(params=[])):
        with pytest.raises(ValueError):
            optim.AdamW(**{**dict(params=p), **bad})
    flat = torch.zeros(100)
    for bad in ([flat, flat], [flat[:60], flat[59:]]):
        with pytest.raises(ValueError, match="overlap"):
            optim.AdamW(bad)
    with pytest.raises(ValueError, match="overlap"):
        optim.AdamW([flat], state=[(torch.zeros(100), flat)])
    optim.AdamW([flat[:60], flat[60:]])
    opt = optim.AdamW(p, bits=[32, 8])
    g = [torch.zeros(3, 5), torch.zeros(7)]
    for bad in (g[:1], [g[0].T, g[1]], [g[0].half(), g[1]], [None, g[1]], 3, g):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(ValueError, match="GPU memory"):
        opt.step(g)
    with pytest.raises(ValueError):
        opt.step(g, grad_factor=torch.zeros(2))
    with pytest.raises(TypeError):
        opt.step(g, lr="fast")
    with pytest.raises(ValueError):
        optim.grad_norm(g, torch.zeros(1), torch.zeros(10, dtype=torch.uint8))


def test_registers_leave_room_for_the_ctas(tmp_path):
    from test_resources import REGISTERS, resources
    found = resources("optim.cu", tmp_path)
    for kernel, threads, ctas in (("adamw_kernelILi24ELb1E", 128, 9), ("adamw_kernelILi24ELb0E", 256, 3)):
        regs = [r for n, r in found.items() if kernel in n]
        assert regs and all(ctas * threads * (-(-r // 8) * 8) <= REGISTERS for r in regs), (kernel, regs)


def test_state_values():
    """What moments() gives for a state in 8 bits."""
    from top_routing_grouped_gb300 import optim
    p = torch.zeros(3, 50)
    m, ms, r, rs = optim.new_state(p, 8)
    assert m.shape == p.shape and ms.shape == (2,) and m.dtype is r.dtype is torch.float8_e4m3fn
    m.copy_(torch.full((3, 50), -1.5)), r.copy_(torch.full((3, 50), 3.0))
    ms.view(torch.uint8).copy_(torch.tensor([127, 130])), rs.view(torch.uint8).copy_(torch.tensor([126, 127]))
    a, b = optim.moments((m, ms, r, rs))
    np.testing.assert_array_equal(a.view(-1).numpy(), [-1.5] * 128 + [-12.0] * 22)
    np.testing.assert_array_equal(b.view(-1).numpy(), [2.25] * 128 + [9.0] * 22)
