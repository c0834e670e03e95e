"""Refusals and host logic of the 8-bit operators, without a GPU: every bad argument is turned
down on the host before any CUDA call (the fake addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_ref as ref


@pytest.fixture(scope="module")
def fp8():
    from top_routing_grouped_gb300 import build as b
    if not b.up_to_date():
        b.build()
    from top_routing_grouped_gb300 import fp8 as m
    return m


P = ctypes.c_void_p
A = [P(4096 * (i + 1)) for i in range(16)]
INVALID, UNSUPPORTED = 1, 2


def test_scale_cols(fp8):
    for c in (1, 127, 128, 129, 512, 513, 2048, 2064, 4096):
        assert fp8.scale_cols(c) == ref.scale_cols(c) and fp8.scale_cols(c) % 4 == 0
        assert -(-c // 128) <= fp8.scale_cols(c) < -(-c // 128) + 4
    assert fp8.scale_cols(0) == 0 and fp8.scale_cols(-5) == 0


def test_reference_rounding_is_torchs():
    """The reference's e4m3 rounding against torch's conversion, over every value and midpoint."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    v = v[torch.isfinite(v)].unique()
    mid = (v[1:] + v[:-1]) / 2
    for t in (v, mid, mid * 1.0001, mid * 0.9999):
        np.testing.assert_array_equal(ref.round_e4m3(t.double().numpy()), t.to(torch.float8_e4m3fn).double().numpy())
    b = ref.scale_byte(np.array([0.0, 448.0, 448.0001, 1.0, np.inf, 2.0 ** -140, 3.4e38]))
    assert b.tolist() == [0, 127, 128, 119, 255, 0, 247]


def test_quantize_refusals(fp8):
    L = fp8._lib
    ok = dict(x=A[0], t=0, rows=4, cols=64, ld=64, br=1, er=4, q=A[1], s=A[2])

    def call(**kw):
        a = {**ok, **kw}
        return L.moe_fp8_quantize(a["x"], a["t"], a["rows"], a["cols"], a["ld"], a["br"], a["er"], a["q"], a["s"], None)

    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(t=5), dict(rows=-1), dict(cols=0), dict(ld=63), dict(br=64),
               dict(x=P(4098)), dict(q=P(4104)), dict(s=P(4097)), dict(br=128, er=0), dict(br=128, er=3)):
        assert call(**kw) == INVALID, kw
    assert call(rows=1 << 40) == UNSUPPORTED
    assert call(rows=0, x=None, q=None, s=None) == 0  # nothing to do


def test_rmsnorm_refusals(fp8):
    L = fp8._lib
    ok = dict(x=A[0], r=A[1], w=A[2], t=1, rows=4, d=64, ldx=64, ldr=64, eps=1e-6, ro=A[3], o=A[4], q=A[5], s=A[6], rs=A[7])

    def call(**kw):
        a = {**ok, **kw}
        return L.moe_rmsnorm(a["x"], a["r"], a["w"], a["t"], a["rows"], a["d"], a["ldx"], a["ldr"], a["eps"], a["ro"], a["o"],
                             a["q"], a["s"], a["rs"], None)

    for kw in (dict(x=None), dict(t=2), dict(rows=-1), dict(d=0), dict(ldx=60), dict(ldr=60), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None), dict(s=None), dict(x=P(4097)), dict(o=P(4097)),
               dict(q=P(4100)), dict(rs=P(4100)), dict(w=P(4100)), dict(ro=None, o=None, q=None, s=None, rs=None),
               dict(ro=A[0], ldx=80), dict(ro=A[1], ldr=80)):
        assert call(**kw) == INVALID, kw
    assert call(d=60000, ldx=60000, ldr=60000) == UNSUPPORTED
    assert call(rows=0) == 0


def test_rmsnorm_backward_refusals(fp8):
    L = fp8._lib
    assert fp8._rmsnorm_ws(0, 64) == 0 and fp8._rmsnorm_ws(-1, 64) == 0 and fp8._rmsnorm_ws(1000, 64) >= 64 * 4
    need = fp8._rmsnorm_ws(1000, 64)
    ok = dict(do=A[0], dt=0, r=A[1], w=A[2], rs=A[3], dr=A[4], t=1, rows=1000, d=64, ld=64, dx=A[5], dw=A[6], ws=A[7], n=need)

    def call(**kw):
        a = {**ok, **kw}
        return L.moe_rmsnorm_backward(a["do"], a["dt"], a["r"], a["w"], a["rs"], a["dr"], a["t"], a["rows"], a["d"], a["ld"],
                                      a["dx"], a["dw"], a["ws"], a["n"], None)

    for kw in (dict(do=None), dict(r=None), dict(rs=None), dict(dx=None), dict(dt=3), dict(t=-1), dict(rows=-1), dict(d=0),
               dict(ld=10), dict(ws=None), dict(ws=P(4224)), dict(n=need - 1), dict(dw=P(4100)), dict(do=P(4098))):
        assert call(**kw) == INVALID, kw
    assert call(d=60000, ld=60000) == UNSUPPORTED


def test_rmsnorm_backward_refuses_overlaps(fp8):
    """dx may be dresidual, dout or r itself (seen where the call stops at a workspace that is too small, its last
    check); anything else that shares a byte with one of them is turned down by name."""
    L = fp8._lib
    rows, d, at = 1000, 64, 1 << 24
    size = {0: 4, 1: 2}

    def call(t=1, dt=1, ld=d, **kw):
        p = dict(do=1 << 28, r=2 << 28, dr=3 << 28, dx=at)
        p.update(kw)
        st = L.moe_rmsnorm_backward(P(p["do"]), dt, P(p["r"]), None, A[3], P(p["dr"]), t, rows, d, ld, P(p["dx"]), A[6], A[7], 0, None)
        return st, L.moe_last_error().decode()

    fine = (INVALID, "workspace too small")
    for kw in (dict(), dict(do=at), dict(r=at), dict(dr=at), dict(do=at, r=at, dr=at), dict(do=at, dt=0, t=0)):
        st, why = call(**kw)
        assert (st, why[:19]) == fine, (kw, why)
    for t in (0, 1):
        bytes_ = rows * d * size[t]
        for name, word in (("do", "dout"), ("r", "r"), ("dr", "dresidual")):
            for off in (16, d * size[t], bytes_ - 16, -16, 16 - bytes_):
                st, why = call(t=t, dt=t, **{name: at + off})
                assert st == INVALID and why.startswith(f"dx overlaps {word}:"), (t, name, off, why)
            for off in (bytes_, -bytes_):
                st, why = call(t=t, dt=t, **{name: at + off})
                assert (st, why[:19]) == fine, (t, name, off, why)
    assert call(do=at, dt=0)[1].startswith("dx overlaps dout")   # another type
    assert call(r=at, ld=80)[1].startswith("dx overlaps r:")     # another pitch


@pytest.mark.parametrize("kw, status", [
    (dict(max_rows=0), "MOE_ERR_INVALID_ARG"), (dict(K=0), "MOE_ERR_INVALID_ARG"), (dict(n=0), "MOE_ERR_INVALID_ARG"),
    (dict(n_experts=0), "MOE_ERR_INVALID_ARG"), (dict(n_experts=129, n_sources=2), "MOE_ERR_INVALID_ARG"),
    (dict(path="tc1"), "MOE_ERR_INVALID_ARG"), (dict(K=72), "MOE_ERR_UNSUPPORTED"), (dict(n=100), "MOE_ERR_UNSUPPORTED"),
    (dict(max_rows=1 << 31), "MOE_ERR_UNSUPPORTED"), (dict(n=1 << 30, n_experts=2), "MOE_ERR_UNSUPPORTED"),
])
def test_plan_refusals(fp8, kw, status):
    a = dict(max_rows=64, K=64, n=64, n_experts=2, n_sources=1, path="auto", **{})
    a.update(kw)
    with pytest.raises(fp8.MoEError) as ei:
        fp8.Fp8MatmulPlan(a["max_rows"], a["K"], a["n"], n_experts=a["n_experts"], n_sources=a["n_sources"], path=a["path"])
    assert status in str(ei.value)
    with pytest.raises(fp8.MoEError) as ei:
        fp8.Fp8ExpertPlan(a["max_rows"], a["K"], a["n_experts"], a["n_sources"], a["n"], path=a["path"])
    assert status in str(ei.value)


def test_simt_plans_take_any_size(fp8):
    assert fp8.Fp8MatmulPlan(3, 5, 7, path="simt").workspace_bytes > 0
    assert fp8.Fp8ExpertPlan(3, 5, 2, 1, 7, path="simt").workspace_bytes > 0


def test_product_refusals(fp8):
    L = fp8._lib
    p, e = fp8.Fp8MatmulPlan(64, 64, 64, n_experts=2), fp8.Fp8ExpertPlan(64, 64, 2, 1, 64)
    n = p.workspace_bytes
    args = dict(seg=A[0], a=A[1], sa=A[2], w=A[3], sw=A[4], out=A[5], ws=A[6], n=n)

    def call(h=p.handle, **kw):
        a = {**args, **kw}
        return L.moe_fp8_matmul(h, a["seg"], a["a"], a["sa"], a["w"], a["sw"], a["out"], a["ws"], a["n"], None)

    for name in ("seg", "a", "sa", "w", "sw", "out"):
        assert call(**{name: None}) == INVALID and call(**{name: P(4104)}) == INVALID, name
    assert call(ws=None) == INVALID and call(ws=P(4224)) == INVALID and call(n=n - 1) == INVALID
    assert call(h=None) == INVALID and call(h=e.handle) == INVALID
    ne = e.workspace_bytes
    for i in range(11):
        b = list(A[:11])
        b[i] = None
        assert L.moe_fp8_expert_forward(e.handle, *b, A[11], ne, None) == INVALID, i
        b[i] = P(4104)
        assert L.moe_fp8_expert_forward(e.handle, *b, A[11], ne, None) == INVALID, i
    assert L.moe_fp8_expert_forward(e.handle, *A[:11], A[11], ne - 1, None) == INVALID
    assert L.moe_fp8_expert_forward(p.handle, *A[:11], A[11], ne, None) == INVALID


def test_checkpoint_refusals(fp8):
    L = fp8._lib
    for i in range(6):
        b = list(A[:6])
        b[i] = None
        assert L.moe_checkpoint_save_rows(b[0], b[1], 4, 64, *b[2:], None) == INVALID, i
        b[i] = P(4104)
        assert L.moe_checkpoint_save_rows(b[0], b[1], 4, 64, *b[2:], None) == INVALID, i
    for i in range(8):
        b = list(A[:8])
        b[i] = P(4104)
        assert L.moe_checkpoint_backward_rows(*b[:5], 4, 64, *b[5:], None) == INVALID, i
        b[i] = None
        if i < 7:  # h may be missing
            assert L.moe_checkpoint_backward_rows(*b[:5], 4, 64, *b[5:], None) == INVALID, i
    for i in range(7):
        b = list(A[:7])
        b[i] = P(4104)
        assert L.moe_checkpoint_restore_rows(*b[:4], 4, 64, *b[4:], None) == INVALID, i
        b[i] = None
        if i < 4:
            assert L.moe_checkpoint_restore_rows(*b[:4], 4, 64, *b[4:], None) == INVALID, i
    assert L.moe_checkpoint_restore_rows(*A[:4], 4, 64, None, None, None, None) == INVALID
    assert L.moe_checkpoint_save_rows(*A[:2], -1, 64, *A[2:6], None) == INVALID
    assert L.moe_checkpoint_save_rows(*A[:2], 4, 0, *A[2:6], None) == INVALID


class OnGpu(torch.Tensor):
    """A host tensor that says it lies in GPU memory: what the binding turns down for other reasons."""
    is_cuda = True


def test_binding_checks_types_shapes_and_layouts(fp8):
    """The binding turns wrong tensors down before their addresses are used."""
    g = lambda t: t.as_subclass(OnGpu)
    x = g(torch.zeros(4, 64))
    q, s = g(torch.zeros(4, 64, dtype=torch.uint8).view(fp8.E4M3)), g(torch.zeros(4, 4, dtype=torch.uint8))
    one = g(torch.ones(4))
    bad = [lambda: fp8.quantize(x.double(), q, s), lambda: fp8.quantize(x, q[:, :32], s), lambda: fp8.quantize(x, x, s),
           lambda: fp8.quantize(x, q, s[:, :1]), lambda: fp8.quantize(x, q, None),
           lambda: fp8.quantize(x.t(), g(torch.zeros(64, 4, dtype=torch.uint8).view(fp8.E4M3)), s),
           lambda: fp8.quantize(x[:1].expand(4, 64), q, s),
           lambda: fp8.rmsnorm(x, g(torch.ones(63)), out=x), lambda: fp8.rmsnorm(x, None, out=g(torch.zeros(64, 4)).t()),
           lambda: fp8.rmsnorm(x, None, residual=x.bfloat16(), out=x), lambda: fp8.rmsnorm(x.view(-1), None, out=x),
           lambda: fp8.rmsnorm_backward(x[:3], x, None, one, x), lambda: fp8.rmsnorm_backward(x, x, None, one[:3], x),
           lambda: fp8.checkpoint_save(x, x, q, s, q, s), lambda: fp8.checkpoint_backward(q, s, q, s, x, x, x),
           lambda: fp8.checkpoint_restore(q, s, q, s, x)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError) as ei:
            f()
        assert "must be a" in str(ei.value), i
    plan = fp8.Fp8MatmulPlan(4, 64, 32)
    w, out = g(torch.zeros(1, 32, 64).to(fp8.E4M3)), g(torch.zeros(4, 32, dtype=torch.bfloat16))
    sw, ws = g(torch.zeros(1, 1, 4, dtype=torch.uint8)), g(torch.zeros(1 << 16, dtype=torch.uint8))
    for args in ((None, q, s, w, s, out, ws), (None, q, s, w, sw, out.float(), ws), (one, q, s, w, sw, out, ws),
                 (None, q[:3], s, w, sw, out, ws), (None, q, s, w, sw, out, ws.float())):
        with pytest.raises(ValueError):
            plan.forward(*args)


def test_binding_refuses_host_memory(fp8):
    """Nothing wrong but where a tensor lies."""
    x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8).view(fp8.E4M3), torch.zeros(4, 4, dtype=torch.uint8)
    g = lambda t: t.as_subclass(OnGpu)
    for args in ((x, g(q), g(s)), (g(x), q, g(s)), (g(x), g(q), s)):
        with pytest.raises(ValueError, match="GPU memory"):
            fp8.quantize(*args)
    with pytest.raises(ValueError, match="GPU memory"):
        fp8.rmsnorm(g(x), torch.ones(64), out=g(x))
    with pytest.raises(ValueError, match="GPU memory"):
        fp8.rmsnorm_backward(g(x), g(x), None, g(torch.ones(4)), g(x), g(torch.ones(64)), torch.zeros(4096, dtype=torch.uint8))


class Elsewhere(torch.Tensor):
    """A tensor without memory that lies on the given device for the binding too."""
    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kwargs=None):
        raise NotImplementedError(f)


class FakeStream:
    cuda_stream, device_index = 0, 1


def binding_calls(fp8):
    """(name, function of a list of tensors and a stream, the tensors' shapes and types) of every call of the
    binding that takes tensors."""
    from top_routing_grouped_gb300 import moe
    f32, bf, f8, u8, i32 = torch.float32, torch.bfloat16, fp8.E4M3, torch.uint8, torch.int32
    T, d, E, F = 4, 64, 2, 32
    x, q, s = ((T, d), f32), ((T, d), f8), ((T, 4), u8)
    b, v, w, ws = ((T, d), bf), ((d,), f32), ((E, 1, 4), u8), ((1 << 20,), u8)
    up, down = ((E, F, d), f8), ((E, d, F), f8)
    mm, ex = fp8.Fp8MatmulPlan(T, d, F, n_experts=E), fp8.Fp8ExpertPlan(T, d, E, 1, F)
    layer = fp8.Fp8MoEPlan(T, 128, 8, 2, 128, has_bias=True)
    lq, lw, lc = ((T, 128), f8), ((8, 128, 128), f8), ((8, 1, 4), u8)
    lx = ((T, 128), bf)
    return [
        ("quantize", fp8.quantize, [x, q, s]),
        ("quantize_weights", fp8.quantize_weights, [((E, F, d), f32), up, w]),
        ("rmsnorm", lambda x, w, r, ro, o, q, s, rs, stream: fp8.rmsnorm(x, w, r, ro, o, q, s, rs, stream=stream),
         [x, v, x, x, x, q, s, ((T,), f32)]),
        ("rmsnorm_backward", fp8.rmsnorm_backward, [x, x, v, ((T,), f32), x, v, ws, x]),
        ("matmul", mm.forward, [((E,), i32), q, s, up, w, ((T, F), bf), ws]),
        ("experts", ex.forward, [((E,), i32), q, s, ((T,), f32), up, w, up, w, down, w, b, ws]),
        ("layer", layer.forward, [lx, lq, s, ((8, 128), bf), ((8,), f32), lw, lc, lw, lc, lw, lc, lx, ws]),
        ("checkpoint_save", fp8.checkpoint_save, [b, b, q, s, q, s]),
        ("checkpoint_restore", fp8.checkpoint_restore, [q, s, q, s, b, b, b]),
        ("checkpoint_backward", fp8.checkpoint_backward, [q, s, q, s, b, b, b, b]),
    ]


@pytest.mark.parametrize("i", range(10))
def test_binding_refuses_each_tensor_elsewhere(fp8, i):
    """Nothing wrong but where one tensor lies, each in turn: in host memory, or on another GPU than the rest; or
    the stream's device."""
    name, f, tensors = binding_calls(fp8)[i]
    for j, (shape, dtype) in enumerate(tensors):
        on = lambda device: [Elsewhere(*t, device if k == j else "cuda:0") for k, t in enumerate(tensors)]
        host = on("cuda:0")
        host[j] = torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype).view(dtype)
        with pytest.raises(ValueError, match="must be in GPU memory"):
            f(*host, stream=None)
        with pytest.raises(ValueError, match="must be on the device of the tensors before it"):
            f(*on("cuda:1"), stream=None)
    with pytest.raises(ValueError, match="stream must be on the tensors' device"):
        f(*[Elsewhere(*t, "cuda:0") for t in tensors], stream=FakeStream())


def test_layer_checkpoint_refuses_other_devices(fp8):
    from top_routing_grouped_gb300 import moe
    p = moe.MoEPlan(64, 128, 8, 2, 128, training=True)
    c = fp8.LayerCheckpoint(p, device="cpu")
    tensor = lambda n, device, dtype=torch.uint8: Elsewhere(n, dtype, device)
    ws = lambda device: tensor((p.workspace_bytes,), device)
    with pytest.raises(ValueError, match="GPU memory"):
        c.save(ws("cuda:0"))
    c.data = tensor((c.data.numel(),), "cuda:0")
    x = lambda device: tensor((64, 128), device, torch.bfloat16)
    for f in (lambda: c.save(ws("cuda:1")), lambda: c.restore(x("cuda:1"), ws("cuda:0")), lambda: c.restore(x("cuda:0"), ws("cuda:1")),
              lambda: c.save(ws("cuda:0"), stream=FakeStream()), lambda: c.restore(x("cuda:0"), ws("cuda:0"), stream=FakeStream()),
              lambda: fp8.Fp8MatmulPlan(4, 64, 32).device_status(ws("cuda:0"), stream=FakeStream())):
        with pytest.raises(ValueError, match="one device"):
            f()


def test_layer_plan_and_forward_refusals(fp8):
    from top_routing_grouped_gb300 import moe
    L = fp8._lib
    p = fp8.Fp8MoEPlan(64, 128, 8, 2, 128)
    p16 = moe.MoEPlan(64, 128, 8, 2, 128)
    assert p.workspace_bytes < p16.workspace_bytes
    n = p.workspace_bytes

    def call(args, h=p.handle, ws=A[14], n=n, bias=None):
        return L.moe_fp8_forward(h, *args[:4], bias, *args[4:], ws, n, None)

    for i in range(11):
        b = list(A[:11])
        b[i] = None
        assert call(b) == INVALID, i
        b[i] = P(4104)
        assert call(b) == INVALID, i
    good = list(A[:11])
    assert call(good, h=p16.handle) == INVALID and call(good, h=None) == INVALID
    assert call(good, ws=None) == INVALID and call(good, ws=P(4224)) == INVALID and call(good, n=n - 1) == INVALID
    pb = fp8.Fp8MoEPlan(64, 128, 8, 2, 128, has_bias=True)
    assert call(good, h=pb.handle, n=pb.workspace_bytes) == INVALID
    # the bf16 entry points turn an 8-bit plan down
    assert L.moe_forward(p.handle, A[0], A[1], None, A[2], A[3], A[4], A[5], A[6], n, None) == INVALID
    for kw in (dict(dtype="f32"), dict(path="simt"), dict(path="tc1"), dict(training=True), dict(test_stall=True)):
        with pytest.raises(moe.MoEError, match="UNSUPPORTED"):
            moe.MoEPlan(64, 128, 8, 2, 128, **{"dtype": "bf16", **kw}, fp8_experts=True)


def test_layer_checkpoint_refusals(fp8):
    from top_routing_grouped_gb300 import moe
    L = fp8._lib
    plain, p = moe.MoEPlan(64, 128, 8, 2, 128), moe.MoEPlan(64, 128, 8, 2, 128, training=True)
    assert L.moe_checkpoint_bytes(None) == 0 and L.moe_checkpoint_bytes(plain.handle) == 0
    c, n = L.moe_checkpoint_bytes(p.handle), p.workspace_bytes
    assert 2 * 64 * 2 * 128 < c < n
    save = lambda h=p.handle, ws=A[0], n=n, ck=A[1], c=c: L.moe_checkpoint_save(h, ws, n, ck, c, None)
    load = lambda h=p.handle, x=A[2], ws=A[0], n=n, ck=A[1], c=c: L.moe_checkpoint_restore(h, x, ck, c, ws, n, None)
    for f in (save, load):
        for kw in (dict(h=None), dict(h=plain.handle), dict(ws=None), dict(ws=P(4224)), dict(n=n - 1), dict(ck=None),
                   dict(ck=P(4224)), dict(c=c - 1)):
            assert f(**kw) == INVALID, kw
    with pytest.raises(ValueError, match="training"):
        fp8.LayerCheckpoint(plain, device="cpu")
