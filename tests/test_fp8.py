"""The 8-bit operators on the GPU against plain 64-bit references, at the sizes, masks and values
where they can go wrong.

Tolerances.  A rounding to type t is off by at most half a step, eps(t)/2 relative to the value:
H[bf16] = 2^-8, H[f32] = 2^-24, H[e4m3] = 2^-4 (2^-10 absolute below 2^-6, in units of the block's
factor).  A sum of K exact products accumulated in fp32 in any order is off by at most K eps
sum|a w| with eps = 2^-23 (one rounding or truncation of the running sum for each term).
Quantising what is given exactly is exact: compared bit for bit."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS32 = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def fp8():
    from top_routing_grouped_gb300 import fp8 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.dtype != torch.uint8 else t.cpu().numpy().astype(np.int64)


def f8(n, *rest):
    return torch.full((n, *rest), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def u8(*shape):
    return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")


def close(got, want, tol, what=""):
    got, want, tol = np.asarray(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan, err_msg=what)
    bad = ~nan & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]}"


# ------------------------------------------------------------------ quantisation

def awkward(n, c, dtype, seed):
    """Values over many magnitudes, with zero blocks, infinities, NaNs, subnormals and maxima at the
    border of two factors."""
    x = torch.randn(n, c, generator=gen(seed)) * torch.exp2(torch.randint(-30, 30, (n, 1), generator=gen(seed + 1)).float())
    x[0] = 0
    if n > 1:
        x[1, : c // 2] = 1e-40
    if n > 2:
        x[2, c // 2] = float("inf")
    if n > 3:
        x[3, c - 1] = float("nan")
    if n > 4:
        x[4] = 0.5
        x[4, 0] = 448.0 * 2.0 ** 3          # exactly the largest value of a factor
    if n > 5:
        x[5] = 0.5
        x[5, c // 3] = -450.0               # the next bf16 above 448
    if n > 6:
        x[6, :] = 3e38
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("n, c, pad", [(1, 1, 0), (9, 16, 0), (7, 130, 3), (300, 128, 8), (33, 2064, 0), (8, 4096, 64),
                                       (1000, 1000, 0)])
def test_quantize_rows_bit_exact(fp8, dtype, n, c, pad):
    x = awkward(n, c + pad, dtype, 3)[:, :c].cuda() if pad == 0 else awkward(n, c + pad, dtype, 3).cuda()[:, :c]
    q, s = f8(n, c), u8(n, fp8.scale_cols(c))
    fp8.quantize(x, q, s)
    wq, ws = ref.quantize(np64(x))
    np.testing.assert_array_equal(np64(s), ws)
    np.testing.assert_array_equal(np64(q), wq)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("E, n, c", [(1, 1, 1), (3, 130, 200), (2, 128, 512), (5, 64, 144)])
def test_quantize_weights_bit_exact(fp8, dtype, E, n, c):
    w = awkward(E * n, c, dtype, 5).view(E, n, c).cuda()
    q, s = f8(E, n, c), u8(E, -(-n // 128), fp8.scale_cols(c))
    fp8.quantize_weights(w, q, s)
    wq, ws = ref.quantize_weights(np64(w))
    np.testing.assert_array_equal(np64(s), ws)
    np.testing.assert_array_equal(np64(q), wq)


def test_zero_rows_do_nothing(fp8):
    e = torch.empty
    fp8.quantize(e(0, 64, device="cuda"), f8(0, 64), u8(0, 4))
    fp8.rmsnorm(e(0, 64, device="cuda"), None, out=e(0, 64, device="cuda"))
    dw = torch.ones(64, device="cuda")
    fp8.rmsnorm_backward(e(0, 64, device="cuda"), e(0, 64, device="cuda"), None, e(0, device="cuda"), e(0, 64, device="cuda"), dw,
                         fp8.rmsnorm_backward_workspace(0, 64))
    assert not dw.any()  # a sum over no rows
    b = lambda: e(0, 64, dtype=BF, device="cuda")
    fp8.checkpoint_save(b(), b(), f8(0, 64), u8(0, 4), f8(0, 64), u8(0, 4))
    fp8.checkpoint_backward(f8(0, 64), u8(0, 4), f8(0, 64), u8(0, 4), b(), b(), b(), b())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ norm

def norm_tol(n64, d, dtype):
    """n = r rstd w in fp32: the mean of d squares is off by at most d eps relative (half of it in
    rstd), and r rstd w, the square root and the division round a handful of times."""
    return np.abs(n64) * ((d / 2 + 8) * EPS32 + (H[dtype] if dtype is not None else 0)) + 1e-37


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("n, d, pad, residual, weight", [
    (1, 1, 0, True, True), (1, 4096, 0, True, True), (5, 100, 3, True, True), (129, 2000, 48, False, True),
    (64, 128, 0, False, False), (700, 512, 8, True, False), (3, 8192, 0, True, True), (2, 12345, 1, True, True),
    (2, 20000, 0, True, True)])
def test_rmsnorm(fp8, dtype, n, d, pad, residual, weight):
    g = gen(11)
    x = (torch.randn(n, d + pad, generator=g) * 3).to(dtype).cuda()[:, :d]
    res = torch.randn(n, d + 2 * pad, generator=g).to(dtype).cuda()[:, :d] if residual else None
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda() if weight else None
    e = lambda: torch.empty(n, d, dtype=dtype, device="cuda")
    r, out, q, s, rstd = e(), e(), f8(n, d), u8(n, fp8.scale_cols(d)), torch.empty(n, device="cuda")
    fp8.rmsnorm(x, w, residual=res, residual_out=r, out=out, q=q, scales=s, rstd=rstd, eps=1e-5)
    want_r = (x.float() + res.float()).to(dtype) if residual else x
    assert torch.equal(r, want_r)
    v = np64(r)
    inv = 1 / np.sqrt((v ** 2).mean(1, keepdims=True) + 1e-5)
    n64 = v * inv * (np64(w) if weight else 1)
    close(np64(rstd), inv[:, 0], inv[:, 0] * (d / 2 + 4) * EPS32, "rstd")
    close(np64(out), n64, norm_tol(n64, d, dtype), "out")
    # the bytes are those of the 64-bit norm unless a maximum lies at a border; the values are
    # within half an e4m3 step of it in the block's own factor
    b, wb = np64(s), ref.quantize(n64)[1]
    kb = -(-d // 128)
    assert (b[:, kb:] == 0).all()
    top = np.abs(np.pad(n64, ((0, 0), (0, kb * 128 - d)))).reshape(n, kb, 128).max(2)
    low, high = ref.scale_byte(top * (1 - d * EPS32)), ref.scale_byte(top * (1 + d * EPS32))
    assert ((b[:, :kb] >= low) & (b[:, :kb] <= high)).all()
    f = np.repeat(ref.scale_value(b[:, :kb]), 128, 1)[:, :d]
    close(np64(q) * f, n64, np.abs(n64) * 2.0 ** -4 + f * 2.0 ** -10 + norm_tol(n64, d, None), "q")
    assert ((b[:, :kb] == wb[:, :kb]).mean() > 0.99) or b.size < 200


def test_rmsnorm_each_output_alone_and_in_place(fp8):
    g = gen(12)
    x, res = (torch.randn(40, 384, generator=g).to(BF).cuda() for _ in range(2))
    w = torch.rand(384, generator=g).cuda()
    e = lambda: torch.empty(40, 384, dtype=BF, device="cuda")
    r, out, q, s, rstd = e(), e(), f8(40, 384), u8(40, 4), torch.empty(40, device="cuda")
    fp8.rmsnorm(x, w, res, r, out, q, s, rstd)
    for kw in (dict(residual_out=e()), dict(out=e()), dict(q=f8(40, 384), scales=u8(40, 4)), dict(rstd=torch.empty(40, device="cuda"))):
        fp8.rmsnorm(x, w, res, **kw)
        for k, t in kw.items():
            want = dict(residual_out=r, out=out, q=q, scales=s, rstd=rstd)[k]
            assert torch.equal(t.view(torch.uint8), want.view(torch.uint8)), k
    for inplace in ("x", "res"):
        xa, ra = x.clone(), res.clone()
        o = e()
        fp8.rmsnorm(xa, w, ra, residual_out=xa if inplace == "x" else ra, out=o)
        assert torch.equal(xa if inplace == "x" else ra, r) and torch.equal(o, out)


def test_rmsnorm_special_rows(fp8):
    """A row of zeros, of one value, of the largest bf16 values, with an infinity, with a NaN."""
    x = torch.randn(6, 300, generator=gen(13))
    x[0] = 0
    x[1] = -2.5
    x[2] = 1e30
    x[3, 7] = float("inf")
    x[4, 299] = float("nan")
    x = x.to(BF).cuda()
    out, q, s = torch.empty_like(x), f8(6, 300), u8(6, 4)
    fp8.rmsnorm(x, None, out=out, q=q, scales=s, eps=1e-6)
    o, b = np64(out), np64(s)
    assert (o[0] == 0).all() and (b[0] == 0).all() and (np64(q)[0] == 0).all()
    close(o[1], np.full(300, -1.0), 2.0 ** -8 + 1e-6)
    # the squares of 1e30 leave fp32: the sum is infinite and rstd 0, as the formula in fp32 has it
    assert (o[2] == 0).all() and (b[2, :3] == 0).all()
    # an infinity: rstd = 0, 0 * inf = NaN at its place and zeros elsewhere; a NaN spreads over its row
    assert np.isnan(o[3, 7]) and (np.delete(o[3], 7) == 0).all() and b[3, 0] == 255 and (b[3, 1:3] == 0).all()
    assert np.isnan(o[4]).all() and (b[4, :3] == 255).all()
    assert np.isfinite(o[5]).all() and (b[5, :3] < 255).all()


@pytest.mark.parametrize("dtype, dout", [(F32, F32), (BF, F32), (BF, BF), (F32, BF)], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("n, d, pad, dres, weight", [(1, 1, 0, False, True), (1, 4096, 0, True, True), (512, 264, 0, True, True),
                                                     (513, 264, 0, True, True), (300, 1000, 5, True, True),
                                                     (2000, 136, 0, False, False), (700, 2048, 8, True, True),
                                                     (3, 12345, 0, True, True)])
def test_rmsnorm_backward_against_the_formula(fp8, dtype, dout, n, d, pad, dres, weight):
    g = gen(14)
    r = (torch.randn(n, d + pad, generator=g) * 2).to(dtype).cuda()[:, :d]
    dn = torch.randn(n, d, generator=g).to(dout).cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda() if weight else None
    dr = torch.randn(n, d, generator=g).to(dtype).cuda() if dres else None
    rstd = (r.double().square().mean(1) + 1e-5).rsqrt().float()
    dx, dw = torch.empty(n, d, dtype=dtype, device="cuda"), torch.empty(d, device="cuda")
    fp8.rmsnorm_backward(dn, r, w, rstd, dx, dw, fp8.rmsnorm_backward_workspace(n, d), dresidual=dr)
    v, inv, do = np64(r), np64(rstd)[:, None], np64(dn)
    gw, xh = do * (np64(w) if weight else 1), v * inv
    m = (gw * xh).mean(1, keepdims=True)
    want = inv * (gw - xh * m) + (np64(dr) if dres else 0)
    # the mean of d products is off by at most (d + 4) eps of the mean of their magnitudes
    mag = np.abs(gw * xh).mean(1, keepdims=True)
    tol = inv * (8 * EPS32 * (np.abs(gw) + np.abs(xh) * np.abs(m)) + np.abs(xh) * mag * (d + 4) * EPS32)
    close(np64(dx), want, tol + (H[dtype] + 2 * EPS32) * np.abs(want) + 2 * EPS32 * (np.abs(np64(dr)) if dres else 0), "dx")
    close(np64(dw), (do * xh).sum(0), (n + 4) * EPS32 * np.abs(do * xh).sum(0), "dweight")
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    fp8.rmsnorm_backward(dn, r, w, rstd, dx2, dw2, fp8.rmsnorm_backward_workspace(n, d), dresidual=dr)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2), "the same call twice gives the same bits"
    if dres:  # in place, and without dweight
        fp8.rmsnorm_backward(dn, r, w, rstd, dr, dresidual=dr)
        assert torch.equal(dr, dx)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("n, d", [(1, 4096), (300, 1000), (512, 264), (512, 97), (513, 264), (2000, 136), (300, 5000), (3, 12345)])
def test_rmsnorm_backward_in_place(fp8, dtype, n, d):
    """dx over dout, over r or over all three: the bits of the call with a tensor of its own, dweight among them."""
    g = gen(16)
    r, dn, dr = ((torch.randn(n, d, generator=g) * 2).to(dtype).cuda() for _ in range(3))
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    rstd = (r.double().square().mean(1) + 1e-5).rsqrt().float()
    ws = fp8.rmsnorm_backward_workspace(n, d)

    def call(dn, r, dx, dr):
        dw = torch.full((d,), 77.0, device="cuda")
        fp8.rmsnorm_backward(dn, r, w, rstd, dx, dw, ws, dresidual=dr)
        return dx, dw

    want = call(dn, r, torch.empty_like(r), dr)
    for over in ("dn", "r"):
        for _ in range(10):
            t = dict(dn=dn.clone(), r=r.clone())
            got = call(t["dn"], t["r"], t[over], dr)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), over
    both = r.clone()  # one tensor for everything
    want = call(r, r, torch.empty_like(r), r)
    got = call(both, both, both, both)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rmsnorm_backward_against_differences(fp8):
    """Central differences of the 64-bit forward, through the kernel's gradients of fp32 inputs.
    With steps of 1e-4 the differences' own error is about 1e-8 of third derivatives of order one;
    the gradients are fp32 results of sums over 96 values: 1e-5 covers both many times over."""
    g = gen(15)
    n, d = 4, 96
    x, w, do = torch.randn(n, d, generator=g), 1 + 0.3 * torch.randn(d, generator=g), torch.randn(n, d, generator=g)
    f = lambda X, W: float((np64(do) * X / np.sqrt((X ** 2).mean(1, keepdims=True) + 1e-5) * W).sum())
    xc = x.cuda()
    rstd = torch.empty(n, device="cuda")
    fp8.rmsnorm(xc, None, rstd=rstd, eps=1e-5)
    dx, dw = torch.empty(n, d, device="cuda"), torch.empty(d, device="cuda")
    fp8.rmsnorm_backward(do.cuda(), xc, w.cuda(), rstd, dx, dw, fp8.rmsnorm_backward_workspace(n, d))
    X, W, h = np64(x), np64(w), 1e-4
    for i, j in [(0, 0), (1, 17), (2, 95), (3, 40)]:
        step = np.zeros_like(X)
        step[i, j] = h
        assert abs((f(X + step, W) - f(X - step, W)) / (2 * h) - float(dx[i, j])) < 1e-5
    for j in (0, 50, 95):
        step = np.zeros_like(W)
        step[j] = h
        assert abs((f(X, W + step) - f(X, W - step)) / (2 * h) - float(dw[j])) < 1e-5


def test_norms_of_several_widths_from_two_threads(fp8):
    """Rows too long for registers, of two widths, from two threads at once: every call is launched, with the bits
    of a call alone.  Each thread has its own stream and tensors."""
    import threading

    def work(d, n=3):
        g = torch.Generator("cuda").manual_seed(d)
        x, do = (torch.randn(n, d, generator=g, device="cuda") for _ in range(2))
        e = lambda: torch.empty(n, d, device="cuda")
        out, dx, rstd, dw = e(), e(), torch.empty(n, device="cuda"), torch.empty(d, device="cuda")
        ws = fp8.rmsnorm_backward_workspace(n, d)
        def once(stream):
            fp8.rmsnorm(x, None, out=out, rstd=rstd, stream=stream)
            fp8.rmsnorm_backward(do, x, None, rstd, dx, dw, ws, stream=stream)
        return once, (out, dx, rstd, dw)

    jobs = {d: work(d) for d in (20000, 49152)}
    torch.cuda.synchronize()
    alone, errors = {}, []
    for d, (once, outs) in jobs.items():
        once(None)
        torch.cuda.synchronize()
        alone[d] = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()

    def loop(once):
        stream = torch.cuda.Stream()
        try:
            for _ in range(2000):
                once(stream)
            stream.synchronize()
        except Exception as e:  # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(once,)) for once, _ in jobs.values()]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for d, (_, outs) in jobs.items():
        for a, b in zip(alone[d], outs):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ products

def make_rows(n, c, seed, std=1.0):
    q, s = ref.quantize(np64(torch.randn(n, c, generator=gen(seed)) * std))
    return q, s


def make_weights(E, n, c, seed):
    return ref.quantize_weights(np64(torch.randn(E, n, c, generator=gen(seed)) * c ** -0.5))


PRODUCTS = [  # segments' rows, E, K, N
    ([1], 1, 16, 16), ([1], 1, 2064, 400), ([128], 1, 128, 256), ([129], 1, 512, 272), ([256], 1, 640, 128),
    ([300], 1, 1024, 1040), ([2177], 1, 144, 96), ([0, 5, 0, 130, 1], 5, 256, 160), ([0, 0, 0], 3, 64, 64),
    ([3, 0, 7, 40, 1, 0, 0, 200], 4, 528, 144),  # two sources
    ([257, 31, 33, 32], 4, 384, 512),
    # more than one unit of work for each SM: the CTA-pair kernels on the "auto" path
    ([1300], 1, 272, 2064), ([129, 0, 700, 300, 1], 5, 528, 1168), ([40, 128, 257, 3, 900, 255], 3, 2064, 816),
    # more units than clusters, one of them with every kind of short group
    ([65, 17, 0, 1, 64, 33, 16, 15], 8, 1552, 2320),
    # K split over pairs of CTAs that take two units each (two segments need two groups of rows)
    ([97, 97, 1], 3, 1040, 3184), ([96, 95, 20], 3, 528, 272),
    # ... over clusters of eight, and a K whose last group of four blocks is short
    ([7], 1, 4176, 144),
]


@pytest.mark.parametrize("path", ["simt", "auto"])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seg, E, K, N", PRODUCTS, ids=lambda v: str(v))
def test_matmul(fp8, path, out, seg, E, K, N):
    n = sum(seg) + 3  # rows past the segments stay as they are
    qa, sa = make_rows(n, K, 21)
    qw, sw = make_weights(E, N, K, 22)
    sa[0] = np.where(sa[0] > 0, np.clip(sa[0] + 9, 0, 254), 0)  # a loud row
    if n > 2:
        sa[2] = np.where(sa[2] > 0, sa[2] - 20, 0)              # a quiet one
    plan = fp8.Fp8MatmulPlan(n, K, N, n_experts=E, n_sources=len(seg) // E, out_dtype="bf16" if out is BF else "f32", path=path)
    ws = torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    (ta, tsa), (tw, tsw) = ref.to_torch(qa, sa), ref.to_torch(qw, sw)
    o = torch.full((n, N), 77.0, dtype=out, device="cuda")
    plan.forward(torch.tensor(seg, dtype=torch.int32, device="cuda"), ta.cuda(), tsa.cuda(), tw.cuda(), tsw.cuda(), o, ws)
    assert plan.device_status(ws) == 0
    m = sum(seg)
    want, mag = ref.matmul(ref.dequantize(qa, sa)[:m], ref.dequantize_w(qw, sw), ref.row_experts(seg, E))
    close(np64(o)[:m], want, H[out] * np.abs(want) + K * EPS32 * mag, "out")
    assert (np64(o)[m:] == 77).all(), "rows past the segments are not written"


CLUSTERS = [  # K split over clusters of 3, 5, 6, 7 and 8 CTAs, which take two or three units each
    ([5000, 9], 2, 1424, 128), ([4000, 0, 1900], 3, 4624, 128), ([2600, 17], 2, 2832, 96), ([2500, 3], 2, 7168, 64),
    ([2100, 95, 5], 3, 4096, 112),
]


@pytest.mark.parametrize("seg, E, K, N", CLUSTERS, ids=lambda v: str(v))
def test_matmul_clusters_take_several_units(fp8, seg, E, K, N):
    test_matmul(fp8, "auto", BF, seg, E, K, N)


@pytest.mark.parametrize("K", [512, 1536, 2560, 8192])
def test_matmul_rows_sum_alike_wherever_they_stand(fp8, K):
    """Equal rows give equal bits, whichever CTA of a cluster adds their parts."""
    n, N = 83, 160
    (qa, sa), (qw, sw) = make_rows(1, K, 51), make_weights(1, N, K, 52)
    plan = fp8.Fp8MatmulPlan(n, K, N, out_dtype="f32")
    o, ws = torch.empty(n, N, device="cuda"), plan.new_workspace()
    (ta, tsa), (tw, tsw) = ref.to_torch(qa, sa), ref.to_torch(qw, sw)
    rows = lambda x: x.expand(n, -1).contiguous().cuda()
    plan.forward(None, rows(ta.view(torch.uint8)).view(ta.dtype), rows(tsa), tw.cuda(), tsw.cuda(), o, ws)
    assert plan.device_status(ws) == 0
    assert (o == o[0]).all()


@pytest.mark.parametrize("path", ["simt", "auto"])
def test_matmul_whole_buffer_without_counts(fp8, path):
    n, K, N = 200, 256, 320
    (qa, sa), (qw, sw) = make_rows(n, K, 23), make_weights(1, N, K, 24)
    plan = fp8.Fp8MatmulPlan(n, K, N, path=path)
    o = torch.empty(n, N, dtype=BF, device="cuda")
    t = [x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qw, sw))]
    ws = plan.new_workspace()
    plan.forward(None, *t, o, ws)
    assert plan.device_status(ws) == 0
    want, mag = ref.matmul(ref.dequantize(qa, sa), ref.dequantize_w(qw, sw), np.zeros(n, int))
    close(np64(o), want, H[BF] * np.abs(want) + K * EPS32 * mag)


def test_matmul_any_size_on_the_simt_path(fp8):
    n, K, N = 37, 131, 77
    (qa, sa), (qw, sw) = make_rows(n, K, 25), make_weights(2, N, K, 26)
    plan = fp8.Fp8MatmulPlan(n, K, N, n_experts=2, out_dtype="f32", path="simt")
    o, ws = torch.empty(n, N, device="cuda"), plan.new_workspace()
    t = [x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qw, sw))]
    plan.forward(torch.tensor([30, 7], dtype=torch.int32, device="cuda"), *t, o, ws)
    assert plan.device_status(ws) == 0
    want, mag = ref.matmul(ref.dequantize(qa, sa), ref.dequantize_w(qw, sw), ref.row_experts([30, 7], 2))
    close(np64(o), want, H[F32] * np.abs(want) + K * EPS32 * mag)


@pytest.mark.parametrize("path", ["simt", "auto"])
def test_matmul_nan_and_extreme_factors_stay_in_their_rows(fp8, path):
    """A NaN value or factor makes its own row NaN and no other; the smallest and largest factors
    give zeros and infinities as fp32 has them."""
    n, K, N = 140, 256, 64
    (qa, sa), (qw, sw) = make_rows(n, K, 27), make_weights(1, N, K, 28)
    ta, tsa = ref.to_torch(qa, sa)
    ta.view(torch.uint8)[3, 200] = 0x7F
    tsa[131, 1] = 255
    tsa[7, :2] = 0
    plan = fp8.Fp8MatmulPlan(n, K, N, out_dtype="f32", path=path)
    o, ws = torch.empty(n, N, device="cuda"), plan.new_workspace()
    tw, tsw = ref.to_torch(qw, sw)
    plan.forward(None, ta.cuda(), tsa.cuda(), tw.cuda(), tsw.cuda(), o, ws)
    assert plan.device_status(ws) == 0
    g = np64(o)
    assert np.isnan(g[[3, 131]]).all() and np.isfinite(np.delete(g, [3, 131], 0)).all()
    assert (np.abs(g[7]) < 1e-30).all()


@pytest.mark.parametrize("path", ["simt", "auto"])
@pytest.mark.parametrize("n, N", [(100, 64), (3000, 1040)], ids=["few rows", "many"])
@pytest.mark.parametrize("seg", [[5, -1, 3], [0.6, 0.3, 0.2], [1 << 30] * 4, [0x7FFFFFFF, 0x7FFFFFFF, 2]],
                         ids=["negative", "too many", "wraps to 0", "wraps to 0 again"])
def test_bad_counts_are_reported_and_compute_nothing(fp8, path, n, N, seg):
    K, E = 128, len(seg)
    seg = [int(c * n) if isinstance(c, float) else c for c in seg]
    (qa, sa), (qw, sw) = make_rows(n, K, 29), make_weights(E, N, K, 30)
    plan = fp8.Fp8MatmulPlan(n, K, N, n_experts=E, path=path)
    o, ws = torch.full((n, N), 5.0, dtype=BF, device="cuda"), plan.new_workspace()
    t = [x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qw, sw))]
    plan.forward(torch.tensor(seg, dtype=torch.int32, device="cuda"), *t, o, ws)
    from top_routing_grouped_gb300 import moe
    assert plan.device_status(ws) == moe.MOE_ERR_INTERNAL
    assert (o == 5).all()
    good = torch.zeros(E, dtype=torch.int32)
    good[0], good[1] = n - 30, 30
    plan.forward(good.cuda(), *t, o, ws)  # the next call is clean
    assert plan.device_status(ws) == 0 and not (o == 5).all(1).any()


EXPERTS = [  # segments' rows, E, d, F
    ([1], 1, 16, 16), ([1, 1, 0, 1, 1], 5, 512, 256), ([0, 0, 0, 0], 2, 64, 64), ([130, 0, 257, 64], 4, 256, 272),
    ([33, 128, 0, 3, 300, 1], 3, 400, 144), ([2100], 1, 128, 400), ([20, 31, 32, 33, 0, 200, 90, 64], 8, 1024, 640),
    ([900, 0, 257, 300], 4, 272, 1168), ([700, 33, 128, 1, 0, 513], 3, 1168, 400),  # CTA pairs on "auto"
]


def expert_rows(x, w1, w3, w2, gates, ex):
    """The expert rows in 64 bits, with the hidden values quantised, and how far a bf16 result may be.

    The hidden value that is quantised is an fp32 one, off by d eps sum|x w| in either factor, so one
    that lies on a border may take the neighbouring e4m3 (a step of at most 2^-3 of it): every
    hidden value within reach of a border adds a step times |w2| to the bound.  A block whose maximum
    is within reach of a factor's border may be rounded in twice the factor: each of its values is then
    half a step of either off, again 2^-3 of it at most (2^-8 of the factor below e4m3's normal
    values)."""
    m, d = x.shape
    w1, w3, w2 = (ref.dequantize_w(*w) for w in (w1, w3, w2))
    F = w1.shape[1]
    a, ma = ref.matmul(x, w1, ex)
    b, mb = ref.matmul(x, w3, ex)
    h = ref.silu(a) * b
    # |silu'| <= 1.1; exp and the quotient are good to 2^-20
    dh = 1.1 * d * EPS32 * ma * np.abs(b) + np.abs(ref.silu(a)) * d * EPS32 * mb + 2.0 ** -20 * np.abs(h)
    qh, sh = ref.quantize(h)
    f = np.repeat(ref.scale_value(sh), 128, 1)[:, :F]
    near = ref.round_e4m3((np.abs(h) - dh) / f) != ref.round_e4m3((np.abs(h) + dh) / f)
    pad = ((0, 0), (0, sh.shape[1] * 128 - F))
    top, dtop = (np.abs(np.pad(v, pad)).reshape(m, -1, 128).max(2) for v in (h, dh))
    border = np.repeat(ref.scale_byte(top - dtop) != ref.scale_byte(top + dtop), 128, 1)[:, :F]
    step = (near | border) * np.maximum(np.abs(h) * 2.0 ** -3, f * np.where(border, 2.0 ** -8, 2.0 ** -9))
    want, mag = ref.matmul(ref.dequantize(qh, sh), w2, ex)
    slack = ref.matmul(step, np.abs(w2), ex)[0]
    g = gates[:, None]
    return g * want, (H[BF] + 2 * EPS32) * np.abs(g * want) + g * (F * EPS32 * mag + slack)


@pytest.mark.parametrize("path", ["simt", "auto"])
@pytest.mark.parametrize("seg, E, d, F", EXPERTS, ids=lambda v: str(v))
def test_experts(fp8, path, seg, E, d, F):
    """y = gate * W2 q(silu(W1 x) * W3 x), q the quantisation to 8 bits."""
    m = sum(seg)
    n = m + 2
    W = len(seg) // E
    (qx, sx) = make_rows(n, d, 31)
    (q1, s1), (q3, s3), (q2, s2) = make_weights(E, F, d, 32), make_weights(E, F, d, 33), make_weights(E, d, F, 34)
    gates = torch.rand(n, generator=gen(35))
    plan = fp8.Fp8ExpertPlan(n, d, E, W, F, path=path)
    ws = torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.full((n, d), 77.0, dtype=BF, device="cuda")
    t = [x.cuda() for p in ((q1, s1), (q3, s3), (q2, s2)) for x in ref.to_torch(*p)]
    tx, tsx = ref.to_torch(qx, sx)
    plan.forward(torch.tensor(seg, dtype=torch.int32, device="cuda"), tx.cuda(), tsx.cuda(), gates.cuda(), *t, y, ws)
    assert plan.device_status(ws) == 0
    assert (np64(y)[m:] == 77).all()
    if m == 0:
        return
    want, tol = expert_rows(ref.dequantize(qx, sx)[:m], (q1, s1), (q3, s3), (q2, s2), np64(gates)[:m], ref.row_experts(seg, E))
    close(np64(y)[:m], want, tol, "y")


@pytest.mark.parametrize("path, seg", [("simt", [40]), ("auto", [40]), ("auto", [300])])
def test_experts_at_the_ends_of_silu(fp8, path, seg):
    """Pre-activations from -300 to 300: SiLU is a itself, or so small that it leaves fp32's normal range."""
    d, F, n = 128, 2048, sum(seg)
    (qx, sx) = make_rows(n, d, 61, std=64.0)
    (q1, s1), (q3, s3), (q2, s2) = make_weights(1, F, d, 62), make_weights(1, F, d, 63), make_weights(1, d, F, 64)
    gates = torch.rand(n, generator=gen(65))
    a = ref.matmul(ref.dequantize(qx, sx), ref.dequantize_w(q1, s1), np.zeros(n, int))[0]
    assert a.min() < -200 and a.max() > 200
    plan = fp8.Fp8ExpertPlan(n, d, 1, 1, F, path=path)
    ws, y = plan.new_workspace(), torch.empty(n, d, dtype=BF, device="cuda")
    t = [x.cuda() for p in ((q1, s1), (q3, s3), (q2, s2)) for x in ref.to_torch(*p)]
    plan.forward(None, *(x.cuda() for x in ref.to_torch(qx, sx)), gates.cuda(), *t, y, ws)
    assert plan.device_status(ws) == 0
    want, tol = expert_rows(ref.dequantize(qx, sx), (q1, s1), (q3, s3), (q2, s2), np64(gates), np.zeros(n, int))
    close(np64(y), want, tol, "y")


# One or few rows and a K of several groups of four blocks: the SwiGLU product's units are shared by clusters of
# 2, 3, 8 and 8 CTAs (16 rows a unit), 8 (32 rows) and 2 and 3 (64 rows).
SPLIT_EXPERTS = [([1], 1, 1024, 256), ([1, 0, 1, 1, 1], 5, 1040, 272), ([1, 1, 0, 1], 2, 4096, 256), ([0, 13, 1], 3, 4096, 400),
                 ([20, 0, 5], 3, 4096, 256), ([50, 3], 2, 1024, 144), ([33, 20, 1], 3, 2320, 256)]


@pytest.mark.parametrize("seg, E, d, F", SPLIT_EXPERTS, ids=lambda v: str(v))
def test_experts_hidden_rows_summed_by_clusters(fp8, seg, E, d, F):
    test_experts(fp8, "auto", seg, E, d, F)


@pytest.mark.parametrize("d", [1024, 4096])
def test_layer_in_8_bits_of_one_wide_token(fp8, d):
    test_layer_in_8_bits(fp8, 1, d, 8, 2, 256, False, False)


# Clusters of 3 to 8 CTAs, some of which take a second unit: the estimate of the units counts one group of rows
# a segment, and two of the three segments have two.
SECOND_UNITS = [(3, 1296, 1408), (4, 1920, 1024), (5, 2320, 896), (6, 2832, 752), (7, 3472, 640), (8, 4000, 624)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("split, K, N", SECOND_UNITS)
def test_matmul_clusters_take_a_second_unit(fp8, out, split, K, N):
    test_matmul(fp8, "auto", out, [97, 97, 1], 3, K, N)


def test_experts_clusters_take_several_units(fp8):
    test_experts(fp8, "auto", [97] * 27 + [2] * 11, 38, 1024, 256)


@pytest.mark.parametrize("path, least", [("simt", 90), ("auto", 87)])
@pytest.mark.parametrize("n", [3, 33, 300])
def test_experts_of_hidden_rows_that_are_all_small(fp8, path, least, n):
    """Pre-activations at the lower end of SiLU, so that nothing larger in a block hides them: a is -80 to
    -least, the same for all hidden columns of a row, and b is 2^14 of either sign (all exact).  The exponential is good
    to 2 + 1.17 |a| steps of 2^-23, and to half a subnormal step of 2^-149 of its 2^-130 at least: 2^-16 in all.
    A hidden value within twice that of a border may take the neighbouring e4m3, a step of 2^-3."""
    d, F = 128, 256
    a = -(80 + np.arange(n) * (least - 80) // max(1, n - 1)).astype(np.float64)
    x = np.zeros((n, d))
    x[:, 0], x[:, 1], x[:, 2] = 10, -a - 80, 1
    w1, w3, w2 = np.zeros((1, F, d)), np.zeros((1, F, d)), np64(torch.randn(1, d, F, generator=gen(67)) * 16)
    w1[:, :, 0], w1[:, :, 1] = -8, -1
    w3[:, :, 2] = 2.0 ** 14 * (1 - 2 * (np.arange(F) % 3 == 0))
    qx, w = ref.quantize(x), [ref.quantize_weights(v) for v in (w1, w3, w2)]
    held, ex = ref.dequantize(*qx), np.zeros(n, int)
    np.testing.assert_array_equal(ref.matmul(held, ref.dequantize_w(*w[0]), ex)[0], np.repeat(a[:, None], F, 1))
    plan = fp8.Fp8ExpertPlan(n, d, 1, 1, F, path=path)
    ws, y = plan.new_workspace(), torch.empty(n, d, dtype=BF, device="cuda")
    t = [v.cuda() for p in w for v in ref.to_torch(*p)]
    plan.forward(None, *(v.cuda() for v in ref.to_torch(*qx)), torch.ones(n, device="cuda"), *t, y, ws)
    assert plan.device_status(ws) == 0
    want, tol = expert_rows(held, *w, np.ones(n), ex)
    h = np.abs(ref.silu(a))[:, None] * np.full((1, F), 2.0 ** 14)
    f = np.repeat(ref.scale_value(ref.quantize(h)[1][:, :F // 128]), 128, 1)
    near = ref.round_e4m3(h * (1 - 2.0 ** -15) / f) != ref.round_e4m3(h * (1 + 2.0 ** -15) / f)
    close(np64(y), want, tol + ref.matmul(near * 2.0 ** -3 * h, np.abs(ref.dequantize_w(*w[2])), ex)[0], "y")
    assert (np.abs(np64(y)).max(1) > 0).all()


def test_experts_paths_agree_on_a_larger_layer(fp8):
    """The tensor-core and SIMT paths on 3000 rows of 16 experts: both round the same sums to the
    same 8 bits but for values at a border, and y to bf16: 2-norm of the difference within 2^-8."""
    g, E, d, F = torch.Generator("cuda").manual_seed(5), 16, 768, 512
    seg = torch.tensor([0, 700, 1, 127, 128, 129, 255, 256, 257, 300, 400, 100, 47, 200, 0, 100], dtype=torch.int32)
    n = int(seg.sum())
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, sx = f8(n, d), u8(n, fp8.scale_cols(d))
    fp8.quantize(rn(n, d), x, sx)
    ws = []
    for r, c in ((F, d), (F, d), (d, F)):
        q, s = f8(E, r, c), u8(E, -(-r // 128), fp8.scale_cols(c))
        fp8.quantize_weights(rn(E, r, c) * c ** -0.5, q, s)
        ws += [q, s]
    gates, ys = torch.rand(n, generator=g, device="cuda"), []
    for path in ("auto", "simt"):
        plan = fp8.Fp8ExpertPlan(n, d, E, 1, F, path=path)
        y, w = torch.empty(n, d, dtype=BF, device="cuda"), plan.new_workspace()
        plan.forward(seg.cuda(), x, sx, gates, *ws, y, w)
        assert plan.device_status(w) == 0
        ys.append(np64(y))
    assert np.linalg.norm(ys[0] - ys[1]) <= 2.0 ** -8 * np.linalg.norm(ys[1])


# ------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("n, F", [(1, 16), (1, 2048), (7, 130), (300, 1072), (1000, 1)])
def test_checkpoint_save_bit_exact(fp8, n, F):
    a, b = awkward(n, F, BF, 41).cuda(), awkward(n, F, BF, 42).flip(0).cuda()
    out = [f8(n, F), u8(n, fp8.scale_cols(F)), f8(n, F), u8(n, fp8.scale_cols(F))]
    fp8.checkpoint_save(a, b, *out)
    for x, (q, s) in ((a, out[:2]), (b, out[2:])):
        wq, ws = ref.quantize(np64(x))
        np.testing.assert_array_equal(np64(s), ws)
        np.testing.assert_array_equal(np64(q), wq)


@pytest.mark.parametrize("n, F", [(1, 16), (1, 2048), (7, 130), (300, 1072), (513, 1)])
def test_checkpoint_backward_against_the_formula(fp8, n, F):
    g = gen(43)
    (qa, sa), (qb, sb) = ref.quantize(np64(torch.randn(n, F, generator=g) * 4)), ref.quantize(np64(torch.randn(n, F, generator=g)))
    dh = torch.randn(n, F, generator=g).to(BF)
    t = [x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qb, sb), dh)]
    da, db, h = (torch.empty(n, F, dtype=BF, device="cuda") for _ in range(3))
    fp8.checkpoint_backward(*t, da, db, h)
    a, b, do = ref.dequantize(qa, sa), ref.dequantize(qb, sb), np64(dh)
    sig = 1 / (1 + np.exp(-a))
    # sigma is good to 2^-20 relative; silu' = sigma (1 + a (1 - sigma)), whose terms may cancel
    mag = sig * (1 + np.abs(a) * (1 - sig) + np.abs(a) * sig * 2)
    close(np64(da), do * b * sig * (1 + a * (1 - sig)), np.abs(do * b) * (mag * 2.0 ** -19 + H[BF] * np.abs(sig * (1 + a * (1 - sig)))), "da")
    for got, want in ((db, do * a * sig), (h, a * sig * b)):
        close(np64(got), want, np.abs(want) * (H[BF] + 2.0 ** -19))
    da2, db2 = t[4].clone(), torch.empty_like(db)
    fp8.checkpoint_backward(*t[:4], da2, da2, db2)  # in place of dh, without h
    assert torch.equal(da2, da) and torch.equal(db2, db)


@pytest.mark.parametrize("n, F", [(1, 16), (7, 130), (300, 1072), (65, 2048)])
def test_checkpoint_restore(fp8, n, F):
    (qa, sa), (qb, sb) = ref.quantize(np64(awkward(n, F, BF, 45))), ref.quantize(np64(torch.randn(n, F, generator=gen(46))))
    t = [x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qb, sb))]
    a, b, h = (torch.empty(n, F, dtype=BF, device="cuda") for _ in range(3))
    fp8.checkpoint_restore(*t, a, b, h)
    va, vb = ref.dequantize(qa, sa), ref.dequantize(qb, sb)
    np.testing.assert_array_equal(np64(a), va)  # four bits times a power of two: exact in bf16
    np.testing.assert_array_equal(np64(b), vb)
    want = ref.silu(va) * vb
    past = np.abs(want) > 3.4e38  # past the largest bf16 and fp32: an infinity
    assert (np64(h)[past] == np.sign(want[past]) * np.inf).all()
    close(np.where(past, 0, np64(h)), np.where(past, 0, want), np.abs(want) * (H[BF] + 2.0 ** -19) + 1e-37, "h")
    for kw in (dict(a=torch.empty_like(a)), dict(b=torch.empty_like(b)), dict(h=torch.empty_like(h))):
        fp8.checkpoint_restore(*t, **kw)
        for k, v in kw.items():
            assert torch.equal(v.view(torch.int16), dict(a=a, b=b, h=h)[k].view(torch.int16))


def test_checkpoint_backward_against_differences(fp8):
    """Central differences of sum(dh * silu(a) * b) in 64 bits at the values the checkpoint holds;
    da, db are bf16: half a step, 2^-8, and 1e-6 for the differences."""
    g, n, F = gen(44), 3, 64
    (qa, sa), (qb, sb) = ref.quantize(np64(torch.randn(n, F, generator=g))), ref.quantize(np64(torch.randn(n, F, generator=g)))
    dh = torch.randn(n, F, generator=g).to(BF)
    da, db = (torch.empty(n, F, dtype=BF, device="cuda") for _ in range(2))
    fp8.checkpoint_backward(*[x.cuda() for x in (*ref.to_torch(qa, sa), *ref.to_torch(qb, sb), dh)], da, db)
    a, b, do, e = ref.dequantize(qa, sa), ref.dequantize(qb, sb), np64(dh), 1e-4
    num_a = do * (ref.silu(a + e) - ref.silu(a - e)) * b / (2 * e)
    num_b = do * ref.silu(a)
    close(np64(da), num_a, H[BF] * np.abs(num_a) + 1e-6)
    close(np64(db), num_b, H[BF] * np.abs(num_b) + 1e-6)


# ------------------------------------------------------------------ streams and graphs

def test_other_streams_and_graph_capture(fp8):
    """The whole serving chain on a side stream, then captured into a CUDA graph and replayed on
    new inputs: the same bits as the eager calls."""
    n, d, F, E = 96, 256, 384, 4
    g = torch.Generator("cuda").manual_seed(9)
    x, res = (torch.randn(n, d, generator=g, device="cuda").to(BF) for _ in range(2))
    w, gates = torch.rand(d, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    ws = []
    for r, c in ((F, d), (F, d), (d, F)):
        q, s = f8(E, r, c), u8(E, -(-r // 128), fp8.scale_cols(c))
        fp8.quantize_weights(torch.randn(E, r, c, generator=g, device="cuda") * c ** -0.5, q, s)
        ws += [q, s]
    seg = torch.tensor([10, 0, 80, 6], dtype=torch.int32, device="cuda")
    plan = fp8.Fp8ExpertPlan(n, d, E, 1, F)
    wsp, q, s, y, r = plan.new_workspace(), f8(n, d), u8(n, 4), torch.empty_like(x), torch.empty_like(x)

    def chain(stream=None):
        fp8.rmsnorm(x, w, res, r, q=q, scales=s, stream=stream)
        plan.forward(seg, q, s, gates, *ws, y, wsp, stream=stream)

    chain()
    torch.cuda.synchronize()
    first = y.clone()
    y.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    chain(side)
    side.synchronize()
    assert torch.equal(first, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    x.copy_(torch.randn(n, d, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    chain()
    torch.cuda.synchronize()
    assert torch.equal(replayed, y) and not torch.equal(first, y)
    assert plan.device_status(wsp) == 0


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("T, d, E, k, F, bias, renorm", [
    (1, 256, 8, 2, 128, False, False), (1, 512, 16, 4, 192, True, True), (300, 192, 8, 3, 320, True, False),
    (130, 128, 32, 2, 64, False, True), (1100, 256, 4, 2, 1152, False, False)])
def test_layer_in_8_bits(fp8, T, d, E, k, F, bias, renorm):
    """moe_fp8_forward: dispatched rows and factors bit for bit, expert rows within the bound of the
    expert stage, and y the sum of its k expert rows in fp32, rounded once."""
    g = gen(51)
    x = torch.randn(T, d, generator=g).to(BF).cuda()
    xq, xs = f8(T, d), u8(T, fp8.scale_cols(d))
    fp8.quantize(x, xq, xs)
    w = [make_weights(E, r, c, 52 + i) for i, (r, c) in enumerate(((F, d), (F, d), (d, F)))]
    tw = [v.cuda() for p in w for v in ref.to_torch(*p)]
    wr = (torch.randn(E, d, generator=g) * d ** -0.5).to(BF).cuda()
    b = torch.linspace(-1, 1, E).cuda() if bias else None
    plan = fp8.Fp8MoEPlan(T, d, E, k, F, has_bias=bias, renorm_gates=renorm, tau=0.7)
    ws = torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.empty(T, d, dtype=BF, device="cuda")
    plan.forward(x, xq, xs, wr, b, *tw, y, ws)
    assert plan.device_status(ws) == 0
    v = plan.views(ws)
    src, gate, pos = (v[n].cpu().numpy() for n in ("perm_src", "gate_perm", "slot_pos"))
    assert torch.equal(v["xp"].view(torch.uint8).cpu(), xq.view(torch.uint8).cpu()[src])
    ex = np.repeat(np.arange(E), v["expert_counts"].cpu().numpy())
    np.testing.assert_array_equal(ex, v["topk_idx"].cpu().numpy().reshape(-1)[v["perm_slot"].cpu().numpy()])
    rows = ref.dequantize(np64(xq), np64(xs))[src]
    want, tol = expert_rows(rows, *w, gate.astype(np.float64), ex)
    yp = np64(v["yp"])
    close(yp, want, tol, "expert rows")
    total, mag = yp[pos.reshape(T, k)].sum(1), np.abs(yp[pos.reshape(T, k)]).sum(1)
    close(np64(y), total, H[BF] * np.abs(total) + k * EPS32 * mag, "y")
    # the same routing as a bf16 plan's on the same x
    from top_routing_grouped_gb300 import moe
    p16 = moe.MoEPlan(T, d, E, k, F, has_bias=bias, renorm_gates=renorm, tau=0.7)
    w16 = p16.new_workspace()
    z = torch.zeros(E, F, d, dtype=BF, device="cuda")
    p16.forward(x, wr, b, z, z, torch.zeros(E, d, F, dtype=BF, device="cuda"), torch.empty_like(y), w16)
    v16 = p16.views(w16)
    for name in ("topk_idx", "topk_gate", "slot_pos", "expert_counts"):
        assert torch.equal(v[name], v16[name]), name
    assert torch.equal(plan.aux_loss(ws), p16.aux_loss(w16))


@pytest.mark.parametrize("T, d, E, k, F", [(1, 1024, 16, 4, 256), (1, 256, 8, 2, 128), (300, 256, 16, 2, 128), (1100, 256, 4, 2, 1152)])
def test_layer_takes_the_gates_of_its_own_call(fp8, T, d, E, k, F):
    """Calls one after another in one workspace, each with a router of its own (other experts, other gates) and
    with NaN where the gates of the call before were: every call's expert rows are those of its own routing, and
    the same call gives the same bits whatever ran before it."""
    g = gen(71)
    x = torch.randn(T, d, generator=g).to(BF).cuda()
    xq, xs = f8(T, d), u8(T, fp8.scale_cols(d))
    fp8.quantize(x, xq, xs)
    w = [make_weights(E, r, c, 72 + i) for i, (r, c) in enumerate(((F, d), (F, d), (d, F)))]
    tw = [v.cuda() for p in w for v in ref.to_torch(*p)]
    routers = [(torch.randn(E, d, generator=g) * d ** -0.5 * s).to(BF).cuda() for s in (1.0, 4.0, 0.25)]
    plan = fp8.Fp8MoEPlan(T, d, E, k, F, tau=0.7)
    ws, y = plan.new_workspace(), torch.empty(T, d, dtype=BF, device="cuda")
    first = []
    for wr in routers:
        plan.views(ws)["gate_perm"].fill_(float("nan"))
        plan.forward(x, xq, xs, wr, None, *tw, y, ws)
        assert plan.device_status(ws) == 0
        v = plan.views(ws)
        src, gate = v["perm_src"].cpu().numpy(), np64(v["gate_perm"])
        np.testing.assert_array_equal(gate, np64(v["topk_gate"]).reshape(-1)[v["perm_slot"].cpu().numpy()])
        ex = np.repeat(np.arange(E), v["expert_counts"].cpu().numpy())
        want, tol = expert_rows(ref.dequantize(np64(xq), np64(xs))[src], *w, gate, ex)
        close(np64(v["yp"]), want, tol, "expert rows")
        first.append((y.clone(), v["yp"].clone()))
    for i in 20 * [0, 1, 2, 1]:
        plan.views(ws)["gate_perm"].fill_(float("nan"))
        plan.forward(x, xq, xs, routers[i], None, *tw, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, first[i][0]) and torch.equal(plan.views(ws)["yp"], first[i][1])
    assert plan.device_status(ws) == 0


@pytest.mark.parametrize("T, d, E, k, F", [(1, 4096, 16, 4, 2048), (300, 1024, 16, 2, 512), (3000, 512, 4, 2, 1152)])
def test_layer_with_the_shortest_limit(fp8, T, d, E, k, F):
    """A limit below the shortest one, 1 ms, is that one, and it runs only while a wait can end: the second
    product, which starts as early as the first, does not report the time until the first has ended."""
    g = torch.Generator("cuda").manual_seed(81)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF)
    xq, xs = f8(T, d), u8(T, fp8.scale_cols(d))
    fp8.quantize(x, xq, xs)
    tw = []
    for r, c in ((F, d), (F, d), (d, F)):
        q, s = f8(E, r, c), u8(E, -(-r // 128), fp8.scale_cols(c))
        fp8.quantize_weights(torch.randn(E, r, c, generator=g, device="cuda") * c ** -0.5, q, s)
        tw += [q, s]
    wr = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    ys = []
    for limit in (1, 0):
        plan = fp8.Fp8MoEPlan(T, d, E, k, F, wait_timeout_ns=limit)
        ws, y = plan.new_workspace(), torch.empty(T, d, dtype=BF, device="cuda")
        plan.forward(x, xq, xs, wr, None, *tw, y, ws)
        assert plan.device_status(ws) == 0
        ys.append(y)
    assert torch.equal(*ys)


def training_layer(moe, T, d, E, k, F, x, w, wr):
    plan = moe.MoEPlan(T, d, E, k, F, training=True)
    ws, y = plan.new_workspace(), torch.empty(T, d, dtype=BF, device="cuda")
    plan.forward(x, wr, None, *w, y, ws)
    return plan, ws


def gradients(plan, x, wr, w, dy, ws):
    T, d, E, F = plan.T, plan.d, plan.E, plan.F
    out = [torch.empty(*s, device="cuda") for s in ((T, d), (E, d), (E, F, d), (E, F, d), (E, d, F))]
    plan.backward(x, wr, None, *w, dy, 0.1, out[0], out[1], None, out[2], out[3], out[4], ws)
    assert plan.device_status(ws) == 0
    return dict(zip(("dx", "dwr", "dw1", "dw3", "dw2"), out))


def test_layer_checkpoint_of_values_that_8_bits_hold(fp8):
    """Inputs whose pre-activations are e4m3 values already (rows of x with a single one, so that a row's
    pre-activations are a column of the weights): the backward from the checkpoint, in a workspace
    that another forward has used, gives the plain backward's gradients bit for bit; dW2 alone is
    taken from the rebuilt hidden rows, silu(a) b to half a bf16 step where the forward's is good to
    one (2^-7), summed over an expert's rows."""
    from top_routing_grouped_gb300 import moe
    T, d, E, k, F = 200, 128, 8, 2, 192
    g = gen(61)
    x = torch.zeros(T, d)
    x[torch.arange(T), torch.randint(0, d, (T,), generator=g)] = 1
    def held(*s):  # e4m3 values of magnitude 2^-5 to 1.75
        return (torch.randint(8, 15, s, generator=g) / 8.0 * torch.exp2(torch.randint(-5, 1, s, generator=g).float())
                * (2 * torch.randint(0, 2, s, generator=g) - 1))
    w = [t.to(BF).cuda() for t in (held(E, F, d), held(E, F, d), torch.randn(E, d, F, generator=g) * F ** -0.5)]
    x, wr = x.to(BF).cuda(), torch.randn(E, d, generator=g).to(BF).cuda()
    dy = torch.randn(T, d, generator=g).to(BF).cuda()
    plan, ws = training_layer(moe, T, d, E, k, F, x, w, wr)
    ckpt = fp8.LayerCheckpoint(plan)
    ckpt.save(ws)
    names = ("topk_idx", "expert_counts", "expert_offsets", "perm_src", "slot_pos", "gate_perm", "xp")
    before = {n: plan.views(ws)[n].clone() for n in names}
    plain = gradients(plan, x, wr, w, dy, ws)
    other = torch.randn(T, d, generator=g).to(BF).cuda()
    plan.forward(other, wr, None, *w, torch.empty(T, d, dtype=BF, device="cuda"), ws)
    ws[: ws.numel() // 2] = 0xFF
    ckpt.restore(x, ws)
    for n in names:
        assert torch.equal(plan.views(ws)[n], before[n]), n
    again = gradients(plan, x, wr, w, dy, ws)
    for n in ("dx", "dwr", "dw1", "dw3"):
        assert torch.equal(plain[n], again[n]), n
    diff, size = np64(again["dw2"] - plain["dw2"]), np64(plain["dw2"])
    assert np.linalg.norm(diff) <= 2.0 ** -7 * np.linalg.norm(size)


def test_layer_checkpoint_of_ordinary_values(fp8):
    """Ordinary values: a kept pre-activation is off by at most 2^-4 of itself, in rms by 2^-4/sqrt(3) of
    it (a uniform error within half a step; less, as the step is a smaller part of most values), and the
    gradients are at most quadratic in them: the gradients' 2-norm error is at most twice that plus
    the bf16 backward's own (1e-2 at most): 0.09.  The routing and what does not depend on the
    pre-activations (the zero gradients of experts without rows) are the plain backward's."""
    from top_routing_grouped_gb300 import moe
    T, d, E, k, F = 300, 256, 16, 3, 320
    g = gen(62)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF).cuda()
    x, wr, dy = rn(T, d), rn(E, d, std=d ** -0.5), rn(T, d)
    w = [rn(E, F, d, std=d ** -0.5), rn(E, F, d, std=d ** -0.5), rn(E, d, F, std=F ** -0.5)]
    plan, ws = training_layer(moe, T, d, E, k, F, x, w, wr)
    ckpt = fp8.LayerCheckpoint(plan)
    ckpt.save(ws)
    plain = gradients(plan, x, wr, w, dy, ws)
    ckpt.restore(x, ws)
    got = gradients(plan, x, wr, w, dy, ws)
    for n in plain:
        err = np.linalg.norm(np64(got[n] - plain[n])) / np.linalg.norm(np64(plain[n]))
        assert 0 < err <= 0.09, (n, err)
    assert ckpt.data.numel() < 0.3 * plan.workspace_bytes


def test_example_serves_and_trains():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    small = ["--tokens", "96", "--layers", "2", "--d", "128", "--experts", "4", "--hidden", "128"]
    # a token alone and in a batch take the same roundings, but the sums' order differs (K split or
    # not), so that values at a border may round the other way: within a bf16 step in the 2-norm
    assert m.main(["serve", *small]) <= 2.0 ** -7
    losses = m.main(["train", *small, "--steps", "6"])
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
