"""The gradients' norm and the step of AdamW against plain 64-bit references.

Tolerances, in units u = 2^-24 (half a step of fp32, relative).  m = b1 m + c1 (f g): the constants, the products
and the sum are rounded: 6 u (|b1 m| + |c1 f g|); v likewise, one rounding more.  r = sqrt(v): half of v's and
2 u of the square root, 6 u.  The update U = lr / bc1 * m / (r / sqrt(bc2) + eps): lr / bc1 has 6 u (expm1 2,
its argument 2, lr and the quotient), 1 / sqrt(bc2) 7 u, the denominator 1 more, the quotient 4 (two steps), the
product 1, m 6 of its terms: 30 u of what U is with |b1 m| + |c1 f g| for m.  p: 4 u |p| (1 - lr wd has two
roundings, the product with p and the sum one) and U's.
What is rounded stochastically grows with the value it is rounded from: the result lies between those that the
reference gives for its value less and plus the tolerance."""
import numpy as np
import pytest
import torch

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def optim():
    from top_routing_grouped_gb300 import optim as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def np64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ references

def words(n, seed, step, tensor, first=0):
    """The random word of every value from `first` (a multiple of 8) on."""
    mask = (1 << 32) - 1

    def mix(x):
        x = x * np.uint64(0x9E3779B1) & np.uint64(mask)
        x = (x ^ x >> np.uint64(16)) * np.uint64(0x6A09E667) & np.uint64(mask)
        x = (x ^ x >> np.uint64(15)) * np.uint64(0xBB67AE85) & np.uint64(mask)
        return x ^ x >> np.uint64(16)
    key = np.uint64(0)
    for part in (seed & mask, seed >> 32, step & mask, tensor):
        key = mix(np.array((int(key) + part) & mask, np.uint64))
    out = np.empty((-(-n // 8), 8), np.uint64)
    out[:, 0] = mix((np.arange(len(out), dtype=np.uint64) + np.uint64(first // 8 + int(key))) & np.uint64(mask))
    for j in range(1, 8):
        out[:, j] = (out[:, j - 1] * np.uint64(0x3C6EF375) + np.uint64(0xA54FF53B)) & np.uint64(mask)
    return out.reshape(-1)[:n].astype(np.int64)


def sr_bf16(x, w):
    """Values [n] in 64 bits with the words' low 16 bits."""
    gap = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
    lo = np.floor(np.abs(x) / gap)
    return np.sign(x) * gap * (lo + ((np.abs(x) / gap - lo) + (w & 0xFFFF) / 65536 >= 1))


def scale_of(top):
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(top / 448))
    e = np.where(top > 448 * np.exp2(e), e + 1, e)
    return np.where(top == 0, -127.0, np.maximum(e, -127))


def blocks(x):
    return np.pad(x, (0, -len(x) % 128)).reshape(-1, 128)


def neighbours(u):
    gap = np.exp2(np.floor(np.log2(np.maximum(u, 2.0 ** -6))) - 3)
    lo = np.floor(u / gap) * gap
    return lo, lo + gap


def sr_m(x, w, e):
    by = np.exp2(np.repeat(e, 128)[:len(x)])
    u = np.abs(x) / by
    lo, hi = neighbours(u)
    return np.sign(x) * by * np.where((u - lo) / (hi - lo) + (w >> 16) / 65536 >= 1, hi, lo)


def sr_r(v, w, e):
    by = np.exp2(np.repeat(e, 128)[:len(v)])
    lo, hi = neighbours(np.sqrt(v) / by)
    up = (v / by ** 2 - lo ** 2) / (hi ** 2 - lo ** 2) > (w >> 8 & 0xFFFF) / 65536
    return by * np.where(up | ((lo == 0) & (v > 0)), hi, lo)


def check_step(before, after, grad, i, *, step, seed, f=1.0, lr=LR, b1=B1, b2=B2, eps=EPS, wd=0.01, optim=None, first=0):
    """One tensor of a step: before / after = (param, master, state) on the CPU."""
    p, w, st = before
    g = np64(grad).reshape(-1) * f
    m, v = (np64(t).reshape(-1) for t in optim.moments(st))
    x = np64(w if w is not None else p).reshape(-1)
    mt, vt = np.abs(b1 * m) + np.abs((1 - b1) * g), b2 * v + (1 - b2) * g * g
    m, v = b1 * m + (1 - b1) * g, vt
    den = np.sqrt(v / (1 - b2 ** step)) + eps
    rate = lr / (1 - b1 ** step)
    tol = U * (4 * np.abs(x) + 30 * rate * mt / den) + 2.0 ** -149
    x = x * (1 - lr * wd) - rate * m / den
    rnd = words(len(x), seed, step, i, first)
    got = np64(after[0]).reshape(-1)
    if w is not None:
        kept = np64(after[1]).reshape(-1)
        assert (np.abs(kept - x) <= tol).all(), "master"
        assert torch.equal(after[0], after[1].to(BF)), "parameter of a master"
    elif p.dtype is F32:
        assert (np.abs(got - x) <= tol).all(), "parameter"
    else:
        assert ((got >= sr_bf16(x - tol, rnd)) & (got <= sr_bf16(x + tol, rnd))).all(), "bf16 parameter"
    if len(st) == 2:
        assert (np.abs(np64(after[2][0]).reshape(-1) - m) <= 6 * U * mt + 2.0 ** -149).all(), "m"
        assert (np.abs(np64(after[2][1]).reshape(-1) - v) <= 7 * U * vt + 2.0 ** -149).all(), "v"
        return
    assert len(after[2][1]) == -(-len(x) // 128)
    vt = 7 * U * vt
    for name, q, s, lo, hi, rounds, top in (("m", after[2][0], after[2][1], m - 6 * U * mt, m + 6 * U * mt, sr_m, np.abs),
                                            ("r", after[2][2], after[2][3], np.maximum(v - vt, 0), v + vt, sr_r, np.sqrt)):
        e = s.view(torch.uint8).cpu().numpy().astype(np.float64) - 127
        # the factor is that of the largest value, which is known to a few u
        t = blocks(top(m if name == "m" else v)).max(1)
        assert ((e >= scale_of(t * (1 - 16 * U))) & (e <= scale_of(t * (1 + 16 * U)))).all(), name + "'s factors"
        val = np64(q).reshape(-1) * np.exp2(np.repeat(e, 128)[:len(x)])
        a, b = rounds(lo, rnd, e), rounds(hi, rnd, e)
        if name == "r":  # of a v at 0 or above: not 0 where the kernel's v is above it
            a = np.where(v > 0, a, np.minimum(a, b))
        assert ((val >= a) & (val <= b)).all(), (name, np.argwhere((val < a) | (val > b))[:3], val[(val < a) | (val > b)][:3], a[(val < a) | (val > b)][:3])


# ------------------------------------------------------------------ the words and the roundings, on the CPU

def test_words_are_even():
    """Each 16-bit field's mean and bits, over values, steps and tensors: within 5 standard deviations of an even distribution."""
    n = 1 << 16
    for fields in ([words(n, 3, 9, 0)], [words(8, 5, s, 1) for s in range(2000)], [words(16, 77 + (s << 33), 1, s) for s in range(1000)]):
        w = np.concatenate(fields)
        for shift in (0, 8, 16):
            h = w >> shift & 0xFFFF
            assert abs(h.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * len(h))
            for bit in range(4, 16):
                assert abs((h >> bit & 1).mean() - 0.5) < 5 * 0.5 / np.sqrt(len(h))


@pytest.mark.parametrize("kind", ["m", "r", "bf16"])
def test_roundings_keep_the_mean(kind):
    """The reference's roundings over all random words' fields: m and a parameter on average, r's square; to one step of 2^-16."""
    g = np.random.default_rng(0)
    every = np.arange(65536, dtype=np.int64)
    for x in np.concatenate([g.uniform(0, 448, 20), g.uniform(0, 0.02, 20), [448.0, 0.0, 2.0 ** -9, 2.0 ** -6]]):
        if kind == "bf16":
            got, gap, want = sr_bf16(np.full(65536, x), every).mean(), max(x, 2.0 ** -126) * 2.0 ** -7, x
        elif kind == "m":
            got, gap, want = sr_m(np.full(65536, x), every << 16, np.zeros(512)).mean(), max(x, 2.0 ** -6) / 8, x
        else:
            if 0 < x < 2.0 ** -9:
                continue  # is kept above 0
            got, gap, want = (sr_r(np.full(65536, x * x), every << 8, np.zeros(512)) ** 2).mean(), max(x, 2.0 ** -6) ** 2 / 2, x * x
        assert abs(got - want) <= gap * 2.0 ** -16 + 1e-12 * want, (kind, x)


# ------------------------------------------------------------------ one step

def make(shape, ptype, gtype, bits, master, seed, optim, offset=0, spread=True):
    """(param, master, state), gradient: on the GPU, `offset` values past an aligned address."""
    g = gen(seed)
    n = int(np.prod(shape))

    def at(t):
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape)
        buf.view(torch.uint8).copy_(t.contiguous().view(torch.uint8).cuda()) if t.dtype.itemsize == 1 else buf.copy_(t)
        return buf
    w = torch.randn(n, generator=g) * 0.1
    big = torch.exp2(torch.randint(-12, 12, (n,), generator=g).float()) if spread else torch.ones(n)
    m, r, gr = torch.randn(n, generator=g) * 1e-3 * big, (torch.rand(n, generator=g) + 0.5) * 1e-3 * big, torch.randn(n, generator=g) * 1e-3 * big
    for t in (m, r, gr):
        t[torch.rand(n, generator=g) < 0.05] = 0
    if n > 300:
        r[128:256] = 0
        gr[128:256] = 0
        m[128:192] = 0
    if bits == 32:
        state = (at(m.view(shape)), at(r.square().view(shape)))
    else:
        state = []
        for v in (m, r):
            e = torch.from_numpy(scale_of(blocks(v.abs().double().numpy()).max(1)))
            q = (v.double() * torch.exp2(-e.repeat_interleave(128)[:n])).float().to(F8)
            state += [at(q.view(shape)), at((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)]
        state = tuple(state)
    return (at(w.to(ptype).view(shape)), at(w.view(shape)) if master else None, state), at(gr.to(gtype).view(shape))


def at_offset(t, offset):
    """A copy on the GPU that begins `offset` values past an aligned address."""
    return torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape).copy_(t)


def copy(b):
    return b[0].cpu().clone(), None if b[1] is None else b[1].cpu().clone(), tuple(t.view(torch.uint8).cpu().clone().view(t.dtype) for t in b[2])


def take(optim, sets, grads, **kw):
    return optim.AdamW([b[0] for b in sets], lr=LR, betas=(B1, B2), eps=EPS, masters=[b[1] for b in sets], state=[b[2] for b in sets], **kw)


KINDS = [(F32, False, 32), (F32, False, 8), (BF, True, 32), (BF, True, 8), (BF, False, 32), (BF, False, 8)]


@gpu
@pytest.mark.parametrize("ptype, master, bits", KINDS)
@pytest.mark.parametrize("gtype", [F32, BF])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_step(optim, ptype, master, bits, gtype, offset):
    shapes = [(1,), (127,), (128,), (129,), (3, 5, 43), (8191,), (8192,), (8193,), (70, 1001), (2, 16384)]
    made = [make(s, ptype, gtype, bits, master, 10 + i, optim, offset) for i, s in enumerate(shapes)]
    sets, grads = [x[0] for x in made], [x[1] for x in made]
    for done, seed, f in ((0, 0, None), (999, 1 << 40 | 12345, 0.37), (10 ** 7, 2 ** 64 - 1, 1.0)):
        before = [copy(b) for b in sets]
        factor = None if f is None else torch.tensor([f], device="cuda")
        opt = take(optim, sets, grads, steps=done, seed=seed, weight_decay=[0.1 * (i % 3) for i in range(len(sets))])
        opt.step(grads, grad_factor=factor)
        assert int(opt.steps) == done + 1 and int(opt._ticket) == 0
        for i, (b, s, gr) in enumerate(zip(before, sets, grads)):
            check_step(b, copy(s), gr, i, step=done + 1, seed=seed, f=1.0 if f is None else float(factor), wd=np.float32(0.1 * (i % 3)), optim=optim)


@gpu
@pytest.mark.parametrize("betas", [(0.0, 0.0), (1e-9, 1e-9), (0.0, 0.999), (0.3, 0.6), (0.5, 0.5), (0.6, 0.4), (0.99, 0.9999)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("offset", [0, 1])
def test_other_betas(optim, betas, bits, offset):
    """Moments that are kept and much larger or smaller than what comes in; 1 - b has one rounding more where b is small."""
    made = [make((5000,), BF, F32, bits, False, 3, optim, offset), make((300,), F32, BF, bits, False, 4, optim, offset)]
    sets, grads = [x[0] for x in made], [x[1] for x in made]
    for scale in (1.0, 2.0 ** -14, 2.0 ** 14):
        now = [g * scale for g in grads] if not offset else [g.mul_(scale) for g in grads]
        before = [copy(b) for b in sets]
        opt = optim.AdamW([b[0] for b in sets], lr=0.02, betas=betas, eps=1e-5, state=[b[2] for b in sets], steps=2, seed=1)
        opt.step(now)
        for i, (b, s, gr) in enumerate(zip(before, sets, now)):
            check_step(b, copy(s), gr, i, step=3, seed=1, lr=0.02, b1=betas[0], b2=betas[1], eps=1e-5, optim=optim)


@gpu
def test_mixed_list_of_many_tensors(optim):
    """More tensors than a launch takes, of all kinds, some without values."""
    made = [make((1 + 37 * i % 300,) if i % 50 else (0, 3), *((F32, F32, 32, False), (BF, F32, 8, False), (BF, BF, 32, True), (F32, BF, 8, False))[i % 4], i, optim)
            for i in range(1001)]
    sets, grads = [x[0] for x in made], [x[1] for x in made]
    before = [copy(b) for b in sets]
    opt = take(optim, sets, grads, seed=5, steps=41)
    opt.step(grads, lr=0.01)
    assert int(opt.steps) == 42 and int(opt._ticket) == 0
    for i, (b, s, gr) in enumerate(zip(before, sets, grads)):
        if gr.numel():
            check_step(b, copy(s), gr, i, step=42, seed=5, lr=0.01, optim=optim)
    empty = optim.AdamW([torch.empty(0, device="cuda")])
    empty.step([torch.empty(0, device="cuda")])
    assert int(empty.steps) == 1


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_first_steps_from_nothing(optim, bits):
    """State of zeros, a gradient of zeros at first, then single values beside much larger ones."""
    p = torch.randn(1000, generator=gen(1)).cuda()
    opt = optim.AdamW([p], lr=LR, bits=bits, weight_decay=0.0)
    was = p.clone()
    opt.step([torch.zeros(1000, device="cuda")])
    assert torch.equal(p, was)  # 0 / (0 + eps)
    assert all((t.view(torch.uint8) == 0).all() for t in opt.state[0])
    g = torch.full((1000,), 1e-12, device="cuda")
    g[::128] = 100.0
    for _ in range(20):
        was = p.clone()
        opt.step([g])
        # every update is a quotient of the value's own moments: at most lr / bc1 * |m| / r, and 8-bit moments are
        # kept in proportion or, under the block's range, with an r that is too large
        assert ((p - was).abs() <= 2 * LR * 8).all() and torch.isfinite(p).all()


@gpu
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_skipped_where_the_factor_is_not_finite(optim, bad):
    made = [make((3000,), BF, F32, b, False, b, optim) for b in (8, 32)]
    sets, grads = [x[0] for x in made], [x[1] for x in made]
    before = [copy(b) for b in sets]
    opt = take(optim, sets, grads, steps=5)
    grads[1][7] = bad
    norm, factor, ws = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), optim.grad_norm_workspace(grads)
    optim.grad_norm(grads, norm, ws, 1.0, factor)
    assert not torch.isfinite(norm) and torch.isnan(factor)
    for f in (factor, torch.tensor([bad], device="cuda")):
        opt.step(grads, grad_factor=f)
        for b, s in zip(before, sets):
            a = copy(s)
            assert torch.equal(a[0], b[0]) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[2], b[2]))
        assert int(opt.steps) == 5
    grads[1][7] = 0
    optim.grad_norm(grads, norm, ws, 1.0, factor)
    opt.step(grads, grad_factor=factor)
    assert int(opt.steps) == 6 and not torch.equal(sets[0][0].cpu(), before[0][0])


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_a_value_that_is_not_finite_stays_in_its_block(optim, bits):
    (p, w, st), g = make((1024,), F32, F32, bits, False, 3, optim)
    g[130], g[700] = float("inf"), float("nan")
    opt = take(optim, [(p, w, st)], [g])
    opt.step([g])
    hit = {130, 700} if bits == 32 else set(range(128, 256)) | set(range(640, 768))
    m, v = optim.moments(opt.state[0])
    bad = set(torch.nonzero(~torch.isfinite(m)).view(-1).tolist()) | set(torch.nonzero(~torch.isfinite(v)).view(-1).tolist())
    assert bad == hit
    assert set(torch.nonzero(~torch.isfinite(p)).view(-1).tolist()) == {130, 700}  # inf / inf


@gpu
def test_captured_step_goes_on(optim):
    """A replayed step counts, draws other words and reads lr; two graphs with a clip each, on another stream."""
    runs = []
    for captured in (False, True):
        torch.manual_seed(0)
        made = [make((5000,), BF, F32, 8, False, 7, optim), make((333,), F32, F32, 32, False, 8, optim)]
        sets, grads = [x[0] for x in made], [x[1] for x in made]
        lr = torch.tensor([1e-2], device="cuda")
        opt = take(optim, sets, grads, seed=9)
        norm, factor, ws = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), optim.grad_norm_workspace(grads)

        def once():
            optim.grad_norm(grads, norm, ws, 0.01, factor)
            opt.step(grads, lr=lr, grad_factor=factor)
        if captured:
            g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.graph(g):
                once()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                for k in range(4):
                    lr.fill_(1e-2 / (k + 1))
                    g.replay()
            s.synchronize()
        else:
            for k in range(4):
                lr.fill_(1e-2 / (k + 1))
                once()
        assert int(opt.steps) == 4
        runs.append([copy(b) for b in sets])
    for a, b in zip(*runs):
        assert torch.equal(a[0], b[0]) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[2], b[2]))


@gpu
def test_small_moments_reach_the_right_value(optim):
    """v of a gradient that is held: b2 = 0.9 and 200 steps of constant g.  Each step moves v by a tenth, a step of e4m3 is
    an eighth of r, a quarter of v: per value the standard deviation is at most 0.25 v / sqrt(0.19) = 0.57 v of one
    step's rounding summed with weights 0.9^i, and of 65536 independent values' mean at most 0.57 / 256 = 0.23 %.  5 of
    them allowed, and 0.9^200 = 7e-10 of the start left."""
    g = torch.linspace(0.5, 1.0, 65536, device="cuda") * 1e-3
    opt = optim.AdamW([torch.zeros(65536, device="cuda")], betas=(0.9, 0.9), bits=8, seed=1)
    for _ in range(200):
        opt.step([g])
    m, v = optim.moments(opt.state[0])
    assert abs(float((v.double() / g.double().square()).mean()) - 1) < 5 * 0.0023
    assert abs(float((m.double() / g.double()).mean()) - 1) < 5 * 0.0023


@gpu
@pytest.mark.parametrize("ptype, master, bits", KINDS)
@pytest.mark.parametrize("gtype", [F32, BF])
def test_a_step_is_the_same_every_time_and_wherever_the_arrays_lie(optim, ptype, master, bits, gtype):
    """Whole vectors and single values; a list that takes one launch and one that takes three, with the tensor at one place in it."""
    results = []
    for offset, others in ((0, 0), (0, 900), (1, 0)):
        made = [make((9001,), ptype, gtype, bits, master, 7, optim, offset), make((2 ** 20,), ptype, gtype, bits, master, 8, optim, offset)]
        more = [make((5,), BF, F32, 8, False, 9, optim) for _ in range(others)]
        opt = take(optim, [x[0] for x in made + more], None, seed=3)
        for _ in range(3):
            opt.step([x[1] for x in made + more])
        results.append([copy(x[0]) for x in made])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a[0], b[0]) and (a[1] is None or torch.equal(a[1], b[1]))
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[2], b[2]))


@gpu
def test_a_step_is_the_same_again(optim):
    results = []
    for _ in range(2):
        made = [make((9000,), BF, F32, 8, False, 7, optim), make((2 ** 20,), BF, F32, 8, False, 8, optim)]
        opt = take(optim, [x[0] for x in made], None, seed=3)
        for _ in range(3):
            opt.step([x[1] for x in made])
        results.append([copy(x[0]) for x in made])
    for a, b in zip(*results):
        assert torch.equal(a[0], b[0]) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[2], b[2]))


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_more_values_than_32_bits_count(optim, bits):
    """The end of a tensor of 2^32 + 5000 values, and its beginning."""
    n = 2 ** 32 + 5000
    if torch.cuda.mem_get_info()[0] < n * 14:
        pytest.skip("not enough memory")
    p, g = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    opt = optim.AdamW([p], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.01, bits=bits, steps=3, seed=11)
    parts = []
    for first in (0, 2 ** 31 - 4096, 2 ** 32 - 4096, n - 5000 // 128 * 128 - 8):
        m = min(4096, n - first)
        (pp, _, st), gg = make((m,), BF, BF, bits, False, first % 97, optim)
        first = first // 128 * 128
        sl = slice(first, first + m)
        p[sl], g[sl] = pp, gg
        views = [t[first // 128:first // 128 + -(-m // 128)] if t.dtype == torch.float8_e8m0fnu else t[sl] for t in opt.state[0]]
        for v, t in zip(views, st):
            v.view(torch.uint8).copy_(t.view(torch.uint8))
        parts.append((first, (p[sl], None, tuple(views)), copy((p[sl], None, tuple(views))), g[sl]))
    opt.step([g])
    for first, after, before, gr in parts:
        check_step(before, copy(after), gr, 0, step=4, seed=11, optim=optim, first=first)
    assert int(torch.count_nonzero(p[8192:2 ** 31 - 8192])) == 0
    norm = torch.zeros(1, device="cuda")
    optim.grad_norm([g], norm, optim.grad_norm_workspace([g]))
    want = sum(float(x[3].double().square().sum()) for x in parts) ** 0.5
    assert abs(float(norm) - want) <= 1e-6 * want


@gpu
def test_two_steps_at_once_and_a_given_stream(optim):
    """Two optimisers on two streams give what they give one after the other."""
    results = []
    for streams in ((None, None), (torch.cuda.Stream(), torch.cuda.Stream())):
        made = [[make((200_001,), BF, F32, 8, False, 20 + j, optim), make((3000,), F32, F32, 32, False, 30 + j, optim)] for j in range(2)]
        opts = [take(optim, [x[0] for x in mm], None, seed=j) for j, mm in enumerate(made)]
        torch.cuda.synchronize()
        for _ in range(10):
            for o, mm, s in zip(opts, made, streams):
                o.step([x[1] for x in mm], stream=s)
        torch.cuda.synchronize()
        assert [int(o.steps) for o in opts] == [10, 10]
        results.append([copy(x[0]) for mm in made for x in mm])
    for a, b in zip(*results):
        assert torch.equal(a[0], b[0]) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[2], b[2]))


@gpu
@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
def test_example_trains_with_it(optimizer):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.main(["train", "--tokens", "96", "--layers", "2", "--d", "128", "--experts", "4", "--hidden", "128", "--steps", "3", "--optimizer", optimizer,
                     "--clip", "1.0"])
    assert len(losses) == 3 and all(np.isfinite(v) for v in losses)


# ------------------------------------------------------------------ the norm

@gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("sizes", [[1], [0], [], [7, 0, 16383, 16384, 16385], [5] * 900, [3_000_001, 12], [40_000_000]])
@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm(optim, dtype, sizes, offset):
    """Each square has one rounding and goes through 4 + 3 + 5 sums in fp32 at most, the rest have 48 bits or more: the sum is
    off by 13 u at most, the norm by half of that and its own rounding."""
    g = torch.Generator(device="cuda").manual_seed(4)
    ts = [(torch.randn(n + offset, generator=g, device="cuda") * 3).to(dtype)[offset:] for n in sizes]
    norm, factor, ws = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), optim.grad_norm_workspace(ts)
    want = float(sum(t.double().square().sum() for t in ts)) ** 0.5
    for most in (1.0, 1e9):
        optim.grad_norm(ts, norm, ws, most, factor)
        assert abs(float(norm) - want) <= 8 * U * want
        assert abs(float(factor) - min(1.0, most / max(want, 1e-300))) <= 10 * U
    optim.grad_norm(ts, norm, ws)
    assert abs(float(norm) - want) <= 8 * U * want


@gpu
def test_grad_norm_is_the_same_every_time(optim):
    ts = [torch.randn(3_000_001, device="cuda"), torch.randn(77, device="cuda").to(BF)]
    seen = set()
    for _ in range(5):
        norm = torch.zeros(1, device="cuda")
        optim.grad_norm(ts, norm, optim.grad_norm_workspace(ts))
        seen.add(float(norm))
    assert len(seen) == 1


@gpu
def test_large_and_small_values(optim):
    for v, want in ((1e18, 1e18 * 10), (1e-15, 1e-14), (2e19, float("inf"))):
        t = [torch.full((100,), v, device="cuda")]
        norm, factor = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        optim.grad_norm(t, norm, optim.grad_norm_workspace(t), 1.0, factor)
        assert float(norm) == want or abs(float(norm) / want - 1) < 1e-5
        assert torch.isnan(factor) == (want == float("inf"))


# ------------------------------------------------------------------ the decay

@gpu
@pytest.mark.parametrize("ptype, master, bits", [(F32, False, 32), (F32, False, 8), (BF, True, 32), (BF, True, 8)])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("lr, wd", [(1e-3, 0.1), (1e-4, 0.01), (1e-5, 0.1), (1e-5, 0.01), (5e-6, 0.01), (1e-6, 0.01), (1.0, 0.3), (1.0, 0.75), (0.5, 3.0), (1e-3, 0.0)])
def test_a_decayed_value_has_one_rounding(optim, ptype, master, bits, offset, lr, wd):
    """p (1 - lr wd) and the update, rounded once: half a step of the result, lr and wd with half a step of fp32 each (2 u of
    the decay), the split of 1 - lr wd (2^-48; 2^-25 where it is below 1 / 2), 30 u of the update as above and two
    more of it and of the decay's second part for their product and sum.  With moments, and with none."""
    (p, w, st), g = make((9001,), ptype, F32, bits, master, 17, optim, offset)
    for still in (False, True):
        if still:
            g.zero_()
            for t in st:
                t.view(torch.uint8).zero_()
        x = np64(w if master else p)
        before = copy((p, w, st))
        m, v = (np64(t) for t in optim.moments(before[2]))
        opt = optim.AdamW([p], lr=lr, betas=(B1, B2), eps=EPS, weight_decay=wd, masters=[w], state=[st], steps=50, seed=2)
        opt.step([g])
        g64 = np64(g)
        mt, v = np.abs(B1 * m) + np.abs((1 - B1) * g64), B2 * v + (1 - B2) * g64 ** 2
        m = B1 * m + (1 - B1) * g64
        den, rate = np.sqrt(v / (1 - B2 ** 51)) + EPS, lr / (1 - B1 ** 51)
        want = x * (1 - lr * wd) - rate * m / den
        half = 2.0 ** -24 * np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))))
        rest = 2.0 ** -25 if lr * wd > 0.5 else 2.0 ** -48
        more = 2 * U * lr * wd * np.abs(x) + 32 * U * rate * mt / den + (rest + 2.0 ** -47) * np.abs(x) + 2.0 ** -149
        got = np64(w if master else p)
        assert (np.abs(got - want) <= half + 1.001 * more).all()
        if master:
            assert torch.equal(p, w.to(BF))


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("wd", [0.0, 0.01, 0.3, 2.0])
@pytest.mark.parametrize("ptype, offset", [(F32, 0), (F32, 1), (BF, 0)])
def test_an_infinite_parameter_stays(optim, bits, wd, ptype, offset):
    """Where 1 - lr wd is above 0; the values beside it change as they would without it."""
    n = 3001
    values, infinite = torch.randn(n, generator=gen(5)).to(ptype), torch.zeros(n, dtype=torch.bool)
    infinite[[3, 200, 2047, 2048, 3000]] = True
    got = []
    for with_it in (True, False):
        p = at_offset(values, offset)
        if with_it:
            p[3], p[200], p[2047], p[2048], p[3000] = (float(s + "inf") for s in "+--+-")
        was = p.clone()
        opt = optim.AdamW([p], lr=0.1, weight_decay=wd, bits=bits, seed=4)
        opt.step([torch.ones(n, device="cuda")])
        if with_it:
            assert torch.equal(p[infinite.cuda()], was[infinite.cuda()])
        got.append(p.cpu())
    assert torch.isfinite(got[1]).all() and torch.equal(got[0][~infinite], got[1][~infinite])


# ------------------------------------------------------------------ large gradients

def below_overflow(v, w, e, sr_r=sr_r):
    """sr_r, but not up to 2^64, whose square fp32 does not hold: 240 of 2^56 is the last value below."""
    r = sr_r(v, w, e)
    return np.where(r >= 2.0 ** 64, 240 * 2.0 ** 56, r)


@gpu
@pytest.mark.parametrize("offset", [0, 1])
def test_a_rounded_v_is_finite_where_v_is(optim, offset, monkeypatch):
    """v in [2.6e38, 3.4e38): in blocks of the factor 2^56 r lies between 224 and 256, the last with a square of 2^128."""
    import sys
    monkeypatch.setattr(sys.modules[__name__], "sr_r", below_overflow)
    n = 4000
    grad = at_offset((torch.linspace(2.6e38, 3.39e38, n, dtype=torch.float64) / 0.999).sqrt().float(), offset)
    grad[1536:2048] *= 1e-3  # blocks of another factor
    p = at_offset(torch.randn(n, generator=gen(1)), offset)
    opt = optim.AdamW([p], lr=LR, betas=(0.3, 1e-3), bits=8, seed=6)
    for step in (1, 2):
        before = copy((p, None, opt.state[0]))
        opt.step([grad])
        after = copy((p, None, opt.state[0]))
        assert all(torch.isfinite(t).all() for t in optim.moments(after[2]))
        check_step(before, after, grad, 0, step=step, seed=6, b1=0.3, b2=1e-3, optim=optim)
        grad.mul_(0.999)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.95), (0.99, 0.999999), (0.3, 0.999)])
def test_gradients_up_to_where_v_overflows(optim, bits, offset, betas, monkeypatch):
    """(1 - b2) g^2 below 3.4e38, g^2 far above it; one block of each size, two steps."""
    import sys
    monkeypatch.setattr(sys.modules[__name__], "sr_r", below_overflow)
    most = 1.8e19 / (1 - betas[1]) ** 0.5  # its square times 1 - b2: 3.24e38
    size = torch.tensor([1.0, 1e10, 1e18, 1.9e19, 3e19, 0.5 * most, 0.98 * most]).repeat_interleave(384)
    p = at_offset(torch.randn(len(size), generator=gen(1)), offset)
    grad = at_offset(size * (torch.rand(len(size), generator=gen(2)) * 0.02 + 0.98) * torch.where(torch.arange(len(size)) % 3 == 0, -1, 1), offset)
    opt = optim.AdamW([p], lr=LR, betas=betas, bits=bits, seed=6)
    for step in (1, 2):
        before = copy((p, None, opt.state[0]))
        if step == 2:
            grad.mul_(0.1)
        opt.step([grad])
        after = copy((p, None, opt.state[0]))
        assert torch.isfinite(p).all() and all(torch.isfinite(t).all() for t in optim.moments(after[2]))
        check_step(before, after, grad, 0, step=step, seed=6, b1=betas[0], b2=betas[1], optim=optim)


# ------------------------------------------------------------------ what all values of a step have in common

@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_all_blocks_of_a_step_take_the_same_number(optim, bits):
    """Moments of zero and gradients of one: every value moves by one number, which hangs on the step's number alone (half as
    many bits of 1 - 0.5^t from one to the next).  The number is raised while a step's thousands of CTAs run."""
    n = 3_000_001
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    opt = optim.AdamW([p], lr=1.0, betas=(0.5, 0.5), weight_decay=0.0, bits=bits)
    for _ in range(20):
        for done in range(12):
            p.zero_(), opt.steps.fill_(done)
            for t in opt.state[0]:
                t.view(torch.uint8).zero_()
            opt.step([g])
            low, high = torch.aminmax(p)
            bc = 1 - 0.5 ** (done + 1)
            assert float(low) == float(high), (done, float(low), float(high))
            assert abs(float(low) + 0.5 / bc / (0.5 / bc) ** 0.5) < 1e-6 and int(opt.steps) == done + 1 and int(opt._ticket) == 0


@gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 50, 1e18, 1.5e19])
def test_grad_norm_of_many_large_values(optim, dtype, offset, size):
    """Squares that fp32 holds, sums that it does not; beside them a tensor that does not show, and one that is not finite.  As
    in test_grad_norm: half of 13 u, and the norm's own rounding."""
    ts = [at_offset((torch.randn(n, generator=gen(n)).clamp(-1.1, 1.1) * size).to(dtype), offset) for n in (77, 8192, 300_001, 5_000_000)]
    ts.insert(2, torch.randn(100_000, device="cuda"))
    norm, factor, ws = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), optim.grad_norm_workspace(ts)
    want = float(sum(t.double().square().sum() for t in ts)) ** 0.5
    optim.grad_norm(ts, norm, ws, 1.0, factor)
    assert abs(float(norm) - want) <= 8 * U * want and abs(float(factor) * want - 1) <= 10 * U
    for bad in (float("nan"), float("inf"), 3e19):
        ts[3][4567] = bad
        optim.grad_norm(ts, norm, ws, 1.0, factor)
        assert not torch.isfinite(norm) and torch.isnan(factor)
