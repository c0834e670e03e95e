"""What is measured of the operators between an expert stage and a training step, and their plain forms.

  dispatch     rows sorted by expert: idx[T, k] gives each token's experts (a value outside [0, E): that
               slot has no row here).  Counts for each expert, each slot's row (stable in slot order, -1
               where it has none), each row's slot, and the tokens' rows and gates in that order
  combine      the way back: out[t] = residual[t] + sum_j gates[t, j] * y[row of (t, j)]; without gates it is
               the gradient of the dispatch
  combine_bwd  its gradient: the rows gates[t, j] * dout[t] in sorted order, and <dout[t], y[row]> for the gates
  adamw        one step over many tensors, in place: moments in fp32, or in 8 bits as m and r = sqrt(v) in
               e4m3 with a power-of-two factor (an e8m0 byte) for 128 consecutive values; bf16 parameters
               with an fp32 master or without.  What is rounded to 8 bits, and a bf16 parameter without
               a master, is rounded up or down by a random number: a hash of seed, step, tensor and index
  grad_norm    the norm of all gradients together and the factor that clips it

Sizes are those of the listed layers (top_routing_grouped_gb300/workloads.py) or generic.
"""
import math

import torch

own = False

DEV = "cuda"
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TYPES = {"bf16": BF, "f32": F32, "e4m3": F8, "i32": torch.int32, "i64": torch.int64}
LR, B1, B2, EPS, DECAY, CLIP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token of large_e64, its 8-bit row to four experts: latency
        dict(name="dispatch_token_e64", op="dispatch", T=1, k=4, E=64, d=4096, dtype="e4m3", idx="i32", skew=0.0, drop=0.0, pad=0),
        # a ragged batch over skewed_e128's experts, half of them on another rank, an odd width out of a wider buffer
        dict(name="dispatch_ragged_e128", op="dispatch", T=1029, k=8, E=128, d=2050, dtype="bf16", idx="i64", skew=1.0, drop=0.5, pad=14),
        # every token of large_e64
        dict(name="dispatch_large_e64", op="dispatch", T=32768, k=4, E=64, d=4096, dtype="bf16", idx="i32", skew=0.05, drop=0.0, pad=0),
        # a handful of decoded tokens of fine_e32
        dict(name="combine_13x2048", op="combine", T=13, k=8, E=32, d=2048, dtype="bf16", out="bf16", gates=True, residual=True, drop=0.0, skew=0.0),
        # every token of large_e64, back into the stream
        dict(name="combine_large_e64", op="combine", T=32768, k=4, E=64, d=4096, dtype="bf16", out="bf16", gates=True, residual=True, drop=0.0, skew=0.05),
        # a short odd batch of fine-tuning in fp32, some slots over their expert's capacity
        dict(name="combine_bwd_f32_777x1000", op="combine_bwd", T=777, k=2, E=8, d=1000, dtype="f32", dout="f32", drop=0.1, skew=0.3),
        # the training step of fine_e32: the layer's backward hands over dout in fp32
        dict(name="combine_bwd_fine_e32", op="combine_bwd", T=8192, k=8, E=32, d=2048, dtype="bf16", dout="f32", drop=0.0, skew=0.0),
        # twelve small blocks of odd widths (60 tensors), clipped: latency
        dict(name="adamw_12_small_blocks", op="adamw", layers=12, d=200, E=4, F=131, param="bf16", grad="f32", bits=32, master=True, clip=True, step=7),
        # the weights of coarse_e8, moments in fp32, fp32 masters
        dict(name="adamw_coarse_e8", op="adamw", layers=1, d=2048, E=8, F=8192, param="bf16", grad="f32", bits=32, master=True, clip=False, step=1000),
        # the weights of two layers of fine_e32, moments in 8 bits, no masters
        dict(name="adamw_8bit_fine_e32", op="adamw", layers=2, d=2048, E=32, F=2048, param="bf16", grad="f32", bits=8, master=False, clip=False, step=1000),
        # the gradients of a few small blocks, ragged
        dict(name="grad_norm_small", op="grad_norm", layers=3, d=264, E=4, F=513, grad="bf16"),
        # the gradients of coarse_e8 as its backward gives them
        dict(name="grad_norm_coarse_e8", op="grad_norm", layers=1, d=2048, E=8, F=8192, grad="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "combine", "combine", "combine_bwd", "combine_bwd", "adamw", "adamw", "grad_norm"])
    while True:
        if op in ("adamw", "grad_norm"):
            c = dict(op=op, layers=_log(rng, 1, 100), d=_log(rng, 16, 4096), E=rng.choice([1, 4, 8, 32, 64]), F=_log(rng, 16, 8192))
            if rng.random() < 0.7:
                c["d"], c["F"] = -(-c["d"] // 8) * 8, -(-c["F"] // 8) * 8
            if c["layers"] * c["E"] * c["d"] * c["F"] > 32 * 2048 * 2048:
                continue
            c["grad"] = rng.choice(["f32", "f32", "bf16"])
            if op == "adamw":
                c["param"] = rng.choice(["bf16", "bf16", "f32"])
                c["bits"] = rng.choice([8, 32])
                c["master"] = c["param"] == "bf16" and rng.random() < 0.5
                c["clip"], c["step"] = rng.random() < 0.4, _log(rng, 1, 100000) - 1
            return c
        E = rng.choice([1, 4, 8, 32, 60, 64, 128, 256])
        c = dict(op=op, T=_log(rng, 1, 32768), k=rng.choice([1, 2, 4, 6, 8, 16]), E=E, d=_log(rng, 16, 8192),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 0.3, 1.0]), drop=rng.choice([0.0, 0.0, 0.1, 0.75]))
        if rng.random() < 0.7:
            c["d"] = -(-c["d"] // 16) * 16
        if c["k"] > E or c["T"] * c["k"] * c["d"] > 32768 * 4 * 2048:
            continue
        if c["T"] * c["k"] < 16:
            c["drop"] = 0.0
        if op == "dispatch":
            c["dtype"], c["idx"] = rng.choice(["bf16", "bf16", "f32", "e4m3"]), rng.choice(["i32", "i64"])
            c["pad"] = rng.choice([0, 0, 16, 6]) if c["dtype"] != "e4m3" else 0
        elif op == "combine":
            c["out"], c["gates"], c["residual"] = rng.choice([c["dtype"], "f32"]), rng.random() < 0.7, rng.random() < 0.5
        else:
            c["dout"] = rng.choice([c["dtype"], "f32"])
        return c


def scale_cols(k):
    """Scale bytes of a row of k values: one for each block of 128, in whole words of four."""
    return (k + 511) // 512 * 4


def _shapes(c):
    """The tensors of a stack of blocks: norm, router and the three matrices of every expert, layer by layer."""
    d, E, F = c["d"], c["E"], c["F"]
    return [(d,), (E, d), (E, F, d), (E, F, d), (E, d, F)] * c["layers"]


def _kinds(c):
    """(shape, parameter's type, bits of its moments, whether it has a master, weight decay): norms stay in fp32."""
    return [((s), F32, 32, False, 0.0) if len(s) == 1 else (s, TYPES[c["param"]], c["bits"], c["master"], DECAY) for s in _shapes(c)]


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1, "i32": 4, "i64": 8}
    if op in ("adamw", "grad_norm"):
        if op == "grad_norm":
            n = sum(math.prod(s) for s in _shapes(c))
            return {"bytes": n * size[c["grad"]] + 8, "flops": 2 * n}
        total = 0
        for s, t, bits, master, _ in _kinds(c):
            n = math.prod(s)
            total += n * ((2 + 8 if master else 2 * (2 if t is BF else 4)) + size[c["grad"]]) + (16 * n if bits == 32 else 4 * n + 4 * -(-n // 128))
        return {"bytes": total, "flops": 16 * sum(math.prod(s) for s in _shapes(c))}
    N, d, e = c["T"] * c["k"], c["d"], size[c["dtype"]]
    rows = N * (1 - c["drop"])
    if op == "dispatch":
        row = d * e + (scale_cols(d) if c["dtype"] == "e4m3" else 0)
        return {"bytes": N * (size[c["idx"]] + 4 + 4 + 4) + 4 * c["E"] + 4 * rows + (c["T"] + rows) * row, "flops": N}
    if op == "combine":
        o = size[c["out"]]
        return {"bytes": N * (8 if c["gates"] else 4) + rows * d * e + c["T"] * d * o * (2 if c["residual"] else 1), "flops": 2 * rows * d}
    return {"bytes": N * 12 + 2 * rows * d * e + c["T"] * d * size[c["dout"]], "flops": 3 * rows * d}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=F32) * std).to(dtype)


def _choice(g, c):
    """Each token's k different experts, a Zipf-like share for each, and dropped slots as -1 or E."""
    T, k, E = c["T"], c["k"], c["E"]
    rank = torch.randperm(E, generator=g, device=DEV)
    like = -c["skew"] * torch.log(rank.to(F32) + 1) - torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    idx = like.topk(k, 1).indices
    gone = torch.rand(T, k, generator=g, device=DEV) < c["drop"]
    return torch.where(gone, torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.5, -1, E), idx)


def _power(amax):
    """The least e with amax <= 448 * 2^e, as the scale's byte e + 127; 0 for a block of zeros."""
    m, x = torch.frexp(amax)
    b = (x - 9 + (m > 0.875).int() + 127).clamp(0, 254)
    return torch.where(amax == 0, torch.zeros_like(b), b)


def _blocks(v):
    """A tensor's values in blocks of 128 consecutive ones, the last filled up with zeros."""
    v = v.reshape(-1)
    return torch.nn.functional.pad(v, (0, -v.numel() % 128)).view(-1, 128)


def _quantize(v):
    """fp32 values -> e4m3 of the same shape and a scale for every 128 consecutive ones."""
    w = _blocks(v)
    b = _power(w.abs().amax(1))
    q = torch.ldexp(w, (127 - b).unsqueeze(1)).reshape(-1)[: v.numel()].view(v.shape).to(F8)
    return q, b.to(torch.uint8).view(E8)


def _factors(s):
    e = s.view(torch.uint8).int() - 127
    return torch.ldexp(torch.ones_like(e, dtype=F32), e)


def _dequantize(q, s):
    return (_blocks(q.to(F32)) * _factors(s).unsqueeze(1)).reshape(-1)[: q.numel()].view(q.shape)


def _pack(tensors, types=None):
    """The tensors as views of one buffer for each type, every one at a multiple of 64 values: (views, buffers)."""
    types = types or [None if t is None else t.dtype for t in tensors]
    at, ends = [], {}
    for t, ty in zip(tensors, types):
        at.append(ends.get(ty, 0))
        ends[ty] = at[-1] if t is None else at[-1] + -(-t.numel() // 64) * 64
    buffers = {ty: torch.zeros(n, device=DEV).to(next(t.dtype for t, u in zip(tensors, types) if u is ty)) for ty, n in ends.items() if n}
    views = [None if t is None else buffers[ty][i:i + t.numel()].view(t.shape) for t, ty, i in zip(tensors, types, at)]
    for v, t in zip(views, tensors):
        if t is not None:
            v.view(torch.uint8).copy_(t.view(torch.uint8))
    return views, list(buffers.values())


def _pack_pairs(pairs):
    """_pack for a list of tensors and (values, scales)."""
    parts = [t if isinstance(t, tuple) else (t, None) for t in pairs]
    (q, bq), (sc, bs) = _pack([x[0] for x in parts]), _pack([x[1] for x in parts])
    return [a if b is None else (a, b) for a, b in zip(q, sc)], bq + bs


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = dict(case=case, seed=seed)
    if op in ("adamw", "grad_norm"):
        gt = TYPES[c["grad"]]
        s["g"] = [_randn(g, *sh, std=2e-3 * (1 + 9 * (i % 5 == 1)), dtype=gt) for i, sh in enumerate(_shapes(c))]
        s["norm"], s["factor"] = (torch.zeros(1, device=DEV) for _ in range(2))
        if op == "adamw":
            s["p"], s["w"], s["m"], s["v"] = [], [], [], []
            for sh, t, bits, master, _ in _kinds(c):
                w = _randn(g, *sh, std=sh[-1] ** -0.5) if len(sh) > 1 else 1 + _randn(g, *sh, std=0.1)
                s["p"].append(w.to(t))
                s["w"].append(w if master else None)
                m, r = _randn(g, *sh, std=5e-4), (_randn(g, *sh).square() * 0.3 + 0.7) * 2e-3
                s["m"].append(_quantize(m) if bits == 8 else m)
                s["v"].append(_quantize(r) if bits == 8 else r.square())
            # a program that saves and loads its state keeps it in a few buffers
            (s["p"], a), (s["w"], b) = _pack(s["p"]), _pack(s["w"])
            (s["m"], m), (s["v"], v) = _pack_pairs(s["m"]), _pack_pairs(s["v"])
            s["kept"] = [*a, *b, *m, *v]
            s["steps"] = torch.full((1,), c["step"], dtype=torch.int64, device=DEV)
        return s
    idx = _choice(g, c)
    T, k, E, d = c["T"], c["k"], c["E"], c["d"]
    s["slot_pos"], s["row_slot"] = (torch.zeros(T, k, dtype=I32, device=DEV), torch.zeros(T * k, dtype=I32, device=DEV))
    s["counts"] = torch.zeros(E, dtype=I32, device=DEV)
    s["gates"] = torch.rand(T, k, generator=g, device=DEV)
    if op == "dispatch":
        s["idx"] = idx.to(TYPES[c["idx"]])
        s["rows"], s["row_gates"] = torch.zeros(T * k, d, device=DEV).to(TYPES[c["dtype"]]), torch.zeros(T * k, device=DEV)
        s["x"] = _randn(g, T, d + c["pad"]).to(TYPES[c["dtype"]])[:, :d]
        if c["dtype"] == "e4m3":
            s["sx"] = torch.randint(118, 122, (T, scale_cols(d)), generator=g, device=DEV, dtype=torch.uint8).view(E8)
            s["srows"] = torch.zeros(T * k, scale_cols(d), dtype=torch.uint8, device=DEV).view(E8)
        return s
    # the rows that a dispatch of this choice has sorted
    s["slot_pos"].copy_(_sorted(idx, E)[1])
    s["y"] = _randn(g, T * k, d, dtype=TYPES[c["dtype"]])
    if op == "combine":
        s["gates"] = s["gates"] if c["gates"] else None
        s["residual"] = _randn(g, T, d, dtype=TYPES[c["out"]]) if c["residual"] else None
        s["out"] = torch.zeros(T, d, dtype=TYPES[c["out"]], device=DEV)
    else:
        s["dout"] = _randn(g, T, d, dtype=TYPES[c["dout"]])
        s["dy"], s["dgates"] = torch.zeros_like(s["y"]), torch.zeros(T, k, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from top_routing_grouped_gb300 import optim, rows

    c, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        if "ws" not in s:  # a user's program keeps it
            s["ws"] = rows.dispatch_workspace(c["T"], c["k"], c["E"])
        rows.dispatch(s["idx"], s["x"], s["counts"], s["slot_pos"], s["rows"], s["ws"], row_slot=s["row_slot"], x_scales=s.get("sx"),
                      row_scales=s.get("srows"), gates=s["gates"], row_gates=s["row_gates"])
        return [s["counts"], s["slot_pos"], s["row_slot"], s["rows"], s.get("srows"), s["row_gates"]]
    if op == "combine":
        rows.combine(s["y"], s["slot_pos"], s["out"], gates=s["gates"], residual=s["residual"])
        return s["out"]
    if op == "combine_bwd":
        rows.combine_backward(s["dout"], s["slot_pos"], s["gates"], y_rows=s["y"], dy_rows=s["dy"], dgates=s["dgates"])
        return [s["dy"], s["dgates"]]
    if "norm_ws" not in s:
        s["norm_ws"] = optim.grad_norm_workspace(s["g"])
    if op == "grad_norm":
        optim.grad_norm(s["g"], s["norm"], s["norm_ws"], max_norm=CLIP, factor=s["factor"])
        return [s["norm"], s["factor"]]
    if "opt" not in s:
        s["opt"] = optim.AdamW(s["p"], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=[k[4] for k in _kinds(c)], masters=s["w"],
                               state=[(*m, *v) if isinstance(m, tuple) else (m, v) for m, v in zip(s["m"], s["v"])], steps=s["steps"], seed=s["seed"])
    if c["clip"]:
        optim.grad_norm(s["g"], s["norm"], s["norm_ws"], max_norm=CLIP, factor=s["factor"])
    s["opt"].step(s["g"], grad_factor=s["factor"] if c["clip"] else None)
    return [*s["kept"], s["steps"], s["norm"]]


def _sorted(idx, E):
    """Counts, each slot's row, each row's slot of a choice of experts."""
    e = idx.reshape(-1).long()
    e = torch.where((e >= 0) & (e < E), e, E)
    counts = torch.bincount(e, minlength=E + 1)[:E]
    order = e.argsort(stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(e < E, rank, -1).view(idx.shape)
    row_slot = torch.where(torch.arange(order.numel(), device=order.device) < counts.sum(), order, -1)
    return counts.to(I32), pos.to(I32), row_slot.to(I32)


WORD = (1 << 32) - 1


def _mix(x):
    """A word's hash, by odd multipliers (the golden ratio's and the roots' of 2 and 3 first 32 bits) and shifts."""
    x = x * 0x9E3779B1 & WORD
    x = (x ^ x >> 16) * 0x6A09E667 & WORD
    x = (x ^ x >> 15) * 0xBB67AE85 & WORD
    return x ^ x >> 16


def _random(n, seed, step, tensor):
    """A 32-bit word for each of a tensor's n values (64-bit integers): a hash for each eight of them, and
    r <- r * A + C from one to the next within the eight."""
    key = _mix((_mix((_mix((_mix(seed & WORD) + (seed >> 32 & WORD)) & WORD) + step) & WORD) + tensor) & WORD)
    r = _mix(torch.arange(-(-n // 8), device=DEV) + key & WORD)
    a, b, steps = 1, 0, []
    for _ in range(8):
        steps.append((a, b))
        a, b = a * 0x3C6EF375 & WORD, b * 0x3C6EF375 + 0xA54FF53B & WORD
    mul, add = torch.tensor(steps, device=DEV).unbind(1)
    return (r[:, None] * mul + add & WORD).view(-1)[:n]


def _round_bf16(v, rnd):
    """To one of the two bf16 neighbours: away from zero where the bits that go, plus 16 random ones, overflow."""
    u = v.reshape(-1).view(I32).long() & WORD
    u = u + torch.where((u >> 23 & 255) == 255, 0, rnd & 0xFFFF) & 0xFFFF0000
    return torch.where(u >> 31 == 1, u - (1 << 32), u).to(I32).view(F32).view(v.shape).to(BF)


def _floor_e4m3(u):
    """The largest e4m3 value at or below u >= 0, and the one after it."""
    step = torch.ldexp(torch.ones_like(u), torch.frexp(u.clamp(min=2.0 ** -6))[1] - 4)
    lo = torch.floor(u / step) * step
    return lo, lo + step


def _round_first(m, rnd):
    """m -> e4m3 and scales, up or down with the probability that keeps the mean."""
    w = _blocks(m)
    b = _power(w.abs().amax(1))
    u = torch.ldexp(w, (127 - b).unsqueeze(1)).reshape(-1)[: m.numel()]
    lo, hi = _floor_e4m3(u.abs())
    q = torch.where((u.abs() - lo) * 65536 + (rnd >> 16) * (hi - lo) >= (hi - lo) * 65536, hi, lo)
    return torch.where(u < 0, -q, q).view(m.shape).to(F8), b.to(torch.uint8).view(E8)


def _round_second(v, rnd):
    """v -> r = sqrt(v) in e4m3 and scales, up or down with the probability that keeps the mean of r^2; never down to 0."""
    r = _blocks(v.sqrt())
    b = _power(r.amax(1))
    by = (127 - b).unsqueeze(1)
    u, u2 = (t.reshape(-1)[: v.numel()] for t in (torch.ldexp(r, by), torch.ldexp(torch.ldexp(_blocks(v), by), by)))
    lo, hi = _floor_e4m3(u)
    up = (u2 - lo * lo) * 65536 > (rnd >> 8 & 0xFFFF) * (hi * hi - lo * lo)
    return torch.where(up | (lo == 0) & (v.reshape(-1) > 0), hi, lo).view(v.shape).to(F8), b.to(torch.uint8).view(E8)


def _grad_norm(s):
    total = torch.stack([t.to(F32).square().sum(dtype=torch.float64) for t in s["g"]]).sum()
    s["norm"].copy_(total.sqrt())
    s["factor"].copy_(CLIP / torch.clamp(total.sqrt(), min=CLIP))


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        counts, pos, row_slot = _sorted(s["idx"], c["E"])
        s["counts"].copy_(counts), s["slot_pos"].copy_(pos), s["row_slot"].copy_(row_slot)
        kept = (pos >= 0).reshape(-1).nonzero().view(-1)
        to, token = pos.view(-1)[kept].long(), kept // c["k"]
        s["rows"].view(torch.uint8)[to] = s["x"].contiguous().view(torch.uint8)[token]
        if "sx" in s:
            s["srows"].view(torch.uint8)[to] = s["sx"].view(torch.uint8)[token]
        s["row_gates"][to] = s["gates"].view(-1)[kept]
        return [s["counts"], s["slot_pos"], s["row_slot"], s["rows"], s.get("srows"), s["row_gates"]]
    if op == "combine":
        at = s["slot_pos"].view(-1).long()
        y = torch.where((at >= 0)[:, None], s["y"][at.clamp(min=0)].to(F32), 0).view(c["T"], c["k"], c["d"])
        out = (y if s["gates"] is None else y * s["gates"][:, :, None]).sum(1)
        s["out"].copy_(out if s["residual"] is None else s["residual"].to(F32) + out)
        return s["out"]
    if op == "combine_bwd":
        kept = (s["slot_pos"].view(-1) >= 0).nonzero().view(-1)
        at, token = s["slot_pos"].view(-1)[kept].long(), kept // c["k"]
        dout = s["dout"].to(F32)[token]
        s["dy"][at] = (s["gates"].view(-1)[kept][:, None] * dout).to(s["dy"].dtype)
        s["dgates"].zero_()
        s["dgates"].view(-1)[kept] = (dout * s["y"][at].to(F32)).sum(1)
        return [s["dy"], s["dgates"]]
    if op == "grad_norm":
        _grad_norm(s)
        return [s["norm"], s["factor"]]
    if c["clip"]:
        _grad_norm(s)
    step = int(s.setdefault("done", c["step"])) + 1
    s["done"] = step
    bc1, bc2 = 1 - B1 ** step, 1 - B2 ** step
    for i, (p, w, gr, (sh, t, bits, master, decay)) in enumerate(zip(s["p"], s["w"], s["g"], _kinds(c))):
        gr = gr.to(F32) * s["factor"] if c["clip"] else gr.to(F32)
        m, v = (_dequantize(*s["m"][i]), _dequantize(*s["v"][i]).square()) if bits == 8 else (s["m"][i], s["v"][i])
        m = B1 * m + (1 - B1) * gr
        v = B2 * v + (1 - B2) * gr * gr
        x = w if master else p.to(F32)
        x = x - LR * decay * x - LR * (m / bc1) / ((v / bc2).sqrt() + EPS)
        if bits == 8 or (t is BF and not master):
            rnd = _random(x.numel(), s["seed"], step, i)
        if bits == 8:
            for kept, new in zip(s["m"][i] + s["v"][i], _round_first(m, rnd) + _round_second(v, rnd)):
                kept.copy_(new)
        else:
            s["m"][i].copy_(m), s["v"][i].copy_(v)
        if master:
            w.copy_(x)
        p.copy_(_round_bf16(x, rnd) if t is BF and not master else x)
    s["steps"] += 1
    return [*s["kept"], s["steps"], s["norm"]]


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_scale(top):
    """2^e, the least with top <= 448 * 2^e, and 2^-127 at least."""
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
    return torch.exp2(torch.where(top == 0, -127.0, e).clamp(-127, 127))


def _exact_words(n, seed, step, tensor):
    def mix(x):
        for mul, shift in ((0x9E3779B1, 16), (0x6A09E667, 15), (0xBB67AE85, 16)):
            x = x * mul % 2 ** 32
            x = x ^ (x // 2 ** shift)
        return x
    key = mix(seed % 2 ** 32)
    for part in (seed // 2 ** 32, step, tensor):
        key = mix((key + part) % 2 ** 32)
    i = torch.arange(n, device=DEV)
    r = mix((torch.div(i, 8, rounding_mode="floor") + key) % 2 ** 32)
    for j in range(1, 8):
        r = torch.where(i % 8 >= j, (r * 0x3C6EF375 + 0xA54FF53B) % 2 ** 32, r)
    return r


def _exact_adamw(c, s, norm, seed):
    step = c["step"] + 1
    f = min(1.0, CLIP / norm) if c["clip"] else 1.0
    ps, ws, ms, vs = [], [], [], []
    for i, (sh, t, bits, master, decay) in enumerate(_kinds(c)):
        g = s["g"][i].double() * f
        if bits == 8:
            m, v = ((q.double().reshape(-1) * sc.double().repeat_interleave(128)[: q.numel()]).view(sh) for q, sc in (s["m"][i], s["v"][i]))
            v = v ** 2
        else:
            m, v = s["m"][i].double(), s["v"][i].double()
        m, v = m + (1 - B1) * (g - m), v + (1 - B2) * (g ** 2 - v)
        x = s["w"][i].double() if master else s["p"][i].double()
        x = x * (1 - LR * decay) - LR * m / (1 - B1 ** step) / (torch.sqrt(v / (1 - B2 ** step)) + EPS)
        words = _exact_words(x.numel(), seed, step, i) if bits == 8 or (t is BF and not master) else None
        if t is BF and not master:
            gap = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126))) - 7)
            part = x.abs() / gap
            lo = torch.floor(part)
            ps.append(torch.sign(x) * gap * (lo + ((part - lo) + (words % 65536).view(sh) / 65536 >= 1)))
        else:
            ps.append(x)
        ws.append(x if master else None)
        if bits == 32:
            ms.append(m), vs.append(v)
            continue
        n, pad = x.numel(), -x.numel() % 128
        for out, val in ((ms, m), (vs, v)):
            root = val if out is ms else val.sqrt()
            sc = _exact_scale(torch.nn.functional.pad(root.reshape(-1).abs(), (0, pad)).view(-1, 128).amax(1))
            each = sc.repeat_interleave(128)[:n].view(sh)
            u = root.abs() / each
            gap = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
            lo = torch.floor(u / gap) * gap
            if out is ms:
                up = (u - lo) / gap + (words // 65536).view(sh) / 65536 >= 1
            else:
                up = (val / each ** 2 - lo ** 2) / ((lo + gap) ** 2 - lo ** 2) > (words // 256 % 65536).view(sh) / 65536
                up = up | ((lo == 0) & (val > 0))
            out.append((torch.sign(root) * torch.where(up, lo + gap, lo), sc))
    kinds = _kinds(c)
    moment = [F8 if k[2] == 8 else F32 for k in kinds]
    kept = _pack(ps, [k[1] for k in kinds])[1] + _pack(ws)[1]
    for moments in (ms, vs):
        parts = [t if isinstance(t, tuple) else (t, None) for t in moments]
        kept += _pack([t[0] for t in parts], moment)[1] + _pack([t[1] for t in parts])[1]
    return [*kept, s["steps"] + 1, torch.full((1,), norm if c["clip"] else 0.0, dtype=torch.float64, device=DEV)]


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("adamw", "grad_norm"):
        norm = math.sqrt(math.fsum(float(torch.dot(t.reshape(-1).double(), t.reshape(-1).double())) for t in s["g"]))
        if op == "grad_norm":
            return [torch.full((1,), v, dtype=torch.float64, device=DEV) for v in (norm, min(1.0, CLIP / norm))]
        return _exact_adamw(c, s, norm, seed)
    T, k, E, d = c["T"], c["k"], c["E"], c["d"]
    if op == "dispatch":
        e = s["idx"].reshape(-1)
        of = [(e == i).nonzero().view(-1) for i in range(E)]
        slots = torch.cat(of)
        n = slots.numel()
        pos, row_slot = torch.full((T * k,), -1, dtype=I32, device=DEV), torch.full((T * k,), -1, dtype=I32, device=DEV)
        pos[slots], row_slot[:n] = torch.arange(n, dtype=I32, device=DEV), slots.to(I32)
        rows, gates = torch.zeros(T * k, d, dtype=torch.float64, device=DEV), torch.zeros(T * k, dtype=torch.float64, device=DEV)
        rows[:n], gates[:n] = s["x"].double()[slots // k], s["gates"].double().view(-1)[slots]
        sc = None
        if "sx" in s:
            sc = torch.full((T * k, scale_cols(d)), 2.0 ** -127, dtype=torch.float64, device=DEV)
            sc[:n] = s["sx"].double()[slots // k]
        return [torch.tensor([v.numel() for v in of], dtype=I32, device=DEV), pos.view(T, k), row_slot, rows, sc, gates]
    has = s["slot_pos"] >= 0
    if op == "combine":
        out = torch.zeros(T, d, dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
        for j in range(k):
            t = has[:, j].nonzero().view(-1)
            y = s["y"][s["slot_pos"][t, j].long()].double()
            out[t] += y if s["gates"] is None else s["gates"][t, j, None].double() * y
        return out
    dy, dg = torch.zeros(T * k, d, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        t = has[:, j].nonzero().view(-1)
        at, dout = s["slot_pos"][t, j].long(), s["dout"][t].double()
        dy[at] = dout * s["gates"][t, j, None].double()
        dg[t, j] = torch.einsum("td,td->t", dout, s["y"][at].double())
    return [dy, dg]
