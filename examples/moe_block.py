"""A stack of pre-norm residual MoE blocks,  r <- r + MoE(norm(r)),  served in 8 bits and trained
with 8-bit activation checkpoints.

  python examples/moe_block.py serve     one batch and then single tokens through the stack
  python examples/moe_block.py train     a few steps on a regression target: SGD, or AdamW over all weights in one
                                         call (--optimizer adamw: fp32 masters and moments; adamw8: moments in
                                         8 bits and no masters), with the gradients clipped (--clip)

Serving: each block's norm adds the block before's output to the stream and writes the
normalised rows once in bf16 (the router's input) and once in e4m3 (the experts'); the experts'
weights are quantised once.  Training: bf16 layers; all blocks share one workspace, and each
leaves an 8-bit checkpoint of its pre-activations for the backward pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_routing_grouped_gb300 import fp8, moe, optim  # noqa: E402

DEV = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def new(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def scales(*shape):
    return new(*shape, dtype=torch.uint8).view(E8M0)


class Weights:
    """Random weights of one block, bf16, and the norm's in fp32."""

    def __init__(self, d, E, F, g):
        def draw(*shape, std):
            return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)
        self.norm = torch.ones(d, device=DEV)
        self.router = draw(E, d, std=d ** -0.5)
        self.w1, self.w3 = draw(E, F, d, std=d ** -0.5), draw(E, F, d, std=d ** -0.5)
        self.w2 = draw(E, d, F, std=F ** -0.5)


class Server:
    """The stack for up to T tokens at a time: weights in 8 bits, one workspace for all blocks."""

    def __init__(self, weights, T, d, E, k, F):
        self.T, self.d = T, d
        self.plan = fp8.Fp8MoEPlan(T, d, E, k, F)
        self.ws = self.plan.new_workspace()
        self.blocks = []
        for w in weights:
            q = []
            for m in (w.w1, w.w3, w.w2):
                qm, sm = new(*m.shape, dtype=E4M3), scales(m.shape[0], (m.shape[1] + 127) // 128, fp8.scale_cols(m.shape[2]))
                fp8.quantize_weights(m, qm, sm)
                q += [qm, sm]
            self.blocks.append((w.norm, w.router, q))
        self.r, self.n, self.y = new(T, d), new(T, d), new(T, d)
        self.q, self.s = new(T, d, dtype=E4M3), scales(T, fp8.scale_cols(d))

    def forward(self, x):
        """x [T, d] bf16 -> the stream after the last block."""
        add = None
        self.r.copy_(x)
        for norm, router, q in self.blocks:
            fp8.rmsnorm(self.r, norm, residual=add, residual_out=None if add is None else self.r, out=self.n, q=self.q,
                        scales=self.s)
            self.plan.forward(self.n, self.q, self.s, router, None, *q, self.y, self.ws)
            add = self.y
        return self.r + self.y


class Trainer:
    """The stack in bf16: one training workspace, a checkpoint and a normalised input a block."""

    def __init__(self, weights, T, d, E, k, F):
        self.weights, self.shape = weights, (T, d, E, k, F)
        self.plan = moe.MoEPlan(T, d, E, k, F, training=True)
        self.ws = self.plan.new_workspace()
        self.norm_ws = fp8.rmsnorm_backward_workspace(T, d)
        L = len(weights)
        self.ckpt = [fp8.LayerCheckpoint(self.plan) for _ in range(L)]
        self.r, self.n = [new(T, d) for _ in range(L)], [new(T, d) for _ in range(L)]
        self.rstd = [new(T, dtype=torch.float32) for _ in range(L)]
        self.y = new(T, d)

    def forward(self, x):
        add = None
        for i, w in enumerate(self.weights):
            src = x if i == 0 else self.r[i - 1]
            fp8.rmsnorm(src, w.norm, residual=add, residual_out=None if add is None else self.r[i], out=self.n[i],
                        rstd=self.rstd[i])
            if add is None:
                self.r[i].copy_(x)
            self.plan.forward(self.n[i], w.router, None, w.w1, w.w3, w.w2, self.y, self.ws)
            self.ckpt[i].save(self.ws)
            add = self.y
        return self.r[-1].float() + self.y.float()

    def backward(self, dout, aux_weight=0.0):
        """Gradients of every block's weights, last block first, from the gradient of the stream's end."""
        T, d, E, k, F = self.shape
        f32 = torch.float32
        dr = dout.to(torch.bfloat16)  # the gradient that reaches the stream
        grads = []
        for i in reversed(range(len(self.weights))):
            w = self.weights[i]
            g = dict(n=new(T, d, dtype=f32), router=new(E, d, dtype=f32), w1=new(E, F, d, dtype=f32),
                     w3=new(E, F, d, dtype=f32), w2=new(E, d, F, dtype=f32), norm=new(d, dtype=f32))
            self.ckpt[i].restore(self.n[i], self.ws)
            self.plan.backward(self.n[i], w.router, None, w.w1, w.w3, w.w2, dr, aux_weight, g["n"], g["router"], None,
                               g["w1"], g["w3"], g["w2"], self.ws)
            nxt = new(T, d)
            fp8.rmsnorm_backward(g["n"], self.r[i], w.norm, self.rstd[i], nxt, g["norm"], self.norm_ws, dresidual=dr)
            dr = nxt
            grads.append(g)
        return grads[::-1], dr


NAMES = ("router", "w1", "w3", "w2", "norm")


class Adam:
    """AdamW over the weights of all blocks: one call for the gradients' norm, one for the step."""

    def __init__(self, weights, lr, bits, clip):
        params = [getattr(w, n) for w in weights for n in NAMES]
        wide = [n == "norm" for _ in weights for n in NAMES]  # norms: fp32, moments in 32 bits, no decay
        self.opt = optim.AdamW(params, lr=lr, weight_decay=[0.0 if n else 0.01 for n in wide], bits=[32 if n else bits for n in wide],
                               masters=[p.float() if bits == 32 and not n else None for p, n in zip(params, wide)])
        self.clip, self.ws = clip, optim.grad_norm_workspace(params)
        self.norm, self.factor = (torch.zeros(1, device=DEV) for _ in range(2))

    def step(self, grads):
        g = [gr[n] for gr in grads for n in NAMES]
        if self.clip:
            optim.grad_norm(g, self.norm, self.ws, max_norm=self.clip, factor=self.factor)
        self.opt.step(g, grad_factor=self.factor if self.clip else None)


def serve(a):
    g = torch.Generator(device=DEV).manual_seed(0)
    ws = [Weights(a.d, a.experts, a.hidden, g) for _ in range(a.layers)]
    x = torch.randn(a.tokens, a.d, generator=g, device=DEV).to(torch.bfloat16)
    batch = Server(ws, a.tokens, a.d, a.experts, a.k, a.hidden).forward(x).clone()
    one = Server(ws, 1, a.d, a.experts, a.k, a.hidden)
    rows = [one.forward(x[t:t + 1]).clone() for t in range(min(4, a.tokens))]
    off = max(float((r - batch[t]).norm() / batch[t].norm()) for t, r in enumerate(rows))
    print(f"served {a.tokens} tokens through {a.layers} blocks; single tokens differ from the batch by {off:.2e} (2-norm)")
    return off


def train(a):
    g = torch.Generator(device=DEV).manual_seed(0)
    ws = [Weights(a.d, a.experts, a.hidden, g) for _ in range(a.layers)]
    x = torch.randn(a.tokens, a.d, generator=g, device=DEV).to(torch.bfloat16)
    target = torch.randn(a.tokens, a.d, generator=g, device=DEV)
    t = Trainer(ws, a.tokens, a.d, a.experts, a.k, a.hidden)
    adam = None if a.optimizer == "sgd" else Adam(ws, a.lr, 8 if a.optimizer == "adamw8" else 32, a.clip)
    losses = []
    for _ in range(a.steps):
        out = t.forward(x)
        diff = out - target
        losses.append(float(0.5 * diff.square().sum(1).mean()))
        grads, _ = t.backward(diff / a.tokens)
        if adam:
            adam.step(grads)
            continue
        for w, gr in zip(ws, grads):
            for name in NAMES:
                p = getattr(w, name)
                p.copy_((p.float() - a.lr * gr[name]).to(p.dtype))
    print(f"loss over {a.steps} steps: {losses[0]:.4f} -> {losses[-1]:.4f}; checkpoint {t.ckpt[0].data.numel() / 2**20:.1f} MiB "
          f"a block, workspace {t.ws.numel() / 2**20:.1f} MiB for all")
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("what", choices=("serve", "train"))
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--k", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--optimizer", choices=("sgd", "adamw", "adamw8"), default="sgd")
    ap.add_argument("--lr", type=float, help="0.2 with SGD, 0.001 with AdamW")
    ap.add_argument("--clip", type=float, default=0.0, help="AdamW: the most that the gradients' norm may be; 0: any")
    a = ap.parse_args(argv)
    if a.lr is None:
        a.lr = 0.2 if a.optimizer == "sgd" else 1e-3
    return serve(a) if a.what == "serve" else train(a)


if __name__ == "__main__":
    main()
