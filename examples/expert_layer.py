"""A mixture-of-experts layer in block-scaled 8 bits, trained on synthetic data.

    python examples/expert_layer.py [--tokens 4096 --hidden 1024 --width 512
                                     --experts 16 --choices 2 --steps 30]

Every product of the experts runs on MXFP8 operands (e4m3, gradients e5m2),
and between the two products the layer keeps gate and up values only in 8
bits for the backward pass.  A step is

  forward   route -> order of rows -> gather -> W1 -> gated activation -> W2
            -> weighted sum back
  backward  the weights' gradient -> gather of the weighted gradient -> W2^T,
            dW2 -> the activation's gradient from its checkpoint -> W1^T, dW1
            -> sum back -> the router's gradient

with no value read back to the host in between: segment sizes stay on the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import block_scaled_precision_blockwise_amd as bsq

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu


def _mx(shape, dtype=E4M3):
    """Empty codes of `shape` and their scales, one per 32 along the last axis."""
    return (torch.empty(shape, dtype=dtype, device="cuda"),
            torch.empty(*shape[:-1], shape[-1] // 32, dtype=E8M0, device="cuda"))


def quantize(x, dtype=E4M3, axis=1):
    """Codes and scales of x [R, C] along its rows, or (axis 0) of its transpose."""
    out = _mx(tuple(x.shape) if axis else tuple(x.shape)[::-1], dtype)
    bsq.bsq_quant_mx(x, *out, axis, bsq.BSQ_E5M2 if dtype == E5M2 else bsq.BSQ_E4M3)
    return out


class ExpertLayer:
    """out[t] = sum over t's choices j of weight_j W2_e (silu(g) u), [g | u] = W1_e x_t.

    Weights are kept in float32 and laid out in 8 bits, both ways round, by
    `lay_out`, once after each update.  Buffers are sized for `tokens`."""

    def __init__(self, tokens, hidden, width, experts, choices, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5  # noqa: E731
        self.T, self.H, self.F, self.E, self.k = tokens, hidden, width, experts, choices
        self.router = new(experts, hidden)
        self.w1, self.w2 = new(experts, 2 * width, hidden), new(experts, hidden, width)
        # segments start at multiples of 128 rows, as the weight gradients need them
        self.cap = bsq.bsq_moe_capacity(tokens * choices, experts, 128)
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.ids, self.pos = i32(tokens, choices), i32(tokens, choices)
        self.offsets, self.counts, self.rows = i32(experts + 1), i32(experts), i32(self.cap)
        self.space = torch.empty(bsq.bsq_moe_plan_workspace_bytes(tokens * choices, experts), dtype=torch.uint8,
                                 device="cuda")
        self.weights = torch.empty(tokens, choices, device="cuda")
        self.lay_out()

    def lay_out(self):
        E, H, F = self.E, self.H, self.F
        both = lambda w: (quantize(w.reshape(-1, w.shape[2])),  # noqa: E731
                          quantize(w.transpose(1, 2).reshape(-1, w.shape[1])))
        view = lambda q, n, m: (q[0].view(E, n, m), q[1].view(E, n, m // 32))  # noqa: E731
        a, at = both(self.w1)
        b, bt = both(self.w2)
        self.q1, self.q1t = view(a, 2 * F, H), view(at, H, 2 * F)
        self.q2, self.q2t = view(b, H, F), view(bt, F, H)

    def forward(self, x):
        """x [T, H] bfloat16 -> out [T, H]; keeps what `backward` reads."""
        T, H, F, cap = self.T, self.H, self.F, self.cap
        bf16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x = x
        self.logits = x.float() @ self.router.t()
        bsq.bsq_moe_route(self.logits, self.ids, self.weights)
        bsq.bsq_moe_plan(self.ids, self.offsets, self.counts, self.rows, self.pos, self.space, align=128)
        # the first product takes its rows from the tokens' codes by `rows`; the
        # ordered and transposed copy is for dW1
        xq = quantize(x)
        self.xt = _mx((H, cap))
        bsq.bsq_moe_gather_mx(x, self.rows, self.k, codes_t=self.xt[0], scales_t=self.xt[1])
        gu = bf16(cap, 2 * F)
        bsq.bsq_moe_matmul(*xq, *self.q1, self.offsets, gu, rows=self.rows, k=self.k)
        h, self.ht, self.kept = _mx((cap, F)), _mx((F, cap)), _mx((cap, 2 * F))
        bsq.bsq_swiglu_mx(gu, *h, *self.ht, *self.kept)
        self.y = bf16(cap, H)
        bsq.bsq_moe_matmul(*h, *self.q2, self.offsets, self.y)
        out = bf16(T, H)
        bsq.bsq_moe_combine(self.y, self.pos, out, weights=self.weights)
        return out

    def backward(self, dout):
        """Gradients (x, router, w1, w2) of dout [T, H] bfloat16."""
        T, H, F, cap = self.T, self.H, self.F, self.cap
        bf16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        dweights = torch.empty(T, self.k, device="cuda")
        bsq.bsq_moe_combine_backward(self.y, self.pos, dout, dweights)
        dy, dyt = _mx((cap, H), E5M2), _mx((H, cap), E5M2)
        bsq.bsq_moe_gather_mx(dout, self.rows, self.k, *dy, *dyt, weights=self.weights)
        dh = bf16(cap, F)
        bsq.bsq_moe_matmul(*dy, *self.q2t, self.offsets, dh)
        dw2 = torch.empty_like(self.w2)
        bsq.bsq_moe_wgrad(*dyt, *self.ht, self.offsets, dw2)
        dgu = bf16(cap, 2 * F)
        bsq.bsq_swiglu_mx_backward(*self.kept, dh, dgu)
        dxr = bf16(cap, H)
        bsq.bsq_moe_matmul(*quantize(dgu, E5M2), *self.q1t, self.offsets, dxr)
        dw1 = torch.empty_like(self.w1)
        bsq.bsq_moe_wgrad(*quantize(dgu, E5M2, axis=0), *self.xt, self.offsets, dw1)
        dx = bf16(T, H)
        bsq.bsq_moe_combine(dxr, self.pos, dx)
        dlogits = torch.empty_like(self.logits)
        bsq.bsq_moe_route_backward(self.logits, self.ids, dweights, dlogits)
        dx = dx.float() + dlogits @ self.router
        return dx, dlogits.t() @ self.x.float(), dw1, dw2

    def update(self, grads, rate):
        """A step of `rate` times each weight's norm down its gradient."""
        for w, g in zip((self.router, self.w1, self.w2), grads[1:]):
            w.sub_(g * (rate * w.norm() / g.norm().clamp_min(1e-30)))
        self.lay_out()


def plain(layer, x):
    """The layer in float32 with autograd, on the layer's choices."""
    ids = layer.ids.long()
    p = torch.softmax(x @ layer.router.t(), 1).gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        g, u = (x[t] @ layer.w1[e].t()).chunk(2, 1)
        out = out.index_add(0, t, p[t, j, None] * ((torch.nn.functional.silu(g) * u) @ layer.w2[e].t()))
    return out


def train(tokens=4096, hidden=1024, width=512, experts=16, choices=2, steps=30, rate=0.02, say=print):
    """Fits the layer to another one's outputs; returns the losses."""
    layer = ExpertLayer(tokens, hidden, width, experts, choices, seed=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    target = ExpertLayer(tokens, hidden, width, experts, choices, seed=2).forward(x).float()
    losses = []
    for step in range(steps):
        out = layer.forward(x).float()
        err = out - target
        losses.append(err.square().mean())
        layer.update(layer.backward((err / tokens).bfloat16()), rate)
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {float(losses[-1]):.5f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, v in (("tokens", 4096), ("hidden", 1024), ("width", 512), ("experts", 16), ("choices", 2), ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=v)
    train(**vars(ap.parse_args()))
