"""The MLP sublayer of a tensor-parallel transformer block, end to end, on one GPU.

W virtual ranks each hold a slice of the two weight matrices.  A rank computes

    a_r = gelu(x W1_r^T + b1_r)          arx_linear, bias and activation in the epilogue
    p_r = a_r W2_r^T                     arx_linear: the rank's partial

and the sublayer ends with the all-reduce's rank-order sum, fused with what
follows it:

    h = residual + dropout(sum_r p_r + b2),  y = layer_norm(h)      arx_reduce_layer_norm

The training step runs the backward passes (arx_layer_norm_bwd,
arx_dropout_add_bwd, arx_linear_bwd), checks them against a 32-bit torch
reference, and repeats the step to show that every bit is the same.  The
serving part captures the sublayer for a few tokens, without dropout, in a
CUDA graph and replays it.

    python examples/tensor_parallel_mlp.py [--ranks W] [--hidden H] [--tokens T] [--dropout P]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_shot_all_gb300 as arx  # noqa: E402

BF16 = torch.bfloat16


class Sublayer:
    """Weights of W ranks, and the buffers and plans of calls on T tokens."""

    def __init__(self, W: int, hidden: int, tokens: int, p: float, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        inner = 4 * hidden // W  # a rank's share of the inner features

        def normal(*shape, scale=1.0, shift=0.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(BF16)

        self.W, self.hidden, self.tokens, self.inner, self.p = W, hidden, tokens, inner, p
        self.w1 = [normal(inner, hidden, scale=hidden ** -0.5) for _ in range(W)]
        self.b1 = [normal(inner, scale=0.1) for _ in range(W)]
        self.w2 = [normal(hidden, inner, scale=(4 * hidden) ** -0.5) for _ in range(W)]
        self.b2 = normal(hidden, scale=0.1)
        self.gain = normal(hidden, scale=0.1, shift=1.0)
        self.shift = normal(hidden, scale=0.1)
        self.rng = torch.tensor([1234, 0], dtype=torch.int64, device="cuda")  # seed, offset

        new = lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        T = tokens
        self.x = new(T, hidden)          # the sublayer's input and residual stream
        self.z = [new(T, inner) for _ in range(W)]
        self.a = [new(T, inner) for _ in range(W)]
        self.partial = [new(T, hidden) for _ in range(W)]
        self.h, self.y = new(T, hidden), new(T, hidden)
        self.mean, self.rstd = new(T, dtype=torch.float32), new(T, dtype=torch.float32)

        # Gradients: the sublayer's output and residual stream come from above.
        self.dy, self.dh_above = new(T, hidden), new(T, hidden)
        self.dh, self.ds, self.dx = new(T, hidden), new(T, hidden), new(T, hidden)
        self.da = new(T, inner)
        self.dpart = [new(T, hidden) for _ in range(W)]
        self.grads = {"gain": new(hidden), "shift": new(hidden), "b2": new(hidden),
                      "w1": [new(inner, hidden) for _ in range(W)], "b1": [new(inner) for _ in range(W)],
                      "w2": [new(hidden, inner) for _ in range(W)]}
        nbytes = max(arx.arx_layer_norm_bwd_workspace_bytes(T, hidden), arx.arx_dropout_add_bwd_workspace_bytes(T, hidden),
                     arx.arx_linear_bwd_workspace_bytes(T, inner), arx.arx_linear_bwd_workspace_bytes(T, hidden))
        self.ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")

    def forward(self, train: bool = True) -> None:
        for r in range(self.W):
            arx.arx_linear(self.x, self.w1[r], self.a[r], bias=self.b1[r], z=self.z[r] if train else None,
                           act=arx.ARX_ACT_GELU)
            arx.arx_linear(self.a[r], self.w2[r], self.partial[r])
        p = self.p if train else 0.0
        arx.arx_reduce_layer_norm(self.partial, self.h, self.y, bias=self.b2, residual=self.x, weight=self.gain,
                                  norm_bias=self.shift, mean=self.mean if train else None,
                                  rstd=self.rstd if train else None, p=p, rng=self.rng if p else None)

    def backward(self) -> None:
        g = self.grads
        # The norm, joined by the gradient that reaches h along the residual stream.
        arx.arx_layer_norm_bwd(self.dy, self.h, self.mean, self.rstd, self.dh, weight=self.gain,
                               dresidual=self.dh_above, dweight=g["gain"], dbias=g["shift"], workspace=self.ws)
        # Every rank's partial has the same gradient; the mask is regenerated from the same state.
        arx.arx_dropout_add_bwd(self.dh, self.ds, self.p, self.rng, dbias=g["b2"], workspace=self.ws)
        for r in range(self.W):
            arx.arx_linear_bwd(self.ds, self.a[r], self.w2[r], dx=self.da, dw=g["w2"][r])
            arx.arx_linear_bwd(self.da, self.x, self.w1[r], dx=self.dpart[r], dw=g["w1"][r], dbias=g["b1"][r],
                               z=self.z[r], act=arx.ARX_ACT_GELU, workspace=self.ws)
        # The ranks' input gradients are one more rank-order all-reduce; the residual's joins it.
        arx.arx_reduce(self.dpart, self.dx)
        arx.arx_dropout_add(self.dx, self.dx, 0.0, residual=self.dh)

    def outputs(self) -> list:
        g = self.grads
        return [self.h, self.y, self.dx, g["gain"], g["shift"], g["b2"], *g["w1"], *g["b1"], *g["w2"]]


def reference(s: Sublayer) -> list:
    """The same step in 32 bits with torch's automatic differentiation."""
    leaf = lambda t: t.float().detach().requires_grad_()  # noqa: E731
    x, gain, shift, b2 = map(leaf, (s.x, s.gain, s.shift, s.b2))
    w1, b1, w2 = ([leaf(t) for t in ts] for ts in (s.w1, s.b1, s.w2))
    total = sum(torch.nn.functional.gelu(x @ w1[r].t() + b1[r]) @ w2[r].t() for r in range(s.W))
    ones = torch.ones(s.tokens, s.hidden, device="cuda")
    mask = torch.empty_like(ones)  # the generator's mask, scaled, from dropout of ones
    arx.arx_dropout_add(ones, mask, s.p, s.rng)
    h = x + (total + b2) * mask
    y = torch.nn.functional.layer_norm(h, (s.hidden,), gain, shift)
    leaves = [x, gain, shift, b2, *w1, *b1, *w2]
    grads = torch.autograd.grad([h, y], leaves, [s.dh_above.float(), s.dy.float()])
    return [h.detach(), y.detach(), *grads]


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--dropout", type=float, default=0.1)
    args = ap.parse_args(argv)
    s = Sublayer(args.ranks, args.hidden, args.tokens, args.dropout)
    for t, scale in ((s.x, 1.0), (s.dy, 0.01), (s.dh_above, 0.01)):
        t.normal_(0.0, scale)

    s.forward()
    s.backward()
    first = [t.clone() for t in s.outputs()]
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    same = all(torch.equal(a, b) for a, b in zip(first, s.outputs()))
    worst = max(float((a.float() - b).norm() / b.norm().clamp_min(1e-30)) for a, b in zip(s.outputs(), reference(s)))
    print(f"training step: {args.ranks} ranks, {args.tokens} tokens, hidden {args.hidden}: same bits twice: {same}; "
          f"largest relative difference from 32 bits: {worst:.2e}")

    # Serving: a few tokens, captured once, replayed on new inputs.
    d = Sublayer(args.ranks, args.hidden, 4, 0.0)
    d.x.normal_()
    d.forward(train=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.forward(train=False)
    d.x.normal_()
    graph.replay()
    replayed = d.y.clone()
    d.forward(train=False)
    torch.cuda.synchronize()
    served = bool(torch.equal(replayed, d.y))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 1e3 / 20
    print(f"serving: 4 tokens, graph replay equals the eager call: {served}; {us:.1f} us for all {args.ranks} ranks")
    return {"same": same, "worst": worst, "served": served}


if __name__ == "__main__":
    main()
