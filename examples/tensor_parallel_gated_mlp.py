"""The gated, root-mean-square-normalised MLP sublayer of a tensor-parallel transformer block, on one GPU.

W virtual ranks each hold a slice of the three weight matrices.  The sublayer takes the
ranks' partials of the one before it (an attention's, say), and

    h = residual + sum_r p_r,  n = rms_norm(h)                  arx_reduce_rms_norm
    a_r = silu(n Wg_r^T) * (n Wu_r^T)                           arx_gated_linear
    q_r = a_r Wd_r^T                                            arx_linear: the rank's partial
    out = h + sum_r q_r,  y = rms_norm(out)                     arx_reduce_rms_norm

The training step runs the backward passes (arx_rms_norm_bwd, arx_linear_bwd,
arx_gated_linear_bwd), checks them against a 32-bit torch reference, and repeats the step
to show that every bit is the same.  The serving part keeps the projections' weights in
8 bits: the norm hands its output to them in 8 bits with a scale for each token, in a
CUDA graph that is replayed.

    python examples/tensor_parallel_gated_mlp.py [--ranks W] [--hidden H] [--tokens T]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_shot_all_gb300 as arx  # noqa: E402

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Sublayer:
    """Weights of W ranks, and the buffers of calls on T tokens."""

    def __init__(self, W: int, hidden: int, tokens: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        inner = 4 * hidden // W  # a rank's share of the inner features

        def normal(*shape, scale=1.0, shift=0.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(BF16)

        self.W, self.hidden, self.tokens, self.inner = W, hidden, tokens, inner
        # A rank's two projections in one buffer, one after the other.
        self.w = [normal(2 * inner, hidden, scale=hidden ** -0.5) for _ in range(W)]
        self.wd = [normal(hidden, inner, scale=(4 * hidden) ** -0.5) for _ in range(W)]
        self.gain = [normal(hidden, scale=0.1, shift=1.0) for _ in range(2)]

        T, new = tokens, lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.partial = [new(T, hidden) for _ in range(W)]  # the sublayer's input
        self.residual = new(T, hidden)
        self.h, self.n, self.out, self.y = (new(T, hidden) for _ in range(4))
        self.rstd = [new(T, dtype=torch.float32) for _ in range(2)]
        self.a, self.zg, self.zu = ([new(T, inner) for _ in range(W)] for _ in range(3))
        self.q = [new(T, hidden) for _ in range(W)]

        # Gradients: the sublayer's output and residual stream come from above.
        self.dy, self.dout_above = new(T, hidden), new(T, hidden)
        self.dout, self.dn, self.dpartial = (new(T, hidden) for _ in range(3))
        self.da = new(T, inner)
        self.dn_r = [new(T, hidden) for _ in range(W)]
        self.grads = {"gain": [new(hidden) for _ in range(2)], "w": [new(2 * inner, hidden) for _ in range(W)],
                      "wd": [new(hidden, inner) for _ in range(W)]}
        nbytes = max(arx.arx_rms_norm_bwd_workspace_bytes(T, hidden), arx.arx_gated_linear_bwd_workspace_bytes(T, inner))
        self.ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")

    def halves(self, w):
        return w[:self.inner], w[self.inner:]

    def forward(self) -> None:
        arx.arx_reduce_rms_norm(self.partial, self.h, self.n, residual=self.residual, weight=self.gain[0], rstd=self.rstd[0])
        for r in range(self.W):
            arx.arx_gated_linear(self.n, *self.halves(self.w[r]), self.a[r], z_gate=self.zg[r], z_up=self.zu[r])
            arx.arx_linear(self.a[r], self.wd[r], self.q[r])
        arx.arx_reduce_rms_norm(self.q, self.out, self.y, residual=self.h, weight=self.gain[1], rstd=self.rstd[1])

    def backward(self) -> None:
        g = self.grads
        # The last norm, joined by the gradient that reaches `out` along the residual stream.
        arx.arx_rms_norm_bwd(self.dy, self.out, self.rstd[1], self.dout, weight=self.gain[1], dresidual=self.dout_above,
                             dweight=g["gain"][1], workspace=self.ws)
        for r in range(self.W):  # every rank's partial has the same gradient
            arx.arx_linear_bwd(self.dout, self.a[r], self.wd[r], dx=self.da, dw=g["wd"][r])
            dw = self.halves(g["w"][r])
            arx.arx_gated_linear_bwd(self.da, self.n, *self.halves(self.w[r]), self.zg[r], self.zu[r], dx=self.dn_r[r],
                                     dw_gate=dw[0], dw_up=dw[1], workspace=self.ws)
        arx.arx_reduce(self.dn_r, self.dn)  # the ranks' input gradients: one more all-reduce
        arx.arx_rms_norm_bwd(self.dn, self.h, self.rstd[0], self.dpartial, weight=self.gain[0], dresidual=self.dout,
                             dweight=g["gain"][0], workspace=self.ws)

    def outputs(self) -> list:
        g = self.grads
        return [self.out, self.y, self.dpartial, *g["gain"], *g["w"], *g["wd"]]


def rms(x, gain):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain


def reference(s: Sublayer) -> list:
    """The same step in 32 bits with torch's automatic differentiation."""
    leaf = lambda t: t.float().detach().requires_grad_()  # noqa: E731
    residual, gain, w, wd = leaf(s.residual), [leaf(t) for t in s.gain], [leaf(t) for t in s.w], [leaf(t) for t in s.wd]
    h = residual + sum(p.float() for p in s.partial)
    n = rms(h, gain[0])
    total = 0
    for r in range(s.W):
        g, u = (n @ w[r].t()).chunk(2, dim=1)
        total = total + (torch.nn.functional.silu(g) * u) @ wd[r].t()
    out = h + total
    y = rms(out, gain[1])
    grads = torch.autograd.grad([out, y], [residual, *gain, *w, *wd], [s.dout_above.float(), s.dy.float()])
    return [out.detach(), y.detach(), *grads]


def eight_bits(rows: int, cols: int):
    """An e4m3 matrix whose rows are on 16 bytes, as the products take them."""
    return torch.empty(rows, -(-cols // 16) * 16, dtype=E4M3, device="cuda")[:, :cols]


class EightBits:
    """Serving: the projections' weights in e4m3 with a scale for each feature, the norm's output in e4m3 too."""

    def __init__(self, s: Sublayer):
        self.s = s
        scale = [w.float().abs().amax(1) / 448 for w in s.w]
        self.w = [eight_bits(*w.shape) for w in s.w]
        for q, w, c in zip(self.w, s.w, scale):
            q.copy_(w.float() / c[:, None])
        self.scale = [s.halves(c) for c in scale]
        self.n = eight_bits(s.tokens, s.hidden)
        self.n_scale = torch.empty(s.tokens, device="cuda")

    def forward(self) -> None:
        s = self.s
        arx.arx_reduce_rms_norm(s.partial, s.h, None, residual=s.residual, weight=s.gain[0], q=self.n, scale=self.n_scale)
        for r in range(s.W):
            arx.arx_gated_linear(self.n, *s.halves(self.w[r]), s.a[r], x_scale=self.n_scale, gate_scale=self.scale[r][0],
                                 up_scale=self.scale[r][1])
            arx.arx_linear(s.a[r], s.wd[r], s.q[r])
        arx.arx_reduce_rms_norm(s.q, s.out, s.y, residual=s.h, weight=s.gain[1])


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=1024)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    s = Sublayer(args.ranks, args.hidden, args.tokens)

    def inputs(s):
        for t, scale in (*((p, args.ranks ** -0.5) for p in s.partial), (s.residual, 1.0), (s.dy, 0.01), (s.dout_above, 0.01)):
            t.normal_(0.0, scale)

    inputs(s)
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
    d = Sublayer(args.ranks, args.hidden, 4)
    e = EightBits(d)
    inputs(d)
    e.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.forward()
    inputs(d)
    graph.replay()
    replayed = d.y.clone()
    e.forward()
    torch.cuda.synchronize()
    served = bool(torch.equal(replayed, d.y))
    d.forward()  # the same in 16 bits
    eight = float((replayed.float() - d.y.float()).norm() / d.y.float().norm())
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 1e3 / 20
    print(f"serving: 4 tokens in 8 bits, graph replay equals the eager call: {served}; from 16 bits {eight:.2e}; "
          f"{us:.1f} us for all {args.ranks} ranks")
    return {"same": same, "worst": worst, "served": served, "eight": eight}


if __name__ == "__main__":
    main()
