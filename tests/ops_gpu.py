"""Shared parts of the GPU tests of the operators around the reduce.

Tolerances are elementwise and derived, not fitted:

* a result rounded once to a type with unit roundoff u is within u * |exact|
  of the value that was rounded, or half the smallest subnormal;
* a sum of n fp32 terms in any order is within n * 2^-24 * sum|term| of exact
  (callers give n, the longest chain of additions through one value, and the
  sum of magnitudes);
* what else enters (a mean's error, an activation's slope) is stated where a
  test adds it.
"""

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
GUARD = 37


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


def strided(t, pad, lead=0):
    """The matrix in a buffer whose rows are ``pad`` elements longer, ``lead`` elements in."""
    r, c = t.shape
    buf = torch.zeros(r * (c + pad) + lead, dtype=t.dtype, device=t.device)
    v = buf[lead:].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


class Out:
    """An output matrix or vector with guard elements around it and between its rows."""

    def __init__(self, shape, dtype, pad=0, lead=0):
        self.shape, self.dtype = tuple(shape), dtype
        r, c = (1, shape[0]) if len(shape) == 1 else shape
        self.lead = GUARD if lead is None else 64 + lead
        self.buf = torch.full((self.lead + r * (c + pad) + GUARD,), 97.0, dtype=dtype, device="cuda")
        body = self.buf[self.lead:self.lead + r * (c + pad)].view(r, c + pad)
        self.t = body[:, :c] if len(shape) == 2 else body[0, :c]
        self.rest = torch.ones_like(self.buf, dtype=torch.bool)
        self.rest[self.lead:self.lead + r * (c + pad)].view(r, c + pad)[:, :c] = False

    def check_guards(self):
        assert bool((self.buf[self.rest] == 97.0).all()), "wrote outside the output"


def assert_close(got, want, extra=0.0, what=""):
    """|got - want| <= u |want| + extra, NaN and infinities in the same places."""
    if isinstance(got, Out):
        got.check_guards()
        got = got.t
    dtype = got.dtype
    g, w = f64(got), np.asarray(want, dtype=np.float64)
    assert g.shape == w.shape, (g.shape, w.shape)
    fine = np.isfinite(w)
    assert np.array_equal(np.isnan(g), np.isnan(w)), f"{what}: NaN in other places"
    assert np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)]), f"{what}: other infinities"
    lim = np.broadcast_to(U[dtype] * np.abs(np.where(fine, w, 0)) * (1 + 2 * U[dtype]) + extra + TINY[dtype], w.shape)
    d = np.abs(np.where(fine, g, 0) - np.where(fine, w, 0))
    if not (d <= lim).all():
        i = np.unravel_index(np.argmax(d / lim), d.shape)
        raise AssertionError(f"{what}: {int((d > lim).sum())} of {d.size} off; worst at {i}: got {g[i]}, "
                             f"want {w[i]}, limit {np.broadcast_to(lim, d.shape)[i]}")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def rng(seed, offset):
    s = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([s(seed), s(offset)], dtype=torch.int64, device="cuda")


def scratch(n):
    return torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")
