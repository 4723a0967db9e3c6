"""The root-mean-square norm and the gated block in 64 bits, from their formulas, on the host.

Test infrastructure: numpy only, none of the package's code.  Inputs are numpy
arrays; results are float64.
"""

import numpy as np

import ops_plain

TOP, LEAST = 448.0, 2.0 ** -126


def rms_norm(h, weight=None, eps=1e-6):
    """(y, scale of each row's 8-bit form, rstd)."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    if weight is not None:
        y = y * weight
    s = np.abs(y).max(1) / TOP  # NaN stays
    return y, np.where(s < LEAST, 1.0, s), rstd


def rms_norm_bwd(dy, h, rstd, weight=None, dresidual=None):
    n = h * rstd[:, None]
    v = dy if weight is None else dy * weight
    dx = rstd[:, None] * (v - n * (v * n).mean(1, keepdims=True))
    return (dx if dresidual is None else dx + dresidual), (dy * n).sum(0)


def gated(x, w_gate, w_up, act, bias_gate=0.0, bias_up=0.0, scales=None):
    """(out, g, u); scales: of x's rows and of either weight's."""
    g, u = x @ w_gate.T, x @ w_up.T
    if scales is not None:
        sx, sg, su = scales
        g, u = g * sx[:, None] * sg, u * sx[:, None] * su
    g, u = g + bias_gate, u + bias_up
    return ops_plain.act(g, act) * u, g, u


def gated_bwd(dout, g, u, x, w_gate, w_up, act):
    """dx, dw_gate, dw_up, dbias_gate, dbias_up."""
    dg, du = dout * u * ops_plain.act_grad(g, act), dout * ops_plain.act(g, act)
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x, dg.sum(0), du.sum(0)
