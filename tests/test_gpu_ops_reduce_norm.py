"""The fused end of a sublayer on the GPU: rank-order sum, bias, dropout, residual, layer norm."""

import numpy as np
import pytest
import torch

import ops_plain as plain
from ops_gpu import E, Out, U, assert_close, bits, f64, make, rng

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _run(arx, W, rows, cols, p=0.0, bias=True, residual=True, norm=True, stats=True, want_h=True, alias=None, lead=0):
    def place(t):
        buf = torch.zeros(t.numel() + lead, dtype=BF16, device="cuda")
        v = buf[lead:].view(t.shape)
        v.copy_(t)
        return v
    slots = [place(make((rows, cols), BF16, 10 + r, W ** -0.5)) for r in range(W)]
    res = place(make((rows, cols), BF16, 3)) if residual else None
    b, w, nb = (make((cols,), BF16, s, 0.3, sh) for s, sh in ((4, 0.0), (5, 1.0), (6, 0.0)))
    s = [f64(x) for x in slots]
    rd = f64(res)
    h, y = Out((rows, cols), BF16, 0, lead), Out((rows, cols), BF16, 0, lead)
    ht, yt = (h.t if want_h else None), y.t
    if alias:
        ht, yt = {"slot": (slots[0], y.t), "residual": (res, y.t), "both": (res, slots[-1])}[alias]
    mean, rstd = Out((rows,), torch.float32), Out((rows,), torch.float32)
    arx.arx_reduce_layer_norm(slots, ht, yt, bias=b if bias else None, residual=res, weight=w if norm else None,
                              norm_bias=nb if norm else None, mean=mean.t if stats else None,
                              rstd=rstd.t if stats else None, p=p, rng=rng(8, 1 << 40) if p else None)
    torch.cuda.synchronize()
    v, mag = sum(s), sum(np.abs(x) for x in s)
    if bias:
        v, mag = v + f64(b), mag + np.abs(f64(b))
    if p:
        k = plain.dropout_scale(rows, cols, p, 8, 1 << 40)
        v, mag = v * k, mag * k
    if residual:
        v, mag = v + rd, mag + np.abs(rd)
    eh = (W + 4) * E * mag                               # additions of the sum, bias, scale and residual
    if want_h:
        assert_close(h if ht is h.t else ht, v, eh, "h")
    wy, wm, wr = plain.layer_norm(v, f64(w) if norm else None, f64(nb) if norm else None)
    n = min(cols, 32 + cols / 32 + 32)
    em = n * E * np.abs(v).mean(1) + eh.mean(1)
    er = 2 * n * E + 2 * em * wr + 8 * E + 2 * eh.max(1) * wr
    if stats:
        assert_close(mean, wm, em, "mean")
        assert_close(rstd, wr, er * wr, "rstd")
    xh = np.abs(v - wm[:, None]) * wr[:, None]
    ey = (em[:, None] + eh) * wr[:, None] + xh * (er[:, None] + 4 * E) + 2 * E * np.abs(v) * wr[:, None]
    if norm:
        ey = ey * np.abs(f64(w)) + 4 * E * (np.abs(f64(w)) * xh + np.abs(f64(nb)))
    assert_close(y if yt is y.t else yt, wy, ey, "y")


@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("cols", [4096, 1001])
def test_every_w(arx, W, cols):
    _run(arx, W, 9, cols)
    _run(arx, W, 9, cols, p=0.25)


@pytest.mark.parametrize("cols", [1, 8, 31, 256, 264, 1000, 1024, 1032, 2048, 2056, 4099, 5000, 8192, 8200, 12345, 16384,
                                  16392, 30000])
def test_columns(arx, cols):
    _run(arx, 3, 6, cols, p=0.1)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 33, 400])
def test_rows(arx, rows):
    _run(arx, 8, rows, 256)
    _run(arx, 2, rows, 4096, p=0.5)


def test_optional_arguments(arx):
    _run(arx, 4, 10, 512, bias=False, residual=False, norm=False, stats=False)
    _run(arx, 4, 10, 512, want_h=False)
    _run(arx, 4, 10, 515, want_h=False, p=0.5)
    _run(arx, 4, 10, 4096, p=1.0)


@pytest.mark.parametrize("lead", [1, 4, 8])
def test_alignment(arx, lead):
    _run(arx, 4, 10, 512, lead=lead, p=0.1)


@pytest.mark.parametrize("alias", ["slot", "residual", "both"])
@pytest.mark.parametrize("cols", [512, 4096, 777, 20000])
def test_in_place(arx, cols, alias):
    _run(arx, 4, 30, cols, p=0.1, alias=alias)


@pytest.mark.parametrize("W", [1, 2, 5, 8])
def test_sum_is_the_reduce_bit_for_bit(arx, W):
    # Without bias, dropout and residual, h rounds the same rank-order sum that arx_reduce rounds.
    rows, cols = 32, 4096
    slots = [make((rows, cols), BF16, r, 10.0 ** (r - 3)) for r in range(W)]
    h, y, out = (torch.empty(rows, cols, dtype=BF16, device="cuda") for _ in range(3))
    arx.arx_reduce_layer_norm(slots, h, y)
    arx.arx_reduce(slots, out)
    torch.cuda.synchronize()
    assert torch.equal(bits(h), bits(out))


def test_same_as_its_parts_in_32_bits_and_its_backward(arx):
    # The fused forward's stored h, mean and rstd feed the backward calls: gradients against 64 bits.
    rows, cols, W, p = 40, 1024, 4, 0.25
    slots = [make((rows, cols), BF16, r) for r in range(W)]
    res = make((rows, cols), BF16, 20)
    w = make((cols,), BF16, 21, 0.2, 1.0)
    h, y = torch.empty_like(res), torch.empty_like(res)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    state = rng(3, 4)
    arx.arx_reduce_layer_norm(slots, h, y, residual=res, weight=w, mean=mean, rstd=rstd, p=p, rng=state)
    dy, dh = make((rows, cols), BF16, 22), make((rows, cols), BF16, 23)
    dx = torch.empty_like(dy)
    arx.arx_layer_norm_bwd(dy, h, mean, rstd, dx, weight=w, dresidual=dh)
    ds = torch.empty_like(dy)
    arx.arx_dropout_add_bwd(dx, ds, p, state)
    torch.cuda.synchronize()
    k = plain.dropout_scale(rows, cols, p, 3, 4)
    v = sum(f64(s) for s in slots) * k + f64(res)
    _, m, r = plain.layer_norm(v)
    want, _, _ = plain.layer_norm_bwd(f64(dy), v, m, r, f64(w), f64(dh))
    # h enters the backward pass rounded: xh moves by u |h| rstd, and dx by about
    # rstd times that times the mean of |q xh| plus |q| / sqrt(cols)-sized sums.
    u = U[BF16]
    q = np.abs(f64(dy) * f64(w))
    move = r[:, None] * u * (np.abs(v) * r[:, None] + np.abs(v).mean(1, keepdims=True) * r[:, None]) * (
        2 * q.mean(1, keepdims=True) + 2 * (q * np.abs(v) * r[:, None]).mean(1, keepdims=True))
    assert_close(dx, want, move + 64 * E * (1 + np.abs(want)), "dx")
    assert_close(ds, f64(dx) * k, 2 * E * np.abs(f64(dx) * k), "ds")


def test_infinities_and_nan_stay_in_their_rows(arx):
    slots = [make((5, 4096), BF16, r) for r in range(3)]
    clean = [s.clone() for s in slots]
    slots[1][2, 17] = float("nan")
    slots[2][4, 4095] = float("inf")
    out = []
    for ss in (slots, clean):
        h, y = torch.empty_like(ss[0]), torch.empty_like(ss[0])
        arx.arx_reduce_layer_norm(ss, h, y)
        out.append((h, y))
    torch.cuda.synchronize()
    for a, b in zip(*out):
        assert torch.equal(bits(a[[0, 1, 3]]), bits(b[[0, 1, 3]]))
    assert torch.isnan(out[0][1][[2, 4]]).all()


def test_plan_and_graph(arx):
    slots = [make((32, 4096), BF16, r) for r in range(8)]
    h, y, h2, y2 = (torch.empty_like(slots[0]) for _ in range(4))
    plan = arx.arx_reduce_layer_norm_plan(slots, h, y, residual=slots[0])
    plan()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        arx.arx_reduce_layer_norm(slots, h2, y2, residual=slots[0])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(h), bits(h2)) and torch.equal(bits(y), bits(y2))
