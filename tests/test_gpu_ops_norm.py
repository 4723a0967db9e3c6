"""Layer norm forward and backward on the GPU against the 64-bit formulas."""

import numpy as np
import pytest
import torch

import ops_plain as plain
from ops_gpu import E, Out, TYPES, U, assert_close, bits, f64, make, scratch, strided

pytestmark = pytest.mark.gpu

# Columns around every switch of the launch rules, whole units of 8 and not, and rows beyond the registers.
COLS = [1, 7, 8, 33, 256, 257, 264, 512, 1000, 1024, 1025, 2048, 2056, 4096, 4099, 5003, 8192, 8200, 16384]
LONG = [16385, 16392, 33000, 40009]


def _forward(arx, rows, cols, dtype, wdtype, pad=0, lead=0, shift=0.0, params=True, eps=1e-5, x=None):
    x = strided(make((rows, cols), dtype, cols + rows, shift=shift) if x is None else x, pad, lead)
    w = make((cols,), wdtype, 1, 0.2, 1.0) if params else None
    b = make((cols,), wdtype, 2, 0.2) if params else None
    y = Out((rows, cols), dtype, pad, lead)
    mean, rstd = Out((rows,), torch.float32), Out((rows,), torch.float32)
    arx.arx_layer_norm(x, y.t, weight=w, bias=b, mean=mean.t, rstd=rstd.t, eps=eps)
    torch.cuda.synchronize()
    xd, wd, bd = f64(x), f64(w), f64(b)
    wy, wm, wr = plain.layer_norm(xd, wd, bd, eps)
    # A row's sums go through at most n additions in a chain; n is bounded by
    # the columns of one thread and the joins over threads and warps.
    n = min(cols, 32 + cols / 32 + 32)
    mag = np.abs(xd).mean(1)
    em = n * E * mag                                    # error of the mean
    spread = 1 / wr
    er = 2 * n * E + 2 * em / spread + 8 * E            # relative error of rstd
    assert_close(mean, wm, em, "mean")
    assert_close(rstd, wr, er * wr, "rstd")
    xh = np.abs(xd - wm[:, None]) * wr[:, None]
    ey = (em[:, None] * wr[:, None] + xh * (er[:, None] + 4 * E) + 2 * E * np.abs(xd) * wr[:, None])
    if params:
        ey = ey * np.abs(wd) + 4 * E * (np.abs(wd) * xh + np.abs(bd))
    assert_close(y, wy, ey, "y")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS + LONG)
def test_forward(arx, cols, dtype):
    _forward(arx, 5, cols, dtype, dtype)


@pytest.mark.parametrize("cols,pad,lead", [(4096, 8, 0), (4096, 3, 0), (1000, 8, 8), (1000, 0, 1), (2048, 1, 5),
                                           (257, 7, 1), (20000, 3, 1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_strides_alignment_and_32_bit_parameters(arx, cols, pad, lead, dtype):
    _forward(arx, 9, cols, dtype, torch.float32, pad, lead)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 700])
def test_forward_rows_and_no_parameters(arx, rows):
    _forward(arx, rows, 256, torch.bfloat16, torch.bfloat16, params=False)
    _forward(arx, rows, 1024, torch.float32, torch.float32, params=False, eps=0.25)


def test_forward_large_mean(arx):
    # A mean 1000 times the spread: the centred second pass keeps the variance.
    _forward(arx, 4, 4096, torch.float32, torch.float32, shift=1000.0)
    _forward(arx, 4, 33000, torch.float32, torch.float32, shift=1000.0)


def test_forward_constant_rows(arx):
    # The spread is zero: (x - mean) is exactly zero for a constant exact in fp32, and y the bias.
    _forward(arx, 3, 512, torch.bfloat16, torch.bfloat16, x=torch.full((3, 512), 3.0, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("cols", [256, 1000, 1001, 4096, 20000])
def test_infinities_and_nan_stay_in_their_rows(arx, cols):
    x = make((6, cols), torch.bfloat16, 3)
    x[1, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4, 0] = -float("inf")
    y = torch.empty_like(x)
    arx.arx_layer_norm(x, y)
    clean = x.clone()
    clean[[1, 3, 4]] = 0
    want = torch.empty_like(x)
    arx.arx_layer_norm(clean, want)
    torch.cuda.synchronize()
    assert torch.isnan(y[[1, 3, 4]]).all()
    assert torch.equal(bits(y[[0, 2, 5]]), bits(want[[0, 2, 5]]))


def _backward(arx, rows, cols, dtype, wdtype, pad=0, lead=0, dres=True, weight=True, grads=True, alias=None):
    x = strided(make((rows, cols), dtype, cols + rows, shift=0.3), pad, lead)
    dy = strided(make((rows, cols), dtype, 5), pad, lead)
    dr = strided(make((rows, cols), dtype, 6), pad, lead) if dres else None
    w = make((cols,), wdtype, 1, 0.2, 1.0) if weight else None
    xd, dyd, wd, drd = f64(x), f64(dy), f64(w), f64(dr)
    mean = make((rows,), torch.float32, 7, 0.01, 0.3)
    rstd = make((rows,), torch.float32, 8, 0.05, 1.0)
    md, rd = f64(mean), f64(rstd)
    dx = Out((rows, cols), dtype, pad, lead)
    target = {"dy": dy, "x": x, "dres": dr}.get(alias, dx.t)
    dw = Out((cols,), wdtype) if grads else None
    db = Out((cols,), wdtype) if grads else None
    ws = scratch(arx.arx_layer_norm_bwd_workspace_bytes(rows, cols))
    arx.arx_layer_norm_bwd(dy, x, mean, rstd, target, weight=w, dresidual=dr, dweight=dw.t if grads else None,
                           dbias=db.t if grads else None, workspace=ws if grads else None)
    torch.cuda.synchronize()
    wdx, wdw, wdb = plain.layer_norm_bwd(dyd, xd, md, rd, wd, drd)
    axh = (np.abs(xd) + np.abs(md)[:, None]) * rd[:, None]   # magnitudes behind xh
    q = np.abs(dyd) * (1 if wd is None else np.abs(wd))
    n = min(cols, 32 + cols / 32 + 32) + 6                    # additions in a chain, and the products' roundings
    r = np.abs(rd)[:, None]
    lim = r * (n * E * q.mean(1, keepdims=True) + (n + 4) * E * axh * (q * axh).mean(1, keepdims=True) * 2
               + 4 * E * q + 4 * E * axh * np.abs((q * axh).mean(1, keepdims=True))) + 4 * E * np.abs(wdx)
    if drd is not None:
        lim = lim + 2 * E * np.abs(drd)
    if alias is None:
        assert_close(dx, wdx, lim, "dx")
    else:
        assert_close(target, wdx, lim, "dx")
    if grads:
        assert_close(dw, wdw, (rows + 6) * E * (np.abs(dyd) * axh).sum(0), "dweight")
        assert_close(db, wdb, rows * E * np.abs(dyd).sum(0), "dbias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS + LONG)
def test_backward(arx, cols, dtype):
    _backward(arx, 11, cols, dtype, dtype, dres=cols % 2 == 0)


@pytest.mark.parametrize("rows,cols", [(1, 64), (2, 256), (305, 264), (2500, 128), (700, 1024), (609, 4096), (37, 8200)])
def test_backward_rows(arx, rows, cols):
    _backward(arx, rows, cols, torch.bfloat16, torch.float32)
    _backward(arx, rows, cols, torch.float32, torch.float32, weight=False)


@pytest.mark.parametrize("cols,pad,lead", [(4096, 8, 0), (4096, 3, 0), (1000, 0, 1), (257, 7, 1), (20000, 3, 1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_strides_and_alignment(arx, cols, pad, lead, dtype):
    _backward(arx, 9, cols, dtype, torch.float32, pad, lead)


@pytest.mark.parametrize("alias", ["dy", "x", "dres"])
@pytest.mark.parametrize("cols", [256, 1000, 1001, 4096, 20000])
def test_backward_in_place(arx, cols, alias):
    _backward(arx, 310, cols, torch.bfloat16, torch.bfloat16, alias=alias)


def test_backward_without_parameter_gradients(arx):
    _backward(arx, 20, 1024, torch.float16, torch.float16, grads=False)
    _backward(arx, 20, 33000, torch.float16, torch.float16, grads=False)


def test_backward_of_no_rows_zeroes_the_parameter_gradients(arx):
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.float32, device="cuda")
    dw, db = Out((100,), torch.bfloat16), Out((100,), torch.bfloat16)
    arx.arx_layer_norm_bwd(x, x, s, s, weight=None, dweight=dw.t, dbias=db.t, workspace=scratch(0))
    assert_close(dw, np.zeros(100))
    assert_close(db, np.zeros(100))


@pytest.mark.parametrize("cols", [24, 1000, 4096])
def test_gradients_against_differences(arx, cols):
    # Central differences of the forward formula in 64 bits: error h^2 / 6 times
    # a third derivative of order 1 (1e-8 here) beside the kernel's fp32 error.
    rows, h = 3, 1e-4
    x, w = make((rows, cols), torch.float32, 9), make((cols,), torch.float32, 10, 0.2, 1.0)
    dy = make((rows, cols), torch.float32, 11)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    arx.arx_layer_norm(x, y, weight=w, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    arx.arx_layer_norm_bwd(dy, x, mean, rstd, dx, weight=w, dweight=dw, dbias=db,
                           workspace=scratch(arx.arx_layer_norm_bwd_workspace_bytes(rows, cols)))
    xd, wd, g = f64(x), f64(w), f64(dy)
    r = np.random.default_rng(0)
    for _ in range(8):
        v, u = r.normal(size=xd.shape), r.normal(size=wd.shape)
        up, dn = ((plain.layer_norm(xd + s * h * v, wd)[0] * g).sum() for s in (1, -1))
        scale = np.sqrt((v * v).sum()) * np.sqrt((f64(dx) ** 2).sum())
        assert abs((up - dn) / (2 * h) - (f64(dx) * v).sum()) < 1e-5 * scale
        up, dn = ((plain.layer_norm(xd, wd + s * h * u)[0] * g).sum() for s in (1, -1))
        assert abs((up - dn) / (2 * h) - (f64(dw) * u).sum()) < 1e-5 * np.sqrt((u * u).sum() * (f64(dw) ** 2).sum())
    assert_close(db, g.sum(0), rows * E * np.abs(g).sum(0))


def test_same_bits_on_every_run_and_plan(arx):
    rows, cols = 2000, 4096
    x, dy = make((rows, cols), torch.bfloat16, 1), make((rows, cols), torch.bfloat16, 2)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    arx.arx_layer_norm(x, torch.empty_like(x), mean=mean, rstd=rstd)
    ws = scratch(arx.arx_layer_norm_bwd_workspace_bytes(rows, cols))
    got = []
    for i in range(3):
        dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        if i < 2:
            arx.arx_layer_norm_bwd(dy, x, mean, rstd, dx, dweight=dw, dbias=db, workspace=ws)
        else:
            arx.arx_layer_norm_bwd_plan(dy, x, mean, rstd, dx, dweight=dw, dbias=db, workspace=ws)()
        torch.cuda.synchronize()
        got.append((bits(dx), bits(dw), bits(db)))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, got[0]))


def test_three_dimensional_and_empty_inputs(arx):
    x = make((3, 5, 64), torch.bfloat16, 1)
    y, z = torch.empty_like(x), torch.empty(15, 64, dtype=x.dtype, device="cuda")
    arx.arx_layer_norm(x, y)
    arx.arx_layer_norm(x.view(15, 64), z)
    assert torch.equal(bits(y.view(15, 64)), bits(z))
    e = x[:0]
    arx.arx_layer_norm(e, e)


def test_offsets_past_32_bits(arx):
    # Five rows 2^30 elements apart: element offsets up to 2^32, byte offsets to 2^33.
    ld, cols = (1 << 30) + 8, 1032
    buf = torch.empty(4 * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((5, cols), (ld, 1))
    src = make((5, cols), torch.bfloat16, 4)
    x.copy_(src)
    y = torch.empty_like(src)
    arx.arx_layer_norm(x, y)
    want = torch.empty_like(src)
    arx.arx_layer_norm(src, want)
    assert torch.equal(bits(y), bits(want))
    arx.arx_layer_norm(src, x)
    assert torch.equal(bits(x), bits(want))


def test_side_stream_and_graph(arx):
    x = make((64, 4096), torch.bfloat16, 1)
    y = torch.empty_like(x)
    want = torch.empty_like(x)
    arx.arx_layer_norm(x, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    arx.arx_layer_norm(x, y, stream=s)
    s.synchronize()
    assert torch.equal(bits(y), bits(want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        arx.arx_layer_norm(x, y)
    x.neg_()
    g.replay()
    arx.arx_layer_norm(x, want)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want))
