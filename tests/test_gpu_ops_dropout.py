"""Dropout with bias and residual on the GPU: the mask bit for bit, the values against 64 bits."""

import numpy as np
import pytest
import torch

import ops_plain as plain
from ops_gpu import E, Out, TYPES, assert_close, bits, f64, make, rng, scratch, strided

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 21), (300, 8), (17, 250), (64, 256), (33, 1000), (10, 4096), (9, 4099), (2000, 72)]
BIG = 0xFEDCBA9876543210  # both halves of seed and offset in use


def _forward(arx, rows, cols, dtype, wdtype, p, pad=0, lead=0, bias=True, residual=True, seed=BIG, offset=BIG ^ 77):
    x = strided(make((rows, cols), dtype, 1), pad, lead)
    r = strided(make((rows, cols), dtype, 2), pad, lead) if residual else None
    b = make((cols,), wdtype, 3) if bias else None
    out = Out((rows, cols), dtype, pad, lead)
    arx.arx_dropout_add(x, out.t, p, rng(seed, offset), bias=b, residual=r)
    torch.cuda.synchronize()
    s = plain.dropout_scale(rows, cols, p, seed, offset)
    xd, bd, rd = f64(x), f64(b), f64(r)
    v = (xd if bd is None else xd + bd) * s
    mag = (np.abs(xd) + (0 if bd is None else np.abs(bd))) * s
    want = v if rd is None else rd + v
    # Three fp32 roundings (bias, scale and the scale's own) and the residual's.
    assert_close(out, want, 3 * E * mag + E * np.abs(want), "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(arx, rows, cols, dtype):
    _forward(arx, rows, cols, dtype, dtype, 0.3)


@pytest.mark.parametrize("p", [0.0, 1e-7, 1 / 65536, 0.1, 0.5, 0.999, 65535 / 65536, 1.0])
@pytest.mark.parametrize("residual", [False, True])
def test_probabilities(arx, p, residual):
    _forward(arx, 40, 256, torch.float32, torch.float32, p, residual=residual)
    _forward(arx, 40, 259, torch.bfloat16, torch.float32, p, bias=False, residual=residual)


@pytest.mark.parametrize("pad,lead", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(arx, pad, lead, dtype):
    _forward(arx, 21, 264, dtype, torch.float32, 0.25, pad, lead)


def test_mask_is_the_published_generator(arx):
    # The element with 16-bit value v is kept at T = v and dropped at T = v + 1.
    rows, cols, seed, offset = 4, 19, 0x299F31D0A4093822, 0x0370734413198A2E
    v = plain.dropout_values(rows, cols, seed, offset)
    x = torch.ones(rows, cols, device="cuda")
    out = torch.empty_like(x)
    for i, j in ((0, 0), (1, 5), (2, 8), (3, 18), (3, 16)):
        for T, kept in ((int(v[i, j]), True), (int(v[i, j]) + 1, False)):
            arx.arx_dropout_add(x, out, T / 65536, rng(seed, offset))
            assert bool(out[i, j] != 0) == kept


def test_infinities_and_nan_in_dropped_places(arx):
    rows, cols, p = 16, 1000, 0.5
    keep = torch.from_numpy(plain.dropout_scale(rows, cols, p, 5, 6) > 0).cuda()
    for dtype in TYPES:
        x = make((rows, cols), dtype, 1)
        bad = x.clone()
        bad[~keep] = float("nan")
        bad[0][~keep[0]] = float("inf")
        a, b = torch.empty_like(x), torch.empty_like(x)
        r = make((rows, cols), dtype, 2)
        arx.arx_dropout_add(x, a, p, rng(5, 6), residual=r)
        arx.arx_dropout_add(bad, b, p, rng(5, 6), residual=r)
        assert torch.equal(bits(a), bits(b))
        arx.arx_dropout_add_bwd(bad, b, p, rng(5, 6))
        assert torch.isfinite(b).all()


def _backward(arx, rows, cols, dtype, wdtype, p, pad=0, lead=0, dbias=True, in_place=False):
    d = strided(make((rows, cols), dtype, 1), pad, lead)
    dd = f64(d)
    dx = Out((rows, cols), dtype, pad, lead)
    db = Out((cols,), wdtype) if dbias else None
    ws = scratch(arx.arx_dropout_add_bwd_workspace_bytes(rows, cols)) if dbias else None
    arx.arx_dropout_add_bwd(d, d if in_place else dx.t, p, rng(BIG, 3), dbias=db.t if dbias else None, workspace=ws)
    torch.cuda.synchronize()
    want = dd * plain.dropout_scale(rows, cols, p, BIG, 3)
    assert_close(d if in_place else dx, want, 2 * E * np.abs(want), "dx")
    if dbias:
        assert_close(db, want.sum(0), (rows + 2) * E * np.abs(want).sum(0), "dbias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(arx, rows, cols, dtype):
    _backward(arx, rows, cols, dtype, dtype, 0.3)


@pytest.mark.parametrize("p", [0.0, 0.5, 1.0])
def test_backward_probabilities_and_forms(arx, p):
    _backward(arx, 300, 264, torch.bfloat16, torch.float32, p)
    _backward(arx, 300, 264, torch.bfloat16, torch.float32, p, in_place=True)
    _backward(arx, 300, 261, torch.float16, torch.float32, p, pad=3, lead=1, in_place=True)
    _backward(arx, 30, 264, torch.bfloat16, torch.float32, p, dbias=False)


def test_bias_gradient_alone_and_of_no_rows(arx):
    d = make((50, 40), torch.float32, 1)
    db = Out((40,), torch.float32)
    arx.arx_dropout_add_bwd(d, None, 0.0, dbias=db.t, workspace=scratch(arx.arx_dropout_add_bwd_workspace_bytes(50, 40)))
    assert_close(db, f64(d).sum(0), 50 * E * np.abs(f64(d)).sum(0))
    db = Out((40,), torch.float32)
    arx.arx_dropout_add_bwd(d[:0], None, 0.0, dbias=db.t, workspace=scratch(0))
    assert_close(db, np.zeros(40))


def test_gradient_against_differences(arx):
    # The forward is linear in x: a difference of two outputs is the gradient up to rounding.
    rows, cols, p = 7, 100, 0.4
    x, v, g = (make((rows, cols), torch.float32, i) for i in (1, 2, 3))
    outs = []
    for s in (1.0, -1.0):
        o = torch.empty_like(x)
        arx.arx_dropout_add(x + s * v, o, p, rng(9, 9), residual=x)
        outs.append(f64(o))
    dx = torch.empty_like(x)
    arx.arx_dropout_add_bwd(g, dx, p, rng(9, 9))
    lhs = ((outs[0] - outs[1]) / 2 * f64(g)).sum()
    rhs = (f64(dx) * f64(v)).sum()
    assert abs(lhs - rhs) < 16 * E * np.sum(np.abs(f64(g)) * (np.abs(outs[0]) + np.abs(outs[1]) + 4))


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("cols", [256, 251])
def test_in_place(arx, cols, target):
    x, r = make((60, cols), torch.bfloat16, 1), make((60, cols), torch.bfloat16, 2)
    want = torch.empty_like(x)
    arx.arx_dropout_add(x, want, 0.2, rng(1, 2), residual=r)
    out = x if target == "x" else r
    arx.arx_dropout_add(x, out, 0.2, rng(1, 2), residual=r)
    assert torch.equal(bits(out), bits(want))


def test_mask_depends_on_row_and_column_alone(arx):
    # Other strides, a narrower matrix and another type see the same mask.
    a = torch.ones(50, 264, device="cuda")
    full = torch.empty_like(a)
    arx.arx_dropout_add(a, full, 0.5, rng(4, 4))
    part = Out((20, 77), torch.bfloat16, 6, 1)
    arx.arx_dropout_add(torch.ones(20, 77, dtype=torch.bfloat16, device="cuda"), part.t, 0.5, rng(4, 4))
    assert torch.equal(part.t != 0, full[:20, :77] != 0)


def test_graph_reads_the_generator_state_at_replay(arx):
    x = torch.ones(32, 512, device="cuda")
    out, want = torch.empty_like(x), torch.empty_like(x)
    state = rng(7, 1)
    arx.arx_dropout_add(x, out, 0.5, state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        arx.arx_dropout_add(x, out, 0.5, state)
    seen = []
    for offset in (2, 3):
        state[1] = offset
        g.replay()
        arx.arx_dropout_add(x, want, 0.5, rng(7, offset))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        seen.append(out.clone())
    assert not torch.equal(*seen)


def test_offsets_past_32_bits(arx):
    ld, cols = (1 << 30) + 8, 512
    buf = torch.empty(4 * ld + cols, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((5, cols), (ld, 1))
    x = make((5, cols), torch.bfloat16, 4)
    want = torch.empty_like(x)
    arx.arx_dropout_add(x, want, 0.5, rng(1, 1))
    arx.arx_dropout_add(x, far, 0.5, rng(1, 1))
    assert torch.equal(bits(far), bits(want))
    far.copy_(x)
    got = torch.empty_like(x)
    arx.arx_dropout_add_bwd(far, got, 0.5, rng(1, 1))
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("rows", [1, 256, 8192, 32768, 32769, 65536, 81921, 116736])
def test_bias_gradient_over_few_and_many_partial_sums(arx, rows):
    # 1 to 456 partial rows, to either side of the 128 up to which they are added in a plain loop;
    # whole numbers, whose sums stay below 2^24, so that every order gives the same.
    g = torch.Generator(device="cuda").manual_seed(rows)
    d = torch.randint(-8, 9, (rows, 8), generator=g, device="cuda").float()
    db = Out((8,), torch.float32)
    arx.arx_dropout_add_bwd(d, None, 0.0, dbias=db.t, workspace=scratch(arx.arx_dropout_add_bwd_workspace_bytes(rows, 8)))
    db.check_guards()
    assert torch.equal(db.t.double(), d.double().sum(0))
