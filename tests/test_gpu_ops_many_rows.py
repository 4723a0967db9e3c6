"""The row operators at rows enough that every block takes several turns.

The kernels for many rows are persistent or walk down chunks of rows: a layer
norm block brings rows in through a ring in shared memory whose slots are used
again, a dropout thread has several rows in flight and goes round.  Each size
here gives a block more turns than its ring has slots and a ragged last one,
for every width at which the launch rules switch, aligned and off 16 bytes.
Tolerances are those of the operators' own test files.
"""

import numpy as np
import pytest
import torch

import test_gpu_ops_dropout as dropout
import test_gpu_ops_linear as linear
import test_gpu_ops_norm as norm
import test_gpu_ops_reduce_norm as reduce_norm
from ops_gpu import TYPES, bits, make, rng, strided

pytestmark = pytest.mark.gpu
BF16, F16, F32 = TYPES

# Rows: where the ring is the form, six turns and a part of one of 152 SMs' blocks
# (three of up to 256 threads to an SM, two above, one of 512), 8, 8, 4, 2, 1, 1, 1
# rows to a block.
RING_ROWS = {256: 22003, 512: 22003, 1024: 11003, 2048: 5503, 4096: 2803, 5120: 1903, 8192: 1003}


def _ring_rows(cols):
    return next(r for c, r in RING_ROWS.items() if cols <= c)


@pytest.mark.parametrize("cols,dtype,wdtype,pad,lead", [
    (200, BF16, F32, 0, 0), (256, F32, F32, 8, 8), (512, F16, F16, 0, 0), (1024, BF16, BF16, 0, 0),
    (1000, F32, F32, 0, 0), (2048, BF16, F32, 8, 0), (4096, F16, F32, 0, 0), (4096, F32, F32, 0, 0),
    (5120, BF16, F32, 0, 0), (8192, BF16, BF16, 0, 0), (8192, F32, F32, 0, 0)])
def test_norm_forward_aligned(arx, cols, dtype, wdtype, pad, lead):
    norm._forward(arx, _ring_rows(cols), cols, dtype, wdtype, pad, lead)


@pytest.mark.parametrize("cols,dtype,wdtype,pad,lead", [
    (61, F16, F32, 0, 1), (250, F32, F32, 3, 0), (257, BF16, F32, 0, 0), (512, BF16, BF16, 1, 3), (515, F32, F32, 0, 0),
    (1001, F16, F16, 0, 5), (2047, BF16, F32, 0, 0), (4093, BF16, BF16, 2, 0), (4099, F16, F32, 0, 0),
    (5003, F32, F32, 0, 1), (8191, BF16, F32, 0, 0), (8191, F32, F32, 0, 3)])
def test_norm_forward_off_16_bytes(arx, cols, dtype, wdtype, pad, lead):
    norm._forward(arx, _ring_rows(cols), cols, dtype, wdtype, pad, lead)


@pytest.mark.parametrize("rows", [608, 609, 1216, 2432, 2433])
@pytest.mark.parametrize("cols", [256, 250, 264, 257, 1024, 3000, 2500])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (BF16, BF16), (F32, F32)])
def test_norm_forward_around_the_switch_of_forms(arx, rows, cols, dtype, wdtype):
    norm._forward(arx, rows, cols, dtype, wdtype)


@pytest.mark.parametrize("rows", [7296, 7297, 14999])
def test_norm_forward_around_the_switch_off_16_bytes(arx, rows):
    norm._forward(arx, rows, 300, F16, F16, pad=1)


@pytest.mark.parametrize("cols,pad,lead", [(256, 0, 0), (257, 0, 0), (1024, 8, 0), (1001, 0, 1), (2047, 0, 0), (4096, 0, 0),
                                           (4099, 0, 0), (5120, 0, 0), (8192, 0, 0), (8191, 0, 0), (16392, 0, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_forward_in_place(arx, cols, pad, lead, dtype):
    rows = _ring_rows(min(cols, 8192))
    x = strided(make((rows, cols), dtype, 1, shift=0.5), pad, lead)
    w, b = make((cols,), torch.float32, 2, 0.2, 1.0), make((cols,), torch.float32, 3)
    want = torch.empty(rows, cols, dtype=dtype, device="cuda")
    strided_want = strided(want, pad, lead)
    arx.arx_layer_norm(x, strided_want, weight=w, bias=b)
    arx.arx_layer_norm(x, x, weight=w, bias=b)
    assert torch.equal(bits(x), bits(strided_want))


def test_norm_many_rows_are_those_of_few(arx):
    # A row's result depends on the row alone within a form: repeated rows come out alike wherever they stand.
    for cols in (256, 257, 2048, 4099, 8192):
        rows = _ring_rows(cols)
        x = make((7, cols), BF16, 4)[torch.arange(rows, device="cuda") % 7].contiguous()
        y = torch.empty_like(x)
        arx.arx_layer_norm(x, y)
        assert torch.equal(y, y[:7][torch.arange(rows, device="cuda") % 7])


# Rows: four turns and a part; two blocks of up to 256 threads to an SM, one above.
BWD_ROWS = {256: 10003, 512: 10003, 1024: 5003, 2048: 2503, 4096: 1303, 16384: 653}


def _bwd_rows(cols):
    return next(r for c, r in BWD_ROWS.items() if cols <= c)


@pytest.mark.parametrize("cols,dtype,wdtype,pad,lead,dres", [
    (200, BF16, F32, 0, 0, True), (512, F16, F16, 0, 0, False), (1024, F32, F32, 8, 8, True), (2048, BF16, BF16, 0, 0, True),
    (4096, BF16, F32, 0, 0, True), (5120, F32, F32, 0, 0, False), (8192, F16, F32, 0, 0, True), (16384, BF16, F32, 0, 0, False)])
def test_norm_backward_aligned(arx, cols, dtype, wdtype, pad, lead, dres):
    norm._backward(arx, _bwd_rows(cols), cols, dtype, wdtype, pad, lead, dres=dres)


@pytest.mark.parametrize("cols,dtype,wdtype,pad,lead,dres", [
    (61, F16, F32, 0, 1, True), (257, BF16, F32, 0, 0, True), (511, F32, F32, 1, 0, False), (1001, BF16, BF16, 0, 3, True),
    (1023, F32, F32, 0, 0, True), (2047, F16, F32, 0, 0, False), (4093, BF16, F32, 2, 1, True), (5003, F32, F32, 0, 0, False),
    (5003, BF16, F32, 0, 0, True), (8191, F16, F16, 0, 0, True), (12001, BF16, F32, 0, 0, False)])
def test_norm_backward_off_16_bytes(arx, cols, dtype, wdtype, pad, lead, dres):
    norm._backward(arx, _bwd_rows(cols), cols, dtype, wdtype, pad, lead, dres=dres)


@pytest.mark.parametrize("alias", ["dy", "x", "dres"])
@pytest.mark.parametrize("cols", [256, 257, 1001, 4096, 4099])
def test_norm_backward_in_place(arx, cols, alias):
    norm._backward(arx, _bwd_rows(cols), cols, BF16, F32, alias=alias)


@pytest.mark.parametrize("cols", [264, 1001, 4096])
def test_norm_backward_parameter_gradients_alone(arx, cols):
    # Without dx there is no barrier of the sums between two rows.
    rows = _bwd_rows(cols)
    x, dy = make((rows, cols), BF16, 1, shift=0.3), make((rows, cols), BF16, 2)
    mean, rstd = make((rows,), F32, 3, 0.01, 0.3), make((rows,), F32, 4, 0.05, 1.0)
    ws = torch.empty(arx.arx_layer_norm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    got = []
    for dx in (torch.empty_like(x), None):
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        arx.arx_layer_norm_bwd(dy, x, mean, rstd, dx, dweight=dw, dbias=db, workspace=ws)
        got.append((bits(dw), bits(db)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---- the fused end: above 608 rows the launch rules give a thread more columns ----------

@pytest.mark.parametrize("cols", [200, 264, 1024, 1032, 2048, 4096, 8192, 16384])
def test_reduce_norm_aligned(arx, cols):
    reduce_norm._run(arx, 3, 609, cols, p=0.25)


@pytest.mark.parametrize("cols", [31, 250, 1001, 2047, 4099, 5003, 8191])
def test_reduce_norm_off_16_bytes(arx, cols):
    reduce_norm._run(arx, 3, 609, cols, p=0.25)


@pytest.mark.parametrize("W", range(1, 9))
def test_reduce_norm_every_w(arx, W):
    for cols in (1000, 2000, 4000, 8000):
        reduce_norm._run(arx, W, 613, cols, p=0.1 if W % 2 else 0.0)


# Rows and columns to either side of each switch of the launch rules.
@pytest.mark.parametrize("W", [1, 4, 6, 7, 8])
@pytest.mark.parametrize("rows,cols", [(1216, 512), (1217, 512), (1217, 264), (2432, 1024), (2433, 1024), (1216, 2048),
                                       (1217, 2048), (608, 4096), (609, 4096), (152, 5120), (153, 5120), (152, 8192),
                                       (153, 8192), (40, 4104), (40, 5128)])
def test_reduce_norm_around_the_switches_of_forms(arx, W, rows, cols):
    reduce_norm._run(arx, W, rows, cols, p=0.25 if W % 2 else 0.0)


@pytest.mark.parametrize("alias", ["slot", "residual", "both"])
@pytest.mark.parametrize("cols", [1024, 2056, 4096, 5000, 8192])
def test_reduce_norm_in_place(arx, cols, alias):
    reduce_norm._run(arx, 4, 701, cols, p=0.1, alias=alias)


def test_reduce_norm_optional_arguments(arx):
    reduce_norm._run(arx, 2, 2003, 1024, bias=False, residual=False, norm=False, stats=False)
    reduce_norm._run(arx, 8, 700, 4096, want_h=False)


# ---- dropout: several rows of a thread in flight, several times round ---------------------

DROPOUT = [(2003, 4096, 0, 0), (2003, 4099, 0, 0), (2003, 4096, 3, 1), (40003, 72, 0, 0), (70001, 21, 0, 0), (1203, 8200, 8, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad,lead", DROPOUT)
def test_dropout_forward(arx, rows, cols, pad, lead, dtype):
    dropout._forward(arx, rows, cols, dtype, F32, 0.3, pad, lead)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad,lead", DROPOUT)
def test_dropout_backward(arx, rows, cols, pad, lead, dtype):
    dropout._backward(arx, rows, cols, dtype, F32, 0.3, pad, lead)
    dropout._backward(arx, rows, cols, dtype, F32, 0.3, pad, lead, dbias=False, in_place=True)


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("cols", [4096, 4099])
def test_dropout_in_place(arx, cols, target):
    x, r = make((2003, cols), BF16, 1), make((2003, cols), BF16, 2)
    want = torch.empty_like(x)
    arx.arx_dropout_add(x, want, 0.2, rng(1, 2), residual=r)
    out = x if target == "x" else r
    arx.arx_dropout_add(x, out, 0.2, rng(1, 2), residual=r)
    assert torch.equal(bits(out), bits(want))


# ---- the activation's gradient, which walks down rows the same way -----------------------

@pytest.mark.parametrize("M,N,K,pad", [(20011, 72, 64, 0), (20011, 72, 64, 3), (3001, 4096, 64, 0), (3001, 4100, 64, 1)])
def test_activation_gradient(arx, M, N, K, pad):
    linear._backward(arx, M, N, K, BF16, "gelu", wdtype=F32, pad=pad, which="xb")
    linear._backward(arx, M, N, K, F16, "silu", pad=pad, which="xb")


def test_turns_are_as_many_as_claimed():
    # The rows above against the grids: 152 SMs of at most three (forward) or two (backward) blocks.
    for cols, rows in RING_ROWS.items():
        per_block = {256: 8, 512: 8, 1024: 4, 2048: 2}.get(cols, 1)
        blocks = 152 * (3 if cols <= 4096 else 2 if cols <= 5120 else 1)
        assert rows > 6 * blocks * per_block and rows % (blocks * per_block)
    for cols, rows in BWD_ROWS.items():
        per_block = {256: 8, 512: 8, 1024: 4, 2048: 2}.get(cols, 1)
        assert rows > 4 * 152 * (2 if cols <= 4096 else 1) * per_block
    assert np.prod([2003, 4096]) > 4 * 152 * 3 * 256 * 8  # more than four rows to a dropout thread
