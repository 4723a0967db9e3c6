"""Host-side checks of the operators around the reduce (no GPU, no kernel launched).

* the 64-bit plain forms are pinned: the generator to its published vectors,
  the gradients to differences of the forward formulas;
* the binding's structs have the layout that a C compiler gives the header's;
* every refusal returns its status before any CUDA call (the addresses are
  fabricated integers: nothing could dereference them);
* the binding refuses tensors of the wrong kind.
"""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import ops_plain as plain
from conftest import ROOT, gpu_available

FAKE = 1 << 40


# ---- the plain forms ----------------------------------------------------------------

def test_generator_matches_the_published_vectors():
    # Known answers of Philox4x32-10, as published with the generator.
    ones = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones,) * 4, (ones, ones), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(plain.philox4x32_10(counter, key)) == want
    # The array form is the same generator, in the documented order.
    v = plain.dropout_values(5, 21, seed=0x299F31D0A4093822, offset=0x0370734413198A2E)
    for row, col in ((0, 0), (4, 20), (3, 7), (2, 8), (1, 13)):
        w = plain.philox4x32_10((col // 8, row, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0))
        j = col % 8
        assert v[row, col] == (w[j // 2] >> (16 * (j % 2))) & 0xFFFF


def test_dropout_values_are_uniform():
    # 2^18 values against p: the kept count is binomial; five standard deviations.
    v = plain.dropout_values(512, 512, seed=11, offset=3)
    for p in (0.1, 0.5, 0.9):
        T = round(65536 * p)
        q = 1 - T / 65536
        assert abs((v >= T).sum() - v.size * q) < 5 * (v.size * q * (1 - q)) ** 0.5


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu", "none"])
def test_activation_gradients_against_differences(name):
    z = np.linspace(-6, 6, 97) + 0.01
    h = 1e-5
    d = (plain.act(z + h, name) - plain.act(z - h, name)) / (2 * h)
    assert np.abs(d - plain.act_grad(z, name)).max() < 1e-8  # h^2 times a third derivative, and rounding / h


def test_layer_norm_gradients_against_differences():
    r = np.random.default_rng(0)
    x, w, b, dy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=7), r.normal(size=(3, 7))
    _, mean, rstd = plain.layer_norm(x, w, b)
    dx, dw, db = plain.layer_norm_bwd(dy, x, mean, rstd, w)
    h = 1e-6
    loss = lambda x, w, b: (plain.layer_norm(x, w, b)[0] * dy).sum()  # noqa: E731
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - dw[j]) < 1e-7
        assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - db[j]) < 1e-7


# ---- the C interface ----------------------------------------------------------------

STRUCTS = ("layer_norm", "layer_norm_bwd", "dropout_add", "dropout_add_bwd", "reduce_layer_norm", "linear",
           "linear_bwd")


def test_struct_layouts_match_the_header(arx, tmp_path):
    cc = shutil.which(os.environ.get("CC", "gcc"))
    assert cc, "a C compiler is needed"
    lines = []
    for op in STRUCTS:
        t = f"arx_{op}_args"
        lines.append(f'printf("{t} %zu\\n", sizeof({t}));')
        lines += [f'printf("{t}.{f} %zu\\n", offsetof({t}, {f}));' for f, _ in getattr(arx, t)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "arx.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c11", "-Wall", str(src), "-I", os.path.join(ROOT, "include"), "-o", exe], check=True)
    got = dict(x.split() for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    for op in STRUCTS:
        t = getattr(arx, f"arx_{op}_args")
        assert int(got[t.__name__]) == ctypes.sizeof(t)
        for f, _ in t._fields_:
            assert int(got[f"{t.__name__}.{f}"]) == getattr(t, f).offset, (t.__name__, f)


def _region(i):
    return FAKE + (i << 32)


def _good(arx, op):
    """Valid arguments of ``op`` with every pointer set."""
    if op == "linear":
        a = arx.arx_linear_args(M=4, N=16, K=8, ldx=8, ldw=8, ldresidual=16, ldout=16, ldz=16, act=2)
        names = "x w bias residual out z status"
    elif op == "linear_bwd":
        a = arx.arx_linear_bwd_args(M=4, N=16, K=8, lddout=16, ldz=16, ldx=8, ldw=8, lddx=8, lddw=8, act=2)
        a.workspace_bytes = arx.arx_linear_bwd_workspace_bytes(4, 16)
        names = "dout z x w dx dw dbias workspace status"
    elif op == "layer_norm":
        a = arx.arx_layer_norm_args(rows=4, cols=16, ldx=16, ldy=16, eps=1e-5)
        names = "x weight bias y mean rstd"
    elif op == "layer_norm_bwd":
        a = arx.arx_layer_norm_bwd_args(rows=4, cols=16, lddy=16, ldx=16, lddresidual=16, lddx=16)
        a.workspace_bytes = arx.arx_layer_norm_bwd_workspace_bytes(4, 16)
        names = "dy x mean rstd weight dresidual dx dweight dbias workspace"
    elif op == "dropout_add":
        a = arx.arx_dropout_add_args(rows=4, cols=16, ldx=16, ldresidual=16, ldout=16, p=0.5)
        names = "x bias residual out rng"
    elif op == "dropout_add_bwd":
        a = arx.arx_dropout_add_bwd_args(rows=4, cols=16, lddout=16, lddx=16, p=0.5)
        a.workspace_bytes = arx.arx_dropout_add_bwd_workspace_bytes(4, 16)
        names = "dout dx dbias rng workspace"
    else:
        a = arx.arx_reduce_layer_norm_args(rows=4, cols=16, W=2, eps=1e-5, p=0.5)
        slots = (ctypes.c_void_p * 2)(_region(20), _region(21))
        a.slots = ctypes.cast(slots, ctypes.c_void_p)
        a._keep = slots
        names = "bias residual weight norm_bias h y mean rstd rng"
    for i, n in enumerate(names.split()):
        setattr(a, n, _region(i))
    return a


def _call(arx, op, a):
    return getattr(arx.lib, f"arx_{op}")(ctypes.byref(a), None)


@pytest.mark.parametrize("op", STRUCTS)
@pytest.mark.skipif(gpu_available(), reason="checks the no-device error path")
def test_valid_arguments_reach_the_launch(arx, op):
    # Nothing is refused, so the call gets as far as CUDA and reports that there is no device.
    assert _call(arx, op, _good(arx, op)) == arx.ARX_ECUDA, arx.arx_last_error()
    assert arx.arx_last_error()


@pytest.mark.parametrize("op", STRUCTS)
def test_null_arguments(arx, op):
    assert getattr(arx.lib, f"arx_{op}")(None, None) == arx.ARX_EINVAL


REFUSED = [
    # op, changes, status, words of the message
    ("layer_norm", {"x": 0}, "EINVAL", "x is null"),
    ("layer_norm", {"y": 0}, "EINVAL", "y is null"),
    ("layer_norm", {"x": FAKE + 1}, "EINVAL", "aligned"),
    ("layer_norm", {"mean": FAKE + 2}, "EINVAL", "aligned"),
    ("layer_norm", {"ldx": 15}, "EINVAL", "leading dimension"),
    ("layer_norm", {"ldx": 1 << 50}, "EINVAL", "leading dimension"),
    ("layer_norm", {"rows": 1 << 31}, "EINVAL", "2^31"),
    ("layer_norm", {"cols": 1 << 31}, "EINVAL", "2^31"),
    ("layer_norm", {"eps": -1.0}, "EINVAL", "eps"),
    ("layer_norm", {"eps": float("nan")}, "EINVAL", "eps"),
    ("layer_norm", {"dtype": 3}, "EINVAL", "dtype"),
    ("layer_norm", {"wdtype": 1}, "EINVAL", "wdtype"),
    ("layer_norm", {"y": _region(0) + 2}, "EOVERLAP", "y overlaps x"),
    ("layer_norm", {"y": _region(1)}, "EOVERLAP", "y overlaps weight"),
    ("layer_norm", {"mean": _region(5)}, "EOVERLAP", "rstd overlaps mean"),
    ("layer_norm", {"y": _region(0), "ldy": 24}, "EOVERLAP", "y overlaps x"),
    ("layer_norm_bwd", {"dy": 0}, "EINVAL", "dy is null"),
    ("layer_norm_bwd", {"mean": 0}, "EINVAL", "mean is null"),
    ("layer_norm_bwd", {"rstd": 0}, "EINVAL", "rstd is null"),
    ("layer_norm_bwd", {"workspace": 0}, "EINVAL", "workspace is null"),
    ("layer_norm_bwd", {"workspace": FAKE + 8}, "EINVAL", "aligned"),
    ("layer_norm_bwd", {"workspace_bytes": 3}, "EINVAL", "need"),
    ("layer_norm_bwd", {"dx": _region(1) + 32}, "EOVERLAP", "dx overlaps x"),
    ("layer_norm_bwd", {"dweight": _region(4)}, "EOVERLAP", "dweight overlaps weight"),
    ("layer_norm_bwd", {"workspace": _region(6)}, "EOVERLAP", "workspace overlaps dx"),
    ("dropout_add", {"p": -0.1}, "EINVAL", "p="),
    ("dropout_add", {"p": 1.1}, "EINVAL", "p="),
    ("dropout_add", {"p": float("nan")}, "EINVAL", "p="),
    ("dropout_add", {"rng": 0}, "EINVAL", "rng is null"),
    ("dropout_add", {"rng": FAKE + 4}, "EINVAL", "rng"),
    ("dropout_add", {"out": _region(2) + 2}, "EOVERLAP", "out overlaps residual"),
    ("dropout_add", {"out": _region(1)}, "EOVERLAP", "out overlaps bias"),
    ("dropout_add", {"out": _region(4)}, "EOVERLAP", "out overlaps rng"),
    ("dropout_add_bwd", {"dout": 0}, "EINVAL", "dout is null"),
    ("dropout_add_bwd", {"workspace": 0}, "EINVAL", "workspace is null"),
    ("dropout_add_bwd", {"dx": _region(0) + 2}, "EOVERLAP", "dx overlaps dout"),
    ("dropout_add_bwd", {"dbias": _region(1)}, "EOVERLAP", "dbias overlaps dx"),
    ("reduce_layer_norm", {"W": 0}, "EINVAL", "W=0"),
    ("reduce_layer_norm", {"W": 9}, "EINVAL", "W=9"),
    ("reduce_layer_norm", {"slots": 0}, "EINVAL", "null pointer array"),
    ("reduce_layer_norm", {"y": 0}, "EINVAL", "y is null"),
    ("reduce_layer_norm", {"rng": 0}, "EINVAL", "rng is null"),
    ("reduce_layer_norm", {"h": _region(5)}, "EOVERLAP", "h overlaps y"),
    ("reduce_layer_norm", {"h": _region(20) + 2}, "EOVERLAP", "h overlaps a slot"),
    ("reduce_layer_norm", {"y": _region(2)}, "EOVERLAP", "y overlaps weight"),
    ("linear", {"x": 0}, "EINVAL", "x is null"),
    ("linear", {"w": 0}, "EINVAL", "w is null"),
    ("linear", {"out": 0}, "EINVAL", "out is null"),
    ("linear", {"dtype": 2, "wdtype": 2}, "EINVAL", "dtype"),
    ("linear", {"act": 5}, "EINVAL", "activation"),
    ("linear", {"act": -1}, "EINVAL", "activation"),
    ("linear", {"ldw": 7}, "EINVAL", "leading dimension"),
    ("linear", {"out": _region(0)}, "EOVERLAP", "out overlaps x"),
    ("linear", {"z": _region(3)}, "EOVERLAP", "z overlaps residual"),
    ("linear", {"z": _region(4)}, "EOVERLAP", "z overlaps out"),
    ("linear", {"out": _region(3), "ldout": 24}, "EOVERLAP", "out overlaps residual"),
    ("linear_bwd", {"z": 0}, "EINVAL", "z is null"),
    ("linear_bwd", {"x": 0}, "EINVAL", "x is null"),
    ("linear_bwd", {"w": 0}, "EINVAL", "w is null"),
    ("linear_bwd", {"workspace_bytes": 16}, "EINVAL", "need"),
    ("linear_bwd", {"dx": _region(0)}, "EOVERLAP", "dx overlaps dout"),
    ("linear_bwd", {"dw": _region(4)}, "EOVERLAP", "dw overlaps dx"),
]


@pytest.mark.parametrize("op,change,status,words", REFUSED, ids=lambda v: str(v)[:40])
def test_refusals(arx, op, change, status, words):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == getattr(arx, "ARX_" + status), arx.arx_last_error()
    assert words in arx.arx_last_error()


@pytest.mark.parametrize("op,change", [
    ("layer_norm", {"rows": 0}), ("layer_norm", {"cols": 0}), ("layer_norm_bwd", {"cols": 0}),
    ("dropout_add", {"rows": 0}), ("reduce_layer_norm", {"rows": 0}), ("linear", {"M": 0}), ("linear", {"N": 0}),
    ("dropout_add_bwd", {"cols": 0}),
    ("linear_bwd", {"dx": 0, "dw": 0, "dbias": 0}), ("layer_norm_bwd", {"dx": 0, "dweight": 0, "dbias": 0})])
def test_nothing_to_do_launches_nothing(arx, op, change):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == arx.ARX_OK


@pytest.mark.skipif(gpu_available(), reason="valid arguments would launch on fabricated addresses")
@pytest.mark.parametrize("op,change", [
    ("layer_norm", {"y": _region(0)}),                                 # in place
    ("layer_norm", {"ldx": 32, "ldy": 32, "y": _region(0) + 32}),      # interleaved views of one buffer
    ("layer_norm", {"rows": 1, "ldx": 0, "ldy": 0}),                   # one row: no leading dimension
    ("layer_norm_bwd", {"dx": _region(0)}), ("layer_norm_bwd", {"dx": _region(1)}),
    ("layer_norm_bwd", {"dx": _region(5)}),
    ("dropout_add", {"out": _region(0)}), ("dropout_add", {"out": _region(2)}),
    ("dropout_add", {"p": 0.0, "rng": 0}), ("dropout_add_bwd", {"dx": _region(0)}),
    ("reduce_layer_norm", {"h": _region(1), "y": _region(20)}), ("reduce_layer_norm", {"h": 0}),
    ("linear", {"out": _region(3)}), ("linear_bwd", {"act": 0, "z": 0, "dbias": 0, "workspace": 0})])
def test_allowed_aliases_and_omissions(arx, op, change):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == arx.ARX_ECUDA, arx.arx_last_error()  # past the checks: no device here


def test_workspace_bytes(arx):
    for f in (arx.arx_layer_norm_bwd_workspace_bytes, arx.arx_dropout_add_bwd_workspace_bytes,
              arx.arx_linear_bwd_workspace_bytes):
        assert f(0, 0) == 0 and f(1 << 31, 8) == 0 and f(8, 1 << 31) == 0
        last = 0
        for rows in (1, 8, 100, 5000):
            n = f(rows, 4096)
            assert n >= last  # more rows never need less
            last = n
    assert arx.arx_linear_bwd_workspace_bytes(10, 13) >= 10 * 16 * 2 + 13 * 4


def test_binding_rejects_tensors_of_the_wrong_kind(arx):
    import torch
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        arx.arx_layer_norm(x, x)
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_layer_norm(x.to(torch.int32), x)
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_linear(x.float(), x.float(), x.float())
    with pytest.raises(ValueError, match="contiguous"):
        arx.arx_layer_norm(x.t(), x)
    with pytest.raises(ValueError, match="overlap"):
        arx.arx_layer_norm(x[:1].expand(4, 16), x)
    with pytest.raises(ValueError, match="equally spaced"):
        arx.arx_layer_norm(torch.zeros(2, 6, 16, dtype=torch.bfloat16)[:, :4], x)
    with pytest.raises(ValueError, match="dimension"):
        arx.arx_dropout_add(x[0], x[0], 0.0)
    with pytest.raises(TypeError, match="bfloat16"):
        arx.arx_reduce_layer_norm([x], x, x.half())
    with pytest.raises(ValueError, match="CUDA tensor"):
        arx.arx_linear_plan(x, x, torch.zeros(4, 4, dtype=torch.bfloat16))


def _odd(arx, op):
    """Operands whose rows are off 16 bytes, at a size where copies of them pay."""
    a = _good(arx, op)
    M, N, K = 1003, 2044, 4100
    a.M, a.N, a.K = M, N, K
    if op == "linear":
        a.ldx = a.ldw = K
        a.ldresidual = a.ldout = a.ldz = N
    else:
        a.lddout = a.ldz = N
        a.ldx = a.ldw = a.lddx = a.lddw = K
        a.workspace_bytes = arx.arx_linear_bwd_workspace_bytes(M, N)
    return a


@pytest.mark.parametrize("op,operand", [("linear", "x"), ("linear_bwd", "w")])
def test_copies_are_asked_for_and_checked(arx, op, operand):
    query, call = getattr(arx.lib, f"arx_{op}_copies_bytes"), getattr(arx.lib, f"arx_{op}")
    a = _odd(arx, op)
    n = query(ctypes.byref(a))
    rows = {"linear": 1003 + 2044, "linear_bwd": 2044}[op]
    assert n == rows * 4104 * 2
    a.copies, a.copies_bytes = _region(40), n - 1
    assert call(ctypes.byref(a), None) == arx.ARX_EINVAL and "copies" in arx.arx_last_error()
    a.copies, a.copies_bytes = _region(40) + 8, n
    assert call(ctypes.byref(a), None) == arx.ARX_EINVAL and "copies not 16-byte aligned" in arx.arx_last_error()
    a.copies = getattr(a, operand)
    assert call(ctypes.byref(a), None) == arx.ARX_EOVERLAP and "copies" in arx.arx_last_error()
    for name in ("ldx", "ldw"):
        setattr(a, name, 4104)
    assert query(ctypes.byref(a)) == 0
    a.M = 1 << 31
    assert query(ctypes.byref(a)) == 0
    assert query(None) == 0
