"""Host-side checks of the root-mean-square norm's and the gated block's entry points (no GPU, no kernel launched).

* the 64-bit plain forms' gradients are pinned to differences of their formulas;
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

import gated_plain as plain
from conftest import ROOT, gpu_available

FAKE = 1 << 40
STRUCTS = ("rms_norm", "rms_norm_bwd", "reduce_rms_norm", "gated_linear", "gated_linear_bwd")


# ---- the plain forms ----------------------------------------------------------------

def test_rms_norm_gradients_against_differences():
    r = np.random.default_rng(0)
    x, w, dy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7))
    _, _, rstd = plain.rms_norm(x, w)
    dx, dw = plain.rms_norm_bwd(dy, x, rstd, w)
    h = 1e-6
    loss = lambda x, w: (plain.rms_norm(x, w)[0] * dy).sum()  # noqa: E731
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7
    assert np.allclose(plain.rms_norm_bwd(dy, x, rstd, w, dy)[0], dx + dy)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_gated_gradients_against_differences(act):
    r = np.random.default_rng(1)
    a = [r.normal(size=s) for s in ((3, 5), (4, 5), (4, 5), (4,), (4,))]  # x, both weights, both biases
    dout = r.normal(size=(3, 4))
    loss = lambda a: (plain.gated(*a[:3], act, *a[3:])[0] * dout).sum()  # noqa: E731
    _, g, u = plain.gated(*a[:3], act, *a[3:])
    grads, h = plain.gated_bwd(dout, g, u, *a[:3], act), 1e-6
    for i, grad in enumerate(grads):
        for at in np.ndindex(a[i].shape):
            up, down = [t.copy() for t in a], [t.copy() for t in a]
            up[i][at] += h
            down[i][at] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - grad[at]) < 1e-7


# ---- the C interface ----------------------------------------------------------------

def test_struct_layouts_match_the_header(arx, tmp_path):
    cc = shutil.which(os.environ.get("CC", "gcc"))
    assert cc, "a C compiler is needed"
    lines = []
    for op in STRUCTS:
        t = f"arx_{op}_args"
        lines.append(f'printf("{t} %zu\\n", sizeof({t}));')
        lines += [f'printf("{t}.{f} %zu\\n", offsetof({t}, {f}));' for f, _ in getattr(arx, t)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "arx.h"\nint main(void) {' + "\n".join(lines)
                   + "return 0; }\n")
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
    if op == "rms_norm":
        a = arx.arx_rms_norm_args(rows=4, cols=16, ldx=16, ldresidual=16, ldh=16, ldy=16, ldq=16, eps=1e-6)
        names = "x residual weight h y q scale rstd"
    elif op == "rms_norm_bwd":
        a = arx.arx_rms_norm_bwd_args(rows=4, cols=16, lddy=16, ldh=16, lddresidual=16, lddx=16)
        a.workspace_bytes = arx.arx_rms_norm_bwd_workspace_bytes(4, 16)
        names = "dy h rstd weight dresidual dx dweight workspace"
    elif op == "gated_linear":
        a = arx.arx_gated_linear_args(M=4, N=16, K=8, ldx=8, ldw_gate=8, ldw_up=8, ldout=16, ldz_gate=16, ldz_up=16, act=4)
        names = "x w_gate w_up bias_gate bias_up out z_gate z_up status"
    elif op == "gated_linear_bwd":
        a = arx.arx_gated_linear_bwd_args(M=4, N=16, K=8, lddout=16, ldz_gate=16, ldz_up=16, ldx=8, ldw_gate=8, ldw_up=8,
                                          lddx=8, lddw_gate=8, lddw_up=8, act=4)
        a.workspace_bytes = arx.arx_gated_linear_bwd_workspace_bytes(4, 16)
        names = "dout z_gate z_up x w_gate w_up dx dw_gate dw_up dbias_gate dbias_up workspace status"
    else:
        a = arx.arx_reduce_rms_norm_args(rows=4, cols=16, ldq=16, W=2, eps=1e-6)
        slots = (ctypes.c_void_p * 2)(_region(20), _region(21))
        a.slots = ctypes.cast(slots, ctypes.c_void_p)
        a._keep = slots
        names = "residual weight h y q scale rstd"
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
    ("rms_norm", {"x": 0}, "EINVAL", "x is null"),
    ("rms_norm", {"y": 0, "q": 0}, "EINVAL", "y and q are null"),
    ("rms_norm", {"scale": 0}, "EINVAL", "scale is null"),
    ("rms_norm", {"x": FAKE + 1}, "EINVAL", "aligned"),
    ("rms_norm", {"scale": FAKE + 2}, "EINVAL", "aligned"),
    ("rms_norm", {"ldx": 15}, "EINVAL", "leading dimension"),
    ("rms_norm", {"ldq": 15}, "EINVAL", "leading dimension 15 of q"),
    ("rms_norm", {"ldh": 1 << 50}, "EINVAL", "leading dimension"),
    ("rms_norm", {"rows": 1 << 31}, "EINVAL", "2^31"),
    ("rms_norm", {"cols": 1 << 31}, "EINVAL", "2^31"),
    ("rms_norm", {"eps": -1.0}, "EINVAL", "eps"),
    ("rms_norm", {"eps": float("nan")}, "EINVAL", "eps"),
    ("rms_norm", {"dtype": 3}, "EINVAL", "dtype"),
    ("rms_norm", {"wdtype": 1}, "EINVAL", "wdtype"),
    ("rms_norm", {"h": _region(0) + 2}, "EOVERLAP", "h overlaps x"),
    ("rms_norm", {"y": _region(3)}, "EOVERLAP", "y overlaps h"),
    ("rms_norm", {"y": _region(2)}, "EOVERLAP", "y overlaps weight"),
    ("rms_norm", {"q": _region(0)}, "EOVERLAP", "q overlaps x"),
    ("rms_norm", {"q": _region(4) + 100}, "EOVERLAP", "q overlaps y"),
    ("rms_norm", {"rstd": _region(6)}, "EOVERLAP", "rstd overlaps scale"),
    ("rms_norm", {"h": _region(1), "ldh": 24}, "EOVERLAP", "h overlaps residual"),
    ("rms_norm_bwd", {"dy": 0}, "EINVAL", "dy is null"),
    ("rms_norm_bwd", {"h": 0}, "EINVAL", "h is null"),
    ("rms_norm_bwd", {"rstd": 0}, "EINVAL", "rstd is null"),
    ("rms_norm_bwd", {"workspace": 0}, "EINVAL", "workspace is null"),
    ("rms_norm_bwd", {"workspace": FAKE + 8}, "EINVAL", "aligned"),
    ("rms_norm_bwd", {"workspace_bytes": 3}, "EINVAL", "need"),
    ("rms_norm_bwd", {"dx": _region(1) + 32}, "EOVERLAP", "dx overlaps h"),
    ("rms_norm_bwd", {"dweight": _region(3)}, "EOVERLAP", "dweight overlaps weight"),
    ("rms_norm_bwd", {"workspace": _region(5)}, "EOVERLAP", "workspace overlaps dx"),
    ("reduce_rms_norm", {"W": 0}, "EINVAL", "W=0"),
    ("reduce_rms_norm", {"W": 9}, "EINVAL", "W=9"),
    ("reduce_rms_norm", {"slots": 0}, "EINVAL", "null pointer array"),
    ("reduce_rms_norm", {"y": 0, "q": 0}, "EINVAL", "y and q are null"),
    ("reduce_rms_norm", {"scale": 0}, "EINVAL", "scale is null"),
    ("reduce_rms_norm", {"eps": -1.0}, "EINVAL", "eps"),
    ("reduce_rms_norm", {"ldq": 8}, "EINVAL", "leading dimension 8 of q"),
    ("reduce_rms_norm", {"h": _region(3)}, "EOVERLAP", "y overlaps h"),
    ("reduce_rms_norm", {"h": _region(20) + 2}, "EOVERLAP", "h overlaps a slot"),
    ("reduce_rms_norm", {"q": _region(21)}, "EOVERLAP", "q overlaps a slot"),
    ("reduce_rms_norm", {"y": _region(1)}, "EOVERLAP", "y overlaps weight"),
    ("gated_linear", {"x": 0}, "EINVAL", "x is null"),
    ("gated_linear", {"w_gate": 0}, "EINVAL", "w_gate is null"),
    ("gated_linear", {"w_up": 0}, "EINVAL", "w_up is null"),
    ("gated_linear", {"out": 0}, "EINVAL", "out is null"),
    ("gated_linear", {"dtype": 2, "out_dtype": 2, "wdtype": 2}, "EINVAL", "dtype"),
    ("gated_linear", {"dtype": 4}, "EINVAL", "dtype"),
    ("gated_linear", {"dtype": 0, "out_dtype": 1}, "EINVAL", "out_dtype 1 is not dtype"),
    ("gated_linear", {"dtype": 3, "out_dtype": 3}, "EINVAL", "dtype"),
    ("gated_linear", {"dtype": 3, "out_dtype": 2}, "EINVAL", "dtype"),
    ("gated_linear", {"dtype": 3, "wdtype": 1}, "EINVAL", "wdtype"),
    ("gated_linear", {"dtype": 3}, "EINVAL", "8-bit x not on rows of 16 bytes"),
    ("gated_linear", {"dtype": 3, "ldx": 16, "ldw_gate": 16, "ldw_up": 24}, "EINVAL", "8-bit w_up not on rows"),
    ("gated_linear", {"dtype": 3, "ldx": 16, "ldw_gate": 16, "ldw_up": 16, "w_gate": _region(1) + 8}, "EINVAL", "8-bit w_gate"),
    ("gated_linear", {"x_scale": _region(30)}, "EINVAL", "scales without 8-bit operands"),
    ("gated_linear", {"up_scale": _region(30)}, "EINVAL", "scales without 8-bit operands"),
    ("gated_linear", {"dtype": 3, "gate_scale": _region(30) + 2}, "EINVAL", "gate_scale not 4-byte aligned"),
    ("gated_linear", {"act": 5}, "EINVAL", "activation"),
    ("gated_linear", {"act": -1}, "EINVAL", "activation"),
    ("gated_linear", {"wait_us": -1}, "EINVAL", "wait_us=-1"),
    ("gated_linear", {"wait_us": 2000001}, "EINVAL", "wait_us=2000001"),
    ("gated_linear", {"N": 1 << 31}, "EINVAL", "2^31"),
    ("gated_linear", {"ldw_up": 7}, "EINVAL", "leading dimension"),
    ("gated_linear", {"x": FAKE + 1}, "EINVAL", "aligned"),
    ("gated_linear", {"out": _region(0)}, "EOVERLAP", "out overlaps x"),
    ("gated_linear", {"z_gate": _region(5)}, "EOVERLAP", "z_gate overlaps out"),
    ("gated_linear", {"z_up": _region(6)}, "EOVERLAP", "z_up overlaps z_gate"),
    ("gated_linear", {"out": _region(4)}, "EOVERLAP", "out overlaps bias_up"),
    ("gated_linear_bwd", {"dout": 0}, "EINVAL", "dout is null"),
    ("gated_linear_bwd", {"z_gate": 0}, "EINVAL", "z_gate is null"),
    ("gated_linear_bwd", {"z_up": 0}, "EINVAL", "z_up is null"),
    ("gated_linear_bwd", {"x": 0}, "EINVAL", "x is null"),
    ("gated_linear_bwd", {"w_up": 0}, "EINVAL", "w_up is null"),
    ("gated_linear_bwd", {"dtype": 3, "wdtype": 3}, "EINVAL", "dtype"),
    ("gated_linear_bwd", {"act": 7}, "EINVAL", "activation"),
    ("gated_linear_bwd", {"wait_us": -5}, "EINVAL", "wait_us=-5"),
    ("gated_linear_bwd", {"workspace": 0}, "EINVAL", "workspace is null"),
    ("gated_linear_bwd", {"workspace_bytes": 16}, "EINVAL", "need"),
    ("gated_linear_bwd", {"dx": _region(0)}, "EOVERLAP", "dx overlaps dout"),
    ("gated_linear_bwd", {"dw_up": _region(7)}, "EOVERLAP", "dw_up overlaps dw_gate"),
    ("gated_linear_bwd", {"workspace": _region(3)}, "EOVERLAP", "workspace overlaps x"),
]


@pytest.mark.parametrize("op,change,status,words", REFUSED, ids=lambda v: str(v)[:40])
def test_refusals(arx, op, change, status, words):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == getattr(arx, "ARX_" + status), arx.arx_last_error()
    assert words in arx.arx_last_error()


@pytest.mark.parametrize("op,change", [
    ("rms_norm", {"rows": 0}), ("rms_norm", {"cols": 0}), ("rms_norm_bwd", {"cols": 0}), ("reduce_rms_norm", {"rows": 0}),
    ("rms_norm_bwd", {"dx": 0, "dweight": 0}), ("gated_linear", {"M": 0}), ("gated_linear", {"N": 0}),
    ("gated_linear_bwd", {"dx": 0, "dw_gate": 0, "dw_up": 0, "dbias_gate": 0, "dbias_up": 0})])
def test_nothing_to_do_launches_nothing(arx, op, change):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == arx.ARX_OK


@pytest.mark.skipif(gpu_available(), reason="valid arguments would launch on fabricated addresses")
@pytest.mark.parametrize("op,change", [
    ("rms_norm", {"h": _region(0)}), ("rms_norm", {"h": _region(1), "y": _region(0)}), ("rms_norm", {"y": _region(1)}),
    ("rms_norm", {"q": 0, "scale": 0}), ("rms_norm", {"y": 0}), ("rms_norm", {"residual": 0, "weight": 0, "h": 0, "rstd": 0}),
    ("rms_norm", {"rows": 1, "ldx": 0, "ldq": 0}),                     # one row: no leading dimension
    ("rms_norm", {"ldq": 17, "q": _region(5) + 3}),                          # bytes at any address
    ("rms_norm_bwd", {"dx": _region(0)}), ("rms_norm_bwd", {"dx": _region(1)}), ("rms_norm_bwd", {"dx": _region(4)}),
    ("rms_norm_bwd", {"dweight": 0, "workspace": 0}), ("rms_norm_bwd", {"rows": 0}),
    ("reduce_rms_norm", {"h": _region(0), "y": _region(20)}), ("reduce_rms_norm", {"h": 0}), ("reduce_rms_norm", {"y": 0}),
    ("gated_linear", {"bias_gate": 0, "z_up": 0, "status": 0}), ("gated_linear", {"w_up": _region(1)}),
    ("gated_linear", {"w_up": _region(1) + 16, "ldw_gate": 16, "ldw_up": 16}),
    ("gated_linear", {"dtype": 3, "out_dtype": 1, "wdtype": 1, "ldx": 16, "ldw_gate": 16, "ldw_up": 16, "x_scale": _region(30)}),
    ("gated_linear", {"K": 0, "x": 0, "w_gate": 0, "w_up": 0}),
    ("gated_linear_bwd", {"dx": 0, "w_gate": 0, "w_up": 0}), ("gated_linear_bwd", {"dw_gate": 0, "dw_up": 0, "x": 0}),
    ("gated_linear_bwd", {"dx": 0, "dw_gate": 0, "dw_up": 0, "x": 0, "w_gate": 0, "w_up": 0})])
def test_allowed_aliases_and_omissions(arx, op, change):
    a = _good(arx, op)
    for k, v in change.items():
        setattr(a, k, v)
    assert _call(arx, op, a) == arx.ARX_ECUDA, arx.arx_last_error()  # past the checks: no device here


def test_workspace_bytes(arx):
    f = arx.arx_rms_norm_bwd_workspace_bytes
    assert f(0, 0) == 0 and f(1 << 31, 8) == 0 and f(8, 1 << 31) == 0
    assert f(1, 4096) == 4096 * 4 and f(100, 4096) < f(5000, 4096) <= f(50000, 4096)

    f = arx.arx_gated_linear_bwd_workspace_bytes
    assert f(0, 0) == 0 and f(1 << 31, 8) == 0 and f(8, 1 << 31) == 0
    assert f(10, 13) >= 2 * (10 * 16 * 2 + 13 * 4) and f(100, 4096) < f(5000, 4096)


@pytest.mark.parametrize("op,operand", [("gated_linear", "w_up"), ("gated_linear_bwd", "w_gate"), ("gated_linear_bwd", "x")])
def test_copies_are_needed_and_checked(arx, op, operand):
    """Operands whose rows are off 16 bytes: the call asks for copies and does nothing without."""
    query, call = getattr(arx.lib, f"arx_{op}_copies_bytes"), getattr(arx.lib, f"arx_{op}")
    a = _good(arx, op)
    a.M, a.N, a.K = M, N, K = 1003, 204, 4100
    for n, _ in a._fields_:
        if n.startswith("ld"):
            setattr(a, n, K if n in ("ldx", "ldw_gate", "ldw_up", "lddx", "lddw_gate", "lddw_up") else N)
    if op == "gated_linear_bwd":
        a.workspace_bytes = arx.arx_gated_linear_bwd_workspace_bytes(M, N)
    n = query(ctypes.byref(a))
    assert n == (M + 2 * N) * 4104 * 2
    assert call(ctypes.byref(a), None) == arx.ARX_EINVAL and f"copies is null, {n} bytes needed" in arx.arx_last_error()
    a.copies, a.copies_bytes = _region(40), n - 1
    assert call(ctypes.byref(a), None) == arx.ARX_EINVAL and "copies" in arx.arx_last_error()
    a.copies, a.copies_bytes = _region(40) + 8, n
    assert call(ctypes.byref(a), None) == arx.ARX_EINVAL and "copies not 16-byte aligned" in arx.arx_last_error()
    a.copies = getattr(a, operand)
    assert call(ctypes.byref(a), None) == arx.ARX_EOVERLAP and "copies" in arx.arx_last_error()
    for name in ("ldx", "ldw_gate", "ldw_up"):
        setattr(a, name, 4104)
    assert query(ctypes.byref(a)) == 0
    a.M = 1 << 31
    assert query(ctypes.byref(a)) == 0
    assert query(None) == 0


def test_one_or_two_rows_of_small_weights_need_no_copies(arx):
    a = _good(arx, "gated_linear")
    a.M, a.K, a.ldx, a.ldw_gate, a.ldw_up = 2, 13, 13, 13, 15
    assert arx.lib.arx_gated_linear_copies_bytes(ctypes.byref(a)) == 0
    a.M = 3
    assert arx.lib.arx_gated_linear_copies_bytes(ctypes.byref(a)) == (3 + 16 + 16) * 16 * 2


def test_binding_rejects_tensors_of_the_wrong_kind(arx):
    import torch
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    q = torch.zeros(4, 16, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA tensor"):
        arx.arx_rms_norm(x, x)
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_rms_norm(q, q)
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_layer_norm(q, q)
    with pytest.raises(TypeError, match="bfloat16"):
        arx.arx_reduce_rms_norm([x.half()], x, x)
    with pytest.raises(ValueError, match="none given"):
        arx.arx_reduce_rms_norm([], x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        arx.arx_rms_norm_plan(x, None, q=q)
    out = torch.zeros(4, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        arx.arx_gated_linear(x, x, x, out)
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_gated_linear(x.float(), x.float(), x.float(), out.float())
    with pytest.raises(TypeError, match="not supported"):
        arx.arx_gated_linear_bwd(q, q, q, q, q, q)
