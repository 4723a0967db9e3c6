"""The tensor-parallel MLP example: its operators together, against torch in 32 bits."""

import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,hidden,tokens,dropout", [(2, 256, 70, 0.1), (8, 512, 33, 0.0), (4, 1024, 300, 0.5)])
def test_sublayer_training_and_serving(arx, ranks, hidden, tokens, dropout):
    spec = importlib.util.spec_from_file_location("tp_mlp", os.path.join(ROOT, "examples", "tensor_parallel_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    got = m.main(["--ranks", str(ranks), "--hidden", str(hidden), "--tokens", str(tokens), "--dropout", str(dropout)])
    assert got["same"] and got["served"]
    # Each result passes at most six roundings to bf16 of values of its own size
    # (z, a, p, h, dz, da or ds, and its own), 2^-9 each in the mean square.
    assert got["worst"] < 6 * 2.0 ** -9
