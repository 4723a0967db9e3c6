"""The gated sublayer end to end: the operators as they are used together, training and serving."""

import importlib.util
import os

import pytest

pytest.importorskip("torch")
from conftest import ROOT  # noqa: E402

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("gated_mlp", os.path.join(ROOT, "examples", "tensor_parallel_gated_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ranks,hidden,tokens", [(2, 512, 96), (4, 1000, 33), (3, 1536, 300)])
def test_training_step_and_serving_graph(arx, ranks, hidden, tokens):
    r = _example().main(["--ranks", str(ranks), "--hidden", str(hidden), "--tokens", str(tokens)])
    assert r["same"] and r["served"]
    # A value passes at most twelve roundings to bf16 on its way (slots, norms, projections, their
    # gradients and the sums), 2^-8 of its size each, most of them independent: sqrt(12) of one
    # in the mean, and never all twelve.
    assert r["worst"] < 12 * 2.0 ** -8
    # e4m3 puts half a step of 2^-4 on both operands of the projections, whose products enter the
    # residual stream through a mean over hundreds of them.
    assert r["eight"] < 2.0 ** -4
