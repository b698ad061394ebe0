"""The example that trains a layer with orthogonalised updates and serves it in
4 bits, end to end on small sizes."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_and_serve_layer",
                                                  os.path.join(ROOT, "examples", "train_and_serve_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("args", [["--format", "mx"], ["--format", "nv", "--four-bit"]])
def test_trains_and_serves(example, args):
    losses, err, apart = example.main(["--steps", "40", "--batch", "256", "--n-in", "300", "--n-out", "200",
                                       "--tokens", "20", *args])
    # an untrained layer answers with 0: the first loss is the outputs' mean
    # square; orthogonalised steps bring all directions down together
    assert losses[-1] < 0.05 * losses[0]
    # two operands of 4 bits, each about 0.1 off: 0.15 together
    assert err < 0.25
    # the same codes and scales, summed by another kernel: bf16 output apart by
    # rounding alone (2^-9)
    assert apart < 4e-3
