"""The helper of the train-and-serve example that needs no GPU."""
import importlib.util
import os

import torch

import dense_gemm_accelerator_gb300 as dga

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_factor():
    spec = importlib.util.spec_from_file_location("train_and_serve_layer", os.path.join(ROOT, "examples", "train_and_serve_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.factor(torch.ones(3), dga.MXFP4) is None
    for largest, want in ((0.0, 1.0), (2688.0, 2.0), (2687.0, 1.0), (-1.0, 2.0 ** -11), (1e-30, 2.0 ** -111)):
        f = example.factor(torch.tensor([[0.0, largest], [0.0, 0.0]]), dga.NVFP4)
        assert f.shape == (1,) and f.dtype == torch.float32 and float(f) == want
