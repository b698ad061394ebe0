"""A fully-connected layer trained with orthogonalised updates, then held and
served in 4 bits.

    python examples/train_and_serve_layer.py [--steps 60] [--format mx|nv]

Y = X W^T + b is fitted to a teacher layer's outputs.  Each step computes the
gradients with linear_backward (or, with --four-bit, its products in 4 bits:
mx_linear_backward), keeps a momentum of the weight's gradient and moves the
weight along the orthogonalised momentum (orthogonalize), whose singular values
are all near one, so that the step's size needs no tuning by layer.  The
trained weight is then quantised once (mx_quantize) and answers a prompt and
single tokens through mx_linear_forward.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_accelerator_gb300 as dga  # noqa: E402


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def factor(x, fmt):
    """An NVFP4 tensor scale (a power of two, so that it rounds nothing; 1 for a zero tensor), or None."""
    if fmt == dga.MXFP4:
        return None
    r = (x.abs().amax().float() / 2688.0).reshape(1)
    return torch.ldexp(torch.ones_like(r), torch.frexp(r).exponent)


def train(steps, batch, n_in, n_out, fmt, four_bit, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn(n_out, n_in, device="cuda", generator=g) / math.sqrt(n_in)
    W = torch.zeros(n_out, n_in, device="cuda")
    b = torch.zeros(n_out, device="cuda")
    momentum = torch.zeros_like(W)
    losses = []
    for step in range(steps):
        X = torch.randn(batch, n_in, device="cuda", generator=g).bfloat16()
        T = dga.linear_forward(X, teacher.bfloat16())
        Y = dga.linear_forward(X, W.bfloat16(), b.bfloat16())
        G = ((Y.float() - T.float()) * (2.0 / batch)).bfloat16()
        if four_bit:
            _, dW, db = dga.mx_linear_backward(X, W.bfloat16(), G, fmt, tensor_scales=(factor(X, fmt), factor(W, fmt), factor(G, fmt)))
        else:
            _, dW, db = dga.linear_backward(X, W.bfloat16(), G)
        momentum.mul_(0.9).add_(dW.float())
        # a step of 1 moves the weight as far as one of its own singular values
        rate = 0.15 * (1 - step / steps)
        W -= rate * dga.orthogonalize(momentum.bfloat16()).float()
        b -= 0.1 * db
        losses.append(float((Y.float() - T.float()).square().mean()))
    return W, b, teacher, losses


def serve(W, b, fmt, tokens, seed=1):
    """Relative errors of the 4-bit layer against the fp32 one, for a prompt and token by token."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(tokens, W.shape[1], device="cuda", generator=g).bfloat16()
    held = dga.mx_quantize(W, fmt, tensor_scale=factor(W, fmt))
    fx, bias = factor(X, fmt), b.bfloat16()
    prompt = dga.mx_linear_forward(X, held, bias, tensor_scale=fx)
    single = torch.cat([dga.mx_linear_forward(X[i:i + 1], held, bias, tensor_scale=fx) for i in range(tokens)])
    exact = X.float() @ W.t() + b
    bytes_held = held.codes.numel() + held.scales.numel()
    return relative(prompt, exact), relative(single, prompt), bytes_held / (2 * W.numel())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=512)
    ap.add_argument("--n-in", type=int, default=1000)
    ap.add_argument("--n-out", type=int, default=700)
    ap.add_argument("--format", choices=("mx", "nv"), default="mx")
    ap.add_argument("--four-bit", action="store_true", help="the gradients' products in 4 bits too")
    ap.add_argument("--tokens", type=int, default=40)
    a = ap.parse_args(argv)
    fmt = dga.MXFP4 if a.format == "mx" else dga.NVFP4
    W, b, teacher, losses = train(a.steps, a.batch, a.n_in, a.n_out, fmt, a.four_bit)
    err, apart, size = serve(W, b, fmt, a.tokens)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.5f} in {a.steps} steps; weight off the teacher's by {relative(W, teacher):.3f}")
    print(f"served in 4 bits ({size:.2f} of the bf16 weight's bytes): {err:.3f} off fp32, token by token {apart:.1e} off the prompt")
    return losses, err, apart


if __name__ == "__main__":
    main()
