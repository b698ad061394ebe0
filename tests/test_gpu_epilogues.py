"""The tensor-core products' stores: with and without a bias and an old C, at sizes and
leading dimensions around the 32 x 32 blocks that leave together.  Small whole numbers,
so that every result is exact but for its rounding to the output's type."""
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "bf16 to fp32", "fp16", "fp16 to fp32", "tf32"])
@pytest.mark.parametrize("M,N,K", [(17, 40, 64), (100, 257, 96), (128, 256, 64), (129, 96, 64), (256, 512, 320), (300, 1000, 72), (545, 321, 128)])
def test_bias_and_old_values(M, N, K, kind):
    dtype = torch.float32 if kind == "tf32" else torch.float16 if "fp16" in kind else torch.bfloat16
    out = torch.float32 if "32" in kind else dtype
    g = torch.Generator(device="cuda").manual_seed(M + N)
    r = lambda lo, *s: torch.randint(lo, -lo + 1, s, device="cuda", generator=g).float()  # noqa: E731
    A, B, bias = r(-3, M, K).to(dtype), r(-3, N, K).to(dtype), r(-8, N).to(out)
    product = A.double() @ B.double().t()
    for pad, off in ((0, 0), (8, 0), (3, 0), (8, 1)):
        for alpha, beta, b in ((1.0, 0.0, None), (1.0, 0.0, bias), (0.5, 1.0, None), (1.0, -2.0, bias), (-2.0, 0.0, bias)):
            old = r(-16, M, N).to(out)
            held = torch.full(((M + 1) * (N + pad) + off + 40,), 7.0, dtype=out, device="cuda")
            C = held[off:off + M * (N + pad)].view(M, N + pad)[:, :N]
            C.copy_(old if beta else torch.full_like(old, float("nan")))
            got = dga.gemm(A, B.t(), C, alpha=alpha, beta=beta, bias=b, tf32=kind == "tf32")
            assert got is C
            want = alpha * product + (beta * old.double() if beta else 0) + (0 if b is None else b.double())
            assert torch.equal(C, want.to(out)), (pad, off, alpha, beta, b is None)
            C.fill_(7.0)
            assert bool((held == 7.0).all())
