"""GPU: what the sums of products with group scales lose, apart from the rounding of their results: exactly cancelling
sums, small groups between large ones, and results beside the nearest bf16 ones."""
import pytest
import torch

import fp8g_ref as ref
from test_gpu_fp8g import DEV, G, product, quantized, tokens

pytestmark = pytest.mark.gpu
BF16 = [(1030, 1000), (4000, 4000)]      # 64 x 128 tiles, 256 x 256 ones


def instruction(a, b, bits):
    """A group's sum as the FP8 matrix instruction makes it (a, b fp64 values of codes, [R, 128] each): of 8 products each
    is cut to a multiple of 2^-bits of the largest power of two that their factors' exponents give.  (Which 8 go
    together does not matter for values that are alike.)"""
    p = a[:, None, :] * b[None, :, :]
    low = lambda v: torch.frexp(v)[1] - 1  # noqa: E731
    e = torch.where(p == 0, torch.full_like(p, -100), (low(a)[:, None, :] + low(b)[None, :, :]).double())
    unit = torch.exp2(e.view(*p.shape[:2], -1, 8).amax(-1, keepdim=True) - bits)
    return ((p.view(*p.shape[:2], -1, 8) / unit).trunc() * unit).sum((-1, -2))


@pytest.mark.parametrize("M,N", BF16)
@pytest.mark.parametrize("e8", [0, 1])
@pytest.mark.parametrize("fa", [0, 1])
def test_cancelling_groups(M, N, e8, fa):
    """[X|-X'] [Y|Y']^T, where X', Y' have X's and Y's columns in another order: nothing, but for what the sums of two
    groups lose.  The instruction keeps 13 bits below the largest of 8
    products: two such losses, and half as much again for the sample; with 12 bits it would be 2.6 times as much."""
    g = torch.Generator().manual_seed(M)
    fmt = ref.TYPE[fa]
    x = (torch.randn(M, G, generator=g) * 100).clamp(-448, 448).to(fmt)
    y = (torch.randn(N, G, generator=g) * 100).clamp(-448, 448).to(ref.TYPE[0])
    perm = torch.randperm(G, generator=g)
    A = torch.cat([x.float(), -x.float()[:, perm]], 1).to(fmt).view(torch.uint8).to(DEV)
    B = torch.cat([y.float(), y.float()[:, perm]], 1).to(ref.TYPE[0]).view(torch.uint8).to(DEV)
    one = (lambda n: torch.full((2, n), 127, dtype=torch.uint8, device=DEV)) if e8 else (lambda n: torch.ones(2, n, device=DEV))
    got = product(A, one(M), B, one(N), M, N, 2 * G, torch.bfloat16, scale=e8, fmt_a=fa).double().cpu()
    a, b = x.float().double()[:200], y.float().double()[:200]
    loss = (instruction(a, b, 13) - a @ b.t()).square().mean().sqrt()
    assert float(got.square().mean().sqrt()) <= 1.5 * 2 ** 0.5 * float(loss)
    # few rows add in fp32: 128 roundings for each group at most
    few = product(A[:64].contiguous(), one(64), B, one(N), 64, N, 2 * G, torch.bfloat16, scale=e8, fmt_a=fa).double().cpu()
    sums = x.float().double()[:64].abs() @ y.float().double().abs().t()
    assert bool((few.abs() <= 2 * G * 2.0 ** -24 * 1.01 * sums).all())


@pytest.mark.parametrize("M,N,K", [(40, 264, 640), (1030, 1000, 640), (4000, 4000, 640)])
@pytest.mark.parametrize("e8", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_small_group_between_large_ones(M, N, K, e8, dtype):
    """Groups are added with fp32's 24 bits: beside +-2^14 one of 2^-9 is kept, also where the instruction adds them."""
    a, b = torch.zeros(M, K), torch.zeros(N, K)
    a[:, 0], a[:, 256 + 5], a[:, 512] = 256.0, 1.0, -256.0
    b[:, 0], b[:, 256 + 5], b[:, 512] = 64.0, 1.0, 64.0
    A, B = (t.to(ref.TYPE[0]).view(torch.uint8).to(DEV) for t in (a, b))
    for small in range(-9, 9):
        sA, sB = torch.full((K // G, M), 127, dtype=torch.uint8), torch.full((K // G, N), 127, dtype=torch.uint8)
        sA[2] = 127 + small
        if not e8:
            sA, sB = torch.exp2(sA.float() - 127), torch.exp2(sB.float() - 127)
        got = product(A, sA.to(DEV), B, sB.to(DEV), M, N, K, dtype, scale=e8)
        assert bool((got == 2.0 ** small).all()), (small, float(got[0, 0]))


@pytest.mark.parametrize("M,N,K,out,form", [s for s in ref.GEMM_FORMS if s[3] == "bf16"] + [(1030, 1000, 8192, "bf16", "SMALL")])
@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("square", [False, True])
def test_bf16_results_are_the_nearest(M, N, K, out, form, e8, square):
    """As a whole a bf16 result is no further from the exact one than the nearest bf16 numbers are, but for the sums: with
    a few values far above the rest the instruction's 13 bits (`instruction` on these inputs) lose up to 3.4e-4 of a
    row of results, a fifth of that rounding.  (A code in 128 off by 3 % would be 2.6e-3.)"""
    A, sA, a = quantized(tokens(M, M, K), e8)
    B, sB, b = quantized(tokens(N, N, K, 0.05), e8, square)
    got = product(A, sA, B, sB, M, N, K, torch.bfloat16, scale=int(e8), square=int(square)).double().cpu()
    want = a @ b.t()
    # row by row, since rows are of very different size
    err, nearest, size = ((t.norm(dim=1)) for t in (got - want, want.bfloat16().double() - want, want))
    assert bool((err <= 1.02 * nearest + 4e-4 * size).all()), float((err / size).max())
