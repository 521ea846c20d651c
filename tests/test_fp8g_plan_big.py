"""The kernels that the largest sizes of the GPU tests of FP8 with group scales take (CPU)."""
import pytest

import fp8g_big as big
import fp8g_ref as ref
from test_fp8g_plan import plan  # noqa: F401


@pytest.mark.parametrize("M,N,K,out,form", big.GEMM)
def test_gemm(plan, M, N, K, out, form):  # noqa: F811
    assert plan("gemm", M, N, K // 128, int(out == "f32")) == form
    assert M * K > 1 << 32


@pytest.mark.parametrize("back,sizes", [(0, s) for s in big.FWD] + [(1, s) for s in big.BWD])
def test_gated_block(plan, back, sizes):  # noqa: F811
    N, H, F, form = sizes
    assert plan("glu", N, F, ref.up(H), back) == form
    assert max(N * ref.up(H) * 128, N * 4 * F, N * ref.up(F) * 128 * (1 + back)) > 1 << 32
