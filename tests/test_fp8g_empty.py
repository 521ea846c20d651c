"""FP8 with group scales where there is nothing to sum: the weight gradients of an empty batch."""
import pytest

import tensor_transformer_mlp_02_amd as tp
from test_block_abi import E_DEV, E_NULL, E_SHAPE, pytestmark  # noqa: F401
from test_fp8g_abi import GEMM, gd, gemm


@pytest.mark.parametrize("kw", [{}, dict(accumulate=1), dict(scale=1), dict(square=1), dict(parts=2), dict(fmt_b=1)])
def test_an_empty_sum(kw):
    none = {k: None for k in GEMM if k != "C"}
    assert gemm(gd(K=0, dtype=tp.TP_F32, **kw), **none) == E_DEV
    assert gemm(gd(K=0, dtype=tp.TP_F32, **kw), **none, C=None) == E_NULL
    assert gemm(gd(K=0, dtype=tp.TP_F32, M=0, **kw), **none, C=None) == E_DEV


def test_is_a_weight_gradient():
    assert gemm(gd(K=0)) == E_SHAPE             # bf16: no sum over tokens
    assert gemm(gd(K=-128, dtype=tp.TP_F32)) == E_SHAPE
