"""Which kernel the gated block takes where the summed index is short beside its values (CPU): the forms that leave
fp32 values in memory and quantize them in a second launch move several times the bytes of those that make the codes in
their tiles, and ask the caller for a workspace of the values' size."""
import pytest

import tensor_transformer_mlp_02_amd as tp
from test_block_abi import pytestmark  # noqa: F401

# us on MI355X: with the fp32 values in memory (few rows' kernel), and with codes made in the tile
FORWARD = [((2048, 128, 1416), (25.8, 15.1)), ((2048, 128, 3584), (45, 25)), ((4096, 128, 3584), (91, 45)),
           ((8192, 128, 1024), (49, 24)), ((8192, 128, 3584), (175, 87)), ((8192, 256, 3584), (200, 101)),
           ((4096, 512, 3584), (130, 61)), ((30000, 128, 512), (103, 45)), ((100000, 128, 128), (90, 45))]
BACKWARD = [((2048, 128, 1416), (27.3, 17.9)), ((2048, 128, 3584), (52, 33)), ((4096, 128, 3584), (98, 63)),
            ((8192, 128, 1024), (57, 35)), ((8192, 128, 3584), (194, 121)), ((8192, 256, 3584), (210, 130)),
            ((4096, 512, 1416), (54, 41)), ((30000, 128, 512), (105, 71)), ((100000, 128, 128), (89, 68))]


@pytest.mark.parametrize("sizes", [s for s, _ in FORWARD])
def test_forward_makes_its_codes_in_the_tile(sizes):
    assert tp.tp_fp8g_glu_fwd_workspace(dict(zip("NHF", sizes))) == 16


@pytest.mark.parametrize("sizes", [s for s, _ in BACKWARD])
def test_backward_makes_its_codes_in_the_tile(sizes):
    assert tp.tp_fp8g_glu_bwd_workspace(dict(zip("NHF", sizes))) == 16


@pytest.mark.parametrize("N,H,F", [(64, 8192, 3584), (100, 1000, 1416), (300, 1000, 1416)])
def test_few_tokens_keep_theirs(N, H, F):
    d = dict(N=N, H=H, F=F)
    assert tp.tp_fp8g_glu_fwd_workspace(d) == N * F * 4 and tp.tp_fp8g_glu_bwd_workspace(d) == N * F * 8
