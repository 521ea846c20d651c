"""GPU: FP8 with group scales on an empty batch, as a rank or an expert without tokens has it."""
import pytest
import torch

import tensor_transformer_mlp_02_amd as tp
from test_gpu_fp8g import DEV, buffer, step_buffers, step_inputs, training_step, untouched

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(5, 20), (200, 264), (1030, 1000), (4000, 3976)])
@pytest.mark.parametrize("kw", [{}, dict(scale=1), dict(square=1), dict(parts=2)])
def test_an_empty_sum_is_zero(M, N, kw):
    C = buffer(M, N, dtype=torch.float32)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    d = dict(M=M, N=N, K=0, dtype=tp.TP_F32, **kw)
    assert bool(C.any())
    tp.tp_fp8g_gemm(d, none, None, none, None, C)
    torch.cuda.synchronize()
    assert not bool(C.any())
    untouched(C)
    C.fill_(3.0)
    tp.tp_fp8g_gemm(dict(d, accumulate=1), none, None, none, None, C)
    torch.cuda.synchronize()
    assert bool((C == 3.0).all())
    untouched(C)


@pytest.mark.parametrize("e8", [False, True])
def test_training_step_without_tokens(e8):
    N, H, F = 0, 264, 392
    ins = step_inputs(N, H, F, 3)
    o = step_buffers(N, H, F, e8)
    for k in ("dB", "dA", "dA_up"):
        o[k].fill_(2.0)
    training_step(N, H, F, *ins, e8, o)
    torch.cuda.synchronize()
    for k in ("dB", "dA", "dA_up"):
        assert bool((o[k] == 2.0).all())
    assert o["Y"].shape == (0, H) and o["dX"].shape == (0, H)


def test_captured_zeros():
    """A weight gradient of no tokens in a graph: zeros after each replay."""
    C = torch.full((130, 264), 5.0, device=DEV)
    d = dict(M=130, N=264, K=0, dtype=tp.TP_F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tp.tp_fp8g_gemm(d, None, None, None, None, C)
    for r in range(3):
        C.fill_(float(r + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert not bool(C.any())
