"""Every gradient of the block norms from a captured graph, bias gradients among them: each replay against the
eager call, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from test_gpu_block_norm import Case  # noqa: E402


@pytest.mark.parametrize("N,H,G,layer", [
    (300, 4096, 1, False), (300, 4096, 1, True), (300, 1032, 300, True),   # more gate rows than workers
    (700, 64, 600, False), (40, 20000, 1, True), (40, 20000, 33, False), (12, 8200, 12, True)])
def test_replays_write_every_gradient(N, H, G, layer):
    c = Case(N, H, G=G, layer=layer, bias=True, seed=N)
    saved = c.saved()
    want = c.backward(saved=saved)
    assert all(want[k] is not None for k in c.GRADS)
    c.check_backward(want)
    ws = torch.empty(tp.tp_block_norm_bwd_workspace(c.desc), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.backward(saved=saved, ws=ws)
    for i in range(3):
        for t in got.values():
            t.fill_(float("nan"))
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        for k in c.GRADS:
            assert torch.equal(got[k], want[k]), (i, k)
        c.backward(saved=saved)     # eager work between the replays
        torch.cuda.synchronize()
