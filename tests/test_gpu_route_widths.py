"""The logits' gradient of large batches for expert counts around those that fill whole lanes, either side of where
tokens share a wavefront: against the definition."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from test_gpu_route import BF16, F32, check_backward, desc, inputs  # noqa: E402


@pytest.mark.parametrize("E", [15, 17, 33, 62, 72, 100, 104, 129, 136, 144, 200, 255, 256])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_of_many_tokens(E, sigmoid, dtype):
    N, K = (4101 if E <= 128 else 7173), 4
    l, _ = inputs(N, E, dtype, masked=True, seed=E)
    g = torch.Generator(device="cuda").manual_seed(E)
    e = torch.randint(-1, E, (N, K), generator=g, device="cuda", dtype=torch.int32)
    up = torch.randn(N, K, generator=g, device="cuda")
    d = desc(N, E, K, sigmoid=sigmoid, renorm=True, dtype=dtype, scale=1.5)
    out = torch.full((N + 1, E), float("nan"), dtype=dtype, device="cuda")
    tp.tp_moe_route_bwd(d, l, e, up, None, 0, out)
    assert bool(torch.isfinite(out[:N]).all()) and bool(torch.isnan(out[N]).all())   # the row behind is left alone
    pick = list(range(0, N, 150)) + [N - 1]
    p = {**d, "N": len(pick)}
    check_backward(p, l[pick].contiguous(), e[pick].contiguous(), up[pick].contiguous(), out=out[pick].contiguous())
