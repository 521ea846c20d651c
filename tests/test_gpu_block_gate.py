"""Block norms with more gate rows than workers and biases: a gate row of few tokens and of many, either side of
where the backward takes another form."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_block_norm import Case  # noqa: E402


@pytest.mark.parametrize("H", [512, 1024, 4096])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("N,G", [(300, 300), (900, 300), (1199, 300), (1200, 300), (1201, 300), (2100, 257), (270, 1000)])
def test_tokens_of_a_gate_row(H, layer, N, G):
    c = Case(N, H, G=G, layer=layer, bias=True, seed=N + H)
    c.check_backward(c.backward())


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("N,G", [(1199, 300), (1200, 300)])
def test_accumulated_and_repeated(layer, N, G):
    c = Case(N, 1024, G=G, layer=layer, bias=True, seed=1)
    a, b = c.backward(), c.backward()
    acc = c.backward(accumulate=True, start=0.25)
    for k in c.GRADS:
        assert torch.equal(a[k], b[k]), k
        if k not in ("dX", "dO"):
            assert torch.equal(acc[k], a[k] + 0.25), k
