"""Which groups of experts stay, where a group's two best choice scores overflow in fp32.

The choice is that of 64-bit arithmetic for any finite bias: experts and, within the bounds of
test_gpu_route.py, weights are compared with oracle/block.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_route import desc, forward, want_forward  # noqa: E402


@pytest.mark.parametrize("N", [50, 4099])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("E,groups,kept", [(16, 4, 2), (64, 8, 3), (512, 16, 4)])
def test_groups_whose_two_best_pass_the_range_of_fp32(N, sign, E, groups, kept):
    """A bias of the size of the largest fp32 takes an expert out (or puts it first): the sum of two such
    scores is still a number, and a group without experts comes after all others."""
    per = E // groups
    for sigmoid in (False, True):
        g = torch.Generator(device="cuda").manual_seed(E)
        l = torch.randn(N, E, generator=g, device="cuda")
        l[:, :per] = -float("inf")                      # the first group has no experts
        b = torch.full((E,), sign * 3e38, device="cuda")
        b[-1] = sign * 2e38                             # the last one has another worth than the rest
        d = desc(N, E, kept * per - 1, groups, kept, 2, sigmoid) if kept * per <= 32 else \
            desc(N, E, 8, groups, kept, 2, sigmoid)
        e, _ = forward(d, l, b)
        pick = list(range(0, N, max(1, N // 50)))
        want, _ = want_forward({**d, "N": len(pick)}, l[pick].contiguous(), b)
        got = e[pick].cpu().numpy()
        assert np.array_equal(got, want), (got[0], want[0])
