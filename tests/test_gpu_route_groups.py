"""Which groups of experts stay, where a group's two best choice scores cancel or overflow in fp32.

The choice is that of 64-bit arithmetic for any finite bias: experts and, within the bounds of
test_gpu_route.py, weights are compared with oracle/block.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_route import check_forward, desc, forward, want_forward  # noqa: E402


def opposed(N, E, groups, B, sigmoid, seed):
    """In every group one expert with the bias B and the rest with -B: a group is worth the sum of two scores,
    nearly the same for all groups (apart by about one rounding of B), while the chosen experts' own scores lie
    further apart than B's rounding."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = E // groups
    step = torch.rand(N, groups, generator=g, device="cuda", dtype=torch.float64).argsort(1).double() / groups
    noise = torch.randn(N, groups, generator=g, device="cuda", dtype=torch.float64) * B * 2.0 ** -22
    unit = 0.25 if sigmoid else 0.5 / groups
    s = torch.full((N, groups, per), 1e-9, device="cuda", dtype=torch.float64)
    s[:, :, 0] = unit * (1 + 0.5 * step)
    s[:, :, 1] = unit * (1 - 0.5 * step) + noise
    s = s.clamp_min(1e-9).view(N, E)
    l = (s / (1 - s)).log() if sigmoid else s.log()
    bias = torch.full((groups, per), -float(B), device="cuda")
    bias[:, 0] = float(B)
    return l.float(), bias.view(-1).contiguous()


SHAPES = [(64, 32, 8), (64, 16, 4), (64, 8, 3), (256, 8, 4), (512, 32, 8)]


@pytest.mark.parametrize("E,groups,kept", SHAPES)
@pytest.mark.parametrize("B", [16, 64, 256])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_of_opposed_biases(E, groups, kept, B, sigmoid):
    # few tokens, and (where groups are whole lanes) as many as share wavefronts
    l, b = opposed(300, E, groups, B, sigmoid, seed=E + groups + B)
    check_forward(desc(300, E, 3, groups, kept, 2, sigmoid, True), l, b)
    N = 7171 if E == 256 else 4099
    l, b = opposed(N, E, groups, B, sigmoid, seed=E + groups + B + 1)
    d = desc(N, E, 3, groups, kept, 2, sigmoid, True)
    e, _ = forward(d, l, b)
    pick = list(range(0, N, 13))
    want, _ = want_forward({**d, "N": len(pick)}, l[pick].contiguous(), b)
    got = e[pick].cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


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
