"""The logits' gradient where scores are near 0 or 1: against the derivative in a form that subtracts nothing
from 1.

With u = 2^-24 and every operation rounded once:
  sigmoid   s (1 - s) = e / (1 + e)^2, e = exp(-|l|): e off by 4 u, the quotient by 10 u with the gradient's own two
            products; a renormalised gradient adds the K scores of its sum and their quotients.  64 u + 4 K u, of
            s (1 - s) times the terms of ds.
  softmax   dl_e = s_e sum_i s_i (ds_e - ds_i).  With c the ds of the largest score m the terms are at most
            s_e (|ds_e| + |c|) (e other than m) and s_e s_i (|ds_i| + |c|) (i other than m), each off by gamma()
            of test_gpu_route.py: the exponentials' rounded arguments and the sums of E terms.
  renormalised  ds_j = (sum_i w_i (t_j - t_i) + t_j 1e-20 / S) / S, in the same way with the largest of the
            chosen."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from oracle import block as ob  # noqa: E402
from test_gpu_route import BF16, F32, HALF, INF, desc, gamma  # noqa: E402

U = 2.0 ** -24


def check(d, logits, expert, up, got):
    """got [N,E] for the weights' gradient up [N,K]; expert in range, none twice."""
    N, E, K = d["N"], d["E"], d["K"]
    l, ex, t = logits.double().cpu().numpy(), expert.cpu().numpy(), up.double().cpu().numpy() * float(np.float32(d["scale"]))
    sig, ren = bool(d["score"]), bool(d["renorm"])
    s, there = ob.scores(l, sig)
    want = ob.route_bwd(l, ex, up.double().cpu().numpy(), sig, ren, float(np.float32(d["scale"])))
    ds, mds = np.zeros((N, E)), np.zeros((N, E))
    for n in range(N):
        v, tn = s[n, ex[n]], t[n]
        if ren:
            S = v.sum() + 1e-20
            m = int(v.argmax())
            k, w = tn[m], v / S
            other = np.arange(K) != m
            ds[n, ex[n]] = ((tn - k) - (w * (tn - k)).sum() + k * (1e-20 / S)) / S
            mds[n, ex[n]] = ((np.abs(tn) + abs(k)) * other + (w * (np.abs(tn) + abs(k)) * other).sum()
                             + abs(k) * 1e-20 / S) / S
        else:
            ds[n, ex[n]], mds[n, ex[n]] = tn, np.abs(tn)
    if sig:
        e = np.where(there, np.exp(-np.abs(np.where(there, l, 0.0))), 0.0)
        mag, g = e / (1 + e) ** 2 * mds, (64 + 4 * K) * U
    else:
        m = np.where(there, l, -np.inf).argmax(1)[:, None]
        rest = np.arange(E)[None] != m
        # (c itself is off by its own terms)
        each = mds + np.take_along_axis(mds, m, 1)
        mag, g = s * (each * rest + (s * each * rest).sum(1, keepdims=True)), 2 * gamma(d, logits)
    got = got.double().cpu().numpy()
    tol = HALF[logits.dtype] * np.abs(want) + g * mag + 1e-37
    over = np.abs(got - want) / tol
    assert over.max() <= 1, (float(over.max()), np.unravel_index(over.argmax(), over.shape), got[over >= over.max()],
                             want[over >= over.max()])


def run(d, logits, expert, up):
    out = torch.full((d["N"], d["E"]), float("nan"), dtype=logits.dtype, device="cuda")
    tp.tp_moe_route_bwd(d, logits, expert, up, None, 0, out)
    return out


def sampled(d, logits, expert, up):
    out = run(d, logits, expert, up)
    N = d["N"]
    pick = list(range(N)) if N < 100 else list(range(0, N, N // 60))
    part = lambda x: x[pick].contiguous()  # noqa: E731
    check({**d, "N": len(pick)}, part(logits), part(expert), part(up), part(out))


# few tokens, and as many as share wavefronts; K of one lane's slots and of several lanes'
SHAPES = [(40, 64, 1), (40, 64, 4), (33, 300, 6), (37, 1000, 32), (4101, 16, 1), (4101, 64, 2), (4101, 100, 16),
          (7173, 256, 8)]


def far_logits(N, E, K, dtype, lo, hi, renorm):
    g = torch.Generator(device="cuda").manual_seed(N + E)
    l = (torch.rand(N, E, generator=g, device="cuda") * (hi - lo) + lo).to(dtype)
    e = l.float().topk(K, dim=1).indices.to(torch.int32)
    sampled(desc(N, E, K, sigmoid=True, renorm=renorm, dtype=dtype, scale=1.5), l, e,
            torch.randn(N, K, generator=g, device="cuda"))


@pytest.mark.parametrize("N,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lo,hi", [(10.0, 60.0), (-60.0, -10.0), (-60.0, 60.0)])
def test_sigmoid_of_far_logits(N, E, K, dtype, lo, hi):
    far_logits(N, E, K, dtype, lo, hi, False)


def one_far_ahead(N, E, K, dtype, renorm):
    g = torch.Generator(device="cuda").manual_seed(N + E)
    l = torch.randn(N, E, generator=g, device="cuda")
    ahead = torch.randint(0, E, (N, 1), generator=g, device="cuda")
    l.scatter_add_(1, ahead, torch.rand(N, 1, generator=g, device="cuda") * 40)
    l[::5, ::3] = -INF                                   # (the one ahead may be out as well)
    l = l.to(dtype)
    e = l.float().topk(K, dim=1).indices.to(torch.int32)
    sampled(desc(N, E, K, renorm=renorm, dtype=dtype, scale=1.5), l, e, torch.randn(N, K, generator=g, device="cuda"))


@pytest.mark.parametrize("N,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_softmax_with_one_expert_far_ahead(N, E, K, dtype):
    one_far_ahead(N, E, K, dtype, False)


@pytest.mark.parametrize("N,E", [(40, 64), (40, 1000), (4101, 128), (7173, 256)])
@pytest.mark.parametrize("K", [1, 4])
def test_softmax_of_nearly_equal_logits(N, E, K):
    """Scores of about 1 / E: the experts that are not chosen get s_e sum_i ds_i s_i, far smaller than any ds.
    Scores: e^x 4 u, a sum of at most 16 terms a lane over 64 lanes 22 u, quotient and product 2 u; twice in the
    result (56 u), with the sum over K slots and the products 10 u more: 80 u of s_e (|ds_e| + sum_i |ds_i| s_i)."""
    g = torch.Generator(device="cuda").manual_seed(N + E + K)
    l = torch.randn(N, E, generator=g, device="cuda") * 0.01
    e = l.topk(K, dim=1).indices.to(torch.int32)
    up = torch.randn(N, K, generator=g, device="cuda")
    got = run(desc(N, E, K, scale=1.5), l, e, up).double()
    s = torch.softmax(l.double(), 1)
    ds = torch.zeros_like(s).scatter_(1, e.long(), up.double() * 1.5)
    want = s * (ds - (ds * s).sum(1, keepdim=True))
    over = (got - want).abs() / (80 * U * s * (ds.abs() + (ds.abs() * s).sum(1, keepdim=True)))
    assert float(over.max()) <= 1, float(over.max())


@pytest.mark.parametrize("N,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_renormalised_weights_of_far_logits(N, E, K, dtype):
    one_far_ahead(N, E, K, dtype, True)
    for lo, hi in ((10.0, 60.0), (-60.0, -10.0), (-60.0, 60.0)):
        far_logits(N, E, K, dtype, lo, hi, True)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("N", [40, 4101])
def test_renormalised_weights_with_one_far_ahead(sigmoid, N):
    """One of the chosen takes almost the whole weight: the gradients of the chosen are small differences."""
    E, K = 64, 4
    g = torch.Generator(device="cuda").manual_seed(N)
    l = torch.randn(N, E, generator=g, device="cuda") - (12.0 if sigmoid else 0.0)
    l.scatter_add_(1, torch.randint(0, E, (N, 1), generator=g, device="cuda"),
                   8 + torch.rand(N, 1, generator=g, device="cuda") * 12)
    e = l.topk(K, dim=1).indices.to(torch.int32)
    sampled(desc(N, E, K, sigmoid=sigmoid, renorm=True, scale=2.5), l, e, torch.randn(N, K, generator=g, device="cuda"))
    # a single weight that is always 1 has no gradient, but for the 1e-20 in its sum
    one = e[:, :1].contiguous()
    d = desc(N, E, 1, sigmoid=sigmoid, renorm=True)
    sampled(d, l, one, torch.ones(N, 1, device="cuda"))
    assert float(run(d, l, one, torch.ones(N, 1, device="cuda")).abs().max()) < 1e-12
