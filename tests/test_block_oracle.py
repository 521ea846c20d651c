"""The 64-bit definitions of the operators around the products, pinned by
something other than themselves: differences, brute force, closed forms."""
import numpy as np
import pytest

from oracle import block as ob


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("G", [0, 1, 2, 5, 7])
def test_norm_backward_against_differences(layer, post, G):
    rng = np.random.default_rng(1)
    N, H = 5, 6
    a, b, eps = 0.8, 0.6, 1e-5
    v = dict(X=rng.normal(size=(N, H)), O=rng.normal(size=(N, H)), w_post=rng.normal(size=H),
             b_post=rng.normal(size=H), gate=rng.normal(size=(G, H)) if G else None,
             w_pre=rng.normal(size=H), b_pre=rng.normal(size=H))
    if not post:
        v["w_post"] = v["b_post"] = None
    cy, ch = rng.normal(size=(N, H)), rng.normal(size=(N, H))

    def loss(u):
        f = ob.norm_fwd(**u, layer=layer, eps=eps, a=a, b=b)
        return (f["Y"] * cy).sum() + (f["Hn"] * ch).sum()

    f = ob.norm_fwd(**v, layer=layer, eps=eps, a=a, b=b)
    g = ob.norm_bwd(cy, ch, f["Y"], v["O"], v["w_post"], v["b_post"], v["gate"], v["w_pre"],
                    f.get("r_post"), f.get("mu_post"), f["r_pre"], f["mu_pre"], layer=layer, a=a, b=b)
    names = {"X": "dX", "O": "dO", "w_post": "dw_post", "b_post": "db_post", "gate": "dgate",
             "w_pre": "dw_pre", "b_pre": "db_pre"}
    for k, name in names.items():
        if v[k] is None:
            continue
        num = np.zeros(v[k].shape)
        for i in np.ndindex(v[k].shape):
            step = 1e-6
            hi, lo = dict(v), dict(v)
            hi[k], lo[k] = v[k].copy(), v[k].copy()
            hi[k][i] += step
            lo[k][i] -= step
            num[i] = (loss(hi) - loss(lo)) / (2 * step)
        # differences: step^2 times a third derivative of size about 10, and 1e-16 * |loss| / step
        np.testing.assert_allclose(g[name], num, rtol=1e-6, atol=1e-7, err_msg=name)


def test_norm_closed_forms():
    x = np.array([[3.0, 4.0]])
    n, r, mu, _ = ob.norm(x, False, np.ones(2), None, 0.0)
    np.testing.assert_allclose(r, 1 / np.sqrt(12.5))
    np.testing.assert_allclose(n, x / np.sqrt(12.5))
    n, r, mu, _ = ob.norm(x, True, np.ones(2), np.array([1.0, 1.0]), 0.0)
    np.testing.assert_allclose(n, [[0.0, 2.0]])
    assert mu[0] == 3.5


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(sigmoid, renorm):
    rng = np.random.default_rng(2)
    l, up = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    l[2, 4] = -np.inf
    expert, w = ob.route_fwd(l, None, 3, sigmoid=sigmoid, renorm=renorm, scale=1.7)
    g = ob.route_bwd(l, expert, up, sigmoid=sigmoid, renorm=renorm, scale=1.7)
    for t, e in np.ndindex(l.shape):
        if not np.isfinite(l[t, e]):
            assert g[t, e] == 0
            continue
        two = []
        for step in (1e-6, -1e-6):
            k = l.copy()
            k[t, e] += step
            ek, wk = ob.route_fwd(k, None, 3, sigmoid=sigmoid, renorm=renorm, scale=1.7)
            assert np.array_equal(ek, expert)
            two.append((wk * up).sum())
        assert abs((two[0] - two[1]) / 2e-6 - g[t, e]) < 1e-8


def test_route_forward_small_cases():
    l = np.array([[0.0, 2.0, 2.0, 1.0]])
    e, w = ob.route_fwd(l, None, 2)
    assert e.tolist() == [[1, 2]]                      # ties: the lower expert first
    assert w[0, 0] == w[0, 1]
    e, w = ob.route_fwd(l, np.array([9.0, 0, 0, 0]), 2, sigmoid=True, renorm=True)
    assert e.tolist() == [[0, 1]]                      # the bias chooses ...
    s = 1 / (1 + np.exp(-np.array([0.0, 2.0])))
    np.testing.assert_allclose(w[0], s / s.sum())      # ... and stays out of the weights
    # two runs of two: the run with the better pair wins, though not the best expert
    l = np.array([[3.0, -9.0, 2.0, 1.9]])
    assert ob.route_fwd(l, None, 1, 2, 1, 1, sigmoid=True)[0].tolist() == [[0]]
    assert ob.route_fwd(l, None, 1, 2, 1, 2, sigmoid=True)[0].tolist() == [[2]]
    # masked: the lowest value of the type, -inf and NaN; all of them
    l = np.array([[-np.inf, ob.LOWEST, np.nan, 0.5], [-np.inf] * 4])
    e, w = ob.route_fwd(l, None, 2)
    assert e.tolist() == [[3, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]


def test_tables_small_case():
    e = np.array([[2, 0], [1, 2], [2, 2], [-1, 5]], np.int32)
    t = ob.route_tables(e, np.arange(8, dtype=np.float32).reshape(4, 2), 1, 2, 10)
    assert t["offsets"].tolist() == [0, 1, 5]
    assert t["row_token"].tolist() == [1, 0, 1, 2, 2] + [-1] * 5
    assert t["row_weight"].tolist() == [2, 0, 3, 4, 5] + [0] * 5
    assert t["tok_ptr"].tolist() == [0, 1, 3, 5, 5]
    assert t["tok_rows"].tolist() == [1, 0, 2, 3, 4] + [-1] * 5
    assert t["slot_row"].tolist() == [[1, -1], [0, 2], [3, 4], [-1, -1]]


def test_adamw_first_step_is_the_sign():
    p, m, v = ob.adamw(np.array([1.0, 1.0]), np.array([0.3, -5.0]), 0.0, 0.0, lr=0.1, beta1=0.9,
                       beta2=0.999, eps=0.0, step=1, wd=0.5)
    np.testing.assert_allclose(p, [1 - 0.05 - 0.1, 1 - 0.05 + 0.1])


def test_e4m3_values():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ob.e4m3(codes), want, equal_nan=True)
    lo, hi = ob.e4m3_neighbours(np.array([1.0, 1.05, -1.05, 448.0, 0.0, 1e-4]))
    assert lo.tolist() == [1.0, 1.0, -1.125, 448.0, 0.0, 0.0]
    assert hi.tolist() == [1.0, 1.125, -1.0, 448.0, 0.0, 2.0 ** -9]


def test_chances_are_even_and_independent():
    n = 1 << 18
    for seed, step, place in ((0, 1, 0), (1, 1, 0), (12345, 7, 3)):
        u, w = ob.chances(seed, step, place, n)
        for x in (u, w):
            # mean of n even chances: standard deviation 0.289 / sqrt(n) = 5.6e-4; 5 of them
            assert abs(x.mean() - 0.5) < 2.9e-3
            counts = np.bincount((x * 64).astype(int), minlength=64)
            # 63 degrees of freedom: mean 63, deviation 11.2
            assert ((counts - n / 64) ** 2 / (n / 64)).sum() < 63 + 6 * 11.3
            for lag in (1, 2, 4, 64, 256):
                r = np.corrcoef(x[:-lag], x[lag:])[0, 1]
                assert abs(r) < 5 / np.sqrt(n), lag
        assert abs(np.corrcoef(u, w)[0, 1]) < 5 / np.sqrt(n)
    a, b = ob.chances(5, 1, 0, n)[0], ob.chances(5, 2, 0, n)[0]
    c = ob.chances(5, 1, 1, n)[0]
    assert abs(np.corrcoef(a, b)[0, 1]) < 5 / np.sqrt(n)
    assert abs(np.corrcoef(a, c)[0, 1]) < 5 / np.sqrt(n)
