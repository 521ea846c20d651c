"""AdamW on the GPU against the 64-bit definition (oracle/block.py).

32-bit states: m and v are two rounded products and a rounded sum of rounded
factors, within 8 * 2^-24 of their terms' magnitudes; the parameter's update
adds a root, two quotients and the descriptor's scalars in fp32: 16 * 2^-24 of
the update, 4 * 2^-24 of the parameter.

8-bit states: a code's value is one of the two E4M3 neighbours of the exact
state over the block's scale, the one that the chance of its element picks:
told only where the chance is further from the border than fp32 arithmetic
reaches (16 steps of the value, 2^-20 of a code's 16 fractions at most)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from oracle import block as ob  # noqa: E402

U = 2.0 ** -24
ALIGN = 256


def f64(t):
    return t.detach().double().cpu().numpy()


def make(counts, bits=32, grad=torch.float32, copy=True, seed=0, fresh=False, wd=0.1, grad_std=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(counts):
        rnd = lambda std: torch.randn(n, generator=g, device="cuda") * std  # noqa: E731
        t = dict(param=rnd(0.05), grad=rnd(grad_std).to(grad), weight_decay=wd if i % 2 == 0 else 0.0)
        t["param_bf16"] = torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda") if copy else None
        m, v = rnd(grad_std * 0.3), rnd(grad_std).square()
        if fresh:
            m, v = torch.zeros_like(m), torch.zeros_like(v)
        if bits == 32:
            t.update(m=m, v=v)
        else:
            blocks = -(-n // 256)
            code = lambda: torch.randint(0, 127, (n,), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
            sign = (torch.randint(0, 2, (n,), generator=g, device="cuda") * 128).to(torch.uint8)
            t.update(m=code() | sign, v=code(),
                     m_scale=torch.rand(blocks, generator=g, device="cuda") * grad_std / 448,
                     v_scale=torch.rand(blocks, generator=g, device="cuda") * grad_std / 448)
            if fresh:
                for k in ("m", "v", "m_scale", "v_scale"):
                    t[k].zero_()
        out.append(t)
    return out


def desc(bits=32, grad=torch.float32, step=3, **kw):
    return {**dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=step, grad_dtype=int(grad == torch.bfloat16),
                   state_bits=bits, seed=77), **kw}


def copy_of(ts):
    return [{k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()} for t in ts]


def check(d, before, after, scale=1.0, places=None):
    """after: the tensors that the step has changed."""
    for i, (b, a) in enumerate(zip(before, after)):
        n = b["param"].numel()
        if n == 0:
            continue
        p0, g = f64(b["param"]), f64(b["grad"]) * scale
        small = d["state_bits"] == 8
        if small:
            m0 = ob.widen(b["m"].cpu().numpy(), f64(b["m_scale"]))
            v0 = ob.widen(b["v"].cpu().numpy(), f64(b["v_scale"])) ** 2
        else:
            m0, v0 = f64(b["m"]), f64(b["v"])
        wd = float(np.float32(b["weight_decay"]))
        p, m, v = ob.adamw(p0, g, m0, v0, lr=d["lr"], beta1=d["beta1"], beta2=d["beta2"], eps=d["eps"],
                           step=d["step"], wd=wd)
        mm = d["beta1"] * np.abs(m0) + (1 - d["beta1"]) * np.abs(g)
        c1, c2 = 1 - d["beta1"] ** d["step"], 1 - d["beta2"] ** d["step"]
        # a bound on a magnitude: |lr|, the rate may be negative
        per = abs(d["lr"]) / c1 / (np.sqrt(v / c2) + d["eps"])
        tol = 4 * U * np.abs(p0) + 24 * U * per * mm + 1e-38
        got = f64(a["param"])
        assert (np.abs(got - p) <= tol).all(), (i, (np.abs(got - p) / tol).max())
        if a["param_bf16"] is not None:
            assert torch.equal(a["param_bf16"], a["param"].to(torch.bfloat16))
        assert torch.equal(a["grad"], b["grad"])
        if not small:
            assert (np.abs(f64(a["m"]) - m) <= 8 * U * mm + 1e-44).all()
            assert (np.abs(f64(a["v"]) - v) <= 8 * U * v + 1e-44).all()
            continue
        place = i if places is None else places[i]
        um, ur = ob.chances(d["seed"], d["step"], place, n)
        for name, x, u in (("m", m, um), ("v", np.sqrt(v), ur)):
            blocks = -(-n // 256)
            pad = np.zeros(blocks * 256)
            pad[:n] = np.abs(x)
            top = pad.reshape(blocks, 256).max(1)
            mag = np.zeros(blocks * 256)
            mag[:n] = mm if name == "m" else np.sqrt(v)
            mtop = mag.reshape(blocks, 256).max(1)
            s = f64(a[name + "_scale"])
            assert (np.abs(s - top / 448) <= 16 * U * mtop / 448 + 1e-44).all(), name
            live = np.repeat(s > 0, 256)[:n]
            t = np.where(live, x / np.where(live, np.repeat(np.maximum(s, 1e-300), 256)[:n], 1.0), 0.0)
            slack = np.where(live, 16 * U * mag[:n] / np.repeat(np.maximum(s, 1e-300), 256)[:n], 0.0) + 2.0 ** -36
            t = np.clip(t, -448, 448)
            val = ob.e4m3(a[name].cpu().numpy())
            lo, hi = ob.e4m3_neighbours(t)
            near = (np.abs(t - lo) <= slack) | (np.abs(t - hi) <= slack)
            ok = (val == lo) | (val == hi) | near
            if name == "v":
                ok |= (x > 0) & (val == 2.0 ** -9)
                assert not ((x > 1e-30) & (val <= 0) & live).any()
            assert ok.all(), (name, np.argwhere(~ok)[:4], t[~ok][:4], val[~ok][:4])
            # which neighbour: up where the fraction left over exceeds 1 - u
            # (of the square for a root: v is what is kept on average)
            gap = np.where(hi > lo, hi - lo, 1.0)
            frac = (t - lo) / gap
            if name == "v":
                frac = frac * (t + lo) / (hi + lo + (hi == 0))
            width = 2 * slack / gap + 2.0 ** -18
            sure = (np.abs(frac - (1 - u)) > width) & ~near & (hi > lo)
            up = frac > 1 - u
            pick = np.where(up, hi, lo)
            if name == "v":
                pick = np.maximum(pick, 2.0 ** -9)
            assert (val == pick)[sure & live].all(), name
            assert sure.mean() > 0.9 or n < 50 or not live.any()


COUNTS = [[1], [0], [5], [255], [256], [257], [1000], [4095, 4096, 4097], [1, 0, 3, 0, 0, 20000, 7], [100003],
          [33] * 50, [4096] * 97 + [1]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_step(counts, bits, grad):
    before = make(counts, bits, grad, seed=len(counts))
    after = copy_of(before)
    d = desc(bits, grad)
    tp.tp_adamw_step(d, after)
    check(d, before, after)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_without_a_copy(bits):
    before = make([300, 5000], bits, copy=False, fresh=True)
    after = copy_of(before)
    d = desc(bits, step=1)
    tp.tp_adamw_step(d, after)
    check(d, before, after)


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars(bits):
    before = make([3000, 17], bits)
    for step, lr, scale in ((1, 1e-2, 0.25), (12, 3e-3, 4.0), (100000, 1e-4, 1.0)):
        after = copy_of(before)
        d = desc(bits, step=step, lr=float(np.float32(lr)))
        tp.tp_adamw_step(desc(bits, step=0, lr=99.0), after, dev_step=torch.tensor([step], dtype=torch.int32, device="cuda"),
                         dev_lr=torch.tensor([lr], device="cuda"), grad_scale=torch.tensor(scale, device="cuda"))
        check(d, before, after, scale=scale)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_overflowed_scale_skips_the_step(bits, scale):
    before = make([3000, 17], bits)
    after = copy_of(before)
    tp.tp_adamw_step(desc(bits), after, grad_scale=torch.tensor(scale, device="cuda"))
    tp.tp_adamw_step(desc(bits), after, dev_step=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for b, a in zip(before, after):
        for k, v in b.items():
            if torch.is_tensor(v) and k != "param_bf16":
                assert torch.equal(v, a[k]), k
            elif k == "param_bf16":
                assert torch.isnan(a[k]).all()


@pytest.mark.parametrize("kw", [dict(beta1=0.0, beta2=0.0), dict(beta1=0.999, beta2=0.9999, step=1), dict(eps=1.0),
                                dict(lr=0.0), dict(lr=-0.1), dict(step=2147483647)])
@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_scalars(kw, bits):
    before = make([2000], bits)
    after = copy_of(before)
    d = desc(bits, **kw)
    tp.tp_adamw_step(d, after)
    check(d, before, after)


@pytest.mark.parametrize("bits", [32, 8])
def test_tiny_huge_and_zero_gradients(bits):
    for std in (0.0, 1e-12, 1e15):
        before = make([700], bits, fresh=True, grad_std=std)
        after = copy_of(before)
        d = desc(bits, step=1)
        tp.tp_adamw_step(d, after)
        check(d, before, after)


def test_nan_and_infinity():
    for bits in (32, 8):
        for bad in (float("nan"), float("inf")):
            ts = make([1024], bits)
            ts[0]["grad"][300] = bad
            clean = make([1024], bits)
            tp.tp_adamw_step(desc(bits), ts)
            tp.tp_adamw_step(desc(bits), clean)
            p, q = ts[0]["param"], clean[0]["param"]
            keep = torch.arange(1024, device="cuda") != 300
            assert torch.equal(p[keep], q[keep]) and torch.isnan(p[300])
            if bits == 8:   # the whole block's states say so
                for name in ("m", "v"):
                    x = ob.widen(ts[0][name].cpu().numpy(), f64(ts[0][name + "_scale"]))
                    assert np.isnan(x[256:512]).all()
                    assert np.isfinite(x[:256]).all() and np.isfinite(x[512:]).all()


def test_rounding_by_chance_keeps_a_slow_average():
    """A state that changes by far less than half a code each step still follows its average."""
    n = 1 << 16
    t = make([n], 8, fresh=True, wd=0.0)[0]
    steps, beta2 = 400, 0.99
    g = torch.full((n,), 1e-2, device="cuda")
    g[::256] = 0.1                                # sets each block's scale
    t["grad"].copy_(g)
    table = tp.tp_adamw_tensors(desc(8), [t])
    for s in range(1, steps + 1):
        tp.tp_adamw_step(desc(8, step=s, beta2=beta2, lr=0.0), table)
    r = ob.widen(t["v"].cpu().numpy(), f64(t["v_scale"]))
    want = 1e-4 * (1 - beta2 ** steps)
    rest = np.ones(n, bool)
    rest[::256] = False
    v = r[rest] ** 2
    # kept on average: the mean of 65280 values scattered by about a third has a deviation of 0.13 %
    assert abs(v.mean() / want - 1) < 0.01
    assert v.std() / want < 0.5


def test_place_in_the_list_and_step_change_the_rounding():
    a, b = make([4096], 8, seed=1)[0], make([4096], 8, seed=1)[0]
    tp.tp_adamw_step(desc(8), [a, b])
    assert torch.equal(a["param"], b["param"]) and not torch.equal(a["m"], b["m"])
    x, y = make([4096], 8, seed=1), make([4096], 8, seed=1)
    tp.tp_adamw_step(desc(8), x)
    tp.tp_adamw_step(desc(8), y)
    assert torch.equal(x[0]["m"], y[0]["m"]) and torch.equal(x[0]["m"], a["m"])
    # an empty tensor keeps its place
    z = make([0], 8) + make([4096], 8, seed=1)
    tp.tp_adamw_step(desc(8), z)
    assert torch.equal(z[1]["m"], b["m"])


@pytest.mark.parametrize("bits", [32, 8])
def test_memory_around_a_tensor_is_left_alone(bits):
    flat = make([4096], bits)[0]
    keep = copy_of([flat])[0]
    lo, n = 256 * 4, 1001
    piece = {k: (v[lo:lo + n] if torch.is_tensor(v) and v.numel() == 4096 else v) for k, v in flat.items()}
    if bits == 8:
        for k in ("m_scale", "v_scale"):
            piece[k] = flat[k][4:8]
    tp.tp_adamw_step(desc(bits), [piece])
    for k, v in flat.items():
        if torch.is_tensor(v):
            s = (4, 8) if v.numel() == 16 else (lo, lo + n)
            for part in (slice(0, s[0]), slice(s[1], None)):
                assert torch.equal(v[part], keep[k][part]) or torch.isnan(v[part]).all(), k


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_graph_follows_the_device_scalars(bits):
    a, b = make([5000, 77], bits), make([5000, 77], bits)
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    lr, scale = torch.tensor([1e-2], device="cuda"), torch.tensor([1.0], device="cuda")
    table = tp.tp_adamw_tensors(desc(bits), a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_adamw_step(desc(bits), table, dev_step=step, dev_lr=lr, grad_scale=scale)
        step.add_(1)
    for s in (1, 2, 3):
        lr.fill_(1e-2 / s)
        scale.fill_(0.5 * s)
        graph.replay()
        torch.cuda.synchronize()
        tp.tp_adamw_step(desc(bits), b, dev_step=torch.tensor([s], dtype=torch.int32, device="cuda"), dev_lr=lr,
                         grad_scale=scale)
        for x, y in zip(a, b):
            for k in x:
                if torch.is_tensor(x[k]):
                    assert torch.equal(x[k], y[k]), (s, k)


def test_more_elements_than_32_bits_count():
    n = (1 << 32) + 3000
    z = lambda d: torch.zeros(n, dtype=d, device="cuda")  # noqa: E731
    t = dict(param=z(torch.float32), grad=z(torch.bfloat16), m=z(torch.uint8), v=z(torch.uint8),
             m_scale=torch.zeros(-(-n // 256), device="cuda"), v_scale=torch.zeros(-(-n // 256), device="cuda"),
             weight_decay=0.0)
    at = [0, 5, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1]
    t["grad"][torch.tensor(at, device="cuda")] = 1.0
    d = desc(8, torch.bfloat16, step=1, eps=1e-4)
    tp.tp_adamw_step(d, [t])
    # m and r are their blocks' largest: exact codes; the parameters move by lr, the others not at all
    assert int((t["param"] != 0).sum()) == len(at)
    for i in at:
        assert abs(float(t["param"][i]) + 1e-2) < 1e-5
        assert int(t["m"][i]) == 0x7e and int(t["v"][i]) == 0x7e


def test_more_elements_than_one_grid_has_threads_for():
    # 8-bit states take 1024 elements a workgroup of 256 threads: from 2^34 elements on a launch
    # would need 2^32 threads.  The first tensor ends behind that, the second begins there.
    n = (1 << 34) + 70000
    if torch.cuda.mem_get_info()[0] < n * 8.5:
        pytest.skip("needs 146 GB of free device memory")
    z = lambda k, d: torch.zeros(k, dtype=d, device="cuda")  # noqa: E731
    ts = [dict(param=z(k, torch.float32), grad=z(k, torch.bfloat16), m=z(k, torch.uint8), v=z(k, torch.uint8),
               m_scale=z(-(-k // 256), torch.float32), v_scale=z(-(-k // 256), torch.float32),
               weight_decay=0.0) for k in (n, 5000)]
    last = ((1 << 24) - 1) * 1024  # first element of the second launch
    at = [0, (1 << 32) - 1, last - 1, last, last + 1023, (1 << 34) - 1, 1 << 34, n - 1]
    ts[0]["grad"][torch.tensor(at, device="cuda")] = 1.0
    ts[1]["grad"][4999] = 1.0
    tp.tp_adamw_step(desc(8, torch.bfloat16, step=1, eps=1e-4), ts)
    for t, places in zip(ts, (at, [4999])):
        # (last + 1023 is 2^34 - 1)
        assert sum(int((part != 0).sum()) for part in t["param"].split(1 << 30)) == len(set(places))
        for i in places:
            assert abs(float(t["param"][i]) + 1e-2) < 1e-5
            assert int(t["m"][i]) == 0x7e and int(t["v"][i]) == 0x7e
    del ts, t
    torch.cuda.empty_cache()
