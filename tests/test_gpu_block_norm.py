"""Block norms on the GPU against the 64-bit definition (oracle/block.py).

Tolerance of an element: half a step of its type relative to the value, plus
gamma times the magnitudes of the terms it is made of, for fp32 arithmetic:
gamma = (H / 4 + 64) * 2^-24 bounds any order of a row's sums (each rounding
is at most 2^-24 relative) with the few operations before and after them, and
(N + 64) * 2^-24 is added for sums over tokens.  sqrt, division and expf-free
arithmetic are correctly rounded, within the 64."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from oracle import block as ob  # noqa: E402

EPS = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, want, mag, dtype, gamma):
    got = host(got).reshape(want.shape)
    assert np.isfinite(got).all(), name
    # the smallest subnormals of the type are rounded absolutely
    tol = HALF[dtype] * np.abs(want) + gamma * mag + 1e-38
    over = np.abs(got - want) / tol
    assert over.max(initial=0.0) <= 1.0, (name, float(over.max()), np.unravel_index(over.argmax(), want.shape))


class Case:
    """One seam's inputs on the GPU and the definition's results."""

    def __init__(self, N, H, G=0, dtype=torch.bfloat16, layer=False, block=True, post=True, pre=True,
                 bias=False, a=1.0, b=0.5, seed=0, big=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.N, self.H, self.G, self.dtype, self.layer, self.a, self.b = N, H, G, dtype, layer, a, b

        def draw(*shape, on=True, shift=0.0, std=1.0):
            x = torch.randn(*shape, generator=g, device="cuda") * std + shift
            return x.to(dtype) if on else None

        self.X = draw(N, H, shift=0.3, std=30.0 if big else 1.0)
        self.O = draw(N, H, on=block, std=0.7)
        post = post and block
        self.w_post, self.b_post = draw(H, on=post, shift=1.0, std=0.3), draw(H, on=post and bias, std=0.3)
        self.gate = draw(G, H, on=G > 0, std=0.5)
        self.w_pre, self.b_pre = draw(H, on=pre, shift=1.0, std=0.3), draw(H, on=pre and bias, std=0.3)
        self.desc = dict(N=N, H=H, gate_rows=G, kind=int(layer), dtype=int(dtype == torch.bfloat16),
                         eps=EPS, res_scale=a, branch_scale=b)
        self.eps = float(np.float32(EPS))
        self.a64, self.b64 = float(np.float32(a)), float(np.float32(b))
        self.gamma = (H / 4 + 64) * 2.0 ** -24
        self.want = ob.norm_fwd(host(self.X), host(self.O), host(self.w_post), host(self.b_post),
                                host(self.gate), host(self.w_pre), host(self.b_pre), layer=layer,
                                eps=self.eps, a=self.a64, b=self.b64) if N else {}
        self.dY, self.dH = draw(N, H, std=0.1), draw(N, H, on=pre, std=0.1)

    def new(self, like, fill=float("nan"), dtype=None):
        return None if like is None else torch.full_like(like, fill, dtype=dtype or like.dtype)

    def stat(self, on):
        return torch.full((2 * self.N if self.layer else self.N,), float("nan"), device="cuda") if on else None

    def forward(self, in_place=False, stats=True):
        Y = None if self.O is None else self.X.clone() if in_place else self.new(self.X)
        Hn = self.new(self.X) if self.w_pre is not None else None
        so = self.stat(stats and self.w_post is not None)
        sp = self.stat(stats and self.w_pre is not None)
        tp.tp_block_norm_fwd(self.desc, Y if in_place else self.X, self.O, self.w_post, self.b_post, self.gate,
                             self.w_pre, self.b_pre, Y, Hn, so, sp)
        return Y, Hn, so, sp

    def check_forward(self, out):
        Y, Hn, so, sp = out
        w, g = self.want, self.gamma
        if Y is not None:
            close("Y", Y, w["Y"], w["mag_Y"], self.dtype, g)
        if Hn is not None:
            close("Hn", Hn, w["Hn"], w["mag_Hn"], self.dtype, g)
        for name, st in (("post", so), ("pre", sp)):
            if st is None:
                continue
            r = w["r_" + name]
            t = host(self.O) if name == "post" else w.get("Y", host(self.X))
            m = np.abs(t) if name == "post" else w.get("mag_Y", np.abs(t))
            # an error of t reaches r through the variance
            close("r_" + name, st[:self.N], r, r * (1 + r * np.sqrt((m ** 2).mean(1))), torch.float32, 2 * g)
            if self.layer:
                close("mu_" + name, st[self.N:], w["mu_" + name], m.mean(1), torch.float32, g)

    def saved(self):
        """Y and the statistics as the forward leaves them, from the definition."""
        def st(name):
            if "r_" + name not in self.want:
                return None
            r = [self.want["r_" + name]] + ([self.want["mu_" + name]] if self.layer else [])
            return torch.tensor(np.concatenate(r), dtype=torch.float32, device="cuda")
        Y = self.X if self.O is None else torch.tensor(self.want["Y"], device="cuda").to(self.dtype)
        return Y, st("post"), st("pre")

    GRADS = ("dX", "dO", "dw_post", "db_post", "dgate", "dw_pre", "db_pre")

    def backward(self, dY=True, db=True, accumulate=False, start=None, saved=None, ws=None):
        Y, so, sp = saved or self.saved()
        f = torch.float32
        o = dict(dX=self.new(self.X), dO=self.new(self.O), dw_post=self.new(self.w_post, dtype=f),
                 db_post=self.new(self.w_post, dtype=f) if db else None, dgate=self.new(self.gate, dtype=f),
                 dw_pre=self.new(self.w_pre, dtype=f), db_pre=self.new(self.w_pre, dtype=f) if db else None)
        if start is not None:
            for k in self.GRADS[2:]:
                if o[k] is not None:
                    o[k].fill_(start)
        nb = tp.tp_block_norm_bwd_workspace(self.desc)
        if ws is None:
            ws = torch.full((nb,), 0xff, dtype=torch.uint8, device="cuda")  # NaN everywhere
        tp.tp_block_norm_bwd(self.desc, self.dY if dY else None, self.dH, Y if self.w_pre is not None else None,
                             self.O, self.w_post, self.b_post, self.gate, self.w_pre, so, sp,
                             *(o[k] for k in self.GRADS), ws, nb, accumulate=accumulate)
        return o

    def check_backward(self, out, dY=True, plus=0.0):
        Y, so, sp = self.saved()
        N = self.N

        def split(st):
            if st is None:
                return None, None
            v = host(st)
            return v[:N], (v[N:] if self.layer else None)

        w = ob.norm_bwd(host(self.dY) if dY else None, host(self.dH), host(Y), host(self.O), host(self.w_post),
                        host(self.b_post), host(self.gate), host(self.w_pre), *split(so), *split(sp),
                        layer=self.layer, a=self.a64, b=self.b64)
        for k in self.GRADS:
            if out[k] is None:
                continue
            row = k in ("dX", "dO")
            # two sums by rows stand behind dO and the post norm's gradients
            gamma = 2 * self.gamma + (0 if row else (N + 64) * 2.0 ** -24)
            close(k, out[k], w[k] + (0 if row else plus), w["mag_" + k] + (0 if row else abs(plus)),
                  self.dtype if row else torch.float32, gamma)


SHAPES = [(1, 8), (3, 24), (2, 64), (67, 512), (5, 520), (33, 1000), (9, 1032), (300, 2048), (4, 2056), (7, 4104),
          (130, 4096), (3, 8192), (5, 8200), (2, 16384), (3, 16392), (2, 40000)]


@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward_and_backward_over_widths(N, H, layer, dtype):
    c = Case(N, H, G=1, dtype=dtype, layer=layer, bias=True, seed=H + N)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("H", [4, 12, 260, 1004, 4100])
@pytest.mark.parametrize("layer", [False, True])
def test_fp32_widths_of_four(H, layer):
    c = Case(37, H, G=3, dtype=torch.float32, layer=layer, bias=True, seed=H)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("G", [0, 1, 2, 3, 7, 64, 255, 256, 257, 1000, 1001, 1300])
@pytest.mark.parametrize("H", [64, 1536])
def test_gate_rows(G, H):
    # fewer rows than workers, about as many, one for each token, more than tokens
    c = Case(1000, H, G=G, layer=G % 2 == 1, bias=True, seed=G)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("N", [1, 63, 65, 500, 40001])
@pytest.mark.parametrize("H,dtype", [(24, torch.bfloat16), (64, torch.bfloat16), (72, torch.bfloat16), (128, torch.bfloat16),
                                     (136, torch.bfloat16), (256, torch.bfloat16), (20, torch.float32), (128, torch.float32)])
@pytest.mark.parametrize("G,bias,layer", [(0, False, False), (1, True, True), (13, False, True), (-1, True, False)])
def test_narrow_rows(N, H, dtype, G, bias, layer):
    # several rows a wavefront, more of them than the grid takes at once; G = -1: a gate a token
    c = Case(N, H, G=N if G < 0 else G, dtype=dtype, layer=layer, bias=bias, seed=N + H)
    c.check_forward(c.forward())
    c.check_backward(c.backward(db=bias))


@pytest.mark.parametrize("G", [7, 20, 33])
@pytest.mark.parametrize("H,dtype", [(16384, torch.bfloat16), (20000, torch.bfloat16), (8192, torch.float32)])
def test_gate_rows_of_wide_rows(G, H, dtype):
    # 20 tokens are 10 workers' work: gate rows for fewer, for more, for more than the tokens
    c = Case(20, H, G=G, dtype=dtype, layer=True, bias=True, seed=G)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


PARTS = [dict(block=False), dict(post=False), dict(pre=False), dict(post=False, pre=False), dict()]


@pytest.mark.parametrize("parts,G,bias,layer", [
    (p, g, b, l) for p, g, b, l in itertools.product(PARTS, (0, 2), (False, True), (False, True))
    if not (g and not p.get("block", True))])
@pytest.mark.parametrize("H", [136, 20000])
def test_parts_left_out(parts, G, bias, layer, H):
    c = Case(6, H, G=G, bias=bias, layer=layer, seed=5, **parts)
    c.check_forward(c.forward())
    c.check_forward(c.forward(stats=False))
    c.check_backward(c.backward(db=bias))
    if parts.get("pre", True):
        c.check_backward(c.backward(dY=False), dY=False)


@pytest.mark.parametrize("H", [4096, 16392])
def test_scales_and_a_large_stream(H):
    c = Case(11, H, G=1, a=0.37, b=-1.8, layer=True, big=True, seed=3)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("H,dtype", [(8200, torch.bfloat16), (16384, torch.bfloat16), (4100, torch.float32),
                                     (8192, torch.float32)])
@pytest.mark.parametrize("G,bias,layer", [(1, False, False), (1, True, True), (600, False, True), (600, True, False)])
def test_several_turns_of_the_widest_rows(H, dtype, G, bias, layer):
    # the widest rows that a workgroup holds, more of them than workgroups
    c = Case(600, H, G=G, dtype=dtype, layer=layer, bias=bias, seed=H)
    c.check_forward(c.forward())
    c.check_backward(c.backward(db=bias))


@pytest.mark.parametrize("H", [64, 256, 8192, 16384, 20000])
def test_stream_updated_in_place(H):
    c = Case(19, H, G=1)
    a, b = c.forward(), c.forward(in_place=True)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("H,N", [(64, 5000), (512, 700), (4096, 300), (20000, 20)])
def test_accumulates_and_repeats_bitwise(H, N):
    for G in (1, 3, N):
        c = Case(N, H, G=G, layer=True, bias=True)
        a, b = c.backward(), c.backward()
        for k in c.GRADS:
            assert torch.equal(a[k], b[k]), k
        acc = c.backward(accumulate=True, start=0.25)
        for k in c.GRADS[2:]:
            assert torch.equal(acc[k], a[k] + 0.25), k   # one more addition, at the end


@pytest.mark.parametrize("G", [0, 1, 5])
@pytest.mark.parametrize("H", [64, 20000])
def test_no_tokens(G, H):
    c = Case(0, H, G=G, bias=True)
    c.forward()
    c.want, c.layer = {}, False
    empty = torch.empty(0, device="cuda")
    out = c.backward(saved=(c.X, empty, empty))
    for k in c.GRADS[2:]:
        if out[k] is not None:
            assert (out[k] == 0).all(), k
    out = c.backward(saved=(c.X, empty, empty), accumulate=True, start=2.0)
    for k in c.GRADS[2:]:
        if out[k] is not None:
            assert (out[k] == 2).all(), k


def test_zero_rows_and_constant_rows_are_finite():
    for layer in (False, True):
        c = Case(4, 264, layer=layer, post=True)
        c.O[1] = 0
        c.X[1] = 0
        c.O[2] = 3
        c.X[2] = 2
        c.want = ob.norm_fwd(host(c.X), host(c.O), host(c.w_post), None, None, host(c.w_pre), None, layer=layer,
                             eps=c.eps, a=c.a64, b=c.b64)
        out = c.forward()
        assert all(torch.isfinite(x).all() for x in out)
        c.check_forward(out)
        c.check_backward(c.backward())


def test_nan_and_infinity_stay_in_their_row():
    c = Case(5, 4096, G=1)
    clean = c.forward()
    c.O[3, 17] = float("nan")
    c.X[1, 5] = float("inf")
    bad = c.forward()
    for x, y in zip(clean, bad):
        for n in (0, 2, 4):
            assert torch.equal(x[n], y[n])
    assert not torch.isfinite(bad[1][3]).any()


def test_rows_past_the_last_are_left_alone():
    for H in (512, 4096, 20000):
        c = Case(7, H, G=1)
        Y, Hn = (torch.full((9, H), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        so, sp = torch.full((9,), 5.0, device="cuda"), torch.full((9,), 5.0, device="cuda")
        tp.tp_block_norm_fwd(c.desc, c.X, c.O, c.w_post, None, c.gate, c.w_pre, None, Y, Hn, so, sp)
        for t in (Y, Hn, so, sp):
            assert (t[7:] == 5).all()
        c.check_forward((Y[:7], Hn[:7], so[:7], sp[:7]))


def test_another_stream_and_a_captured_graph():
    c = Case(300, 4096, G=1, seed=8)
    want_f, want_b = c.forward(), c.backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.forward()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want_f))
    ws = torch.empty(tp.tp_block_norm_bwd_workspace(c.desc), dtype=torch.uint8, device="cuda")
    saved = c.saved()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf = c.forward()
        gb = c.backward(saved=saved, ws=ws)
    for _ in range(3):
        for t in list(gf) + list(gb.values()):
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(gf, want_f))
        for k in c.GRADS:
            if k.startswith("db"):
                continue
            assert torch.equal(gb[k], want_b[k]), k


def test_long_batch_past_32_bit_offsets():
    # 2^32 bytes and elements: sampled rows either side
    H, N = 8192, (1 << 19) + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(N, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    Hn = torch.zeros_like(X)
    tp.tp_block_norm_fwd(dict(N=N, H=H), X, None, None, None, None, w, None, None, Hn)
    pick = [0, 1, (1 << 18) - 1, 1 << 18, (1 << 18) + 1, (1 << 19) - 1, 1 << 19, N - 1]
    x = host(X[pick])
    want, _, _, mag = ob.norm(x, False, np.ones(H), None, float(np.float32(EPS)))
    close("Hn", Hn[pick], want, mag, torch.bfloat16, (H / 4 + 64) * 2.0 ** -24)


def test_backward_past_32_bit_offsets():
    H, N = 8192, (1 << 19) + 3
    g = torch.Generator(device="cuda").manual_seed(2)
    bf = lambda: torch.empty(N, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    X, dY, dH = bf(), bf(), bf()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    r = torch.empty(N, device="cuda")
    Hn = torch.empty_like(X)
    d = dict(N=N, H=H)
    tp.tp_block_norm_fwd(d, X, None, None, None, None, w, None, None, Hn, None, r)
    dX, dw = Hn.fill_(float("nan")), torch.empty(H, device="cuda")
    nb = tp.tp_block_norm_bwd_workspace(d)
    tp.tp_block_norm_bwd(d, dY, dH, X, None, None, None, None, w, None, r, dX, None, None, None, None, dw, None,
                         torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    pick = [0, 1, (1 << 18) - 1, 1 << 18, (1 << 18) + 1, (1 << 19) - 1, 1 << 19, N - 1]
    want = ob.norm_bwd(host(dY[pick]), host(dH[pick]), host(X[pick]), None, None, None, None, np.ones(H), None, None,
                       host(r[pick]), None, layer=False, a=1.0, b=1.0)
    close("dX", dX[pick], want["dX"], want["mag_dX"], torch.bfloat16, (H / 2 + 128) * 2.0 ** -24)
    # sums of half a million terms of size 1, in chains of 2049 and 256: far below 1e-5 of their magnitudes
    part = torch.zeros(H, dtype=torch.float64, device="cuda")
    mag = torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, N, 1 << 15):
        t = dH[i:i + (1 << 15)].double() * X[i:i + (1 << 15)].double() * r[i:i + (1 << 15), None].double()
        part += t.sum(0)
        mag += t.abs().sum(0)
    assert bool(((dw.double() - part).abs() <= (2049 + 256 + 64) * 2.0 ** -24 * mag).all())
