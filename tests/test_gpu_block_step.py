"""One training step of a mixture-of-experts block, every operator in its
place: norm, routing, dispatch tables, permute, grouped experts with offsets in
device memory, combine, the seam to the next block with its gate, the way back
through all of them, and the AdamW step on what they left.

Checked against 64-bit autograd on the same inputs (bf16 bar of the parity
tests: a chain of bf16 roundings), and replayed from a captured graph."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402
from oracle import block as ob  # noqa: E402
from parity import TOL, assert_close  # noqa: E402

BF = tp.TP_BF16
A, B, EPS = 1.0, 0.5, 1e-5


class Block:
    def __init__(self, N=300, H=264, F=136, E=8, K=2, groups=4, kept=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.N, self.H, self.F, self.E, self.K = N, H, F, E, K
        rnd = lambda *s, std=1.0, shift=0.0, dt=torch.bfloat16: (  # noqa: E731
            torch.randn(*s, generator=g, device="cuda") * std + shift).to(dt)
        self.X = rnd(N, H)
        self.w_in, self.w_post, self.w_next = rnd(H, std=0.1, shift=1), rnd(H, std=0.1, shift=1), rnd(H, std=0.1, shift=1)
        self.gate = rnd(1, H, std=0.5)
        self.Wr = rnd(H, E, std=H ** -0.5, dt=torch.float32)
        self.bias = rnd(E, std=0.05, dt=torch.float32)
        self.Wg, self.Wu, self.Wd = rnd(E, H, F, std=H ** -0.5), rnd(E, H, F, std=H ** -0.5), rnd(E, F, H, std=F ** -0.5)
        self.dY, self.dNext = rnd(N, H, std=1e-2), rnd(N, H, std=1e-2)
        self.nin = dict(N=N, H=H, dtype=BF, eps=EPS)
        self.seam = dict(N=N, H=H, gate_rows=1, dtype=BF, eps=EPS, res_scale=A, branch_scale=B)
        self.route = dict(N=N, E=E, K=K, groups=groups, groups_kept=kept, group_best=2, score=tp.TP_SCORE_SIGMOID,
                          renorm=1, scale=2.0)
        self.expert = dict(H=H, F=F, E=E, dtype=BF)
        R = self.R = N * K
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.Hn, self.O, self.Y, self.Next = bf(N, H), bf(N, H), bf(N, H), bf(N, H)
        self.st_in, self.st_post, self.st_next = f32(N), f32(N), f32(N)
        self.logits, self.dlogits = f32(N, E), f32(N, E)
        self.e, self.w = i32(N, K), f32(N, K)
        self.tab = dict(offsets=i32(E + 1), row_token=i32(R), row_weight=f32(R), tok_ptr=i32(N + 1), tok_rows=i32(R),
                        slot_row=i32(N, K))
        self.Xp, self.Yp, self.Z, self.Ha = bf(R, H), bf(R, H), bf(R, 2 * F), bf(R, F)
        self.dRes, self.dO, self.dYp, self.dXp, self.dHn, self.dX = bf(N, H), bf(N, H), bf(R, H), bf(R, H), bf(N, H), bf(N, H)
        self.dw_rows = f32(R)
        self.grads = dict(w_in=f32(H), w_post=f32(H), w_next=f32(H), gate=f32(1, H), Wr=f32(H, E), Wg=f32(E, H, F),
                          Wu=f32(E, H, F), Wd=f32(E, F, H))
        byte = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = [(byte(n), n) for n in (tp.tp_moe_route_tables_workspace(N, K, E),
                                          tp.tp_block_norm_bwd_workspace(self.seam),
                                          tp.tp_block_norm_bwd_workspace(self.nin),
                                          tp.tp_grouped_expert_devoff_workspace(self.expert, R))]
        # the optimizer's side: fp32 main copies, states, and the bf16 weights that the products read
        self.main = {k: getattr(self, k).float().clone() for k in self.grads}
        self.states = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.main.items()}
        self.adam = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=1)
        self.table = tp.tp_adamw_tensors(self.adam, [
            dict(param=self.main[k], param_bf16=getattr(self, k) if getattr(self, k).dtype == torch.bfloat16 else None,
                 grad=v, m=self.states[k][0], v=self.states[k][1], weight_decay=0.1 if v.dim() > 1 else 0.0)
            for k, v in self.grads.items()])

    def forward(self):
        N, H, K, E, R = self.N, self.H, self.K, self.E, self.R
        tp.tp_block_norm_fwd(self.nin, self.X, None, None, None, None, self.w_in, None, None, self.Hn, None, self.st_in)
        torch.matmul(self.Hn.float(), self.Wr, out=self.logits)
        tp.tp_moe_route_fwd(self.route, self.logits, self.bias, self.e, self.w)
        tp.tp_moe_route_tables(N, K, 0, E, R, self.e, self.w, *self.tab.values(), *self.ws[0])
        t = self.tab
        tp.tp_moe_permute(BF, N, H, R, t["row_token"], self.Hn, self.Xp)
        tp.tp_grouped_expert_fwd_devoff(self.expert, R, t["offsets"], self.Xp, self.Wg, self.Wu, self.Wd, self.Z,
                                        self.Ha, self.Yp)
        tp.tp_moe_combine(BF, N, H, R, t["tok_ptr"], t["tok_rows"], t["row_weight"], self.Yp, self.O)
        tp.tp_block_norm_fwd(self.seam, self.X, self.O, self.w_post, None, self.gate, self.w_next, None, self.Y,
                             self.Next, self.st_post, self.st_next)

    def backward(self):
        N, H, R, t, g = self.N, self.H, self.R, self.tab, self.grads
        tp.tp_block_norm_bwd(self.seam, self.dY, self.dNext, self.Y, self.O, self.w_post, None, self.gate, self.w_next,
                             self.st_post, self.st_next, self.dRes, self.dO, g["w_post"], None, g["gate"], g["w_next"],
                             None, *self.ws[1])
        tp.tp_moe_combine_bwd(BF, N, H, R, t["row_token"], t["row_weight"], self.dO, self.Yp, self.dYp, self.dw_rows)
        tp.tp_grouped_expert_bwd_devoff(self.expert, R, t["offsets"], self.Xp, self.Wg, self.Wu, self.Wd, self.Z,
                                        self.Ha, self.dYp, self.dXp, g["Wg"], g["Wu"], g["Wd"], *self.ws[3])
        tp.tp_moe_route_bwd(self.route, self.logits, self.e, self.dw_rows, t["slot_row"], R, self.dlogits)
        torch.matmul(self.Hn.float().t(), self.dlogits, out=g["Wr"])
        tp.tp_moe_combine(BF, N, H, R, t["tok_ptr"], t["tok_rows"], None, self.dXp, self.dHn)
        self.dHn.copy_(self.dHn.float() + self.dlogits @ self.Wr.t())
        tp.tp_block_norm_bwd(self.nin, self.dRes, self.dHn, self.X, None, None, None, None, self.w_in, None, self.st_in,
                             self.dX, None, None, None, None, g["w_in"], None, *self.ws[2])

    def step(self):
        tp.tp_adamw_step(self.adam, self.table)


def reference(b):
    """The same block in 64 bits, differentiated by torch; the experts chosen are b's."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    leaves = {k: d(getattr(b, k)).requires_grad_(True) for k in ("X", "w_in", "w_post", "w_next", "gate", "Wr", "Wg", "Wu", "Wd")}
    norm = lambda x, w: x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * w  # noqa: E731
    L = leaves
    hn = norm(L["X"], L["w_in"])
    s = torch.sigmoid(hn @ L["Wr"])
    e = b.e.long().cpu()
    w = s.gather(1, e)
    w = 2.0 * w / (w.sum(1, keepdim=True) + 1e-20)
    out = torch.zeros_like(L["X"])
    for k in range(b.E):
        tok, slot = (e == k).nonzero(as_tuple=True)
        x = hn[tok]
        h = torch.nn.functional.silu(x @ L["Wg"][k]) * (x @ L["Wu"][k])
        out = out.index_add(0, tok, w[tok, slot][:, None] * (h @ L["Wd"][k]))
    y = A * L["X"] + B * L["gate"] * norm(out, L["w_post"])
    nxt = norm(y, L["w_next"])
    ((y * d(b.dY)).sum() + (nxt * d(b.dNext)).sum()).backward()
    return dict(Hn=hn, O=out, Y=y, Next=nxt, w=w), {k: v.grad for k, v in leaves.items()}


@pytest.mark.parametrize("N,H,F,E,K,groups,kept", [(300, 264, 136, 8, 2, 4, 2), (1, 64, 32, 4, 2, 1, 1),
                                                   (1025, 512, 256, 16, 4, 4, 2)])
def test_training_step(N, H, F, E, K, groups, kept):
    b = Block(N, H, F, E, K, groups, kept)
    b.forward()
    b.backward()
    want_e, _ = ob.route_fwd(b.logits.double().cpu().numpy(), b.bias.cpu().numpy(), K, groups, kept, 2, True, True, 2.0)
    assert np.array_equal(b.e.cpu().numpy(), want_e)
    outs, grads = reference(b)
    tol = TOL[BF]
    np64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    for k, v in outs.items():
        assert_close(k, np64(getattr(b, k)), np64(v), tol)
    assert_close("dX", np64(b.dX), np64(grads["X"]), tol)
    for k, v in b.grads.items():
        assert_close("d" + k, np64(v), np64(grads[k]), tol)
    before = {k: v.clone() for k, v in b.main.items()}
    b.step()
    for k, v in b.grads.items():
        wd = 0.1 if v.dim() > 1 else 0.0
        p, m, s = ob.adamw(np64(before[k]), np64(v), 0.0, 0.0, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=1, wd=float(np.float32(wd)))
        # the first step moves by lr at most: 24 roundings of it, 4 of the parameter
        assert (np.abs(np64(b.main[k]) - p) <= 2.0 ** -24 * (4 * np.abs(np64(before[k])) + 24 * 1e-2)).all(), k
        if getattr(b, k).dtype == torch.bfloat16:
            assert torch.equal(getattr(b, k), b.main[k].to(torch.bfloat16)), k
    # the weights that the products read have moved
    y = b.Y.clone()
    b.forward()
    assert not torch.equal(y, b.Y)


def test_captured_steps_equal_eager_ones():
    eager, captured = Block(seed=3), Block(seed=3)
    # a step before the capture (the libraries' first calls set themselves up), undone
    keep = {k: v.clone() for k, v in captured.main.items()}
    weights = {k: getattr(captured, k).clone() for k in captured.grads}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.forward()
        captured.backward()
        captured.step()
    torch.cuda.current_stream().wait_stream(side)
    for k, v in keep.items():
        captured.main[k].copy_(v)
        getattr(captured, k).copy_(weights[k])
        for s in captured.states[k]:
            s.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.forward()
        captured.backward()
        captured.step()
    for i in range(3):
        X = torch.randn(eager.N, eager.H, device="cuda").to(torch.bfloat16)
        for b in (eager, captured):
            b.X.copy_(X)
        eager.forward()
        eager.backward()
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("Next", "e", "w", "dX", "dlogits"):
            assert torch.equal(getattr(eager, k), getattr(captured, k)), (i, k)
        for k in eager.grads:
            assert torch.equal(eager.grads[k], captured.grads[k]), (i, k)
            assert torch.equal(eager.main[k], captured.main[k]), (i, k)
