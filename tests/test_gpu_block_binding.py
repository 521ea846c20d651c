"""The binding's two routes to an entry point, its compiled step and the Python loop: the same results, the same
refusals, and the compiled one in use where it is built."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import tensor_transformer_mlp_02_amd as tp  # noqa: E402

N, H, E, K = 70, 264, 16, 2


def call_each(stream=None):
    """One call of every operator on the same inputs; all the outputs."""
    g = torch.Generator(device="cuda").manual_seed(5)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    f32 = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = {}
    d = dict(N=N, H=H, gate_rows=1, branch_scale=0.5)
    X, O, w1, w2, gate, dY, dH = bf(N, H), bf(N, H), bf(H), bf(H), bf(1, H), bf(N, H), bf(N, H)
    out.update(Y=torch.zeros_like(X), Hn=torch.zeros_like(X), so=f32(N), sp=f32(N))
    tp.tp_block_norm_fwd(d, X, O, w1, None, gate, w2, None, out["Y"], out["Hn"], out["so"], out["sp"], stream=stream)
    nb = tp.tp_block_norm_bwd_workspace(d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out.update(dX=torch.zeros_like(X), dO=torch.zeros_like(X), dw1=f32(H), dgate=f32(1, H), dw2=f32(H))
    tp.tp_block_norm_bwd(d, dY, dH, out["Y"], O, w1, None, gate, w2, out["so"], out["sp"], out["dX"], out["dO"], out["dw1"],
                         None, out["dgate"], out["dw2"], None, ws, nb, accumulate=False, stream=stream)
    r = dict(N=N, E=E, K=K, score=tp.TP_SCORE_SIGMOID, renorm=1)
    logits, bias = torch.randn(N, E, generator=g, device="cuda"), torch.randn(E, generator=g, device="cuda")
    out.update(e=i32(N, K), w=f32(N, K), dl=f32(N, E))
    tp.tp_moe_route_fwd(r, logits, bias, out["e"], out["w"], stream=stream)
    out.update(offsets=i32(E + 1), row_token=i32(N * K), row_weight=f32(N * K), tok_ptr=i32(N + 1), tok_rows=i32(N * K),
               slot_row=i32(N, K))
    tb = tp.tp_moe_route_tables_workspace(N, K, E)
    tp.tp_moe_route_tables(N, K, 0, E, N * K, out["e"], out["w"], *(out[k] for k in (
        "offsets", "row_token", "row_weight", "tok_ptr", "tok_rows", "slot_row")), torch.empty(
            max(16, tb), dtype=torch.uint8, device="cuda"), tb, stream=stream)
    tp.tp_moe_route_bwd(r, logits, out["e"], torch.ones(N, K, device="cuda"), None, 0, out["dl"], stream=stream)
    a = dict(lr=1e-2, step=2)
    t = dict(param=torch.randn(1000, generator=g, device="cuda"), grad=torch.randn(1000, generator=g, device="cuda"),
             m=torch.zeros(1000, device="cuda"), v=torch.zeros(1000, device="cuda"),
             param_bf16=torch.zeros(1000, dtype=torch.bfloat16, device="cuda"))
    tp.tp_adamw_step(a, [t], grad_scale=torch.ones(1, device="cuda"), stream=stream)
    out.update(t)
    out["permuted"] = torch.zeros(N * K, H, dtype=torch.bfloat16, device="cuda")   # an entry point of tpmlp.h
    tp.tp_moe_permute(tp.TP_BF16, N, H, N * K, out["row_token"], X, out["permuted"], stream=stream)
    torch.cuda.synchronize()
    return out


class Counting:
    def __init__(self, module):
        self.module, self.done, self.passed_on = module, 0, 0

    def _count(self, result):
        self.done += result is not None
        self.passed_on += result is None
        return result

    def call(self, *a):
        return self._count(self.module.call(*a))

    def addresses(self, *a):
        return self._count(self.module.addresses(*a))


def test_the_compiled_step_is_in_use():
    assert tp._marshaller(), "_marshal is not built or not usable"


def test_both_routes_give_the_same(monkeypatch):
    module = tp._marshaller()
    spy = Counting(module)
    monkeypatch.setattr(tp, "_compiled", spy)
    first = call_each()
    # six calls of one step, the AdamW call's scalars among them, and the addresses of tp_moe_permute
    assert spy.done >= 7 and spy.passed_on == 0
    monkeypatch.setattr(tp, "_compiled", False)
    second = call_each()
    for k in first:
        assert torch.equal(first[k], second[k]), k


@pytest.mark.parametrize("compiled", [True, False])
def test_both_routes_take_a_stream(monkeypatch, compiled):
    want = call_each()
    if not compiled:
        monkeypatch.setattr(tp, "_compiled", False)
    s = torch.cuda.current_stream()
    for stream in (s, s.cuda_stream):
        got = call_each(stream)
        for k in want:
            assert torch.equal(want[k], got[k]), k


@pytest.mark.parametrize("compiled", [True, False])
def test_both_routes_refuse_the_same(monkeypatch, compiled):
    if not compiled:
        monkeypatch.setattr(tp, "_compiled", False)
    x, w = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda"), torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)

    def norm(X=x, weight=w, Hn=y, H=H):
        tp.tp_block_norm_fwd(dict(N=N, H=H), X, None, None, None, None, weight, None, None, Hn)

    for kw, what in ((dict(X=x.float()), "X must be a torch.bfloat16"), (dict(X=x.cpu()), "X must be a GPU tensor"),
                     (dict(X=x.t()), "X must be contiguous"), (dict(Hn=y[:-1]), "Hn holds"),
                     (dict(weight=w[:-8]), "w_pre holds")):
        with pytest.raises(ValueError, match=what):
            norm(**kw)
    with pytest.raises(tp.TpError) as err:
        norm(H=H - 4)
    assert err.value.status == 2 and "multiple of 8" in err.value.message
    norm()
