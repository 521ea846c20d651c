"""GPU: products with an E5M2 operand (gradients) in each of the kernels, and a training step whose gradients are E5M2,
against the formulas in 64 bits."""
import pytest
import torch

import fp8g_ref as ref
import tensor_transformer_mlp_02_amd as tp
from test_gpu_fp8g import (G, RESULTS, buffer, check_product, product, quantized, step_buffers, step_inputs, tokens,
                           untouched)

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMATS = [(1, 0), (0, 1)]


@pytest.mark.parametrize("M,N,K,out,form", ref.GEMM_FORMS)
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("square", [False, True])
def test_gemm(M, N, K, out, form, fa, fb, e8, square):
    A, sA, a = quantized(tokens(1, M, K), e8, fmt=fa)
    B, sB, b = quantized(tokens(2, N, K, 0.05), e8, square, fb)
    C = product(A, sA, B, sB, M, N, K, TYPES[out], scale=int(e8), square=int(square), fmt_a=fa, fmt_b=fb)
    check_product(C, a, b, TYPES[out])
    untouched(C)


@pytest.mark.parametrize("M,N,K,out,form", [s for s in ref.GEMM_FORMS if s[3] == "f32"])
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("e8", [False, True])
def test_gemm_accumulate(M, N, K, out, form, fa, fb, e8):
    A, sA, a = quantized(tokens(3, M, K), e8, fmt=fa)
    B, sB, b = quantized(tokens(4, N, K), e8, fmt=fb)
    before = tokens(5, M, N)
    C = buffer(M, N, dtype=torch.float32)
    C.copy_(before)
    product(A, sA, B, sB, M, N, K, torch.float32, C, scale=int(e8), accumulate=1, fmt_a=fa, fmt_b=fb)
    check_product(C, a, b, torch.float32, before.double())
    untouched(C)


@pytest.mark.parametrize("M,N,K,out,form", ref.GEMM_FORMS)
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("e8", [False, True])
def test_gemm_parts(M, N, K, out, form, fa, fb, e8):
    A, sA, a = quantized(tokens(6, M, 2 * K), e8, fmt=fa)
    B, sB, b = quantized(tokens(7, N, K), e8, True, fb)
    B2, sB2, b2 = quantized(tokens(8, N, K), e8, True, fb)
    C = buffer(M, N, dtype=TYPES[out])
    tp.tp_fp8g_gemm(dict(M=M, N=N, K=K, parts=2, scale=int(e8), square=1, dtype=int(out == "bf16"), fmt_a=fa, fmt_b=fb),
                    A, sA, B, sB, C, B2, sB2)
    check_product(C, a, torch.cat([b, b2], 1), TYPES[out])
    untouched(C)


@pytest.mark.parametrize("N,H,F", [(5, 136, 200), (200, 264, 392), (2100, 1032, 1416)])
@pytest.mark.parametrize("e8", [False, True])
def test_training_step(N, H, F, e8):
    """The whole block against 64 bits without quantization.  An E4M3 quantization leaves at most 2^-4 of a value, an
    E5M2 one 2^-3: Y passes four of the first; a gradient at most five, two of which (dY, dZ) are E5M2."""
    X, dY, Wg, Wu, B = step_inputs(N, H, F, 3)
    o, e = step_buffers(N, H, F, e8), int(e8)
    qd = lambda r, c, **kw: dict(rows=r, cols=c, scale=e, **kw)  # noqa: E731
    tp.tp_fp8g_quantize(qd(N, H), X, o["Xq"], o["sX"], o["Xq_t"], o["sX_t"])
    for w, r, c, k in ((Wg, H, F, "g"), (Wu, H, F, "u"), (B, F, H, "b")):
        tp.tp_fp8g_quantize(qd(r, c, square=1), w, o["W" + k], o["sW" + k], o["W" + k + "t"], o["sW" + k + "t"])
    d, ws = dict(N=N, H=H, F=F, scale=e), o["ws"]
    tp.tp_fp8g_glu_fwd(d, o["Xq"], o["sX"], o["Wgt"], o["sWgt"], o["Wut"], o["sWut"], o["Z"], None, o["Hq"], o["sH"], o["Hq_t"],
                       o["sH_t"], ws, ws.numel())
    pf, pn = ref.up(F) * G, ref.up(N) * G
    tp.tp_fp8g_gemm(dict(M=N, N=H, K=pf, scale=e, square=1), o["Hq"], o["sH"], o["Wbt"], o["sWbt"], o["Y"])
    tp.tp_fp8g_quantize(qd(N, H, fmt=1), dY, o["dYq"], o["sdY"], o["dYq_t"], o["sdY_t"])
    tp.tp_fp8g_glu_bwd(dict(d, fmt=1), o["dYq"], o["sdY"], o["Wb"], o["sWb"], o["Z"], o["dZ"], o["sdZ"], o["dZ_t"], o["sdZ_t"],
                       ws, ws.numel())
    tp.tp_fp8g_gemm(dict(M=N, N=H, K=pf, scale=e, square=1, parts=2, fmt_a=1), o["dZ"], o["sdZ"], o["Wg"], o["sWg"], o["dX"],
                    o["Wu"], o["sWu"])
    acc = dict(K=pn, scale=e, dtype=tp.TP_F32, accumulate=1, fmt_b=1)
    tp.tp_fp8g_gemm(dict(acc, M=F, N=H), o["Hq_t"], o["sH_t"], o["dYq_t"], o["sdY_t"], o["dB"])
    tp.tp_fp8g_gemm(dict(acc, M=H, N=F), o["Xq_t"], o["sX_t"], o["dZ_t"][0], o["sdZ_t"][0], o["dA"])
    tp.tp_fp8g_gemm(dict(acc, M=H, N=F), o["Xq_t"], o["sX_t"], o["dZ_t"][1], o["sdZ_t"][1], o["dA_up"])
    x, dy, wg, wu, b = (t.double().cpu() for t in (X, dY, Wg, Wu, B))
    g, u = x @ wg, x @ wu
    act, slope = ref.gate(0, g)
    h, dh = act * u, dy @ b.t()
    dg, du = dh * u * slope, dh * act
    want = dict(Y=h @ b, dX=dg @ wg.t() + du @ wu.t(), dB=h.t() @ dy, dA=x.t() @ dg, dA_up=x.t() @ du)
    for k in RESULTS:
        rel = float((o[k].double().cpu() - want[k]).norm() / want[k].norm())
        assert rel <= (4 if k == "Y" else 7) * 2.0 ** -4, (k, rel)
