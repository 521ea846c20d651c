"""GPU: the gated block where the summed index is one or two groups, in each of its kernels, against the formulas in
64 bits."""
import pytest
import torch

import fp8g_ref as ref
from test_gpu_fp8g import (BF16, DEV, G, check_codes, glu_bwd, glu_bwd_reference, glu_fwd, glu_inputs, glu_reference, quantized,
                           tokens)

pytestmark = pytest.mark.gpu
# (few rows; 128 x 128 tiles; 256-row tiles)
SIZES = [(300, 128, 512), (1000, 128, 1416), (600, 8, 1416), (4100, 128, 1416), (4100, 200, 3592)]


@pytest.mark.parametrize("N,H,F", SIZES)
@pytest.mark.parametrize("gate,e8", [(0, False), (1, True)])
def test_glu_fwd(N, H, F, gate, e8):
    X, Wg, Wu = glu_inputs(N, H, F, e8, N)
    o = glu_fwd(N, H, F, gate, e8, X, Wg, Wu)
    g, u, h, eg, eu, eh = glu_reference(gate, X, Wg, Wu)
    z = o["Z"].double().cpu()
    for got, want, e in ((z[:, :F], g, eg), (z[:, F:], u, eu), (o["H"].double().cpu(), h, eh)):
        assert bool(((got - want).abs() <= BF16 * 1.01 * want.abs() + 2 * e + 1e-38).all())
    check_codes(o["Hq"], o["sH"], h, eh, e8)
    check_codes(o["Hq_t"], o["sH_t"], h.t().contiguous(), eh.t().contiguous(), e8)


@pytest.mark.parametrize("N,H,F", SIZES)
@pytest.mark.parametrize("gate,e8,fmt", [(0, False, 0), (1, True, 1)])
def test_glu_bwd(N, H, F, gate, e8, fmt):
    dY = quantized(tokens(N + 1, N, H, 1e-3), e8, fmt=fmt)
    B = quantized(tokens(N + 2, F, H, 0.05), e8, True)
    Z = (tokens(N + 3, N, 2 * F) * 0.5).to(torch.bfloat16).to(DEV)
    q, s, q_t, s_t = glu_bwd(N, H, F, gate, e8, fmt, dY, B, Z)
    dg, du, eg, eu = glu_bwd_reference(gate, dY, B, Z, F)
    pf, gf = ref.up(F) * G, ref.up(F)
    for k, (d, e) in enumerate(((dg, eg), (du, eu))):
        check_codes(q[:, k * pf:(k + 1) * pf].contiguous(), s[k * gf:(k + 1) * gf].contiguous(), d, e, e8, fmt)
        check_codes(q_t[k], s_t[k], d.t().contiguous(), e.t().contiguous(), e8, fmt)
