"""GPU: FP8 with group scales at the ends of its ranges, against the formulas in 64 bits: power-of-two scales beside
fp32's largest and smallest values; more workgroups than a launch has; offsets past 2^32."""
import pytest
import torch

import fp8g_big as big
import fp8g_ref as ref
import tensor_transformer_mlp_02_amd as tp
from test_gpu_fp8g import (BF16, DEV, G, check_codes, check_product, glu_bwd, glu_bwd_reference, glu_fwd,
                           glu_inputs, glu_reference, product, quantized, tokens)

pytestmark = pytest.mark.gpu
FLT_MAX = 3.4028234663852886e38


@pytest.fixture(scope="module", autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


# a few rows; then each of the kernels (fp8g_ref.GEMM_FORMS)
SIZES = [(8, 264, 256, "f32"), (8, 264, 256, "bf16")] + [s[:4] for s in ref.GEMM_FORMS]


# --- power-of-two scales ------------------------------------------------------
def check_far(got, a, b, out):
    """As check_product, with what fp32 and bf16 cannot hold below their smallest normal numbers: a product and its
    addition are each off by at most fp32's smallest step 2^-149, of a quarter of them (the widened scales are
    halves) 4 times that, 2 K of them; a bf16 result by half its smallest step, 2^-134."""
    want = a @ b.t()
    small = 8 * a.shape[1] * 2.0 ** -149
    if out == "bf16":
        bound = BF16 * want.abs() * 1.01 + ref.few_bits_error(a, b) + small + 2.0 ** -134
    else:
        bound = ref.sum_error(a, b) + small
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("M,N,K,out", SIZES)
@pytest.mark.parametrize("far", ["A", "B"])
def test_largest_values(M, N, K, out, far):
    """FLT_MAX has the code 256 and the scale 2^120: 2^128, whose products with small numbers are ordinary ones."""
    a, b = tokens(1, M, K) * 2.0 ** -70, tokens(2, N, K) * 2.0 ** -70
    t = a if far == "A" else b
    t[3, 1], t[5, G + 2], t[-1] = FLT_MAX, -FLT_MAX, FLT_MAX
    A, sA, a = quantized(a, True)
    B, sB, b = quantized(b, True)
    assert float((a if far == "A" else b).abs().max()) == 2.0 ** 128
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    check_far(product(A, sA, B, sB, M, N, K, dtype, scale=1), a, b, out)


@pytest.mark.parametrize("M,N,K,out", SIZES)
@pytest.mark.parametrize("fmt", [0, 1])
def test_smallest_codes(M, N, K, out, fmt):
    """The smallest code of the smallest scale that a group has, against a large number: exact."""
    byte, code = (19, 2.0 ** -9) if fmt == 0 else (12, 2.0 ** -16)
    A, sA = torch.ones(M, K, dtype=torch.uint8, device=DEV), torch.full((K // G, M), byte, dtype=torch.uint8, device=DEV)
    B, sB = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV), torch.full((K // G, N), 127 + 100, dtype=torch.uint8, device=DEV)
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    got = product(A, sA, B, sB, M, N, K, dtype, scale=1, fmt_a=fmt).double()
    want = torch.tensor(K * code * 2.0 ** (byte - 127 + 100), dtype=torch.float64)
    assert bool((got == want.to(dtype).double().item()).all()), (float(got[0, 0]), float(want))


@pytest.mark.parametrize("N,H,F", [(9, 264, 392)] + [s[:3] for s in ref.FWD_FORMS])
def test_largest_values_glu_fwd(N, H, F):
    x = tokens(N, N, H)
    x[3, 1], x[-1, 2] = FLT_MAX, -FLT_MAX
    X = quantized(x, True)
    Wg, Wu = (quantized(tokens(N + k, F, H, 0.3 / H ** 0.5) * 2.0 ** -90, True, True) for k in (1, 2))
    o = glu_fwd(N, H, F, 0, True, X, Wg, Wu)
    g, u, h, eg, eu, eh = glu_reference(0, X, Wg, Wu)
    z = o["Z"].double().cpu()
    for got, want, e in ((z[:, :F], g, eg), (z[:, F:], u, eu), (o["H"].double().cpu(), h, eh)):
        assert bool(((got - want).abs() <= BF16 * 1.01 * want.abs() + 2 * e + 1e-38).all())
    check_codes(o["Hq"], o["sH"], h, eh, True)
    check_codes(o["Hq_t"], o["sH_t"], h.t().contiguous(), eh.t().contiguous(), True)


@pytest.mark.parametrize("N,H,F", [(9, 264, 392)] + [s[:3] for s in ref.BWD_FORMS])
def test_largest_values_glu_bwd(N, H, F):
    dy = tokens(N + 1, N, H) * 2.0 ** 60
    dy[3, 1], dy[-1, 2] = FLT_MAX, -FLT_MAX
    dY = quantized(dy, True)
    B = quantized(tokens(N + 2, F, H, 0.05) * 2.0 ** -90, True, True)
    Z = (tokens(N + 3, N, 2 * F) * 0.5).to(torch.bfloat16).to(DEV)
    q, s, q_t, s_t = glu_bwd(N, H, F, 0, True, 0, dY, B, Z)
    dg, du, eg, eu = glu_bwd_reference(0, dY, B, Z, F)
    pf, gf = ref.up(F) * G, ref.up(F)
    for k, (d, e) in enumerate(((dg, eg), (du, eu))):
        check_codes(q[:, k * pf:(k + 1) * pf].contiguous(), s[k * gf:(k + 1) * gf].contiguous(), d, e, True)
        check_codes(q_t[k], s_t[k], d.t().contiguous(), e.t().contiguous(), True)


# --- more workgroups than a launch has ----------------------------------------
def memory_for(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"{gib} GiB of device memory")


# 2^24 workgroups of 256 threads (a launch ends below 2^32 threads), few rows' kernel; 2^23, the 64 x 128 tiles'
@pytest.mark.parametrize("M,N", [((1 << 30) - 5, 8), ((1 << 28) + 1000, 136)])
def test_gemm_of_many_workgroups(M, N):
    memory_for(200)
    K, tail = G, 200
    A = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    sA = torch.full((1, M), 127, dtype=torch.uint8, device=DEV)
    B, sB, b = quantized(tokens(2, N, K), True, True)
    C = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    # beside the first and the last row, and beside the borders between launches
    step = (1 << 22) * 64 // ref.up(N)
    places = [0, M - tail] + [r - tail // 2 for r in range(step, M, step)]
    rows = {}
    for i, r in enumerate(p for p in places if 0 <= p <= M - tail):
        q, s, rows[r] = quantized(tokens(10 + i, tail, K), True)
        A[r:r + tail], sA[:, r:r + tail] = q, s
    product(A, sA, B, sB, M, N, K, torch.bfloat16, C, scale=1, square=1)
    for r, a in rows.items():
        check_product(C[r:r + tail], a, b, torch.bfloat16)
        C[r:r + tail] = 0
    for part in C.split(1 << 26):
        assert not bool(part.any())


# --- offsets past 2^32 bytes ---------------------------------------------------
TAIL = 300


def empty(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


def nothing(*tensors):
    for t in tensors:
        for part in t.split(max(1, (1 << 30) // max(1, t[0].numel()))):
            assert not bool(part.any())


def ones(*tensors):
    for t in tensors:
        assert bool((t == 1).all())


@pytest.mark.parametrize("square", [0, 1])
def test_quantize_both_past_32_bits(square):
    rows, cols, n = 600_000, 8192, 3 * G + 64     # (the last groups of 128 rows, the last of them half a group)
    memory_for(40)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = tokens(7, n, cols).to(torch.bfloat16)
    x[-n:] = tail.to(DEV)
    gr, gc, pr = ref.up(rows), ref.up(cols), ref.up(rows) * G
    q, q_t = empty(rows, cols), empty(cols, pr)
    s, s_t = (empty(*d, dtype=torch.float32) for d in (((gr, gc), (gc, gr)) if square else ((gc, rows), (gr, cols))))
    tp.tp_fp8g_quantize(dict(rows=rows, cols=cols, square=square), x, q, s, q_t, s_t)
    m = ref.up(n)
    cq, _, cs = ref.quantize(tail.float(), 0, False, bool(square))
    assert torch.equal(q[-n:].cpu(), cq.view(torch.uint8)) and torch.equal((s[-m:] if square else s[:, -n:]).cpu(), cs)
    cq, _, cs = ref.quantize(tail.float().t().contiguous(), 0, False, bool(square))
    assert torch.equal(q_t[:, -m * G:].cpu(), cq.view(torch.uint8)) and torch.equal((s_t[:, -m:] if square else s_t[-m:]).cpu(), cs)
    nothing(q[:-n], q_t[:, :-m * G])
    ones(*((s[:-m], s_t[:, :-m]) if square else (s[:, :-n], s_t[:-m])))


@pytest.mark.parametrize("M,N,K,out,form", big.GEMM)
@pytest.mark.parametrize("square", [0, 1])
def test_gemm_past_32_bits(M, N, K, out, form, square):
    memory_for(80)
    A, sA = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.ones(K // G, M, device=DEV)
    q, s, a = quantized(tokens(13, TAIL, K))
    A[-TAIL:], sA[:, -TAIL:] = q, s
    B, sB, b = quantized(tokens(14, N, K), square=bool(square))
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    C = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    product(A, sA, B, sB, M, N, K, dtype, C, square=square)
    check_product(C[-TAIL:], a, b, dtype)
    nothing(C[:-TAIL])


@pytest.mark.parametrize("N,H,F,form", big.FWD)
def test_glu_fwd_past_32_bits(N, H, F, form):
    memory_for(120)
    (q, s, x), Wg, Wu = glu_inputs(TAIL, H, F, False, 1)
    X, sX = torch.zeros(N, ref.up(H) * G, dtype=torch.uint8, device=DEV), torch.ones(ref.up(H), N, device=DEV)
    X[-TAIL:], sX[:, -TAIL:] = q, s
    gf, gn = ref.up(F), ref.up(N)
    Z, Hb, Hq, sH = (empty(N, 2 * F, dtype=torch.bfloat16), empty(N, F, dtype=torch.bfloat16), empty(N, gf * G),
                     empty(gf, N, dtype=torch.float32))
    Hq_t, sH_t = empty(F, gn * G), empty(gn, F, dtype=torch.float32)
    d = dict(N=N, H=H, F=F)
    n = tp.tp_fp8g_glu_fwd_workspace(d)
    tp.tp_fp8g_glu_fwd(d, X, sX, Wg[0], Wg[1], Wu[0], Wu[1], Z, Hb, Hq, sH, Hq_t, sH_t, empty(n), n)
    g, u, h, eg, eu, eh = glu_reference(0, (q, s, x), Wg, Wu)
    z = Z[-TAIL:].double().cpu()
    for got, want, e in ((z[:, :F], g, eg), (z[:, F:], u, eu), (Hb[-TAIL:].double().cpu(), h, eh)):
        assert bool(((got - want).abs() <= BF16 * 1.01 * want.abs() + 2 * e + 1e-38).all())
    check_codes(Hq[-TAIL:], sH[:, -TAIL:].contiguous(), h, eh, False)
    # the groups of 128 tokens that the last ones are in
    m = gn - (N - TAIL) // G
    lead = N - TAIL - (gn - m) * G
    ht, et = (torch.cat([torch.zeros(lead, F, dtype=torch.float64), t]).t().contiguous() for t in (h, eh))
    check_codes(Hq_t[:, -m * G:].contiguous(), sH_t[-m:].contiguous(), ht, et, False)
    nothing(Z[:-TAIL], Hb[:-TAIL], Hq[:-TAIL], Hq_t[:, :-m * G])
    ones(sH[:, :-TAIL], sH_t[:-m])


@pytest.mark.parametrize("N,H,F,form", big.BWD)
def test_glu_bwd_past_32_bits(N, H, F, form):
    memory_for(120)
    q, s, y = quantized(tokens(1, TAIL, H, 1e-3))
    B = quantized(tokens(2, F, H, 0.05), False, True)
    z = (tokens(3, TAIL, 2 * F) * 0.5).to(torch.bfloat16).to(DEV)
    dY, sdY = torch.zeros(N, ref.up(H) * G, dtype=torch.uint8, device=DEV), torch.ones(ref.up(H), N, device=DEV)
    Z = torch.zeros(N, 2 * F, dtype=torch.bfloat16, device=DEV)
    dY[-TAIL:], sdY[:, -TAIL:], Z[-TAIL:] = q, s, z
    gf, gn, pf = ref.up(F), ref.up(N), ref.up(F) * G
    dZ, sdZ = empty(N, 2 * pf), empty(2 * gf, N, dtype=torch.float32)
    dZ_t, sdZ_t = empty(2, F, gn * G), empty(2, gn, F, dtype=torch.float32)
    d = dict(N=N, H=H, F=F)
    n = tp.tp_fp8g_glu_bwd_workspace(d)
    tp.tp_fp8g_glu_bwd(d, dY, sdY, B[0], B[1], Z, dZ, sdZ, dZ_t, sdZ_t, empty(n), n)
    dg, du, eg, eu = glu_bwd_reference(0, (q, s, y), B, z, F)
    m = gn - (N - TAIL) // G
    lead = N - TAIL - (gn - m) * G
    for k, (v, e) in enumerate(((dg, eg), (du, eu))):
        check_codes(dZ[-TAIL:, k * pf:(k + 1) * pf].contiguous(), sdZ[k * gf:(k + 1) * gf, -TAIL:].contiguous(), v, e, False)
        vt, et = (torch.cat([torch.zeros(lead, F, dtype=torch.float64), t]).t().contiguous() for t in (v, e))
        check_codes(dZ_t[k, :, -m * G:].contiguous(), sdZ_t[k, -m:].contiguous(), vt, et, False)
        nothing(dZ_t[k, :, :-m * G])
    nothing(dZ[:-TAIL])
    ones(sdZ[:, :-TAIL], sdZ_t[:, :-m])
