"""FP8 with group scales in 64 bits, from the formulas of include/tpmlp_fp8g.h (CPU)."""
import torch

G = 128
FMAX = {0: 448.0, 1: 57344.0}
TYPE = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


def up(n):
    return -(-n // G)


def padded(x, rows=False):
    r, c = x.shape
    out = torch.zeros((up(r) * G if rows else r), up(c) * G, dtype=x.dtype)
    out[:r, :c] = x
    return out


def scale_of(top, fmt, e8):
    """(multiplier, fp32 scale, stored scale) of fp32 maxima, each operation rounded as the header says."""
    fmax = torch.tensor(FMAX[fmt], dtype=torch.float32)
    bad = ~torch.isfinite(top)
    some = (top > 2.0 ** -100) & ~bad
    a = torch.where(some, top, fmax)
    if e8:
        p = torch.ceil(torch.log2(a.double() / float(fmax)))
        p = torch.where(a.double() / 2.0 ** p > float(fmax), p + 1, p)
        p = torch.where(a.double() / 2.0 ** (p - 1) <= float(fmax), p - 1, p)
        stored = (p + 127).to(torch.uint8)
        s, inv = (2.0 ** p).float(), (2.0 ** -p).float()
        stored = torch.where(bad, torch.full_like(stored, 255), torch.where(some, stored, torch.full_like(stored, 127)))
        s = torch.where(bad, torch.full_like(s, float("nan")), torch.where(some, s, torch.ones_like(s)))
        return torch.where(some, inv, torch.zeros_like(inv)), s, stored
    s = torch.where(bad, torch.full_like(a, float("nan")), a / fmax)
    return torch.where(some, fmax / a, torch.zeros_like(a)), s, s


def code(y, fmt):
    """The code (its value, fp64) nearest to fp32 y, ties to even, saturated."""
    return y.clamp(-FMAX[fmt], FMAX[fmt]).to(TYPE[fmt])


def largest(x, dim):
    """Largest magnitude; NaN where there is one."""
    m = x.abs().amax(dim)
    return torch.where(torch.isnan(x).sum(dim) > 0, torch.full_like(m, float("nan")), m)


def quantize(x, fmt=0, e8=False, square=False):
    """(codes [R, P(C)] as float8, fp32 scales, stored scales) of fp32 x."""
    R = x.shape[0]
    if square:
        v = padded(x, True)
        v = v.view(v.shape[0] // G, G, -1, G)
        inv, s, stored = scale_of(largest(v, (1, 3)), fmt, e8)
        m = inv[:, None, :, None]
    else:
        v = padded(x).view(R, -1, G)
        inv, s, stored = scale_of(largest(v, 2), fmt, e8)
        m = inv[:, :, None]
        s, stored = s.t().contiguous(), stored.t().contiguous()
    y = torch.where(m > 0, v * m, torch.zeros_like(v))
    q = code(y, fmt).view(-1, up(x.shape[1]) * G)[:R]
    return q, s, stored


def values(q, s, square=False, fmt=0):
    """fp64 values of codes (float8 or bytes) with fp32 or E8M0 scales."""
    v = (q if q.dtype == TYPE[fmt] else q.view(TYPE[fmt])).float().double()
    if s.dtype == torch.uint8:
        s = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=torch.float64), 2.0 ** (s.double() - 127))
    s = s.double()
    R, C = v.shape
    if square:
        return v * s.repeat_interleave(G, 0)[:R].repeat_interleave(G, 1)[:, :C]
    return v * s.t().repeat_interleave(G, 1)


def gate(name, g):
    """Activation and derivative (name 0: SiLU, 1: GeLU in its tanh form)."""
    if name == 0:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c, k = (2 / torch.pi) ** 0.5, 0.044715
    # (1 + tanh z) / 2 = sigmoid(2 z), which far below zero is no difference of near equals
    z = 2 * c * (g + k * g ** 3)
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    return g * s, s + g * 2 * s * r * c * (1 + 3 * k * g * g)


def sum_error(A, B):
    """How far an fp32 sum of A B^T may be off, element by element.  In a group the products are exact
    in fp32 and added one by one or in a tree: at most 128 roundings; then one rounding for the group's
    scale and one for its addition, for each group; 4 for what comes after."""
    groups = A.shape[1] // G
    return (G + 2 * groups + 4) * 2.0 ** -24 * (A.abs() @ B.abs().t())


def few_bits_error(A, B):
    """The same for the FP8 instruction's sums: of 8 products each may lose what lies 13 bits below the
    largest (2^-13 of it; a product may be twice the power of two that goes by, so 2^-12), and
    8 of them, against their sum of magnitudes: 2^-9."""
    return 2.0 ** -9 * (A.abs() @ B.abs().t()) + sum_error(A, B)


# Sizes at which each of the kernels is taken (tests/test_fp8g_plan.py holds them to that): ragged in every dimension
GEMM_FORMS = [(300, 1000, 640, "f32", "FEW"), (65, 2056, 1152, "bf16", "FEW"), (1030, 1000, 384, "bf16", "SMALL"),
              (2000, 2040, 1152, "f32", "SMALL"), (2100, 2056, 384, "bf16", "SMALL"), (4100, 2056, 640, "f32", "SMALL"),
              (4000, 4000, 640, "bf16", "LARGE"), (4000, 3976, 640, "f32", "LARGE")]
FWD_FORMS = [(300, 2056, 1416, "FEW"), (500, 264, 1416, "SMALL"), (2000, 520, 1032, "GROUP"), (4100, 136, 1416, "LARGE")]
BWD_FORMS = [(500, 264, 1416, "FEW"), (1000, 1032, 1416, "SMALL"), (2000, 520, 1032, "GROUP"), (6000, 1032, 2056, "LARGE")]
