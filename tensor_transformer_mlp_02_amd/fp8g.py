"""Binding of FP8 with group scales (declared in include/tpmlp_fp8g.h): the
quantizer, the product, the gated feed-forward block's projections and their
gradient.

Argument marshalling only, as in the package's ``__init__``.  Codes are
1-byte tensors (uint8 or a float8 type), scales float32 (TP_GROUP_F32) or
1-byte (TP_GROUP_E8M0) ones.
"""
from __future__ import annotations

import ctypes

from . import TP_BF16, _elt, _vp
from . import lib as _base_lib
from .block import _as, _call, _defaults, _entry, _i32, _i64, _sz

__all__ = [
    "TP_GROUP_F32", "TP_GROUP_E8M0", "TP_FP8G_GROUP", "TP_GATE_SILU", "TP_GATE_GELU_TANH",
    "tp_fp8g_quant_desc", "tp_fp8g_gemm_desc", "tp_fp8g_glu_desc",
    "tp_fp8g_quantize", "tp_fp8g_gemm", "tp_fp8g_glu_fwd", "tp_fp8g_glu_fwd_workspace",
    "tp_fp8g_glu_bwd", "tp_fp8g_glu_bwd_workspace",
]

TP_GROUP_F32, TP_GROUP_E8M0 = 0, 1
TP_GATE_SILU, TP_GATE_GELU_TANH = 0, 1
TP_FP8G_GROUP = 128


class tp_fp8g_quant_desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("dtype", _i32), ("fmt", _i32), ("scale", _i32),
                ("square", _i32)]


class tp_fp8g_gemm_desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("parts", _i32), ("fmt_a", _i32),
                ("fmt_b", _i32), ("scale", _i32), ("square", _i32), ("dtype", _i32),
                ("accumulate", _i32)]


class tp_fp8g_glu_desc(ctypes.Structure):
    _fields_ = [("N", _i64), ("H", _i64), ("F", _i64), ("gate", _i32), ("scale", _i32),
                ("fmt", _i32)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is None:
        L = _base_lib()
        for name, args, res in (
                ("tp_fp8g_quantize", [_vp] * 7, ctypes.c_int),
                ("tp_fp8g_gemm", [_vp] * 9, ctypes.c_int),
                ("tp_fp8g_glu_fwd_workspace", [_vp], _sz),
                ("tp_fp8g_glu_fwd", [_vp] * 14 + [_sz, _vp], ctypes.c_int),
                ("tp_fp8g_glu_bwd_workspace", [_vp], _sz),
                ("tp_fp8g_glu_bwd", [_vp] * 11 + [_sz, _vp], ctypes.c_int)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
            _entry[name] = ctypes.cast(fn, _vp).value
        _ready = L
    return _ready


def _run(name: str, args: tuple, stream) -> int:
    if _ready is None:
        _lib()
    return _call(name, args, stream)


_QUANT = _defaults(tp_fp8g_quant_desc, dtype=TP_BF16)
_GEMM = _defaults(tp_fp8g_gemm_desc, parts=1, dtype=TP_BF16)
_GLU = _defaults(tp_fp8g_glu_desc)


def _up(n: int) -> int:
    return -(-n // TP_FP8G_GROUP)


class _Scales:
    """A descriptor's scales as items: their bytes, and their element type."""

    def __init__(self, scale: int):
        self.size, self.type = (4, ("float32",)) if scale == TP_GROUP_F32 else (1, ())

    def __call__(self, t, count: int, name: str) -> tuple:
        return (t, count * self.size, name, *self.type)


def tp_fp8g_quantize(desc, x, q, s, q_t=None, s_t=None, stream=None) -> int:
    """Codes and scales of x along its rows (q, s), of its transpose (q_t, s_t), or both.  ``desc``:
    rows, cols and, with their defaults, dtype TP_BF16, fmt TP_FP8_E4M3, scale TP_GROUP_F32,
    square 0."""
    d = _as(tp_fp8g_quant_desc, desc, _QUANT)
    r, c, sc = d.rows, d.cols, _Scales(d.scale)
    gr, gc = _up(r), _up(c)
    return _run("tp_fp8g_quantize", (
        ctypes.addressof(d), (x, r * c * _elt(d.dtype), "x", "bfloat16" if d.dtype == TP_BF16 else "float32"),
        (q, r * gc * 128, "q"), sc(s, (gr if d.square else r) * gc, "s"),
        (q_t, c * gr * 128, "q_t"), sc(s_t, (gc if d.square else c) * gr, "s_t")), stream)


def tp_fp8g_gemm(desc, A, sA, B, sB, C, B2=None, sB2=None, stream=None) -> int:
    """C = A B^T of codes (parts 2: [A_0|A_1] [B|B2]^T).  ``desc``: M, N, K and, with their defaults,
    parts 1, fmt_a and fmt_b TP_FP8_E4M3, scale TP_GROUP_F32, square 0, dtype TP_BF16,
    accumulate 0."""
    d = _as(tp_fp8g_gemm_desc, desc, _GEMM)
    m, n, k, p, sc = d.M, d.N, d.K, d.parts, _Scales(d.scale)
    kg = _up(k)
    sb = (_up(n) if d.square else n) * kg
    return _run("tp_fp8g_gemm", (
        ctypes.addressof(d), (A, m * k * p, "A"), sc(sA, m * kg * p, "sA"), (B, n * k, "B"),
        sc(sB, sb, "sB"), (B2, n * k, "B2"), sc(sB2, sb, "sB2"),
        (C, m * n * _elt(d.dtype), "C", "bfloat16" if d.dtype == TP_BF16 else "float32")), stream)


def _glu(desc) -> tp_fp8g_glu_desc:
    return _as(tp_fp8g_glu_desc, desc, _GLU)


def tp_fp8g_glu_fwd_workspace(desc) -> int:
    return int(_lib().tp_fp8g_glu_fwd_workspace(ctypes.byref(_glu(desc))))


def tp_fp8g_glu_fwd(desc, X, sX, Wg, sWg, Wu, sWu, Z_save, H_act, Hq, sH, Hq_t, sH_t, workspace,
                    ws_bytes: int, stream=None) -> int:
    """G = X Wg^T, U = X Wu^T, H = act(G) U; Z_save = [G|U], H_act, and the codes of H along its rows
    (Hq, sH) and along the tokens (Hq_t, sH_t), each of them optional.  ``desc``: N, H, F and, with
    their defaults, gate TP_GATE_SILU, scale TP_GROUP_F32, fmt TP_FP8_E4M3."""
    d = _glu(desc)
    n, f, gh, gf, gn, sc = d.N, d.F, _up(d.H), _up(d.F), _up(d.N), _Scales(d.scale)
    return _run("tp_fp8g_glu_fwd", (
        ctypes.addressof(d), (X, n * gh * 128, "X"), sc(sX, n * gh, "sX"), (Wg, f * gh * 128, "Wg"),
        sc(sWg, gf * gh, "sWg"), (Wu, f * gh * 128, "Wu"), sc(sWu, gf * gh, "sWu"),
        (Z_save, n * f * 4, "Z_save", "bfloat16"), (H_act, n * f * 2, "H_act", "bfloat16"),
        (Hq, n * gf * 128, "Hq"), sc(sH, n * gf, "sH"), (Hq_t, f * gn * 128, "Hq_t"),
        sc(sH_t, f * gn, "sH_t"), (workspace, int(ws_bytes), "workspace"), int(ws_bytes)), stream)


def tp_fp8g_glu_bwd_workspace(desc) -> int:
    return int(_lib().tp_fp8g_glu_bwd_workspace(ctypes.byref(_glu(desc))))


def tp_fp8g_glu_bwd(desc, dY, sdY, B, sB, Z_save, dZ, sdZ, dZ_t, sdZ_t, workspace, ws_bytes: int,
                    stream=None) -> int:
    """dH = dY B^T, dG = dH U act'(G), dU = dH act(G): the codes of [dG|dU] along their rows (dZ, sdZ)
    and along the tokens (dZ_t, sdZ_t), either pair optional.  ``desc`` as the forward's; fmt is that
    of dY and dZ."""
    d = _glu(desc)
    n, f, gh, gf, gn, sc = d.N, d.F, _up(d.H), _up(d.F), _up(d.N), _Scales(d.scale)
    return _run("tp_fp8g_glu_bwd", (
        ctypes.addressof(d), (dY, n * gh * 128, "dY"), sc(sdY, n * gh, "sdY"), (B, f * gh * 128, "B"),
        sc(sB, gf * gh, "sB"), (Z_save, n * f * 4, "Z_save", "bfloat16"), (dZ, n * 2 * gf * 128, "dZ"),
        sc(sdZ, n * 2 * gf, "sdZ"), (dZ_t, 2 * f * gn * 128, "dZ_t"), sc(sdZ_t, 2 * f * gn, "sdZ_t"),
        (workspace, int(ws_bytes), "workspace"), int(ws_bytes)), stream)
