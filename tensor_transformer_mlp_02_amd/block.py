"""Binding of the operators around the products (declared in
include/tpmlp_block.h): block norms, routing to experts, AdamW.

Argument marshalling only, as in the package's ``__init__``: device tensors
or raw addresses in, the C entry point of the same name called on the
current HIP stream, ``TpError`` on a nonzero status.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import TP_BF16, _check, _current_device, _elt, _marshaller, _ptr, _sized, _stream, _vp
from . import lib as _base_lib

__all__ = [
    "TP_NORM_RMS", "TP_NORM_LAYER", "TP_SCORE_SOFTMAX", "TP_SCORE_SIGMOID", "TP_ADAMW_BLOCK",
    "tp_norm_desc", "tp_route_desc", "tp_adamw_desc", "tp_adamw_tensor",
    "tp_block_norm_fwd", "tp_block_norm_bwd", "tp_block_norm_bwd_workspace",
    "tp_moe_route_fwd", "tp_moe_route_bwd", "tp_moe_route_tables",
    "tp_moe_route_tables_workspace", "tp_adamw_tensors", "tp_adamw_step",
]

TP_NORM_RMS, TP_NORM_LAYER = 0, 1
TP_SCORE_SOFTMAX, TP_SCORE_SIGMOID = 0, 1
TP_ADAMW_BLOCK = 256

_i32, _i64, _f32, _f64, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                               ctypes.c_size_t)


class tp_norm_desc(ctypes.Structure):
    _fields_ = [("N", _i64), ("H", _i64), ("gate_rows", _i64), ("kind", _i32), ("dtype", _i32),
                ("eps", _f32), ("res_scale", _f32), ("branch_scale", _f32)]


class tp_route_desc(ctypes.Structure):
    _fields_ = [("N", _i64), ("E", _i32), ("K", _i32), ("groups", _i32), ("groups_kept", _i32),
                ("group_best", _i32), ("score", _i32), ("renorm", _i32), ("dtype", _i32),
                ("scale", _f32)]


class tp_adamw_desc(ctypes.Structure):
    _fields_ = [("lr", _f64), ("beta1", _f64), ("beta2", _f64), ("eps", _f64), ("step", _i32),
                ("grad_dtype", _i32), ("state_bits", _i32), ("seed", ctypes.c_uint32)]


class tp_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("param_bf16", _vp), ("grad", _vp), ("m", _vp), ("v", _vp),
                ("m_scale", _vp), ("v_scale", _vp), ("count", _i64), ("weight_decay", _f32),
                ("reserved", _i32)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is None:
        L = _base_lib()
        ND = RD = AD = AT = _vp  # structures, by address
        for name, args, res in (
                ("tp_block_norm_fwd", [ND] + [_vp] * 12, ctypes.c_int),
                ("tp_block_norm_bwd_workspace", [ND], _sz),
                ("tp_block_norm_bwd", [ND] + [_vp] * 18 + [_sz, _i32, _vp], ctypes.c_int),
                ("tp_moe_route_fwd", [RD] + [_vp] * 5, ctypes.c_int),
                ("tp_moe_route_bwd", [RD] + [_vp] * 4 + [_i64, _vp, _vp], ctypes.c_int),
                ("tp_moe_route_tables_workspace", [_i64, _i32, _i32], _sz),
                ("tp_moe_route_tables", [_i64, _i32, _i32, _i32, _i64] + [_vp] * 9 + [_sz, _vp],
                 ctypes.c_int),
                ("tp_adamw_step", [AD, _i32, AT] + [_vp] * 4, ctypes.c_int)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
            _entry[name] = ctypes.cast(fn, _vp).value
        _ready = L
    return _ready


_entry = {}


def _call(name: str, args: tuple, stream) -> int:
    """Entry point `name` with args (items as _sized takes them, ints, None) and the stream."""
    L = _ready or _lib()
    if stream is not None:
        stream = _stream(stream)
    m = _marshaller()
    rc = m.call(name, _entry[name], args, stream) if m else None
    if rc is None:
        rc = getattr(L, name)(*[_sized([a])[0] if isinstance(a, tuple) else a for a in args],
                              _stream(stream))
    return rc if rc == 0 else _check(rc)


def _defaults(cls, **given):
    """Every field of a descriptor in its order, 0 where nothing else is the default."""
    return {name: given.get(name, 0) for name, _ in cls._fields_}


_NORM = _defaults(tp_norm_desc, kind=TP_NORM_RMS, dtype=TP_BF16, eps=1e-5, res_scale=1.0,
                  branch_scale=1.0)
_ROUTE = _defaults(tp_route_desc, groups=1, groups_kept=1, group_best=1, score=TP_SCORE_SOFTMAX,
                   scale=1.0)
_ADAMW = _defaults(tp_adamw_desc, beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_bits=32)


def _as(cls, desc, defaults):
    if isinstance(desc, cls):
        return desc
    fields = {**defaults, **desc}   # in the structure's order
    if len(fields) != len(defaults):
        raise TypeError(f"{cls.__name__} has no field {sorted(fields.keys() - defaults.keys())}")
    return cls(*fields.values())


def _norm(desc) -> tp_norm_desc:
    return _as(tp_norm_desc, desc, _NORM)


def _route(desc) -> tp_route_desc:
    return _as(tp_route_desc, desc, _ROUTE)


def _adamw(desc) -> tp_adamw_desc:
    return _as(tp_adamw_desc, desc, _ADAMW)


def _type(d) -> str:
    return "bfloat16" if d.dtype == TP_BF16 else "float32"


def _norm_sizes(d: tp_norm_desc):
    # (a negative size asks for nothing here: the library refuses it)
    n, h = d.N, d.H
    vec = h * _elt(d.dtype)
    return _type(d), n * vec, vec, d.gate_rows * vec, h * 4, d.gate_rows * h * 4, n * (8 if d.kind else 4)


def tp_block_norm_fwd(desc, X, O, w_post, b_post, gate, w_pre, b_pre, Y, Hn, stat_post=None,
                      stat_pre=None, stream=None) -> int:
    """Y = res_scale X + branch_scale gate norm(O), Hn = norm(Y).  ``desc``: N, H and, with their
    defaults, gate_rows 0, kind TP_NORM_RMS, dtype TP_BF16, eps 1e-5, res_scale 1, branch_scale 1."""
    d = _norm(desc)
    t, rows, vec, gate_n, _, _, stat = _norm_sizes(d)
    return _call("tp_block_norm_fwd", (
        ctypes.addressof(d), (X, rows, "X", t), (O, rows, "O", t), (w_post, vec, "w_post", t),
        (b_post, vec, "b_post", t), (gate, gate_n, "gate", t), (w_pre, vec, "w_pre", t),
        (b_pre, vec, "b_pre", t), (Y, rows, "Y", t), (Hn, rows, "Hn", t),
        (stat_post, stat, "stat_post", "float32"), (stat_pre, stat, "stat_pre", "float32")), stream)


def tp_block_norm_bwd_workspace(desc) -> int:
    return int(_lib().tp_block_norm_bwd_workspace(ctypes.byref(_norm(desc))))


def tp_block_norm_bwd(desc, dY, dHn, Y, O, w_post, b_post, gate, w_pre, stat_post, stat_pre, dX,
                      dO, dw_post, db_post, dgate, dw_pre, db_pre, workspace, ws_bytes: int,
                      accumulate: bool = False, stream=None) -> int:
    """Gradients of tp_block_norm_fwd from its Y (X where O is None), O and statistics;
    accumulate=True adds into the fp32 gradients."""
    d = _norm(desc)
    t, rows, vec, gate_n, out, gate_out, stat = _norm_sizes(d)
    return _call("tp_block_norm_bwd", (
        ctypes.addressof(d), (dY, rows, "dY", t), (dHn, rows, "dHn", t), (Y, rows, "Y", t), (O, rows, "O", t),
        (w_post, vec, "w_post", t), (b_post, vec, "b_post", t), (gate, gate_n, "gate", t),
        (w_pre, vec, "w_pre", t), (stat_post, stat, "stat_post", "float32"),
        (stat_pre, stat, "stat_pre", "float32"), (dX, rows, "dX", t), (dO, rows, "dO", t),
        (dw_post, out, "dw_post", "float32"), (db_post, out, "db_post", "float32"),
        (dgate, gate_out, "dgate", "float32"), (dw_pre, out, "dw_pre", "float32"),
        (db_pre, out, "db_pre", "float32"), (workspace, int(ws_bytes), "workspace"),
        int(ws_bytes), 1 if accumulate else 0), stream)


def tp_moe_route_fwd(desc, logits, bias, topk_expert, topk_weight, stream=None) -> int:
    """The K experts of each token and their weights.  ``desc``: N, E, K and, with their defaults,
    groups 1, groups_kept 1, group_best 1, score TP_SCORE_SOFTMAX, renorm 0, dtype TP_F32, scale 1."""
    d = _route(desc)
    n, e, k, t = d.N, d.E, d.K, _type(d)
    return _call("tp_moe_route_fwd", (
        ctypes.addressof(d), (logits, n * e * _elt(d.dtype), "logits", t),
        (bias, e * 4, "bias", "float32"), (topk_expert, n * k * 4, "topk_expert", "int32"),
        (topk_weight, n * k * 4, "topk_weight", "float32")), stream)


def tp_moe_route_bwd(desc, logits, topk_expert, d_weight, slot_row, R: int, dlogits,
                     stream=None) -> int:
    """dlogits from the weights' gradient: d_weight [N,K] with slot_row None, else [R] by rows."""
    d = _route(desc)
    n, e, k, t = d.N, d.E, d.K, _type(d)
    dw = n * k * 4 if slot_row is None else int(R) * 4
    whole = n * e * _elt(d.dtype)
    return _call("tp_moe_route_bwd", (
        ctypes.addressof(d), (logits, whole, "logits", t),
        (topk_expert, n * k * 4, "topk_expert", "int32"), (d_weight, dw, "d_weight", "float32"),
        (slot_row, n * k * 4, "slot_row", "int32"), int(R), (dlogits, whole, "dlogits", t)), stream)


def tp_moe_route_tables_workspace(N: int, K: int, n_local: int) -> int:
    return int(_lib().tp_moe_route_tables_workspace(int(N), int(K), int(n_local)))


def tp_moe_route_tables(N: int, K: int, first_expert: int, n_local: int, R: int, topk_expert,
                        topk_weight, offsets, row_token, row_weight, tok_ptr, tok_rows, slot_row,
                        workspace, ws_bytes: int, stream=None) -> int:
    """Dispatch tables of the experts [first_expert, first_expert + n_local), on the device."""
    N, K, first_expert, n_local, R, ws_bytes = (int(N), int(K), int(first_expert), int(n_local),
                                                int(R), int(ws_bytes))
    n, r = N * 4, R * 4
    nk = n * K
    return _call("tp_moe_route_tables", (
        N, K, first_expert, n_local, R, (topk_expert, nk, "topk_expert", "int32"),
        (topk_weight, nk, "topk_weight", "float32"),
        (offsets, (n_local + 1) * 4, "offsets", "int32"), (row_token, r, "row_token", "int32"),
        (row_weight, r, "row_weight", "float32"), (tok_ptr, n + 4, "tok_ptr", "int32"),
        (tok_rows, r, "tok_rows", "int32"), (slot_row, nk, "slot_row", "int32"),
        (workspace, ws_bytes, "workspace"), ws_bytes), stream)


class AdamwTensors:
    """The tensors of a step as the library reads them, laid out once.  Holds on to the tensors;
    they have to keep their memory (no resize) while the table is in use."""

    def __init__(self, desc, tensors):
        d = _adamw(desc)
        small = d.state_bits == 8
        self.formats = (d.grad_dtype, d.state_bits)
        self.n = len(tensors)
        self.array = (tp_adamw_tensor * max(1, self.n))()
        self.address = ctypes.addressof(self.array)
        self.tensors = [dict(t) for t in tensors]
        self.device = None
        state = None if small else "float32"
        for i, t in enumerate(self.tensors):
            count = t.get("count")
            count = t["param"].numel() if count is None else int(count)
            blocks = -(-max(count, 0) // TP_ADAMW_BLOCK)
            for name, nbytes, dtype in (
                    ("param", count * 4, "float32"), ("param_bf16", count * 2, "bfloat16"),
                    ("grad", count * _elt(d.grad_dtype),
                     "bfloat16" if d.grad_dtype == TP_BF16 else "float32"),
                    ("m", count if small else count * 4, state),
                    ("v", count if small else count * 4, state),
                    ("m_scale", blocks * 4, "float32"), ("v_scale", blocks * 4, "float32")):
                x = t.get(name)
                if small and name in ("m", "v") and getattr(x, "dtype", None) is not None \
                        and x.element_size() != 1:
                    raise ValueError(f"{name} of tensor {i} must have one byte an element")
                setattr(self.array[i], name,
                        _ptr(x, max(nbytes, 0), f"{name} of tensor {i}", dtype))
                if self.device is None and hasattr(x, "device"):
                    self.device = x.device.index
            self.array[i].count = count
            self.array[i].weight_decay = float(t.get("weight_decay", 0.0))


def tp_adamw_tensors(desc, tensors) -> AdamwTensors:
    """The table of a step: ``tensors`` is a list of dicts with param (float32), grad, m, v and,
    where there, param_bf16, m_scale, v_scale, weight_decay (0), count (param's elements).  The
    types are those of ``desc`` (grad_dtype, state_bits)."""
    return AdamwTensors(desc, tensors)


def tp_adamw_step(desc, tensors, dev_step=None, dev_lr=None, grad_scale=None,
                  stream=None) -> int:
    """One AdamW step over ``tensors`` (tp_adamw_tensors, or the list it takes).  ``desc``: lr and,
    with their defaults, beta1 0.9, beta2 0.999, eps 1e-8, step 1, grad_dtype TP_F32,
    state_bits 32, seed 0.  dev_step (int32), dev_lr, grad_scale (float32): device scalars."""
    d = _adamw(desc)
    t = tensors if isinstance(tensors, AdamwTensors) else AdamwTensors(d, tensors)
    if t.formats != (d.grad_dtype, d.state_bits):
        raise ValueError(f"the table is for (grad_dtype, state_bits) = {t.formats}")
    if t.device is not None and _current_device() != t.device:
        raise ValueError(f"the table is on cuda:{t.device}, the current device is "
                         f"cuda:{_current_device()}")
    return _call("tp_adamw_step", (
        ctypes.addressof(d), t.n, t.address, (dev_step, 4, "dev_step", "int32"),
        (dev_lr, 4, "dev_lr", "float32"), (grad_scale, 4, "grad_scale", "float32")), stream)
