"""Argument checks of the operators around the products, on the CPU: every
refusal documented in include/tpmlp_block.h, before any GPU call."""
import ctypes
import math
import os
import re

import pytest

import tensor_transformer_mlp_02_amd as tp

try:
    import torch
    _gpu = torch.cuda.device_count() > 0
except ImportError:
    _gpu = False
# arguments that pass every check would reach a kernel with made-up addresses
pytestmark = pytest.mark.skipif(_gpu, reason="the accepted calls must end at the missing GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tpmlp_block.h")
E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_DEV, E_HIP, E_ALIAS = range(1, 9)


def addr(k, off=0):
    """Fake device addresses, 1 TiB apart (never dereferenced)."""
    return (1 << 44) + (k << 40) + off


def status(fn, *a, **kw):
    try:
        fn(*a, **kw)
    except tp.TpError as e:
        assert e.message
        return e.status
    return 0


def test_exports_every_declared_function():
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+(tp_\w+)\s*\(", text, re.M)))
    assert len(names) == 8, names
    for n in names:
        assert hasattr(tp.lib(), n) and n in tp.__all__, n


# --- block norms -------------------------------------------------------------
def nd(**kw):
    return {**dict(N=12, H=64, gate_rows=3, kind=tp.TP_NORM_LAYER, dtype=tp.TP_BF16, eps=1e-5,
                   res_scale=1.0, branch_scale=0.5), **kw}


FWD = dict(X=addr(1), O=addr(2), w_post=addr(3), b_post=addr(4), gate=addr(5), w_pre=addr(6),
           b_pre=addr(7), Y=addr(8), Hn=addr(9), stat_post=addr(10), stat_pre=addr(11))


def fwd(desc=None, **kw):
    return status(tp.tp_block_norm_fwd, desc or nd(), **{**FWD, **kw})


PURE = dict(O=None, w_post=None, b_post=None, gate=None, Y=None, stat_post=None)


@pytest.mark.parametrize("desc,want", [
    (nd(dtype=3), E_DTYPE), (nd(kind=2), E_DTYPE), (nd(N=-1), E_SHAPE), (nd(H=0), E_SHAPE),
    (nd(H=12), E_SHAPE), (nd(H=6, dtype=tp.TP_F32), E_SHAPE), (nd(H=(1 << 21) + 8), E_SHAPE),
    (nd(N=(1 << 30) + 1), E_SHAPE), (nd(gate_rows=-1), E_SHAPE), (nd(eps=0.0), E_SHAPE),
    (nd(eps=math.inf), E_SHAPE), (nd(eps=math.nan), E_SHAPE), (nd(res_scale=math.nan), E_SHAPE),
    (nd(branch_scale=math.inf), E_SHAPE), (nd(), E_DEV), (nd(N=0), E_DEV)])
def test_norm_descriptor(desc, want):
    assert fwd(desc) == want
    assert bwd(desc) == want


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), E_NULL), (dict(Y=None), E_NULL), (dict(Hn=None), E_NULL),
    (dict(w_post=None), E_NULL), (dict(w_pre=None), E_NULL), (dict(gate=None), E_NULL),
    (dict(w_post=None, b_post=None), E_SHAPE),               # its statistics are still asked for
    (dict(w_pre=None, b_pre=None), E_SHAPE),
    (dict(w_pre=None, b_pre=None, Hn=None, stat_pre=None), E_DEV),   # no norm after the sum
    (dict(O=None), E_SHAPE), (dict(X=addr(1, 8)), E_ALIGN), (dict(stat_pre=addr(11, 2)), E_ALIGN),
    (dict(stat_pre=addr(11, 4)), E_DEV), (dict(b_post=None, b_pre=None, stat_post=None,
                                               stat_pre=None), E_DEV),
    (dict(Y=addr(1)), E_DEV),                                # the stream updated in place
    (dict(Y=addr(1, 16)), E_ALIAS), (dict(Y=addr(2)), E_ALIAS), (dict(Hn=addr(1)), E_ALIAS),
    (dict(Hn=addr(8)), E_ALIAS), (dict(stat_pre=addr(10, 95)), E_ALIGN),
    (dict(stat_pre=addr(10, 92)), E_ALIAS), (dict(stat_pre=addr(10, 96)), E_DEV)])
def test_norm_forward_buffers(kw, want):
    assert fwd(**kw) == want


def test_norm_without_a_block():
    assert fwd(nd(gate_rows=0), **PURE) == E_DEV
    assert fwd(nd(gate_rows=0), **{**PURE, "w_pre": None, "b_pre": None}) == E_NULL
    assert fwd(nd(), **PURE) == E_SHAPE
    assert fwd(nd(N=0), X=None, O=None, Y=None, Hn=None) == E_DEV   # empty tensors have no address


BWD = dict(dY=addr(1), dHn=addr(2), Y=addr(3), O=addr(4), w_post=addr(5), b_post=addr(6),
           gate=addr(7), w_pre=addr(8), stat_post=addr(9), stat_pre=addr(10), dX=addr(11),
           dO=addr(12), dw_post=addr(13), db_post=addr(14), dgate=addr(15), dw_pre=addr(16),
           db_pre=addr(17), workspace=addr(18))


def bwd(desc=None, ws_bytes=None, accumulate=False, **kw):
    d = desc or nd()
    if ws_bytes is None:
        ws_bytes = tp.tp_block_norm_bwd_workspace(d)
    return status(tp.tp_block_norm_bwd, d, ws_bytes=ws_bytes, accumulate=accumulate, **{**BWD, **kw})


@pytest.mark.parametrize("kw,want", [
    (dict(dHn=None), E_NULL), (dict(Y=None), E_NULL), (dict(dX=None), E_NULL),
    (dict(dO=None), E_NULL), (dict(dw_post=None), E_NULL), (dict(dw_pre=None), E_NULL),
    (dict(dgate=None), E_NULL), (dict(gate=None), E_NULL), (dict(stat_post=None), E_NULL),
    (dict(stat_pre=None), E_NULL), (dict(w_post=None, b_post=None), E_SHAPE),
    (dict(dY=None), E_DEV), (dict(db_post=None, db_pre=None, b_post=None), E_DEV),
    (dict(w_pre=None), E_SHAPE), (dict(O=None), E_SHAPE), (dict(dX=addr(1)), E_ALIAS),
    (dict(dO=addr(4)), E_ALIAS), (dict(dw_pre=addr(13, 128)), E_ALIAS),
    (dict(dw_pre=addr(13, 256)), E_DEV), (dict(dw_pre=addr(16, 4)), E_ALIGN),
    (dict(workspace=None), E_WS), (dict(workspace=addr(18, 4)), E_ALIGN),
    (dict(workspace=addr(2)), E_ALIAS), (dict(ws_bytes=16), E_WS)])
def test_norm_backward_buffers(kw, want):
    assert bwd(**kw) == want


def test_norm_backward_optional_parts():
    gone = dict(w_pre=None, dHn=None, Y=None, stat_pre=None, dw_pre=None, db_pre=None)
    assert bwd(**gone) == E_DEV
    assert bwd(**gone, dY=None) == E_NULL           # no gradient at all
    pure = dict(O=None, w_post=None, b_post=None, gate=None, stat_post=None, dO=None,
                dw_post=None, db_post=None, dgate=None)
    assert bwd(nd(gate_rows=0), **pure) == E_DEV
    assert status(tp.tp_block_norm_bwd, nd(), ws_bytes=1 << 30, accumulate=True, **BWD) == E_DEV
    assert tp.tp_block_norm_bwd_workspace(nd(H=7)) == 0


# --- routing -----------------------------------------------------------------
def rd(**kw):
    return {**dict(N=10, E=64, K=4, groups=8, groups_kept=2, group_best=2,
                   score=tp.TP_SCORE_SIGMOID, renorm=1, dtype=tp.TP_F32, scale=1.0), **kw}


def route(desc=None, **kw):
    return status(tp.tp_moe_route_fwd, desc or rd(),
                  **{**dict(logits=addr(1), bias=addr(2), topk_expert=addr(3),
                            topk_weight=addr(4)), **kw})


def route_bwd(desc=None, **kw):
    return status(tp.tp_moe_route_bwd, desc or rd(),
                  **{**dict(logits=addr(1), topk_expert=addr(2), d_weight=addr(3),
                            slot_row=addr(4), R=40, dlogits=addr(5)), **kw})


@pytest.mark.parametrize("desc,want", [
    (rd(dtype=2), E_DTYPE), (rd(score=2), E_DTYPE), (rd(E=0), E_SHAPE), (rd(E=1025), E_SHAPE),
    (rd(K=0), E_SHAPE), (rd(K=33, groups=1, groups_kept=1), E_SHAPE), (rd(K=17), E_SHAPE),
    (rd(K=16), E_DEV), (rd(groups=0), E_SHAPE), (rd(groups=7), E_SHAPE), (rd(groups=128, E=128), E_SHAPE),
    (rd(groups_kept=0), E_SHAPE), (rd(groups_kept=9), E_SHAPE), (rd(group_best=0), E_SHAPE),
    (rd(group_best=3), E_SHAPE), (rd(renorm=2), E_SHAPE), (rd(scale=math.inf), E_SHAPE),
    (rd(N=-1), E_SHAPE), (rd(N=1 << 31), E_SHAPE), (rd(N=0), E_DEV), (rd(), E_DEV)])
def test_route_descriptor(desc, want):
    assert route(desc) == want
    assert route_bwd(desc) == want


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), E_NULL), (dict(topk_expert=None), E_NULL), (dict(topk_weight=None), E_NULL),
    (dict(bias=None), E_DEV), (dict(logits=addr(1, 4)), E_ALIGN), (dict(bias=addr(2, 2)), E_ALIGN),
    (dict(topk_weight=addr(4, 4)), E_DEV), (dict(topk_weight=addr(1, 16)), E_ALIAS),
    (dict(topk_weight=addr(3, 8)), E_ALIAS)])
def test_route_forward_buffers(kw, want):
    assert route(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), E_NULL), (dict(topk_expert=None), E_NULL), (dict(d_weight=None), E_NULL),
    (dict(dlogits=None), E_NULL), (dict(slot_row=None), E_DEV), (dict(R=0, d_weight=None), E_DEV),
    (dict(R=-1), E_SHAPE), (dict(dlogits=addr(1)), E_ALIAS), (dict(dlogits=addr(3)), E_ALIAS),
    (dict(d_weight=addr(3, 1)), E_ALIGN), (dict(dlogits=addr(5, 8)), E_ALIGN)])
def test_route_backward_buffers(kw, want):
    assert route_bwd(**kw) == want


def tables(ws_bytes=None, **kw):
    a = {**dict(N=10, K=4, first_expert=8, n_local=16, R=40, topk_expert=addr(1),
                topk_weight=addr(2), offsets=addr(3), row_token=addr(4), row_weight=addr(5),
                tok_ptr=addr(6), tok_rows=addr(7), slot_row=addr(8), workspace=addr(9)), **kw}
    if ws_bytes is None:
        ws_bytes = tp.tp_moe_route_tables_workspace(a["N"], a["K"], a["n_local"])
    return status(tp.tp_moe_route_tables, ws_bytes=ws_bytes, **a)


@pytest.mark.parametrize("kw,want", [
    (dict(), E_DEV), (dict(N=0, R=0), E_DEV), (dict(N=-1), E_SHAPE), (dict(K=0), E_SHAPE),
    (dict(K=33), E_SHAPE), (dict(n_local=0), E_SHAPE), (dict(n_local=1025), E_SHAPE),
    (dict(first_expert=-1), E_SHAPE), (dict(R=39), E_SHAPE), (dict(R=1 << 31), E_SHAPE),
    (dict(N=1 << 29, R=1 << 31), E_SHAPE), (dict(topk_expert=None), E_NULL),
    (dict(topk_weight=None), E_NULL), (dict(row_weight=None), E_NULL),
    (dict(topk_weight=None, row_weight=None), E_DEV), (dict(offsets=None), E_NULL),
    (dict(tok_ptr=None), E_NULL), (dict(tok_rows=None), E_NULL), (dict(slot_row=None), E_NULL),
    (dict(row_token=None), E_NULL), (dict(workspace=None), E_WS), (dict(ws_bytes=4), E_WS),
    (dict(workspace=addr(9, 4)), E_ALIGN), (dict(offsets=addr(3, 2)), E_ALIGN),
    (dict(tok_rows=addr(4, 4)), E_ALIAS), (dict(slot_row=addr(1)), E_ALIAS),
    (dict(workspace=addr(6)), E_ALIAS)])
def test_tables_arguments(kw, want):
    assert tables(**kw) == want


def test_tables_workspace_of_bad_shapes_is_zero():
    assert tp.tp_moe_route_tables_workspace(-1, 2, 8) == 0
    assert tp.tp_moe_route_tables_workspace(4, 99, 8) == 0


# --- AdamW -------------------------------------------------------------------
def ad(**kw):
    return {**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_dtype=tp.TP_F32,
                   state_bits=32, seed=0), **kw}


def tensor(k=0, off=0, bits=32, count=1000, **kw):
    t = dict(param=addr(8 * k + 1, off), grad=addr(8 * k + 2, off), m=addr(8 * k + 3, off),
             v=addr(8 * k + 4, off), param_bf16=addr(8 * k + 5, off), count=count)
    if bits == 8:
        t.update(m_scale=addr(8 * k + 6, off), v_scale=addr(8 * k + 7, off))
    return {**t, **kw}


def step(desc=None, tensors=None, **kw):
    return status(tp.tp_adamw_step, desc or ad(), [tensor()] if tensors is None else tensors, **kw)


@pytest.mark.parametrize("desc,want", [
    (ad(), E_DEV), (ad(grad_dtype=2), E_DTYPE), (ad(state_bits=16), E_DTYPE), (ad(lr=math.inf), E_SHAPE),
    (ad(beta1=1.0), E_SHAPE), (ad(beta1=-0.1), E_SHAPE), (ad(beta2=math.nan), E_SHAPE),
    (ad(beta1=0.0, beta2=0.0), E_DEV), (ad(eps=0.0), E_SHAPE), (ad(eps=1e-40), E_SHAPE),
    (ad(step=0), E_SHAPE)])
def test_adamw_descriptor(desc, want):
    assert step(desc) == want


def test_adamw_device_scalars():
    assert step(ad(step=0), dev_step=addr(90)) == E_DEV
    assert step(dev_lr=addr(90, 2)) == E_ALIGN
    assert step(grad_scale=addr(90, 4)) == E_DEV
    assert step(grad_scale=addr(1, 400)) == E_ALIAS    # inside param


@pytest.mark.parametrize("t,want", [
    (tensor(param=None), E_NULL), (tensor(grad=None), E_NULL), (tensor(m=None), E_NULL),
    (tensor(v=None), E_NULL), (tensor(param_bf16=None), E_DEV), (tensor(off=8), E_ALIGN),
    (tensor(count=-1), E_SHAPE), (tensor(count=(1 << 40) + 1), E_SHAPE),
    (tensor(count=0, param=None, grad=None, m=None, v=None), E_DEV),
    (tensor(weight_decay=math.nan), E_SHAPE), (tensor(bits=8), E_SHAPE),
    (tensor(m=addr(4)), E_ALIAS), (tensor(param_bf16=addr(1)), E_ALIAS)])
def test_adamw_tensor(t, want):
    assert step(tensors=[t]) == want
    assert step(tensors=[tensor(9), t]) == want


def test_adamw_many_tensors():
    assert step(tensors=[]) == E_DEV
    assert step(tensors=[tensor(k) for k in range(200)]) == E_DEV
    # in the list's order, out of order, and overlapping either way
    flat = [tensor(0, 4096 * k) for k in range(20)]
    assert step(tensors=flat) == E_DEV
    assert step(tensors=flat[::-1]) == E_DEV
    assert step(tensors=flat + [tensor(0, 4096 * 7)]) == E_ALIAS
    assert step(tensors=[tensor(0, 4096 * k, count=1025) for k in range(3)]) == E_ALIAS


def test_adamw_8bit_tensors():
    d = ad(state_bits=8)
    assert step(d, [tensor(bits=8)]) == E_DEV
    assert step(d, [tensor()]) == E_NULL                           # the scales
    assert step(d, [tensor(bits=8, m_scale=addr(6, 4))]) == E_DEV  # 4-byte aligned
    assert step(d, [tensor(bits=8, v_scale=addr(6, 12))]) == E_ALIAS   # 4 blocks: 16 bytes
    assert step(d, [tensor(bits=8, v_scale=addr(6, 16))]) == E_DEV


def test_adamw_reserved_field_and_null_table():
    L = tp.lib()
    tp.tp_adamw_step   # binds the argument types
    assert step() == E_DEV
    d = tp.tp_adamw_desc(**ad())
    assert L.tp_adamw_step(None, 0, None, None, None, None, None) == E_NULL
    assert L.tp_adamw_step(ctypes.byref(d), 1, None, None, None, None, None) == E_NULL
    assert L.tp_adamw_step(ctypes.byref(d), -1, None, None, None, None, None) == E_SHAPE
    assert L.tp_adamw_step(ctypes.byref(d), 65537, None, None, None, None, None) == E_SHAPE
    t = (tp.tp_adamw_tensor * 1)()
    t[0].reserved = 1
    assert L.tp_adamw_step(ctypes.byref(d), 1, t, None, None, None, None) == E_SHAPE


# --- the binding's own checks ------------------------------------------------
def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(12, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tp.tp_block_norm_fwd(nd(), **{**FWD, "X": x})
    with pytest.raises(ValueError):
        tp.tp_block_norm_fwd(nd(), **{**FWD, "stat_pre": torch.zeros(24, dtype=torch.float64)})
    with pytest.raises(ValueError):
        tp.tp_moe_route_fwd(rd(), addr(1), None, torch.zeros(40, dtype=torch.int64), addr(4))
    with pytest.raises(ValueError):
        tp.tp_adamw_tensors(ad(), [tensor(grad=torch.zeros(1000, dtype=torch.bfloat16))])
    with pytest.raises(ValueError):
        tp.tp_adamw_tensors(ad(state_bits=8), [tensor(bits=8, m=torch.zeros(1000))])
    table = tp.tp_adamw_tensors(ad(), [tensor()])
    with pytest.raises(ValueError):
        tp.tp_adamw_step(ad(state_bits=8), table)


def test_tensors_of_another_type_are_refused():
    torch = pytest.importorskip("torch")
    wide, slim = torch.zeros(12, 64), torch.zeros(12, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="X must be a torch.bfloat16"):
        tp.tp_block_norm_fwd(nd(), **{**FWD, "X": wide})
    with pytest.raises(ValueError, match="dHn must be a torch.float32"):
        tp.tp_block_norm_bwd(nd(dtype=tp.TP_F32), ws_bytes=1 << 20, **{**BWD, "dHn": slim})
    with pytest.raises(ValueError, match="logits must be a torch.float32"):
        tp.tp_moe_route_fwd(rd(dtype=tp.TP_F32), slim, None, addr(3), addr(4))
    with pytest.raises(ValueError, match="dlogits must be a torch.bfloat16"):
        tp.tp_moe_route_bwd(rd(dtype=tp.TP_BF16), addr(1), addr(2), addr(3), None, 0, wide)


def test_descriptors_take_their_fields_by_name():
    for desc in (dict(E=8, N=2, K=1, scales=2.0), dict(N=2, K=1, E=8, group=2)):
        with pytest.raises(TypeError, match="no field"):
            tp.tp_moe_route_fwd(desc, addr(1), None, addr(3), addr(4))
    with pytest.raises(TypeError, match="no field"):
        tp.tp_adamw_step(dict(lr=1e-3, beta3=0.9), [])
    from tensor_transformer_mlp_02_amd import block
    d = block._norm(dict(H=64, N=3, eps=0.5))   # whatever their order
    assert (d.N, d.H, d.eps, d.dtype, d.res_scale, d.gate_rows) == (3, 64, 0.5, tp.TP_BF16, 1.0, 0)
    assert block._norm(d) is d
