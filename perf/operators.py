"""The operators around the shard's and the experts' products, as workloads: the block norms with their
gate and residual scale, routing to experts with its dispatch tables, and the AdamW step.

A case is a dict of plain values; `prepare` makes what a training or serving program has in hand before
the call, `run` makes one pass: the plain form in elementary torch operations, or, with `own` set, the
framework's entry points.  `exact` is the same result from the definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_LOWEST = -3.3895313892515355e38  # the lowest finite bfloat16: a logit at or below it is masked out
_BLOCK = 256                      # elements that share one scale of an 8-bit state
_FMAX = 448.0                     # largest finite E4M3 value


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # one generated token's residual seam of the SwiGLU shard's width: latency only
        dict(name="norm_fwd_one_token", op="norm_fwd", N=1, H=8192, dtype="bf16", kind="rms", post=True, gate_rows=0,
             bias=False),
        # the SwiGLU shard's tokens: sandwich norm, a learned gate a channel, the next block's norm
        dict(name="norm_fwd_4096x8192", op="norm_fwd", N=4096, H=8192, dtype="bf16", kind="rms", post=True, gate_rows=1,
             bias=False),
        # the GeLU shard's tokens in training
        dict(name="norm_bwd_8192x4096", op="norm_bwd", N=8192, H=4096, dtype="bf16", kind="rms", post=True, gate_rows=1,
             bias=False),
        # fp32, LayerNorm with biases, an odd width, a gate for each of 3 sequences
        dict(name="norm_bwd_odd_f32", op="norm_bwd", N=999, H=1004, dtype="f32", kind="layer", post=True, gate_rows=3,
             bias=True),
        # a decode batch: few tokens over many experts in groups
        dict(name="route_fwd_8_tokens", op="route_fwd", N=8, E=256, K=8, score="sigmoid", bias=True, groups=8, kept=4,
             best=2, renorm=True, dtype="f32", first=0, local=32, masked=False),
        # the grouped experts' workload: top 2 of 64, 8 of them on this rank
        dict(name="route_fwd_16384_top2", op="route_fwd", N=16384, E=64, K=2, score="softmax", bias=False, groups=1,
             kept=1, best=1, renorm=False, dtype="f32", first=0, local=8, masked=False),
        # a training batch with a balance bias, groups, odd tokens and some experts masked
        dict(name="route_fwd_8191_groups", op="route_fwd", N=8191, E=256, K=8, score="sigmoid", bias=True, groups=8,
             kept=4, best=2, renorm=True, dtype="f32", first=64, local=64, masked=True),
        # their gradients: from the rows' weight gradients, as the combine's backward leaves them
        dict(name="route_bwd_16384_top2", op="route_bwd", N=16384, E=64, K=2, score="softmax", bias=False, groups=1,
             kept=1, best=1, renorm=False, dtype="f32", first=0, local=8, masked=False),
        dict(name="route_bwd_8191_renorm", op="route_bwd", N=8191, E=256, K=8, score="softmax", bias=False, groups=1,
             kept=1, best=1, renorm=True, dtype="bf16", first=0, local=256, masked=True),
        # many small tensors (norm weights, biases, a router): few launches count
        dict(name="adamw_small_tensors", op="adamw", shapes=",".join(["4096"] * 24 + ["1001"] * 8 + ["64x1004"] * 4 + ["1"]),
             bits=32, grad="f32", copy=True, step=1),
        # the SwiGLU shard's three weights
        dict(name="adamw_swiglu_shard", op="adamw", shapes="8192x3584,8192x3584,3584x8192", bits=32, grad="f32", copy=True,
             step=1000),
        # the grouped experts' weights and their norms, states in 8 bits
        dict(name="adamw_experts_8bit", op="adamw", shapes="8x4096x1408,8x4096x1408,8x1408x4096,4096,4096,64x1001", bits=8,
             grad="f32", copy=True, step=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "route_fwd", "route_bwd", "adamw"])
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        step = 8 if dtype == "bf16" else 4
        H = max(1, _log(rng, 64, 8192) // step) * step
        N = _log(rng, 1, max(2, (4096 * 8192 // (1 if dtype == "bf16" else 2)) // H))
        seqs = rng.choice([2, 3, 4])
        gate = rng.choice([0, 1, seqs, N])
        if gate == seqs:
            N = -(-N // seqs) * seqs
        return dict(op=op, N=N, H=H, dtype=dtype, kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.7,
                    gate_rows=gate, bias=rng.random() < 0.4)
    if op.startswith("route"):
        E, groups, kept = rng.choice([(8, 1, 1), (60, 1, 1), (64, 1, 1), (64, 8, 3), (128, 1, 1), (160, 8, 3), (256, 8, 4),
                                      (256, 1, 1), (384, 1, 1), (512, 16, 4)])
        K = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= kept * (E // groups)])
        N = _log(rng, 1, 16384 * 256 // E if E > 64 else 32768)
        local = rng.choice([E, max(1, E // 4), max(1, E // 8)]) if N > 64 else E
        return dict(op=op, N=N, E=E, K=K,
                    score=rng.choice(["softmax", "sigmoid"]), bias=op == "route_fwd" and rng.random() < 0.5, groups=groups,
                    kept=kept, best=rng.choice([1, 2]), renorm=K > 1 and rng.random() < 0.5, dtype=rng.choice(["f32", "f32", "bf16"]),
                    first=rng.randrange(0, E - local + 1), local=local, masked=rng.random() < 0.3)
    left, shapes = _log(rng, 1000, 80_000_000), []
    for _ in range(rng.randrange(1, 40)):
        n = min(left, _log(rng, 1, max(2, left)))
        if n < 1:
            break
        shapes.append(str(n))
        left -= n
    return dict(op=op, shapes=",".join(shapes), bits=rng.choice([8, 32]), grad=rng.choice(["f32", "f32", "bf16"]),
                copy=rng.random() < 0.7, step=_log(rng, 1, 100000))


def _counts(case):
    return [math.prod(int(d) for d in s.split("x")) for s in case["shapes"].split(",")]


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, e = case["N"] * case["H"], 2 if case["dtype"] == "bf16" else 4
        gate = case["gate_rows"] * case["H"]
        vec = case["H"] * ((2 if case["post"] else 1) * (2 if case["bias"] else 1))
        if op == "norm_fwd":
            return {"bytes": (4 * n + gate + vec) * e + 12 * case["N"], "flops": 14 * n}
        return {"bytes": (6 * n + gate + vec) * e + 4 * (gate + vec) + 12 * case["N"], "flops": 40 * n}
    if op.startswith("route"):
        N, E, K = case["N"], case["E"], case["K"]
        e = 2 if case["dtype"] == "bf16" else 4
        rows = N * K * case["local"] / E
        if op == "route_fwd":  # logits once; experts, weights, the slots' rows; the tables of the rows on this rank
            return {"bytes": N * E * e + 12 * N * K + 4 * N + 12 * rows + 4 * case["local"], "flops": N * E * (8 + K)}
        return {"bytes": 2 * N * E * e + 8 * N * K + 4 * rows, "flops": N * E * 10}
    n = sum(_counts(case))
    each = 8 + (4 if case["grad"] == "f32" else 2) + (2 if case["copy"] else 0) + (16 if case["bits"] == 32 else 4)
    return {"bytes": n * each, "flops": 16 * n}


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
_DEV = "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, device=_DEV, dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    op = case["op"]
    if op.startswith("norm"):
        return _prepare_norm(case, g)
    if op.startswith("route"):
        return _prepare_route(case, g)
    return _prepare_adamw(case, g, seed)


def _prepare_norm(case, g):
    N, H, dt = case["N"], case["H"], _TYPES[case["dtype"]]
    layer = case["kind"] == "layer"
    st = dict(case=case, desc=dict(N=N, H=H, gate_rows=case["gate_rows"], kind=int(layer), dtype=int(dt == torch.bfloat16),
                                   eps=1e-5, res_scale=1.0, branch_scale=0.5))
    # a residual stream has a few channels much larger than the rest
    wide = 1 + 15 * (torch.rand(H, device=_DEV, generator=g) < 0.01).float()
    X = _normal(g, N, H) * wide
    O = _normal(g, N, H, std=0.7)
    vec = lambda on: (1 + _normal(g, H, std=0.1)).to(dt) if on else None  # noqa: E731
    st["w_post"], st["w_pre"] = vec(case["post"]), vec(True)
    st["b_post"] = _normal(g, H, std=0.1, dtype=dt) if case["post"] and case["bias"] else None
    st["b_pre"] = _normal(g, H, std=0.1, dtype=dt) if case["bias"] else None
    st["gate"] = _normal(g, case["gate_rows"], H, std=0.5, dtype=dt) if case["gate_rows"] else None
    st["O"] = O.to(dt)
    new = lambda *s, d=dt: torch.empty(s, device=_DEV, dtype=d)  # noqa: E731
    stat = 2 * N if layer else N
    if case["op"] == "norm_fwd":
        st["X"] = X.to(dt)
        st["Y"], st["Hn"] = new(N, H), new(N, H)
        st["stat_post"] = new(stat, d=torch.float32) if case["post"] else None
        st["stat_pre"] = new(stat, d=torch.float32)
        return st
    # the backward has the forward's y and statistics, and the gradients from above
    y = X + 0.5 * O
    st["Y"] = y.to(dt)

    def stats(t):
        t = t.float()
        mean = t.mean(1) if layer else t.new_zeros(N)
        r = ((t - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
        return torch.cat([r, mean]) if layer else r

    st["stat_post"], st["stat_pre"] = stats(st["O"]) if case["post"] else None, stats(st["Y"])
    st["dY"], st["dHn"] = _normal(g, N, H, std=1e-2, dtype=dt), _normal(g, N, H, std=1e-2, dtype=dt)
    st["dX"], st["dO"] = new(N, H), new(N, H)
    f = torch.float32
    st["dw_post"] = new(H, d=f) if case["post"] else None
    st["db_post"] = new(H, d=f) if st["b_post"] is not None else None
    st["dgate"] = new(case["gate_rows"], H, d=f) if case["gate_rows"] else None
    st["dw_pre"] = new(H, d=f)
    st["db_pre"] = new(H, d=f) if case["bias"] else None
    return st


def _prepare_route(case, g):
    N, E, K, dt = case["N"], case["E"], case["K"], _TYPES[case["dtype"]]
    st = dict(case=case, desc=dict(N=N, E=E, K=K, groups=case["groups"], groups_kept=case["kept"], group_best=case["best"],
                                   score=int(case["score"] == "sigmoid"), renorm=int(case["renorm"]),
                                   dtype=int(dt == torch.bfloat16), scale=2.5 if case["renorm"] else 1.0))
    logits = _normal(g, N, E)
    if case["masked"]:  # experts that are switched off for some tokens, and tokens that are padding
        off = torch.rand(N, E, device=_DEV, generator=g) < 0.05
        off |= torch.rand(N, 1, device=_DEV, generator=g) < 0.02
        logits = logits.masked_fill(off, -math.inf)
    st["logits"] = logits.to(dt)
    st["bias"] = _normal(g, E, std=0.05) if case["bias"] else None
    i32 = lambda *s: torch.empty(s, device=_DEV, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: torch.empty(s, device=_DEV, dtype=torch.float32)  # noqa: E731
    if case["op"] == "route_fwd":
        R = N * K
        st.update(expert=i32(N, K), weight=f32(N, K), offsets=i32(case["local"] + 1), row_token=i32(R), row_weight=f32(R),
                  tok_ptr=i32(N + 1), tok_rows=i32(R), slot_row=i32(N, K))
        return st
    best, expert = st["logits"].float().topk(K, dim=1)
    expert = expert.masked_fill(best <= _LOWEST, -1)
    on = (expert >= case["first"]) & (expert < case["first"] + case["local"])
    rows = torch.randperm(N * K, device=_DEV, generator=g).view(N, K)
    st["R"] = N * K
    st["expert"] = expert.to(torch.int32)
    st["slot_row"] = rows.masked_fill(~on, -1).to(torch.int32)
    st["d_weight"] = _normal(g, N * K, std=1e-2)
    st["dlogits"] = torch.empty(N, E, device=_DEV, dtype=dt)
    return st


_KINDS = ("param", "param_bf16", "m", "v", "m_scale", "v_scale")


def _slices(case):
    """Where each tensor starts in the program's flat buffers (whole blocks apart), and their length."""
    at, starts = 0, []
    for n in _counts(case):
        starts.append(at)
        at += -(-n // _BLOCK) * _BLOCK
    return starts, at


def _prepare_adamw(case, g, seed):
    # parameters, gradients and states live in flat buffers, a tensor being a piece of each
    starts, total = _slices(case)
    st = dict(case=case, desc=dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=case["step"], seed=seed & 0xffffffff,
                                   grad_dtype=int(case["grad"] == "bf16"), state_bits=case["bits"]), tensors=[])
    st["grad_scale"] = torch.tensor(0.5, device=_DEV)  # the clip factor, computed on the device
    used = torch.zeros(total, device=_DEV)
    size = torch.ones(total, device=_DEV)
    for a, n in zip(starts, _counts(case)):
        used[a:a + n] = 1
        size[a:a + n] = 1e-3 * torch.rand(1, device=_DEV, generator=g)
    flat = dict(param=_normal(g, total, std=0.02) * used)
    grad = (_normal(g, total) * size * used).to(_TYPES[case["grad"]])
    m, r = _normal(g, total) * size * 0.3 * used, (_normal(g, total).abs() * 0.7 + 0.1) * size * used
    if case["step"] == 1:  # before the first step the states are zeros
        m, r = torch.zeros_like(m), torch.zeros_like(r)
    flat["param_bf16"] = flat["param"].to(torch.bfloat16) if case["copy"] else None
    if case["bits"] == 32:
        flat.update(m=m, v=r * r, m_scale=None, v_scale=None)
    else:
        for name, x in (("m", m), ("v", r)):
            b = x.view(-1, _BLOCK)
            scale = b.abs().amax(1) / _FMAX
            flat[name] = (b / scale.clamp_min(1e-38)[:, None]).to(torch.float8_e4m3fn).view(-1)
            flat[name + "_scale"] = scale
    st["flat"] = flat
    for a, n in zip(starts, _counts(case)):
        t = {k: None if flat[k] is None else flat[k][a // _BLOCK:-(-(a + n) // _BLOCK)] if k.endswith("scale")
             else flat[k][a:a + n] for k in _KINDS}
        st["tensors"].append(dict(t, grad=grad[a:a + n], weight_decay=0.1 if n > 5000 else 0.0))
    return st


# ---------------------------------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "norm_fwd":
        return _own_norm_fwd(state) if own else _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _own_norm_bwd(state) if own else _plain_norm_bwd(state)
    if op == "route_fwd":
        return _own_route_fwd(state) if own else _plain_route_fwd(state)
    if op == "route_bwd":
        return _own_route_bwd(state) if own else _plain_route_bwd(state)
    return _own_adamw(state) if own else _plain_adamw(state)


def _lib():
    import tensor_transformer_mlp_02_amd as tp
    return tp


def _workspace(st, size):
    """A scratch buffer that the program keeps from its first pass on."""
    if "workspace" not in st:
        st["ws_bytes"] = size(_lib())
        st["workspace"] = torch.empty(max(16, st["ws_bytes"]), dtype=torch.uint8, device=_DEV)
    return st["workspace"], st["ws_bytes"]


# --- block norms -------------------------------------------------------------------------------------
def _norm(t, layer, w, b, eps):
    mean = t.mean(1, keepdim=True) if layer else torch.zeros_like(t[:, :1])
    c = t - mean if layer else t
    r = torch.rsqrt(c.square().mean(1, keepdim=True) + eps)
    n = c * r * w.float()
    stat = torch.cat([r.view(-1), mean.view(-1)]) if layer else r.view(-1)
    return (n + b.float() if b is not None else n), stat


def _gate_rows(st):
    """The gate's row for each token, as a view or a gather."""
    d, gate = st["desc"], st["gate"].float()
    if d["gate_rows"] in (1, d["N"]):
        return gate
    return gate.repeat(-(-d["N"] // d["gate_rows"]), 1)[:d["N"]]


def _plain_norm_fwd(st):
    d, layer = st["desc"], st["desc"]["kind"] == 1
    u, stat_post = st["O"].float(), None
    if st["w_post"] is not None:
        u, stat_post = _norm(u, layer, st["w_post"], st["b_post"], d["eps"])
    if st["gate"] is not None:
        u = u * _gate_rows(st)
    y = st["X"].float() * d["res_scale"] + u * d["branch_scale"]
    h, stat_pre = _norm(y, layer, st["w_pre"], st["b_pre"], d["eps"])
    dt = st["X"].dtype
    return dict(Y=y.to(dt), Hn=h.to(dt), stat_post=stat_post, stat_pre=stat_pre)


def _own_norm_fwd(st):
    _lib().tp_block_norm_fwd(st["desc"], st["X"], st["O"], st["w_post"], st["b_post"], st["gate"], st["w_pre"],
                             st["b_pre"], st["Y"], st["Hn"], st["stat_post"], st["stat_pre"])
    return dict(Y=st["Y"], Hn=st["Hn"], stat_post=st["stat_post"], stat_pre=st["stat_pre"])


def _stats(stat, N, layer):
    return stat[:N, None], (stat[N:, None] if layer else 0.0)


def _plain_norm_bwd(st):
    d, layer = st["desc"], st["desc"]["kind"] == 1
    N, dt = d["N"], st["Y"].dtype
    out = {}
    # through the norm before the next block
    r, mean = _stats(st["stat_pre"], N, layer)
    xh = (st["Y"].float() - mean) * r if layer else st["Y"].float() * r
    dh = st["dHn"].float()
    out["dw_pre"] = (dh * xh).sum(0)
    if st["db_pre"] is not None:
        out["db_pre"] = dh.sum(0)
    p = dh * st["w_pre"].float()
    dt_y = p - xh * (p * xh).mean(1, keepdim=True)
    if layer:
        dt_y = dt_y - p.mean(1, keepdim=True)
    dyt = st["dY"].float() + r * dt_y
    out["dX"] = (dyt * d["res_scale"]).to(dt)
    # through the gate and the norm after the block
    o, post = st["O"].float(), st["w_post"] is not None
    if post:
        ro, mo = _stats(st["stat_post"], N, layer)
        oh = (o - mo) * ro if layer else o * ro
        u = oh * st["w_post"].float()
        if st["b_post"] is not None:
            u = u + st["b_post"].float()
    else:
        u = o
    du = dyt * d["branch_scale"]
    if st["gate"] is not None:
        G = d["gate_rows"]
        out["dgate"] = (du * u).view(N // G, G, -1).sum(0)
        du = du * _gate_rows(st)
    if post:
        out["dw_post"] = (du * oh).sum(0)
        if st["db_post"] is not None:
            out["db_post"] = du.sum(0)
        q = du * st["w_post"].float()
        do = q - oh * (q * oh).mean(1, keepdim=True)
        if layer:
            do = do - q.mean(1, keepdim=True)
        du = do * ro
    out["dO"] = du.to(dt)
    return out


def _own_norm_bwd(st):
    ws, nb = _workspace(st, lambda tp: tp.tp_block_norm_bwd_workspace(st["desc"]))
    names = ("dX", "dO", "dw_post", "db_post", "dgate", "dw_pre", "db_pre")
    _lib().tp_block_norm_bwd(st["desc"], st["dY"], st["dHn"], st["Y"], st["O"], st["w_post"], st["b_post"], st["gate"],
                             st["w_pre"], st["stat_post"], st["stat_pre"], *(st[n] for n in names), ws, nb)
    return {n: st[n] for n in names if st[n] is not None}


# --- routing -----------------------------------------------------------------------------------------
def _scores(logits, score, wide):
    """Scores of the experts and which of them are there; wide: in 64 bits, where choices hang on them."""
    l = logits.to(wide)
    there = l > _LOWEST
    l = l.clamp(max=3.4028234663852886e38)
    if score == 1:
        return torch.sigmoid(l).masked_fill(~there, 0.0), there
    l = l.masked_fill(~there, -math.inf)
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(there.any(1, keepdim=True), top, torch.zeros_like(top)))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300 if wide == torch.float64 else 1e-30), there


def _plain_route_fwd(st):
    case, d = st["case"], st["desc"]
    N, E, K = d["N"], d["E"], d["K"]
    s, there = _scores(st["logits"], d["score"], torch.float64)
    c = s if st["bias"] is None else s + st["bias"].double()
    c = c.masked_fill(~there, -math.inf)
    key = c if st["bias"] is not None else st["logits"].double().masked_fill(~there, -math.inf)
    G = d["groups"]
    if G > 1:
        best = c.view(N, G, E // G).topk(min(d["group_best"], E // G), dim=2).values
        best = torch.where(torch.isinf(best) & (torch.arange(best.shape[2], device=_DEV) > 0), torch.zeros_like(best), best)
        order = best.sum(2).sort(dim=1, descending=True, stable=True).indices[:, :d["groups_kept"]]
        keep = torch.zeros(N, G, dtype=torch.bool, device=_DEV).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    value, expert = key.sort(dim=1, descending=True, stable=True)
    value, expert = value[:, :K], expert[:, :K]
    w = s.gather(1, expert).masked_fill(value == -math.inf, 0.0)
    expert = expert.masked_fill(value == -math.inf, -1)
    if d["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = (w * d["scale"]).float()
    # the rows on this rank, ordered by (expert, token, slot)
    R, first, local = N * K, case["first"], case["local"]
    flat = expert.reshape(-1) - first
    on = (flat >= 0) & (flat < local)
    order = torch.where(on, flat, local).sort(stable=True).indices
    count = torch.bincount(torch.where(on, flat, local), minlength=local + 1)[:local]
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    at = torch.arange(R, device=_DEV)
    kept = at < offsets[-1]
    row_token = torch.where(kept, order // K, -1)
    row_weight = torch.where(kept, w.reshape(-1)[order], 0.0)
    slot_row = torch.empty(R, dtype=torch.int64, device=_DEV).scatter_(0, order, torch.where(kept, at, -1))
    # each token's rows, ascending
    tok_ptr = torch.cat([count.new_zeros(1), on.view(N, K).sum(1).cumsum(0)])
    tok_rows = torch.where(kept, torch.where(kept, row_token, N).sort(stable=True).indices, -1)
    i = torch.int32
    return dict(expert=expert.to(i), weight=w, offsets=offsets.to(i), row_token=row_token.to(i), row_weight=row_weight,
                tok_ptr=tok_ptr.to(i), tok_rows=tok_rows.to(i), slot_row=slot_row.view(N, K).to(i))


def _own_route_fwd(st):
    tp, case, d = _lib(), st["case"], st["desc"]
    N, K = d["N"], d["K"]
    ws, nb = _workspace(st, lambda tp: tp.tp_moe_route_tables_workspace(N, K, case["local"]))
    tp.tp_moe_route_fwd(d, st["logits"], st["bias"], st["expert"], st["weight"])
    tp.tp_moe_route_tables(N, K, case["first"], case["local"], N * K, st["expert"], st["weight"], st["offsets"],
                           st["row_token"], st["row_weight"], st["tok_ptr"], st["tok_rows"], st["slot_row"], ws, nb)
    return {n: st[n] for n in ("expert", "weight", "offsets", "row_token", "row_weight", "tok_ptr", "tok_rows", "slot_row")}


def _plain_route_bwd(st):
    d = st["desc"]
    s, there = _scores(st["logits"], d["score"], torch.float32)
    expert, rows = st["expert"].long(), st["slot_row"].long()
    t = st["d_weight"][rows.clamp_min(0)].masked_fill(rows < 0, 0.0) * d["scale"]
    on = expert >= 0
    chosen = s.gather(1, expert.clamp_min(0)).masked_fill(~on, 0.0)
    if d["renorm"]:
        total = chosen.sum(1, keepdim=True) + 1e-20
        t = (t - (t * chosen / total).sum(1, keepdim=True)) / total
    t = t.masked_fill(~on, 0.0)
    ds = torch.zeros_like(s).scatter_add_(1, expert.clamp_min(0), t)
    if d["score"] == 1:
        dl = s * (1 - s) * ds
    else:
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _own_route_bwd(st):
    _lib().tp_moe_route_bwd(st["desc"], st["logits"], st["expert"], st["d_weight"], st["slot_row"], st["R"], st["dlogits"])
    return st["dlogits"]


# --- AdamW -------------------------------------------------------------------------------------------
def _mix(x):
    """32 bits in 64-bit integers, mixed: two multiplications by the fractions of sqrt 2 and sqrt 3."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xffffffff
    return x ^ (x >> 16)


def _random(seed, step, k, n):
    """Two fractions in [0, 1) of 16 bits for each of n elements of tensor k."""
    key = _mix((_mix((_mix(seed) + step) & 0xffffffff) + k) & 0xffffffff)
    i = torch.arange(n, device=_DEV)
    h = _mix(((i & 0xffffffff) ^ key) + (i >> 32) & 0xffffffff)
    return (h & 0xffff).float() / 65536, (h >> 16).float() / 65536


def _power_of_two(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _to_8bit(x, u, root):
    """E4M3 values and block scales of x: rounded down or up by chance u, x (a root: its square) unbiased."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % _BLOCK)).view(-1, _BLOCK)
    top = b.abs().amax(1)
    # divisions in 64 bits, rounded once: correctly rounded, whatever the type's own division does
    some = top > 2.0 ** -100
    scale = torch.where(some, (top.double() / _FMAX).float(), 0.0)
    inv = torch.where(some, (_FMAX / top.double().clamp_min(1e-300)).float(), 0.0)
    t = (b * inv[:, None]).view(-1)[:n]
    e = torch.frexp(t.abs()).exponent.clamp_min(-5) - 4  # the step between E4M3 values is 2^e
    t = t * _power_of_two(-e)
    if root:
        k = torch.floor(t)
        odd = 2 * k + 1  # up with the chance (t^2 - k^2) / ((k + 1)^2 - k^2)
        k = k + ((t - k) * (t + k) + u * odd >= odd)
        k = torch.where(x > 0, k.clamp_min(1.0), k)  # a positive root stays positive
    else:
        k = torch.floor(t + u)
    return (k * _power_of_two(e)).clamp(-_FMAX, _FMAX).to(torch.float8_e4m3fn), scale


def _plain_adamw(st):
    d, gs, ts = st["desc"], st["grad_scale"], st["tensors"]
    b1, b2, lr, eps = d["beta1"], d["beta2"], d["lr"], d["eps"]
    c1, c2 = 1 - b1 ** d["step"], 1 - b2 ** d["step"]
    p = [t["param"] for t in ts]
    if d["state_bits"] == 32:
        g = torch._foreach_mul([t["grad"].float() for t in ts], gs)
        m, v = [t["m"] for t in ts], [t["v"] for t in ts]
        torch._foreach_mul_(m, b1)
        torch._foreach_add_(m, torch._foreach_mul(g, 1 - b1))
        torch._foreach_mul_(v, b2)
        torch._foreach_mul_(g, g)
        torch._foreach_add_(v, torch._foreach_mul(g, 1 - b2))
        root = torch._foreach_sqrt(v)
    else:
        m, root = [], []
        for k, t in enumerate(ts):
            n = t["param"].numel()
            g = t["grad"].float() * gs
            old = [t[a].float() * t[a + "_scale"].repeat_interleave(_BLOCK)[:n] for a in ("m", "v")]
            m.append(old[0] * b1 + g * (1 - b1))
            root.append((old[1] * old[1] * b2 + g * g * (1 - b2)).double().sqrt().float())
            u = _random(d["seed"], d["step"], k, n)
            for a, x, c in (("m", m[-1], u[0]), ("v", root[-1], u[1])):
                code, scale = _to_8bit(x, c, a == "v")
                t[a].copy_(code)
                t[a + "_scale"].copy_(scale)
    torch._foreach_mul_(p, [1 - lr * t["weight_decay"] for t in ts])
    torch._foreach_div_(root, math.sqrt(c2))
    torch._foreach_add_(root, eps)
    step = torch._foreach_div(m, root)
    torch._foreach_mul_(step, lr / c1)
    torch._foreach_sub_(p, step)
    if ts[0]["param_bf16"] is not None:
        torch._foreach_copy_([t["param_bf16"] for t in ts], p)
    return st["flat"]


def _own_adamw(st):
    tp = _lib()
    if "table" not in st:
        st["table"] = tp.tp_adamw_tensors(st["desc"], st["tensors"])  # laid out once, as a program keeps it
    tp.tp_adamw_step(st["desc"], st["table"], grad_scale=st["grad_scale"])
    return st["flat"]


# ---------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        return _exact_norm_fwd(st)
    if op == "norm_bwd":
        return _exact_norm_bwd(st)
    if op == "route_fwd":
        return _exact_route_fwd(st)
    if op == "route_bwd":
        return _exact_route_bwd(st)
    return _exact_adamw(st)


def _exact_graph(st, leaves):
    """y, h and the statistics as a graph in 64 bits over `leaves` (X, O and the weights)."""
    d = st["desc"]
    L = {k: None if v is None else v.double() for k, v in leaves.items()}

    def norm(t, w, b):
        mean = t.sum(1, keepdim=True) / d["H"] if d["kind"] == 1 else t.new_zeros(t.shape[0], 1)
        var = ((t - mean) ** 2).sum(1, keepdim=True) / d["H"]
        r = 1 / (var + d["eps"]).sqrt()
        n = (t - mean) * r * w
        return (n if b is None else n + b), (torch.cat([r, mean]) if d["kind"] == 1 else r).reshape(-1)

    u, stat_post = L["O"], None
    if L["w_post"] is not None:
        u, stat_post = norm(u, L["w_post"], L["b_post"])
    if L["gate"] is not None:
        u = u * L["gate"][torch.arange(d["N"], device=u.device) % d["gate_rows"]]
    y = d["res_scale"] * L["X"] + d["branch_scale"] * u
    return y, norm, stat_post, L


def _exact_norm_fwd(st):
    y, norm, stat_post, L = _exact_graph(st, {k: st[k] for k in ("X", "O", "w_post", "b_post", "gate", "w_pre", "b_pre")})
    h, stat_pre = norm(y, L["w_pre"], L["b_pre"])
    return dict(Y=y, Hn=h, stat_post=stat_post, stat_pre=stat_pre)


def _exact_norm_bwd(st):
    """Term by term from the stored y, O and statistics; a row's mean and 1/std are constants of the call."""
    d = st["desc"]
    N, H, layer = d["N"], d["H"], d["kind"] == 1
    w64 = lambda n: None if st[n] is None else st[n].to(torch.float64)  # noqa: E731

    def back(grad_out, x, stat, w):
        r = stat[:N].reshape(N, 1)
        hat = (x - (stat[N:].reshape(N, 1) if layer else 0)) * r
        gw = grad_out * w
        along = torch.einsum("nh,nh->n", gw, hat)[:, None] / H
        flat = gw.sum(1, keepdim=True) / H if layer else 0
        return (gw - hat * along - flat) * r, hat

    out = {}
    dh, y, o = w64("dHn"), w64("Y"), w64("O")
    through, hat = back(dh, y, w64("stat_pre"), w64("w_pre"))
    out["dw_pre"] = torch.einsum("nh,nh->h", dh, hat)
    if st["db_pre"] is not None:
        out["db_pre"] = dh.sum(0)
    total = w64("dY") + through
    del through, hat, dh, y
    out["dX"] = total * d["res_scale"]
    total = total * d["branch_scale"]
    rows = torch.arange(N, device=total.device) % max(1, d["gate_rows"])
    gate = w64("gate")
    du = total if gate is None else total * gate[rows]
    u = o
    if st["w_post"] is not None:
        out["dO"], hat = back(du, o, w64("stat_post"), w64("w_post"))
        out["dw_post"] = torch.einsum("nh,nh->h", du, hat)
        u = hat * w64("w_post")
        if st["b_post"] is not None:
            out["db_post"] = du.sum(0)
            u = u + w64("b_post")
    else:
        out["dO"] = du
    if gate is not None:
        out["dgate"] = torch.zeros_like(gate).index_add_(0, rows, total * u)
    return out


def _exact_route_fwd(st):
    """The weights of the chosen experts, by repeated search of the largest; whole numbers have no such value."""
    d = st["desc"]
    N, E = d["N"], d["E"]
    l = st["logits"].double()
    off = l <= _LOWEST
    if d["score"] == 1:
        s = 1 / (1 + torch.exp(-l))
    else:
        z = torch.where(off, torch.full_like(l, -1e9), l)
        z = torch.exp(z - z.max(1, keepdim=True)[0])
        s = z / z.sum(1, keepdim=True)
    s = torch.where(off, torch.zeros_like(s), s)
    c = s + (0 if st["bias"] is None else st["bias"].double())
    c = torch.where(off, torch.full_like(c, -1e6), c)  # no choice score comes near this
    per = E // d["groups"]
    if d["groups"] > 1:
        a = c.reshape(N, d["groups"], per)
        a = torch.sort(a, dim=2)[0].flip(2)[:, :, :min(d["group_best"], per)]
        lead, more = a[:, :, 0], a[:, :, 1:]
        worth = lead + torch.where(more > -1e5, more, torch.zeros_like(more)).sum(2)
        for _ in range(d["groups_kept"]):
            g = worth.argmax(1, keepdim=True)
            worth.scatter_(1, g, -1e9)
        c = torch.where((worth > -5e8).repeat_interleave(per, 1), torch.full_like(c, -1e6), c)
    picks = []
    for _ in range(d["K"]):
        top, e = c.max(1, keepdim=True)
        picks.append(torch.where(top > -1e5, s.gather(1, e), torch.zeros_like(top)))
        c = c.scatter(1, e, -1e6)
    w = torch.cat(picks, 1)
    if d["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    none = ("expert", "offsets", "row_token", "row_weight", "tok_ptr", "tok_rows", "slot_row")
    return dict(weight=w * d["scale"], **{n: None for n in none})


def _exact_route_bwd(st):
    """Differences of the definition, as torch derives them in 64 bits on the whole graph."""
    d = st["desc"]
    rows, expert = st["slot_row"].long(), st["expert"].long()
    up = torch.where(rows >= 0, st["d_weight"].double()[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64, device=_DEV))
    l = st["logits"].double()
    off = l <= _LOWEST
    l = torch.where(off, torch.zeros_like(l), l).requires_grad_(True)
    on = (~off).double()
    if d["score"] == 1:
        s = on / (1 + torch.exp(-l))
    else:
        z = torch.exp(l - l.detach().max(1, keepdim=True)[0]) * on
        s = z / (z.sum(1, keepdim=True) + (on.sum(1, keepdim=True) == 0))
    w = s.gather(1, expert.clamp(min=0)) * (expert >= 0)
    if d["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    (w * up * d["scale"]).sum().backward()
    return l.grad


def _exact_adamw(st):
    d, flat = st["desc"], st["flat"]
    wide = {k: torch.zeros(flat["param"].numel(), dtype=torch.float64, device=_DEV) for k in ("param", "m", "v")}
    g0 = float(st["grad_scale"])
    starts, _ = _slices(st["case"])
    for a, t in zip(starts, st["tensors"]):
        n = t["param"].numel()
        g = t["grad"].double() * g0
        if d["state_bits"] == 32:
            m, v = t["m"].double(), t["v"].double()
        else:
            whole = lambda k: t[k].double() * t[k + "_scale"].double().repeat_interleave(_BLOCK)[:n]  # noqa: E731
            m, v = whole("m"), whole("v") ** 2
        m = d["beta1"] * m + (1 - d["beta1"]) * g
        v = d["beta2"] * v + (1 - d["beta2"]) * g ** 2
        hat = (m / (1 - d["beta1"] ** d["step"])) / ((v / (1 - d["beta2"] ** d["step"])) ** 0.5 + d["eps"])
        p = t["param"].double()
        wide["param"][a:a + n] = p - d["lr"] * (hat + t["weight_decay"] * p)
        wide["m"][a:a + n], wide["v"][a:a + n] = m, v
    full = d["state_bits"] == 32  # an 8-bit state is rounded by chance: no value in 64 bits stands for it
    return dict(param=wide["param"], param_bf16=None if flat["param_bf16"] is None else wide["param"],
                m=wide["m"] if full else None, v=wide["v"] if full else None, m_scale=None, v_scale=None)
