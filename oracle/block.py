"""The operators around the products, in 64-bit numpy (test infrastructure).

Plain definitions, one step at a time, sharing no code with the library.  The
norm functions also return, for each output, the sum of the magnitudes of the
terms it is made of: what a rounding error of fp32 arithmetic is relative to.
"""
from __future__ import annotations

import numpy as np

f64 = np.float64


def _zero(x, like):
    return np.zeros_like(like) if x is None else x


def norm(t, layer, w, b, eps, mag=None):
    """((t - mu) r) w + b by rows -> (result, r, mu, magnitudes); mag: those of t."""
    mag = np.abs(t) if mag is None else mag
    mu = t.mean(1, keepdims=True) if layer else np.zeros((t.shape[0], 1))
    r = 1.0 / np.sqrt(((t - mu) ** 2).mean(1, keepdims=True) + eps)
    out = (t - mu) * r * w
    # an error of t reaches r through the variance
    spread = 1.0 + r * np.sqrt((mag ** 2).mean(1, keepdims=True))
    m = (mag + np.abs(mu)) * r * np.abs(w) + np.abs(out) * spread
    if b is not None:
        out, m = out + b, m + np.abs(b)
    return out, r[:, 0], mu[:, 0], m


def norm_fwd(X, O, w_post, b_post, gate, w_pre, b_pre, *, layer, eps, a, b):
    """-> dict of Y, Hn, r and mu of both norms, and the magnitudes of Y and Hn."""
    out = {}
    y, my = X, np.abs(X)
    if O is not None:
        u, mu_ = O, np.abs(O)
        if w_post is not None:
            u, out["r_post"], out["mu_post"], mu_ = norm(O, layer, w_post, b_post, eps)
        if gate is not None:
            g = gate[np.arange(X.shape[0]) % gate.shape[0]]
            u, mu_ = g * u, np.abs(g) * mu_
        y, my = a * X + b * u, np.abs(a * X) + np.abs(b) * mu_
        out["Y"], out["mag_Y"] = y, my
    if w_pre is not None:
        out["Hn"], out["r_pre"], out["mu_pre"], out["mag_Hn"] = norm(y, layer, w_pre, b_pre, eps, my)
    return out


def norm_bwd(dY, dH, Y, O, w_post, b_post, gate, w_pre, r_post, mu_post, r_pre, mu_pre, *, layer,
             a, b):
    """-> dict of the gradients and their magnitudes ("mag_" + name)."""
    N = Y.shape[0] if Y is not None else O.shape[0]
    out = {}

    def put(name, value, mag):
        out[name], out["mag_" + name] = value, mag

    def back(p, mag_p, t, r, mu):
        """r (p - mean p - th mean(p th))"""
        th, mth = (t - mu) * r, (np.abs(t) + np.abs(mu)) * r
        m1 = (p * th).mean(1, keepdims=True)
        mm1 = (mag_p * mth).mean(1, keepdims=True)
        m2 = p.mean(1, keepdims=True) if layer else 0.0
        mm2 = mag_p.mean(1, keepdims=True) if layer else 0.0
        return r * (p - m2 - th * m1), r * (mag_p + mm2 + mth * mm1), th, mth

    col = lambda x: np.asarray(x, f64).reshape(N, 1)  # noqa: E731
    D = _zero(dY, dH if dH is not None else O).astype(f64)
    mD = np.abs(D)
    if w_pre is not None:
        p = dH * w_pre
        mu = col(mu_pre) if layer else 0.0
        e, me, yh, myh = back(p, np.abs(p), Y, col(r_pre), mu)
        put("dw_pre", (dH * yh).sum(0), (np.abs(dH) * myh).sum(0))
        put("db_pre", dH.sum(0), np.abs(dH).sum(0))
        D, mD = D + e, mD + me
    if O is None:
        put("dX", D, mD)
        return out
    put("dX", a * D, np.abs(a) * mD)
    du, mdu = b * D, np.abs(b) * mD
    mu = col(mu_post) if layer and w_post is not None else 0.0
    if w_post is not None:
        oh, moh = (O - mu) * col(r_post), (np.abs(O) + np.abs(mu)) * col(r_post)
        u, mu_ = oh * w_post + _zero(b_post, w_post), moh * np.abs(w_post) + np.abs(_zero(b_post, w_post))
    else:
        u, mu_ = O, np.abs(O)
    if gate is not None:
        rows = np.arange(N) % gate.shape[0]
        dg, mdg = np.zeros(gate.shape), np.zeros(gate.shape)
        np.add.at(dg, rows, du * u)
        np.add.at(mdg, rows, mdu * mu_)
        put("dgate", dg, mdg)
        du, mdu = du * gate[rows], mdu * np.abs(gate[rows])
    if w_post is not None:
        put("dw_post", (du * oh).sum(0), (mdu * moh).sum(0))
        put("db_post", du.sum(0), mdu.sum(0))
        q, mq = du * w_post, mdu * np.abs(w_post)
        du, mdu, _, _ = back(q, mq, O, col(r_post), mu)
    put("dO", du, mdu)
    return out


# ---------------------------------------------------------------------------
LOWEST = -3.3895313892515355e38  # of finite bf16


def scores(logits, sigmoid):
    """-> (scores, which experts are there)"""
    l = np.asarray(logits, f64)
    there = l > LOWEST  # False for NaN
    l = np.minimum(np.where(there, l, 0.0), np.finfo(np.float32).max)
    with np.errstate(over="ignore"):
        if sigmoid:
            return np.where(there, 1.0 / (1.0 + np.exp(-l)), 0.0), there
        top = np.max(np.where(there, l, -np.inf), axis=1, keepdims=True, initial=-np.inf)
        e = np.where(there, np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0), there


def route_fwd(logits, bias, K, groups=1, kept=1, best=1, sigmoid=False, renorm=False, scale=1.0):
    """Token by token -> (expert [N,K] int32, weight [N,K] float64)."""
    s, there = scores(logits, sigmoid)
    N, E = s.shape
    expert, weight = np.full((N, K), -1, np.int32), np.zeros((N, K))
    per = E // groups
    for t in range(N):
        c = s[t] + (0.0 if bias is None else np.asarray(bias, f64))
        order = c if bias is not None else np.asarray(logits[t], f64)
        alive = [e for e in range(E) if there[t, e]]
        if groups > 1:
            worth = []
            for g in range(groups):
                top = sorted((c[e] for e in range(g * per, (g + 1) * per) if there[t, e]),
                             reverse=True)[:best]
                worth.append(sum(top) if top else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-worth[g], g))[:kept]
            alive = [e for e in alive if e // per in keep]
        chosen = sorted(alive, key=lambda e: (-order[e], e))[:K]
        total = sum(s[t, e] for e in chosen) + 1e-20
        for j, e in enumerate(chosen):
            expert[t, j] = e
            weight[t, j] = scale * (s[t, e] / total if renorm else s[t, e])
    return expert, weight


def route_bwd(logits, expert, d_weight, sigmoid=False, renorm=False, scale=1.0):
    """dlogits from the gradient of the weights [N,K] (0 for a slot without one)."""
    s, there = scores(logits, sigmoid)
    N, E = s.shape
    out = np.zeros((N, E))
    e = np.where(there, np.exp(-np.abs(np.where(there, np.asarray(logits, f64), 0.0))), 0.0)
    slope = e / (1 + e) ** 2  # s (1 - s) of a sigmoid, without 1 - s
    for t in range(N):
        on = [j for j in range(expert.shape[1]) if 0 <= expert[t, j] < E]
        total = sum(s[t, expert[t, j]] for j in on) + 1e-20
        up = {j: scale * float(d_weight[t, j]) for j in on}
        if renorm and on:  # up_j - sum_i up_i s_i / total, the largest score's up taken out of both
            k = up[max(on, key=lambda j: s[t, expert[t, j]])]
            mean = sum((up[j] - k) * s[t, expert[t, j]] for j in on) / total
            up = {j: ((up[j] - k) - mean + k * (1e-20 / total)) / total for j in on}
        ds = np.zeros(E)
        for j in on:
            ds[expert[t, j]] += up[j]
        if sigmoid:
            out[t] = slope[t] * ds
        else:  # ds - sum ds s, the largest score's ds taken out of both: nothing cancels where it is nearly 1
            ds = ds - ds[s[t].argmax()]
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


def route_tables(expert, weight, first, n_local, R):
    """The dispatch tables, pair by pair."""
    N, K = expert.shape
    rows = sorted((int(expert[t, j]) - first, t, j) for t in range(N) for j in range(K)
                  if first <= int(expert[t, j]) < first + n_local)
    offsets = np.zeros(n_local + 1, np.int32)
    row_token, tok_rows = np.full(R, -1, np.int32), np.full(R, -1, np.int32)
    row_weight, slot_row = np.zeros(R, np.float32), np.full((N, K), -1, np.int32)
    lists = [[] for _ in range(N)]
    for r, (e, t, j) in enumerate(rows):
        offsets[e + 1:] += 1
        row_token[r], slot_row[t, j] = t, r
        row_weight[r] = 0.0 if weight is None else weight[t, j]
        lists[t].append(r)
    tok_ptr = np.cumsum([0] + [len(x) for x in lists]).astype(np.int32)
    tok_rows[:len(rows)] = [r for x in lists for r in x]
    return dict(offsets=offsets, row_token=row_token, row_weight=row_weight, tok_ptr=tok_ptr,
                tok_rows=tok_rows, slot_row=slot_row)


# ---------------------------------------------------------------------------
BLOCK, FMAX = 256, 448.0


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, step, wd):
    """-> (p, m, v) after the step"""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = m / (1 - beta1 ** step) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * wd * p - lr * hat, m, v


def e4m3(codes):
    """Values of E4M3 codes (OCP: no infinities, 0x7f / 0xff NaN)."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    sign, e, f = np.where(c >> 7, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where((c & 127) == 127, np.nan, sign * v)


def e4m3_neighbours(x):
    """The E4M3 values just below and just above each x of magnitude at most 448."""
    values = np.unique(e4m3([c for c in range(256) if c & 127 != 127]))
    i = np.clip(np.searchsorted(values, x, side="right") - 1, 0, len(values) - 1)
    lo = values[i]
    return lo, np.where(lo == x, lo, values[np.minimum(i + 1, len(values) - 1)])


def widen(codes, scales):
    """A state of 8 bits as fp64: code * its block's scale."""
    n = len(codes)
    return e4m3(codes) * np.repeat(np.asarray(scales, f64), BLOCK)[:n]


def _mix(x):
    x = np.asarray(x, np.uint64)
    M = np.uint64(0xffffffff)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & M
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & M
    return x ^ (x >> np.uint64(16))


def chances(seed, step, place, n, start=0):
    """The two chances in [0, 1) of elements start .. start+n-1 of tensor `place`."""
    M = np.uint64(0xffffffff)
    key = _mix((_mix((_mix(seed) + np.uint64(step)) & M) + np.uint64(place)) & M)
    i = np.arange(start, start + n, dtype=np.uint64)
    h = _mix((((i & M) ^ key) + (i >> np.uint64(32))) & M)
    return (h & np.uint64(0xffff)).astype(f64) / 65536, (h >> np.uint64(16)).astype(f64) / 65536
