"""Plain statements in 64 bits of linear attention with a decay for each head (forward, gradients,
decode step) and of the group norm with an activation.  TEST INFRASTRUCTURE ONLY, like the rest of
this package; numpy, token by token."""
from __future__ import annotations

import numpy as np


def _decays(g, batch, L, H):
    """(a, starts anew) as [batch, L, H]."""
    g = np.broadcast_to(np.asarray(g, np.float64), (batch, L, H))
    start = g * np.log2(np.e) < -150.0
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(start, 0.0, np.exp(np.where(start, 0.0, g))), start


def _kept(a, start, S):
    with np.errstate(invalid="ignore"):
        return np.where(start[..., None, None], 0.0, a[..., None, None] * S)


def _heads(t, H):
    """[..., Hk, width] with each head's own row."""
    return np.repeat(np.asarray(t, np.float64), H // t.shape[-2], axis=-2)


def linear_fwd(q, k, v, g, scale=1.0, S0=None):
    """(o [B, L, H, V], last state [B, H, K, V])."""
    B, L, H, V = v.shape
    q, k, v = _heads(q, H), _heads(k, H), np.asarray(v, np.float64)
    a, start = _decays(g, B, L, H)
    S = np.zeros((B, H, q.shape[-1], V)) if S0 is None else np.asarray(S0, np.float64)
    o = np.empty(v.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(L):
            S = _kept(a[:, t], start[:, t], S) + k[:, t, :, :, None] * v[:, t, :, None, :]
            o[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
    return o, S


def linear_bwd(q, k, v, g, do, scale=1.0, S0=None, dlast=None):
    """Gradients; dlog_decay as [B, L, H] whatever the shape of g."""
    B, L, H, V = v.shape
    Hk, K = q.shape[-2:]
    qh, kh, v, do = _heads(q, H), _heads(k, H), np.asarray(v, np.float64), np.asarray(do, np.float64)
    a, start = _decays(g, B, L, H)
    S = np.zeros((B, H, K, V)) if S0 is None else np.asarray(S0, np.float64)
    states = [S]
    for t in range(L):
        S = _kept(a[:, t], start[:, t], S) + kh[:, t, :, :, None] * v[:, t, :, None, :]
        states.append(S)
    R = np.zeros((B, H, K, V)) if dlast is None else np.asarray(dlast, np.float64)
    dq, dk, dv, dg = np.empty((B, L, H, K)), np.empty((B, L, H, K)), np.empty(v.shape), np.empty((B, L, H))
    for t in range(L - 1, -1, -1):
        R = R + scale * qh[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * (states[t + 1] * do[:, t, :, None, :]).sum(-1)
        dk[:, t] = (R * v[:, t, :, None, :]).sum(-1)
        dv[:, t] = (R * kh[:, t, :, :, None]).sum(-2)
        dg[:, t] = (R * _kept(a[:, t], start[:, t], states[t])).sum((-1, -2))
        R = _kept(a[:, t], start[:, t], R)
    share = lambda d: d.reshape(B, L, Hk, H // Hk, K).sum(3)                          # noqa: E731
    return dict(dq=share(dq), dk=share(dk), dv=dv, dlog_decay=dg, dinitial_state=R)


def linear_decay_parts(q, k, v, g, do, scale=1.0, S0=None, dlast=None, chunk=64):
    """dlog_decay [B, L, H] by chunks, what passes a token's decay: "pairs" of its chunk that lie on both sides of it;
    sums over "x" [B, L, H] from it on, of the state S before the chunk with the chunk's tokens; sums over "y" before it,
    of the chunk's tokens with the gradient R behind the chunk; "through" [B, chunks, H], S with R.  Also
    "starts", whether any token of a chunk starts anew, "log2" of its decay and "least" of its tokens'; "beside", <S, R> behind
    each chunk."""
    B, L, H, V = v.shape
    qh, kh, v, do = _heads(q, H), _heads(k, H), np.asarray(v, np.float64), np.asarray(do, np.float64)
    a, start = _decays(g, B, L, H)
    K, n = qh.shape[-1], -(-L // chunk)
    S = np.zeros((B, H, K, V)) if S0 is None else np.asarray(S0, np.float64)
    R = np.zeros((B, H, K, V)) if dlast is None else np.asarray(dlast, np.float64)
    at_start, at_end = [], [None] * n
    for t in range(L):
        if t % chunk == 0:
            at_start.append(S)
        S = _kept(a[:, t], start[:, t], S) + kh[:, t, :, :, None] * v[:, t, :, None, :]
    at_start.append(S)
    for t in range(L - 1, -1, -1):
        if t == L - 1 or (t + 1) % chunk == 0:
            at_end[t // chunk] = R
        R = _kept(a[:, t], start[:, t], R + scale * qh[:, t, :, :, None] * do[:, t, :, None, :])
    out = {k: np.zeros((B, L, H)) for k in ("pairs", "x", "y")}
    out.update({k: np.zeros((B, n, H)) for k in ("through", "log2", "least", "beside")}, starts=np.zeros((B, n, H), bool))
    for c in range(n):
        r = slice(c * chunk, min(L, (c + 1) * chunk))
        m = r.stop - r.start
        begins = start[:, r].cumsum(1)                        # how often it has begun, per token
        with np.errstate(divide="ignore"):
            log = np.where(start[:, r], 0.0, np.log(np.where(start[:, r], 1.0, a[:, r]))).cumsum(1)
        P = np.exp(np.minimum(log[:, :, None] - log[:, None], 700.0)) * (begins[:, :, None] == begins[:, None])
        P *= np.tril(np.ones((m, m)))[None, :, :, None]
        f = np.exp(log) * (begins == 0)
        w = np.exp(log[:, -1:] - log) * (begins == begins[:, -1:])
        M = scale * P * np.einsum("bihk,bjhk->bijh", qh[:, r], kh[:, r]) * np.einsum("bihv,bjhv->bijh", do[:, r], v[:, r])
        for t in range(m):
            out["pairs"][:, r.start + t] = M[:, t:, :t].sum((1, 2))
        out["x"][:, r] = scale * f * np.einsum("bihk,bhkv,bihv->bih", qh[:, r], at_start[c], do[:, r])
        out["y"][:, r] = w * np.einsum("bjhk,bhkv,bjhv->bjh", kh[:, r], at_end[c], v[:, r])
        out["starts"][:, c] = start[:, r].any(1)
        out["log2"][:, c] = log[:, -1] * np.log2(np.e)
        with np.errstate(divide="ignore"):
            out["least"][:, c] = np.log2(np.where(start[:, r], 1.0, a[:, r])).min(1)
        out["through"][:, c] = np.where(out["starts"][:, c], 0.0, np.exp(log[:, -1]) * (at_start[c] * at_end[c]).sum((-1, -2)))
        out["beside"][:, c] = (at_start[c + 1] * at_end[c]).sum((-1, -2))
    total = np.array(out["pairs"])
    for c in range(n):
        r = slice(c * chunk, min(L, (c + 1) * chunk))
        x, y = out["x"][:, r], out["y"][:, r]
        total[:, r] += x[:, ::-1].cumsum(1)[:, ::-1] + out["through"][:, c:c + 1]
        total[:, r.start + 1:r.stop] += y[:, :-1].cumsum(1)
    out["dlog_decay"] = np.where(start, 0.0, total)
    return out


def linear_step(q, k, v, g, S, scale=1.0):
    """One token from states S [B, H, K, V]: (o [B, H, V], new states)."""
    o, S = linear_fwd(q[:, None], k[:, None], v[:, None], np.broadcast_to(g, v.shape[:2])[:, None], scale, S)
    return o[:, 0], S


def _act(t, silu):
    """(act, act')"""
    if not silu:
        return t, np.ones_like(t)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-t))
    return t * s, s + t * s * (1.0 - s)


def group_norm(x, groups, weight=None, bias=None, z=None, eps=1e-5, silu=True, dy=None):
    """y [..., C], or with dy the gradients dx, dz, dweight, dbias, and as xh, r, u what they are
    formed of ((x - mean) / sqrt(var + eps), 1 / sqrt(var + eps), the gradient of xh)."""
    x = np.asarray(x, np.float64)
    C = x.shape[-1]
    xg = x.reshape(x.shape[:-1] + (groups, C // groups))
    xc = xg - xg.mean(-1, keepdims=True)
    var = (xc * xc).mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    xh = (xc * r).reshape(x.shape)
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    n = xh * w + (0.0 if bias is None else np.asarray(bias, np.float64))
    e = n if z is None else np.asarray(z, np.float64)
    act, slope = _act(e, silu)
    if dy is None:
        return act if z is None else n * act
    dy = np.asarray(dy, np.float64)
    dn = dy * (slope if z is None else act)
    out = {} if z is None else {"dz": dy * n * slope}
    lead = tuple(range(x.ndim - 1))
    out.update(dweight=(dn * xh).sum(lead), dbias=dn.sum(lead))
    u = (dn * w).reshape(xg.shape)
    hat = xh.reshape(xg.shape)
    # u - mean(u) - xh mean(u xh) with the part along xh written out: a group of two channels has
    # nothing else
    unit = np.where(var > 0, xc / np.sqrt(np.where(var > 0, var, 1.0)), 0.0)
    uc = u - u.mean(-1, keepdims=True)
    along = (uc * unit).mean(-1, keepdims=True)
    across = uc - unit * along if C // groups > 2 else np.zeros_like(uc)
    if C // groups == 2:
        across = np.where(var > 0, across, uc)
    out["dx"] = (r * (across + unit * along * (eps * r * r))).reshape(x.shape)
    out.update(xh=xh, r=np.broadcast_to(r, xg.shape).reshape(x.shape), u=u.reshape(x.shape), hat=hat)
    return out
