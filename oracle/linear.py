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
