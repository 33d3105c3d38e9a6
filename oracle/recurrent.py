"""Plain statements in 64 bits of the gated linear recurrence (forward and gradients) and of
the 8-bit state cache with the decode steps on it.  TEST INFRASTRUCTURE ONLY, like the rest of
this package; numpy, token by token."""
from __future__ import annotations

import numpy as np


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _softplus(x):
    return np.log1p(np.exp(-np.abs(x))) + np.maximum(x, 0.0)


def gated_token(x, r, g, lam, c, clear=None):
    """(a, m, log a, v, sigmoid(r), sigmoid(g)) of tokens; ``clear`` marks the first of a sequence."""
    x, r, g, lam = (np.asarray(v, np.float64) for v in (x, r, g, lam))
    s, sg = _sigmoid(r), _sigmoid(g)
    la = -c * _softplus(lam) * s
    a, m = np.exp(la), np.sqrt(-np.expm1(2 * la))
    if clear is not None:
        a, m = np.where(clear[..., None], 0.0, a), np.where(clear[..., None], 1.0, m)
    return a, m, la, sg * x, s, sg


def gated_fwd(x, r, g, lam, c=8.0, h0=None, reset=None):
    """(states [B, L, D], last state [B, D])."""
    B, L, D = x.shape
    a, m, _, v, _, _ = gated_token(x, r, g, lam, c, reset)
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    y = np.empty((B, L, D))
    for t in range(L):
        # a cleared token takes nothing from the state, whatever it holds
        kept = a[:, t] * h if reset is None else np.where(reset[:, t, None], 0.0, a[:, t] * h)
        h = kept + m[:, t] * v[:, t]
        y[:, t] = h
    return y, h


def gated_bwd(x, r, g, lam, dy, c=8.0, h0=None, reset=None, dlast=None):
    """Gradients, and as ``dlam_abs`` the sum of the magnitudes that dlam adds up."""
    B, L, D = x.shape
    a, m, la, v, s, sg = gated_token(x, r, g, lam, c, reset)
    y, _ = gated_fwd(x, r, g, lam, c, h0, reset)
    first = np.zeros((B, 1, D)) if h0 is None else np.asarray(h0, np.float64)[:, None]
    before = np.concatenate([first, y], 1)[:, :L]
    adj = np.zeros((B, D)) if dlast is None else np.asarray(dlast, np.float64).copy()
    out = {k: np.empty((B, L, D)) for k in ("dx", "dr", "dg")}
    lam = np.asarray(lam, np.float64)
    rho = _sigmoid(lam) / _softplus(lam)
    dlam, mag = np.zeros(D), np.zeros(D)
    for t in range(L - 1, -1, -1):
        adj = adj + np.asarray(dy[:, t], np.float64)
        with np.errstate(divide="ignore", invalid="ignore"):
            w = np.where(m[:, t] > 0, la[:, t] / m[:, t], 0.0)
        e = adj * a[:, t] * (la[:, t] * before[:, t] - a[:, t] * w * v[:, t])
        out["dx"][:, t] = adj * m[:, t] * sg[:, t]
        out["dg"][:, t] = adj * m[:, t] * v[:, t] * (1 - sg[:, t])
        out["dr"][:, t] = e * (1 - s[:, t])
        dlam += e.sum(0) * rho
        mag += (np.abs(adj) * a[:, t] * (np.abs(la[:, t] * before[:, t]) + np.abs(a[:, t] * w * v[:, t]))).sum(0) * rho
        adj = a[:, t] * adj
    out.update(dlam=dlam, dlam_abs=mag, dinitial_state=adj)
    return out


def cache_bits(seed, count, rows, row_len):
    """The 16-bit numbers of the cache's stochastic rounding, [count, rows, row_len]."""
    mask = (1 << 32) - 1
    row = np.arange(count * rows, dtype=np.uint64)

    def mix(v):                                            # whole numbers below 2^32, held in 64 bits
        v = v ^ (v >> np.uint64(16))
        v = (v * np.uint64(0xBB67AE85)) & np.uint64(mask)
        return v ^ (v >> np.uint64(15))

    seed = int(seed) & ((1 << 64) - 1)
    key = mix(np.uint64(seed & mask) ^ ((row * np.uint64(0x9E3779B9)) & np.uint64(mask)))
    key = mix(key ^ np.uint64(seed >> 32))
    pair = np.arange((row_len + 1) // 2, dtype=np.uint64)
    w = mix((key[:, None] + pair * np.uint64(0x9E3779B9)) & np.uint64(mask))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(count, rows, -1)
    return bits[..., :row_len].astype(np.int64)


def as_rows(states, row_len):
    """States [count, elems] as [count, rows, row_len]; the last row is filled up with zeros."""
    count, elems = states.shape
    rows = -(-elems // row_len)
    out = np.zeros((count, rows * row_len))
    out[:, :elems] = states
    return out.reshape(count, rows, row_len)


def cache_code(h, seed=None):
    """(code before rounding down, scale) of rows [count, rows, row_len] of finite values: the code
    is its floor, cut to -127 .. 127."""
    h = np.asarray(h, np.float64)
    amax = np.abs(h).max(-1)
    held = amax >= 2.0 ** -100
    off = 0.5 if seed is None else (cache_bits(seed, *h.shape) + 0.5) / 65536.0
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(held[..., None], h * 127.0 / amax[..., None], 0.0)
    return np.where(held[..., None], t + off, 0.0), np.where(held, amax / 127.0, 0.0)


def step(h, u, delta, A, B, C, Dskip=None, z=None, euler=False, softplus=False, bias=None):
    """One token of the selective scan from states h [B, D, N]: (y [B, D], new states)."""
    h, u, delta, A, B, C = (np.asarray(v, np.float64) for v in (h, u, delta, A, B, C))
    dt = np.broadcast_to(delta, u.shape) + (0.0 if bias is None else np.asarray(bias, np.float64))
    if softplus:
        dt = _softplus(dt)
    da = dt[..., None] * A
    with np.errstate(divide="ignore", invalid="ignore"):
        drive = dt[..., None] if euler else np.where(A == 0, dt[..., None], np.expm1(da) / A)
    h = np.exp(da) * h + drive * B[:, None, :] * u[..., None]
    y = (h * C[:, None, :]).sum(-1)
    if Dskip is not None:
        y = y + np.asarray(Dskip, np.float64) * u
    if z is not None:
        z = np.asarray(z, np.float64)
        y = y * z * _sigmoid(z)
    return y, h
