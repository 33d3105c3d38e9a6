"""Group norm with an activation on the GPU against its 64-bit statement.

Tolerances.  The mean of `width` values is off by at most log2(width) + 32 roundings of their largest
magnitude (a thread adds up to 32, the threads' sums are joined in pairs), so a centred value is off by
n 2^-24 max|x|, n = log2(width) + 40; divided by the standard deviation that is n 2^-24 c with
c = 1 + max|x| r, r = 1 / sqrt(var + eps), and the same for what r itself is off by, times |xh|.  The
activation's slope is below 1.1 and its exp and reciprocal add 2^-21.  Results are rounded: 2^-8 of them in
bf16."""
import numpy as np
import pytest

from oracle import linear as orc

pytestmark = pytest.mark.gpu

#         batch, L, groups, width
SIZES = [(1, 1, 1, 1), (2, 3, 5, 2), (1, 7, 3, 3), (3, 5, 4, 8), (2, 33, 24, 64), (1, 130, 40, 64), (2, 9, 7, 65),
         (1, 17, 2, 257), (1, 5, 3, 512), (2, 3, 1, 1000), (1, 3, 2, 2048), (1, 3, 2, 2049), (1, 2, 1, 2560), (1, 2, 2, 8192),
         (1, 1, 1, 8191), (700, 1, 3, 16), (1, 600, 1, 128), (3, 1000, 2, 96)]


def _torch():
    import torch
    return torch


def dev(a, io="f32"):
    t = _torch()
    if a is None:
        return None
    v = t.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return v.to(t.bfloat16) if io == "bf16" else v


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf(a, io):
    t = _torch()
    a = np.asarray(a, np.float32)
    return t.from_numpy(a).to(t.bfloat16).float().numpy() if io == "bf16" else a


def near(got, ref, bound, what):
    got = host(got) if hasattr(got, "detach") else got
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(got == ref, 0.0, np.abs(got - ref) / bound)
    print("%s: %.3f of the bound" % (what, r.max(initial=0.0)))
    assert r.max(initial=0.0) <= 1.0, "%s: %.3g of the bound" % (what, r.max())


def inputs(size, io, gate, affine, seed=0):
    B, L, G, W = size
    rng = np.random.default_rng(seed)
    C = G * W
    i = {"x": bf(rng.standard_normal((B, L, C)) * np.exp(rng.standard_normal((B, L, 1))) + rng.standard_normal(C), io),
         "dy": bf(rng.standard_normal((B, L, C)), io), "z": bf(rng.standard_normal((B, L, C)), io) if gate else None}
    i["weight"] = (1 + 0.3 * rng.standard_normal(C)).astype(np.float32) if affine != "none" else None
    i["bias"] = rng.standard_normal(C).astype(np.float32) if affine == "both" else None
    return i


def check(i, size, io, silu, y=None, d=None, eps=1e-5):
    B, L, G, W = size
    kw = dict(groups=G, weight=i["weight"], bias=i["bias"], z=i["z"], eps=eps, silu=silu)
    g = orc.group_norm(i["x"], dy=i["dy"], **kw)
    u24, half = 2.0 ** -24, 2.0 ** -8 if io == "bf16" else 2.0 ** -24
    top = lambda a: np.repeat(np.abs(a).reshape(B, L, G, W).max(-1), W, -1)           # noqa: E731
    n = np.log2(W) + 40
    c = n * u24 * (1 + top(i["x"]) * g["r"])                 # what xh is off by, beside |xh| c
    w = 1.0 if i["weight"] is None else np.abs(i["weight"].astype(np.float64))
    b = 0.0 if i["bias"] is None else np.abs(i["bias"].astype(np.float64))
    xh = np.abs(g["xh"])
    off_n = w * c * (1 + xh) + 2 * u24 * (w * xh + b)
    mag_n = w * xh + b
    z = None if i["z"] is None else np.abs(i["z"].astype(np.float64))
    if y is not None:
        ref = orc.group_norm(i["x"], **kw)
        gate = 1.1 if z is None else z
        near(y, ref, half * np.abs(ref) + gate * (off_n + 2.0 ** -21 * mag_n), "y")
    if d is None:
        return
    dy = np.abs(i["dy"].astype(np.float64))
    # act' lies within 1.1 and its slope within 1/2 (silu)
    off_dn = dy * ((0.5 * off_n + 2.0 ** -21 * 1.1) if z is None else 2.0 ** -21 * z)
    mag_dn = dy * (1.1 if z is None else z)
    lead = (0, 1)
    rows = (B * L + 64) * u24
    for name, on, off in (("dweight", xh, off_dn * xh + mag_dn * c * (1 + xh)), ("dbias", 1.0, off_dn)):
        given = i["weight" if name == "dweight" else "bias"]
        assert (name in d) == (given is not None)
        if given is not None:
            near(d[name], g[name], (off + rows * mag_dn * on).sum(lead) + 2 * u24 * np.abs(g[name]), name)
    assert ("dz" in d) == (z is not None)
    if z is not None:
        near(d["dz"], g["dz"], half * np.abs(g["dz"]) + dy * (1.1 * off_n + 2.0 ** -21 * 1.1 * mag_n), "dz")
    # dx = r (u - mean(u) - xh mean(u xh)): |u| up to mag_dn w, and its mean with n roundings
    mu, ou = mag_dn * w, off_dn * w
    off = top(ou) * (2 + xh) + top(mu) * n * u24 * (2 + 2 * xh) + top(mu) * (c * (1 + xh) * (1 + xh) + xh * top(c * (1 + xh)))
    near(d["dx"], g["dx"], half * np.abs(g["dx"]) + g["r"] * off * 2, "dx")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("activation,affine", [("silu", "both"), ("none", "both"), ("silu", "none"), ("silu", "weight")])
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_backward(size, activation, affine, gate, io):
    import selective_state_space_s6_amd as ss
    i = inputs(size, io, gate, affine, seed=sum(size))
    kw = dict(groups=size[2], activation=activation)
    v = {k: dev(a, io if k in ("x", "z", "dy") else "f32") for k, a in i.items()}
    y = ss.group_norm_fwd(v["x"], v["weight"], v["bias"], v["z"], **kw)
    check(i, size, io, activation == "silu", y=y)
    d = ss.group_norm_bwd(v["x"], v["weight"], v["bias"], v["z"], dy=v["dy"], **kw)
    check(i, size, io, activation == "silu", d=d)
