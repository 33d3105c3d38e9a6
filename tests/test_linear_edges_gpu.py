"""Linear attention and the group norm on the GPU at their edges: values that are not finite, layouts and strides,
empty calls, offsets beyond 32 bits, streams, workspaces, captured calls.  Bounds as in test_linear_gpu.py and
test_norm_gpu.py."""
import ctypes

import numpy as np
import pytest

from oracle import linear as orc
from tests import test_linear_gpu as lin
from tests import test_norm_gpu as nrm

pytestmark = pytest.mark.gpu

dev, host, inputs = lin.dev, lin.host, lin.inputs


def _torch():
    import torch
    return torch


def _ss():
    import selective_state_space_s6_amd as ss
    return ss


def tensors(i, io):
    v = {k: dev(i[k], io) for k in ("q", "k", "v", "do")}
    v.update(g=dev(i["g"]), S0=dev(i["S0"]), dlast=dev(i["dlast"]))
    return v


def fwd(v, i, **kw):
    return _ss().linear_attention_fwd(v["q"], v["k"], v["v"], v["g"], scale=i["scale"], initial_state=v["S0"],
                                      return_last_state=True, **kw)


def bwd(v, i, **kw):
    return _ss().linear_attention_bwd(v["q"], v["k"], v["v"], v["g"], do=v["do"], scale=i["scale"], initial_state=v["S0"],
                                      dlast_state=v["dlast"], **kw)


def same(a, b):
    t = _torch()
    return all(t.equal(x, y) for x, y in zip(a, b)) if not isinstance(a, dict) else set(a) == set(b) and all(
        t.equal(a[k], b[k]) for k in a)


# ---------------------------------------------------------------------- pairs of heads, segments, widths apart

#          batch, L, H, Hk, K, V: two heads a workgroup and segments; K and V of different kernels; one token less than a
#          chunk, one more than a segment
WIDE_APART = [(1, 1100, 4, 1, 64, 64), (2, 705, 4, 2, 128, 32), (1, 640, 6, 3, 200, 64), (1, 900, 2, 2, 256, 16),
              (1, 900, 2, 2, 16, 256), (1, 449, 2, 1, 1, 64), (1, 385, 2, 2, 64, 1), (3, 127, 8, 2, 7, 3), (1, 2049, 2, 2, 8, 8)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", WIDE_APART)
def test_pairs_and_segments(size, io):
    i = inputs(size, io, seed=21, decay="packed")
    v = tensors(i, io)
    o, last = fwd(v, i)
    lin.check_forward(i, size, io, o, last)
    lin.check_backward(i, size, io, bwd(v, i))
    d = bwd(v, i, decay_grad=False)
    assert "dlog_decay" not in d
    full = bwd(v, i)
    assert _torch().equal(d["dv"], full["dv"])
    lin.check_backward(i, size, io, dict(d, dlog_decay=full["dlog_decay"]))


@pytest.mark.parametrize("size", [(1, 90, 2, 1, 24, 40), (1, 330, 2, 2, 16, 16)])
def test_gradients_against_differences(size):
    """The loss <do, o> + <dlast, last> is linear in each of q, k, v and the initial state, so its difference over any step
    is the gradient's product with it, up to rounding alone: n 2^-24 of the magnitudes on either side (test_linear_gpu.py).
    In the decays a central difference is off by its own remainder too, which the 64-bit statement gives."""
    B, L, H, Hk, K, V = size
    i = inputs(size, "f32", seed=31, decay="token")
    rng = np.random.default_rng(5)
    d = bwd(tensors(i, "f32"), i)
    n = (K + V + L / 16 + 100) * 2.0 ** -24 * 2
    loss = lambda o, last: (host(o) * i["do"]).sum() + (host(last) * i["dlast"]).sum()       # noqa: E731
    oracle_run = lambda j: orc.linear_fwd(*(j[a] for a in "qkvg"), j["scale"], j["S0"])      # noqa: E731
    exact = lambda j: (lambda o, s: (o * i["do"]).sum() + (s * i["dlast"]).sum())(*oracle_run(j))    # noqa: E731
    size_of = lambda j: (lambda o, s: (o * np.abs(i["do"])).sum() + (s * np.abs(i["dlast"])).sum())(*oracle_run(lin.absolute(j)))    # noqa: E731
    base = loss(*fwd(tensors(i, "f32"), i))
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dinitial_state")):
        step = host(d[key])
        step /= np.sqrt((step ** 2).mean())                    # along the gradient, of size one
        j = dict(i, **{name: (i[name] + step).astype(np.float32)})
        step = j[name].astype(np.float64) - i[name]
        diff, grad = loss(*fwd(tensors(j, "f32"), j)) - base, (host(d[key]) * step).sum()
        bound = n * (size_of(i) + size_of(j) + size_of(dict(i, **{name: np.abs(step)})))
        assert abs(diff - grad) <= bound, (name, diff, grad, bound)
        assert abs(grad) > 10 * bound, name                    # the bound says something
    step = 2e-2 * rng.uniform(-1, 1, i["g"].shape)
    up, dn = (dict(i, g=(i["g"] + s * step).astype(np.float32)) for s in (1, -1))
    step = (up["g"].astype(np.float64) - dn["g"]) / 2
    diff = (loss(*fwd(tensors(up, "f32"), up)) - loss(*fwd(tensors(dn, "f32"), dn))) / 2
    grad = (host(d["dlog_decay"]) * step).sum()
    ref = (orc.linear_bwd(i["q"], i["k"], i["v"], i["g"], i["do"], i["scale"], i["S0"], i["dlast"])["dlog_decay"] * step).sum()
    mid = dict(i, g=((up["g"].astype(np.float64) + dn["g"]) / 2).astype(np.float32))
    rest = abs((exact(up) - exact(dn)) / 2 - ref) + n * size_of(mid)
    # the decays' gradient is off by n 2^-24 of the magnitudes that pass each of L tokens
    bound = rest + n * (size_of(up) + size_of(dn)) + n * np.abs(step).max() * L * size_of(i)
    assert abs(diff - grad) <= bound, (diff, grad, bound)


# ---------------------------------------------------------------------- values that are not finite

def near_where_finite(got, ref, bound, what):
    """Equal where the reference is not finite (NaN or the same infinity), near elsewhere."""
    got = host(got)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)), "%s: finite elsewhere at %d" % (what, (fine != np.isfinite(got)).sum())
    lin.near(np.where(fine, got, 0.0), np.where(fine, ref, 0.0), np.where(np.isfinite(bound), bound, 1e30), what)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["v", "k", "S0", "v then start", "S0 then start", "last token", "whole document"])
@pytest.mark.parametrize("size", [(2, 150, 2, 2, 32, 48), (1, 700, 2, 1, 64, 130), (1, 900, 4, 1, 40, 64)])
def test_what_is_not_finite_stays_where_it_belongs(size, where, io):
    """Only what depends on such a value is not finite: not the tokens before it, not the document behind, not the
    other columns; in segments (long sequences of few heads) as in one walk."""
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=7, decay="token")
    bad = {"v": np.inf, "k": np.nan, "v then start": -np.inf}.get(where, np.inf)
    if where in ("v", "v then start", "whole document"):
        i["v"][0, 70:80 if where == "whole document" else 71, 0, 3 % V] = bad
    if where == "k":
        i["k"][0, 70, 0, 1] = bad
    if where.startswith("S0"):
        i["S0"][0, 0, 2, 5] = np.inf
    if where == "last token":
        i["v"][0, L - 1, 0, 1] = np.inf
    if where in ("v then start", "whole document"):
        i["g"][:, 100] = -np.inf
        i["g"][:, 60] = -np.inf
    if where == "S0 then start":
        i["g"][:, 65] = -np.inf
    v = tensors(i, io)
    o, last = fwd(v, i)
    with np.errstate(invalid="ignore", over="ignore"):
        ro, rl = orc.linear_fwd(i["q"], i["k"], i["v"], i["g"], i["scale"], i["S0"])
        clean = {k: np.nan_to_num(a, nan=1.0, posinf=1.0, neginf=-1.0) if k in ("q", "k", "v", "S0") else a for k, a in i.items()}
        mo, ml = orc.linear_fwd(*(lin.absolute(clean)[a] for a in "qkvg"), i["scale"], np.abs(clean["S0"]))
    n, mixed, out = lin.units(size, io)
    near_where_finite(o, ro, out * np.abs(ro) + mixed * mo, where + " o")
    near_where_finite(last, rl, n * ml, where + " last_state")
    # an infinity whose sign nothing disputes stays one
    if where == "S0":
        assert np.array_equal(np.isinf(host(last)), np.isinf(rl))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 150, 2, 2, 32, 48), (1, 900, 2, 1, 64, 64)])
def test_gradients_of_a_document_next_to_one_that_is_not_finite(size, io):
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=8, decay="token")
    cut = [40, 90]
    for c in cut:
        i["g"][:, c] = -np.inf
    clean = bwd(tensors(i, io), i)
    for name, value in (("v", np.inf), ("do", np.nan), ("k", -np.inf), ("q", np.inf)):
        j = dict(i, **{name: i[name].copy()})
        j[name][0, 50] = value
        d = bwd(tensors(j, io), j)
        for k in ("dq", "dk", "dv"):
            a, b = host(d[k]), host(clean[k])
            # (no gradient holds its own operand: dq none of q, dk none of k, dv none of v)
            assert np.isfinite(a[0, 40:90]).all() == (k == "d" + name), (name, k)
            # the other documents: the same up to rounding (a chunk that holds part of this one is walked token by token)
            scale = np.abs(b).max()
            tol = (2.0 ** -7 + 2.0 ** -7 if io == "bf16" else 2e-5) * scale
            for part in (np.s_[0, :40], np.s_[0, 90:], np.s_[1:]):
                assert np.isfinite(a[part]).all() and np.abs(a[part] - b[part]).max(initial=0.0) <= tol, (name, k)
        assert np.isfinite(host(d["dinitial_state"])).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name,value", [("v", np.inf), ("do", np.nan), ("k", -np.inf), ("q", np.inf)])
def test_decay_gradient_of_documents_next_to_one_that_is_not_finite(name, value, io):
    """Documents that lie across segments, one of them not finite: the others' gradients are the same."""
    size = (1, 900, 2, 1, 64, 64)
    i = inputs(size, io, seed=9, decay="token")
    for c in (400, 640, 800):
        i["g"][:, c] = -np.inf
    clean = bwd(tensors(i, io), i)
    lin.check_backward(i, size, io, clean)
    j = dict(i, **{name: i[name].copy()})
    j[name][0, 700] = value
    got = bwd(tensors(j, io), j)["dlog_decay"]
    assert not np.isfinite(host(got)[0, 640:800]).all()
    got[:, 640:800] = clean["dlog_decay"][:, 640:800]
    lin.check_backward(i, size, io, dict(clean, dlog_decay=got))


def test_sums_that_leave_the_range():
    """Products beyond fp32's largest value are infinite, whatever lies beside them."""
    i = inputs((1, 130, 1, 1, 16, 16), "f32", seed=2, decay="fixed")
    i["k"][0, 5] = 1e30
    i["v"][0, 5, 0, 4] = 1e30
    o, _ = fwd(tensors(i, "f32"), i)
    o = host(o)
    assert np.isfinite(o[0, :5]).all() and not np.isfinite(o[0, 5:, 0, 4]).any()
    assert np.isfinite(np.delete(o, 4, -1)).all()


def test_group_norm_keeps_what_is_not_finite_in_its_group():
    t = _torch()
    x = t.randn(3, 4, 4 * 64, device="cuda")
    x[1, 2, 64:128][7] = float("nan")
    y = host(_ss().group_norm_fwd(x, groups=4)).reshape(3, 4, 4, 64)
    hit = np.zeros((3, 4, 4), bool)
    hit[1, 2, 1] = True
    assert np.array_equal(np.isnan(y).all(-1), hit) and np.array_equal(np.isnan(y).any(-1), hit)
    # no spread at all: the bias
    b = t.arange(64, device="cuda", dtype=t.float32)
    y = _ss().group_norm_fwd(t.full((5, 64), 3.0, device="cuda"), None, b, groups=2, activation="none")
    assert t.equal(y, b.expand(5, 64))


# ---------------------------------------------------------------------- layouts

LAYOUTS = ["heads first", "time first", "one tensor", "room between", "off by one", "expanded"]


def laid_out(name, shape, io, values=None, outputs=False):
    """A tensor of this shape in another layout, holding values."""
    t = _torch()
    dtype = t.bfloat16 if io == "bf16" else t.float32
    B, L, H, W = shape
    if name == "heads first":
        x = t.zeros(B, H, L, W, dtype=dtype, device="cuda").transpose(1, 2)
    elif name == "time first":
        x = t.zeros(L, B, H, W, dtype=dtype, device="cuda").transpose(0, 1)
    elif name == "one tensor":
        x = t.zeros(B, L, H, 3 * W + 1, dtype=dtype, device="cuda")[..., W:2 * W]
    elif name == "room between":
        x = t.zeros(B, L + 3, H + 1, W + 5, dtype=dtype, device="cuda")[:, 1:L + 1, 1:, 2:W + 2]
    elif name == "off by one":
        x = t.zeros(B * L * H * W + 1, dtype=dtype, device="cuda")[1:].view(shape)
    else:
        x = t.zeros(shape, dtype=dtype, device="cuda")
    if values is not None:
        x.copy_(dev(values, io))
    return x


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [(2, 130, 4, 2, 64, 64), (2, 70, 3, 3, 37, 83), (1, 1030, 2, 1, 128, 130)])
def test_layouts(size, layout, io):
    """The same bits as from contiguous tensors, and nothing written beside the output."""
    t, ss = _torch(), _ss()
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=11, decay="token")
    v = tensors(i, io)
    want, wlast = fwd(v, i)
    wgrad = bwd(v, i)
    q, k, x, do = (laid_out(layout, i[n].shape, io, i[n]) for n in ("q", "k", "v", "do"))
    if layout == "expanded":
        x, do, q = x[:1, :1].expand(B, L, H, V), do[:, :, :1].expand(B, L, H, V), q[:, :, :1].expand(B, L, Hk, K)
        c = dict(v, q=q.contiguous(), v=x.contiguous(), do=do.contiguous())
        want, wlast = fwd(c, i)
        wgrad = bwd(c, i)
    g = dev(i["g"]).permute(2, 0, 1).contiguous().permute(1, 2, 0)
    room = laid_out(layout, (B, L, H, V), io)
    whole = room._base if room._base is not None else room
    whole.fill_(3.0)
    before = whole.clone()
    o, last = ss.linear_attention_fwd(q, k, x, g, scale=i["scale"], initial_state=v["S0"], o=room, return_last_state=True)
    assert t.equal(o, want) and t.equal(last, wlast)
    o.fill_(3.0)
    assert t.equal(whole, before)
    grads = ss.linear_attention_bwd(q, k, x, g, do=do, scale=i["scale"], initial_state=v["S0"], dlast_state=v["dlast"])
    assert same(grads, wgrad)


def test_a_decay_for_all_tokens_is_the_decay_of_each():
    t = _torch()
    size = (2, 140, 4, 2, 32, 48)
    i = inputs(size, "f32", seed=1, decay="fixed")
    v = tensors(i, "f32")
    e = dict(v, g=v["g"].expand(2, 140, 4))
    assert same(fwd(v, i), fwd(e, i))
    a, b = bwd(v, i), bwd(e, i)
    assert all(t.equal(a[k], b[k]) for k in ("dq", "dk", "dv", "dinitial_state"))
    ref = b["dlog_decay"].double().sum((0, 1))
    # one rounding of each token's, and of the sum
    assert (a["dlog_decay"].double() - ref).abs().max() <= 2.0 ** -24 * (b["dlog_decay"].double().abs().sum((0, 1)).max() + ref.abs().max())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C,groups", [(96, 4), (75, 3), (520, 1)])
def test_norm_layouts(io, C, groups):
    t, ss = _torch(), _ss()
    B, L = 3, 7
    i = nrm.inputs((B, L, groups, C // groups), io, True, "both", seed=4)
    v = {k: dev(a, io if k in ("x", "z", "dy") else "f32") for k, a in i.items()}
    args = (v["weight"], v["bias"])
    want = ss.group_norm_fwd(v["x"], *args, v["z"], groups=groups)
    grads = ss.group_norm_bwd(v["x"], *args, v["z"], dy=v["dy"], groups=groups)
    for name in LAYOUTS[1:]:
        lay = lambda a: laid_out(name, (B, L, 1, C), io, None if a is None else a.reshape(B, L, 1, C))[:, :, 0]     # noqa: E731
        x, z, dy = lay(i["x"]), lay(i["z"]), lay(i["dy"])
        room = lay(None)
        whole = room._base if room._base is not None else room
        whole.fill_(3.0)
        before = whole.clone()
        y = ss.group_norm_fwd(x, *args, z, groups=groups, y=room)
        # (another alignment sums a group in another order)
        nrm.check(i, (B, L, groups, C // groups), io, True, y=y)
        y.fill_(3.0)
        assert t.equal(whole, before)
        nrm.check(i, (B, L, groups, C // groups), io, True, d=ss.group_norm_bwd(x, *args, z, dy=dy, groups=groups))
    x, z = v["x"].clone(), v["z"].clone()
    assert t.equal(ss.group_norm_fwd(x, *args, z, groups=groups, y=x), want) and t.equal(x, want)
    x = v["x"].clone()
    assert t.equal(ss.group_norm_fwd(x, *args, z, groups=groups, y=z), want) and t.equal(z, want) and t.equal(x, v["x"])
    rows = lambda a: a.reshape(B * L, C)                                                # noqa: E731
    assert t.equal(ss.group_norm_fwd(rows(v["x"]), *args, rows(v["z"]), groups=groups), rows(want))
    one = v["x"][:1, :1].expand(B, L, C)
    assert same(ss.group_norm_bwd(one, *args, v["z"], dy=v["dy"], groups=groups),
                ss.group_norm_bwd(one.contiguous(), *args, v["z"], dy=v["dy"], groups=groups))
    assert t.equal(grads["dx"], ss.group_norm_bwd(v["x"], *args, v["z"], dy=v["dy"], groups=groups)["dx"])


# ---------------------------------------------------------------------- empty calls, one buffer for two

def test_empty_calls():
    t, ss = _torch(), _ss()
    new = lambda *s: t.randn(*s, device="cuda")                                         # noqa: E731
    S0, dlast, g = new(2, 3, 4, 5), new(2, 3, 4, 5), new(2, 0, 3)
    q, v = new(2, 0, 3, 4), new(2, 0, 3, 5)
    o, last = ss.linear_attention_fwd(q, q, v, g, initial_state=S0, return_last_state=True)
    assert o.shape == (2, 0, 3, 5) and t.equal(last, S0)
    _, last = ss.linear_attention_fwd(q, q, v, g, return_last_state=True)
    assert not last.any()
    d = ss.linear_attention_bwd(q, q, v, -new(3).abs(), do=v, initial_state=S0, dlast_state=dlast)
    assert t.equal(d["dinitial_state"], dlast) and not d["dlog_decay"].any() and d["dq"].shape == q.shape
    d = ss.linear_attention_bwd(q, q, v, g, do=v, initial_state=S0)
    assert not d["dinitial_state"].any()
    o, last = ss.linear_attention_fwd(q[:0].reshape(0, 5, 3, 4), q[:0].reshape(0, 5, 3, 4), v[:0].reshape(0, 5, 3, 5), -new(3).abs(),
                                      return_last_state=True)
    assert o.shape == (0, 5, 3, 5) and last.shape == (0, 3, 4, 5)
    o = ss.linear_attention_step(q[:0, 0:1].reshape(0, 3, 4), q[:0, 0:1].reshape(0, 3, 4), v[:0, 0:1].reshape(0, 3, 5), -new(3).abs(),
                                 state=S0)
    assert o.shape == (0, 3, 5)
    x, w = new(0, 6), new(6)
    assert ss.group_norm_fwd(x, groups=2).shape == (0, 6)
    d = ss.group_norm_bwd(x, w, w, dy=x, groups=2)
    assert not d["dweight"].any() and not d["dbias"].any()


def test_a_state_that_is_continued_in_place():
    t, ss = _torch(), _ss()
    for size in ((2, 100, 2, 2, 32, 48), (1, 1000, 2, 2, 64, 64)):
        i = inputs(size, "f32", seed=3)
        v = tensors(i, "f32")
        o, last = fwd(v, i)
        state = v["S0"].clone()
        o2, _ = ss.linear_attention_fwd(v["q"], v["k"], v["v"], v["g"], scale=i["scale"], initial_state=state, last_state=state)
        assert t.equal(o2, o) and t.equal(state, last)
        # the C entry point allows it for the gradients too
        d = bwd(v, i)
        B, L, H, Hk, K, V = size
        dims = ss.LinattnDims()
        ss.lib().linear_attention_dims_init(ctypes.byref(dims), ss.SELSCAN_F32, B, L, H, Hk, K, V)
        dims.scale = i["scale"]
        both, out = v["dlast"].clone(), {k: t.empty_like(d[k]) for k in ("dq", "dk", "dv", "dlog_decay")}
        st = ss.lib().linear_attention_bwd(v["q"].data_ptr(), v["k"].data_ptr(), v["v"].data_ptr(), v["g"].data_ptr(), v["S0"].data_ptr(),
                                           v["do"].data_ptr(), both.data_ptr(), out["dq"].data_ptr(), out["dk"].data_ptr(),
                                           out["dv"].data_ptr(), out["dlog_decay"].data_ptr(), both.data_ptr(), ctypes.byref(dims),
                                           None, 0, t.cuda.current_stream().cuda_stream)
        assert st == 0
        t.cuda.synchronize()
        assert t.equal(both, d["dinitial_state"]) and all(t.equal(out[k], d[k]) for k in out)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2048, 2049, 4099, 8191, 8192])
def test_wide_groups_in_place(width, io):
    """Four wavefronts a group, whose last piece may begin within the one before's: y in the place of x, or of z."""
    t, ss = _torch(), _ss()
    size = (2, 3, 2, width)
    i = nrm.inputs(size, io, True, "both", seed=6)
    v = {k: dev(a, io if k in ("x", "z", "dy") else "f32") for k, a in i.items()}
    args = (v["weight"], v["bias"])
    want = ss.group_norm_fwd(v["x"], *args, v["z"], groups=2)
    nrm.check(i, size, io, True, y=want)
    nrm.check(i, size, io, True, d=ss.group_norm_bwd(v["x"], *args, v["z"], dy=v["dy"], groups=2))
    for n in range(3):
        x, z = v["x"].clone(), v["z"].clone()
        assert t.equal(ss.group_norm_fwd(x, *args, v["z"], groups=2, y=x), want)
        assert t.equal(ss.group_norm_fwd(v["x"], *args, z, groups=2, y=z), want) and t.equal(z, want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_padded_rows(io):
    """Keys of zero and a log decay of zero behind a sequence's end leave its state as it was."""
    ends = [37, 64, 150, 1]
    size = (4, 150, 2, 1, 32, 48)
    i = inputs(size, io, seed=13, decay="token")
    for b, n in enumerate(ends):
        i["k"][b, n:] = 0.0
        i["g"][b, n:] = 0.0
    _, last = fwd(tensors(i, io), i)
    for b, n in enumerate(ends):
        j = {k: a[b:b + 1, :n] if k in ("q", "k", "v", "do", "g") else a[b:b + 1] if k in ("S0", "dlast") else a for k, a in i.items()}
        _, rl = orc.linear_fwd(*(j[a] for a in "qkvg"), i["scale"], j["S0"])
        _, ml = orc.linear_fwd(*(lin.absolute(j)[a] for a in "qkvg"), i["scale"], np.abs(j["S0"]))
        lin.near(last[b:b + 1], rl, lin.units(size, io)[0] * ml, "row %d" % b)


def test_slots_read_twice():
    t, ss = _torch(), _ss()
    H, K, V = 2, 24, 37
    state = t.randn(6, H, K, V, device="cuda")
    before = state.clone()
    q, k, v = (t.randn(4, H, w, device="cuda") for w in (K, K, V))
    ids = lambda *a: t.tensor(a, dtype=t.int32, device="cuda")                          # noqa: E731
    o = t.full((4, H, V), 7.0, device="cuda")
    ss.linear_attention_step(q, k, v, -t.rand(H, device="cuda"), state=state, o=o, read_slots=ids(1, 1, 1, 1), write_slots=ids(0, 3, 5, -1))
    assert t.equal(state[[1, 2, 4]], before[[1, 2, 4]]) and (o[3] == 7.0).all() and not (o[:3] == 7.0).any()
    assert not t.equal(state[0], state[5])


# ---------------------------------------------------------------------- offsets beyond 32 bits

def test_tokens_and_rows_far_apart():
    t = _torch()
    B, L, H, K, V = 2, 600, 1, 8, 16
    size = (B, L, H, 1, K, V)
    i = inputs(size, "bf16", seed=4)
    v = tensors(i, "bf16")
    want, wlast = fwd(v, i)
    wgrad = bwd(v, i)
    # tokens 2^22 elements apart, batch rows interleaved: 2.5e9 elements of two bytes
    buf = t.empty(L << 22, dtype=t.bfloat16, device="cuda")
    far = lambda x, at: buf.as_strided(x.shape, (x.shape[-1] + 64, 1 << 22, x.shape[-1], 1), at).copy_(x)    # noqa: E731
    j = dict(v, q=far(v["q"], 0), k=far(v["k"], 1000), v=far(v["v"], 2000), do=far(v["do"], 3000))
    o, last = fwd(j, i, o=buf.as_strided((B, L, H, V), (100, 1 << 22, V, 1), 4000))
    assert t.equal(o, want) and t.equal(last, wlast)
    assert same(bwd(j, i), wgrad)
    x = v["v"].reshape(B, L, V)
    assert t.equal(_ss().group_norm_fwd(j["v"][:, :, 0], groups=2), _ss().group_norm_fwd(x, groups=2))


def test_a_slot_far_into_the_states():
    t, ss = _torch(), _ss()
    H, K, V, slots = 64, 128, 128, 2100                       # 2.2e9 values
    state = t.empty(slots, H, K, V, device="cuda")
    q, k = t.randn(2, 2, H, K, device="cuda")
    v, g = t.randn(2, H, V, device="cuda"), -t.rand(H, device="cuda")
    near_, ids = t.randn(2, H, K, V, device="cuda"), t.tensor([2099, 2060], dtype=t.int32, device="cuda")
    state[ids.long()] = near_
    o = ss.linear_attention_step(q, k, v, g, state=state, read_slots=ids, write_slots=ids)
    want = ss.linear_attention_step(q, k, v, g, state=near_)
    assert t.equal(o, want) and t.equal(state[ids.long()], near_)


# ---------------------------------------------------------------------- streams, workspaces, captured calls

@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_repeats_streams_and_workspaces(io):
    t, ss = _torch(), _ss()
    for size in ((2, 100, 4, 2, 40, 64), (1, 1500, 2, 2, 64, 64)):
        i = inputs(size, io, seed=5, decay="packed")
        v = tensors(i, io)
        want, grads = fwd(v, i), bwd(v, i)
        assert same(fwd(v, i), want) and same(bwd(v, i), grads)
        t.cuda.synchronize()
        side = t.cuda.Stream()
        a, b = fwd(v, i, stream=side), bwd(v, i, stream=side)
        c = fwd(v, i, stream=side.cuda_stream)
        # two calls at once, a stream each
        other = t.cuda.Stream()
        d, e = bwd(v, i, stream=other), bwd(v, i, stream=side)
        t.cuda.synchronize()
        assert same(a, want) and same(b, grads) and same(c, want) and same(d, grads) and same(e, grads)
        ws = t.full((1 << 28,), 255, dtype=t.uint8, device="cuda")                      # what it holds is of no account
        assert same(fwd(v, i, workspace=ws), want) and same(bwd(v, i, workspace=ws), grads)
    i = nrm.inputs((4, 50, 3, 40), io, True, "both")
    x = {k: dev(a, io if k in ("x", "z", "dy") else "f32") for k, a in i.items()}
    run = lambda **kw: ss.group_norm_bwd(x["x"], x["weight"], x["bias"], x["z"], dy=x["dy"], groups=3, **kw)     # noqa: E731
    want = run()
    t.cuda.synchronize()
    got = run(stream=side)
    t.cuda.synchronize()
    assert same(got, want) and same(run(workspace=t.full((1 << 24,), 255, dtype=t.uint8, device="cuda")), want)


def test_the_library_s_own_allocation():
    """Without a workspace the C entry points take one in the stream's order."""
    t, ss = _torch(), _ss()
    size = (1, 1500, 2, 2, 64, 64)
    i = inputs(size, "f32", seed=6)
    v = tensors(i, "f32")
    want, last = fwd(v, i)
    B, L, H, Hk, K, V = size
    dims = ss.LinattnDims()
    ss.lib().linear_attention_dims_init(ctypes.byref(dims), ss.SELSCAN_F32, B, L, H, Hk, K, V)
    dims.scale = i["scale"]
    assert ss.lib().linear_attention_workspace_size(ctypes.byref(dims)) > 0
    o, s = t.empty_like(want), t.empty_like(last)
    st = ss.lib().linear_attention_fwd(v["q"].data_ptr(), v["k"].data_ptr(), v["v"].data_ptr(), v["g"].data_ptr(), o.data_ptr(),
                                       v["S0"].data_ptr(), s.data_ptr(), ctypes.byref(dims), None, 0,
                                       t.cuda.current_stream().cuda_stream)
    t.cuda.synchronize()
    assert st == 0 and t.equal(o, want) and t.equal(s, last)


@pytest.mark.parametrize("size", [(2, 100, 4, 2, 40, 64), (1, 1500, 2, 2, 64, 64)])
def test_captured_calls(size):
    """Replayed several times on changed inputs, with eager work between: every replay as the eager call."""
    t, ss = _torch(), _ss()
    B, L, H, Hk, K, V = size
    i = inputs(size, "bf16", seed=9, decay="packed")
    v = tensors(i, "bf16")
    z, w = t.randn(B, L, H * V, device="cuda").bfloat16(), t.rand(H * V, device="cuda") + 0.5

    def layer():
        o, last = fwd(v, i)
        y = ss.group_norm_fwd(o.view(B, L, H * V), w, None, z, groups=H)
        d = ss.group_norm_bwd(o.view(B, L, H * V), w, None, z, dy=y, groups=H)
        grads = ss.linear_attention_bwd(v["q"], v["k"], v["v"], v["g"], do=d["dx"].view(B, L, H, V), scale=i["scale"],
                                        initial_state=v["S0"], dlast_state=v["dlast"])
        return dict(grads, o=o, last=last, y=y, dz=d["dz"], dw=d["dweight"])

    layer()
    t.cuda.synchronize()
    graph, other = t.cuda.CUDAGraph(), t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = layer()
    with t.cuda.graph(other):
        more = layer()
    for n in range(3):
        v["q"].normal_()
        v["v"].normal_()
        want = layer()
        t.cuda.synchronize()
        graph.replay()
        other.replay()
        t.cuda.synchronize()
        assert same(got, want) and same(more, want), n
    # decoding steps
    state, o = t.randn(2 * B, H, K, V, device="cuda"), t.empty(B, H, V, dtype=t.bfloat16, device="cuda")
    q, k, x = t.randn(B, Hk, K, device="cuda").bfloat16(), t.randn(B, Hk, K, device="cuda").bfloat16(), t.randn(B, H, V, device="cuda").bfloat16()
    g, ids = -t.rand(H, device="cuda"), t.arange(B, dtype=t.int32, device="cuda")
    step = lambda s, o: ss.linear_attention_step(q, k, x, g, state=s, o=o, read_slots=ids, write_slots=ids)      # noqa: E731
    eager, eo = state.clone(), o.clone()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(state, o)
    for n in range(3):
        graph.replay()
        step(eager, eo)
        t.cuda.synchronize()
        assert t.equal(state, eager) and t.equal(o, eo), n
        q.normal_()


# ---------------------------------------------------------------------- refusals of the binding

def test_refusals():
    t, ss = _torch(), _ss()
    new = lambda *s, **kw: t.zeros(*s, device="cuda", **kw)                              # noqa: E731
    q, v, g = new(2, 5, 2, 8), new(2, 5, 4, 6), new(4)
    with pytest.raises(TypeError):
        ss.linear_attention_fwd(q, q.bfloat16(), v, g)
    with pytest.raises(TypeError):
        ss.linear_attention_fwd(q, q, v, g.bfloat16())
    with pytest.raises(TypeError):
        ss.linear_attention_fwd(q.half(), q.half(), v.half(), g)
    for bad in (new(3), new(2, 5, 3), new(2, 4, 4), new(5, 4)):
        with pytest.raises(ValueError):
            ss.linear_attention_fwd(q, q, v, bad)
    for args in ((q, new(2, 5, 2, 9), v), (q, q, new(2, 5, 3, 6)), (q, q, new(2, 4, 4, 6)), (q[0], q[0], v[0]),
                 (q.transpose(2, 3), q.transpose(2, 3), v), (q.cpu(), q, v)):
        with pytest.raises(ValueError):
            ss.linear_attention_fwd(*args, g)
    with pytest.raises(ValueError):
        ss.linear_attention_fwd(q, q, v, g, initial_state=new(2, 4, 6, 8))
    with pytest.raises(ValueError):
        ss.linear_attention_fwd(q, q, v, g, initial_state=new(2, 4, 6, 8).transpose(2, 3))
    with pytest.raises(ss.SelscanError):
        ss.linear_attention_fwd(q, q, v, g, o=new(1, 5, 4, 6).expand(2, 5, 4, 6))
    with pytest.raises(ss.SelscanError):
        ss.linear_attention_fwd(new(2, 5, 2, 257), new(2, 5, 2, 257), v, g)
    with pytest.raises(ss.SelscanError):
        ss.linear_attention_fwd(q, q, v, g, scale=float("nan"))
    with pytest.raises(ValueError):
        ss.linear_attention_bwd(q, q, v, g, do=new(2, 5, 4, 7))
    with pytest.raises(ss.SelscanError):
        ss.linear_attention_fwd(new(1, 2000, 2, 8), new(1, 2000, 2, 8), new(1, 2000, 4, 6), g, workspace=new(64, dtype=t.uint8))
    s = new(3, 4, 8, 6)
    with pytest.raises(TypeError):
        ss.linear_attention_step(q[:, 0], q[:, 0], v[:, 0], g, state=s, read_slots=new(2, dtype=t.int64))
    with pytest.raises(ValueError):
        ss.linear_attention_step(q[:, 0], q[:, 0], v[:, 0], g, state=s, write_slots=new(3, dtype=t.int32))
    with pytest.raises(ValueError):
        ss.linear_attention_step(q[:, 0], q[:, 0], v[:, 0], g, state=new(3, 4, 6, 8))
    with pytest.raises(ss.SelscanError):
        ss.linear_attention_step(q[:, 0], q[:, 0], v[:, 0], g, state=s[:1])              # slots 0, 1 must exist
    x = new(3, 12)
    for kw in (dict(groups=5), dict(groups=0), dict(groups=3, eps=0.0)):
        with pytest.raises(ss.SelscanError):
            ss.group_norm_fwd(x, **kw)
    with pytest.raises(KeyError):
        ss.group_norm_fwd(x, groups=3, activation="relu")
    with pytest.raises(ValueError):
        ss.group_norm_fwd(x, new(11), groups=3)
    with pytest.raises(TypeError):
        ss.group_norm_fwd(x, new(12, dtype=t.float64), groups=3)
    with pytest.raises(ValueError):
        ss.group_norm_fwd(new(12, 3).t(), groups=3)
    with pytest.raises(ValueError):
        ss.group_norm_fwd(new(2, 2, 3, 12), groups=3)
