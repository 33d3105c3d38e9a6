"""The 64-bit statements of linear attention and of the group norm, against differences, the pairwise
form and closed forms (CPU)."""
import numpy as np
import pytest

from oracle import linear as orc


def inputs(B=2, L=9, H=4, Hk=2, K=3, V=5, seed=0, decay="token"):
    rng = np.random.default_rng(seed)
    q, k = rng.standard_normal((2, B, L, Hk, K))
    v, do = rng.standard_normal((2, B, L, H, V))
    S0, dlast = rng.standard_normal((2, B, H, K, V))
    g = -np.exp(rng.standard_normal(H if decay == "fixed" else (B, L, H)))
    if decay == "packed":
        g[rng.random((B, L)) < 0.3] = -np.inf
    return dict(q=q, k=k, v=v, g=g), do, S0, dlast


@pytest.mark.parametrize("decay", ["fixed", "token", "packed"])
def test_forward_is_the_pairwise_form(decay):
    i, _, S0, _ = inputs(decay=decay)
    o, last = orc.linear_fwd(**i, scale=0.3, S0=S0)
    B, L, H, V = i["v"].shape
    a = np.exp(np.broadcast_to(i["g"], (B, L, H)))
    for b in range(B):
        for h in range(H):
            q, k = i["q"][b, :, h // 2], i["k"][b, :, h // 2]
            for t in range(L):
                want = np.prod(a[b, :t + 1, h]) * q[t] @ S0[b, h]
                for j in range(t + 1):
                    want = want + np.prod(a[b, j + 1:t + 1, h]) * (q[t] @ k[j]) * i["v"][b, j, h]
                assert np.allclose(o[b, t, h], 0.3 * want, rtol=0, atol=1e-12)
            end = np.prod(a[b, :, h]) * S0[b, h]
            for j in range(L):
                end = end + np.prod(a[b, j + 1:, h]) * np.outer(k[j], i["v"][b, j, h])
            assert np.allclose(last[b, h], end, rtol=0, atol=1e-12)


@pytest.mark.parametrize("decay", ["fixed", "token", "packed"])
def test_gradients_against_differences(decay):
    i, do, S0, dlast = inputs(L=6, seed=2, decay=decay)
    grads = orc.linear_bwd(**i, do=do, scale=0.7, S0=S0, dlast=dlast)
    if decay == "fixed":
        grads["dlog_decay"] = grads["dlog_decay"].sum((0, 1))

    def loss(**kw):
        a = dict(i, S0=S0)
        a.update(kw)
        o, last = orc.linear_fwd(**a, scale=0.7)
        return (o * do).sum() + (last * dlast).sum()

    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("S0", "dinitial_state")):
        base = dict(i, S0=S0)[name]
        for at in np.ndindex(*base.shape):
            if not np.isfinite(base[at]):
                assert grads[key][at] == 0.0
                continue
            up, dn = base.copy(), base.copy()
            up[at] += 1e-5
            dn[at] -= 1e-5
            want = (loss(**{name: up}) - loss(**{name: dn})) / 2e-5
            # central differences: 1e-10 of the third derivative, 1e-16 / 1e-5 of the loss
            assert abs(grads[key][at] - want) < 1e-7 * (1 + abs(want)), (name, at)


def test_a_start_keeps_out_what_is_not_finite():
    i, _, S0, _ = inputs(decay="token")
    i["v"][:, 2] = np.inf
    S0[:] = np.nan
    i["g"][:, 4] = -np.inf
    o, last = orc.linear_fwd(**i, S0=S0)
    assert not np.isfinite(o[:, :4]).any() and np.isfinite(o[:, 4:]).all() and np.isfinite(last).all()


def test_step_continues_the_sequence():
    i, _, S0, _ = inputs(decay="packed")
    o, last = orc.linear_fwd(**i, S0=S0)
    S = S0
    for t in range(i["v"].shape[1]):
        y, S = orc.linear_step(i["q"][:, t], i["k"][:, t], i["v"][:, t], i["g"][:, t], S)
        assert np.allclose(y, o[:, t], rtol=0, atol=1e-13)
    assert np.allclose(S, last, rtol=0, atol=1e-13)


@pytest.mark.parametrize("width", [1, 2, 3, 7])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_norm_gradients_against_differences(width, gate, silu):
    rng = np.random.default_rng(width)
    C = 2 * width
    p = dict(x=rng.standard_normal((3, C)), weight=rng.standard_normal(C), bias=rng.standard_normal(C))
    if gate:
        p["z"] = rng.standard_normal((3, C))
    dy = rng.standard_normal((3, C))
    grads = orc.group_norm(groups=2, eps=0.1, silu=silu, dy=dy, **p)
    for name in p:
        for at in np.ndindex(*p[name].shape):
            side = []
            for d in (1e-5, -1e-5):
                a = p[name].copy()
                a[at] += d
                side.append((orc.group_norm(groups=2, eps=0.1, silu=silu, **dict(p, **{name: a})) * dy).sum())
            want = (side[0] - side[1]) / 2e-5
            assert abs(grads["d" + name][at] - want) < 1e-7 * (1 + abs(want)), (name, at)


def test_norm_closed_forms():
    y = orc.group_norm(np.array([[1.0, -1.0, 3.0, 3.0]]), 2, eps=1e-30, silu=False)
    assert np.allclose(y, [[1, -1, 0, 0]], rtol=0, atol=1e-12)
    y = orc.group_norm(np.array([[1.0, -1.0]]), 1, z=np.array([[0.0, 2.0]]), eps=1e-30)
    assert np.allclose(y, [[0, -2 / (1 + np.exp(-2.0))]], rtol=0, atol=1e-12)
