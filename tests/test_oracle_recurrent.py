"""The 64-bit statements of the gated recurrence and of the state cache, against differences,
closed forms and counts (CPU)."""
import numpy as np
import pytest

from oracle import recurrent as orc


def inputs(B, L, D, seed=0, reset=False):
    rng = np.random.default_rng(seed)
    x, r, g, dy = (rng.standard_normal((B, L, D)) for _ in range(4))
    lam = rng.uniform(-5, 1, D)
    marks = rng.random((B, L)) < 0.3 if reset else None
    return x, r, g, lam, dy, rng.standard_normal((B, D)), rng.standard_normal((B, D)), marks


def test_variance_is_kept():
    """With unit-variance input through an open gate the state's variance stays one."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 60, 1))
    h0 = rng.standard_normal((400, 1))
    y, _ = orc.gated_fwd(x, np.zeros_like(x), np.full_like(x, 40.0), np.array([-2.0]), h0=h0)
    assert abs(y[:, -1].var() - 1.0) < 4 * np.sqrt(2 / 400)   # four deviations of a variance of 400 samples


def test_reset_cuts_the_sequence():
    x, r, g, lam, _, h0, _, _ = inputs(2, 12, 5)
    marks = np.zeros((2, 12), bool)
    marks[:, 7] = True
    y, last = orc.gated_fwd(x, r, g, lam, h0=h0, reset=marks)
    tail, tail_last = orc.gated_fwd(x[:, 8:], r[:, 8:], g[:, 8:], lam, h0=x[:, 7] / (1 + np.exp(-g[:, 7])))
    assert np.allclose(y[:, 8:], tail, rtol=0, atol=1e-14) and np.allclose(last, tail_last, rtol=0, atol=1e-14)


@pytest.mark.parametrize("reset", [False, True])
def test_gradients_against_differences(reset):
    x, r, g, lam, dy, h0, dlast, marks = inputs(2, 9, 3, seed=2, reset=reset)
    grads = orc.gated_bwd(x, r, g, lam, dy, h0=h0, reset=marks, dlast=dlast)

    def loss(**kw):
        a = dict(x=x, r=r, g=g, lam=lam, h0=h0)
        a.update(kw)
        y, last = orc.gated_fwd(a["x"], a["r"], a["g"], a["lam"], h0=a["h0"], reset=marks)
        return (y * dy).sum() + (last * dlast).sum()

    for name, key in (("x", "dx"), ("r", "dr"), ("g", "dg"), ("lam", "dlam"), ("h0", "dinitial_state")):
        base = {"x": x, "r": r, "g": g, "lam": lam, "h0": h0}[name]
        for i in np.ndindex(*base.shape):
            up, dn = base.copy(), base.copy()
            up[i] += 1e-5
            dn[i] -= 1e-5
            fd = (loss(**{name: up}) - loss(**{name: dn})) / 2e-5
            assert abs(fd - grads[key][i]) <= 1e-7 * (1 + abs(fd)), (name, i)


def test_gradients_stay_finite_where_the_decay_is_one():
    x, r, g, lam, dy, h0, dlast, _ = inputs(1, 6, 2, seed=3)
    grads = orc.gated_bwd(x, np.full_like(r, -800.0), g, lam, dy, h0=h0, dlast=dlast)
    assert all(np.all(np.isfinite(v)) for v in grads.values())
    assert np.allclose(grads["dinitial_state"], dlast + dy.sum(1), rtol=0, atol=1e-12)


def test_cache_bits_look_uniform():
    """Counts of the top four bits of 2^18 numbers: each of 16 bins within six deviations; the
    mean of the numbers within six; neighbours, rows and seeds uncorrelated within six."""
    n = 1 << 18
    b = orc.cache_bits(77, 64, 64, 64)
    counts = np.bincount((b >> 12).ravel(), minlength=16)
    assert np.all(np.abs(counts - n / 16) < 6 * np.sqrt(n / 16))
    u = (b + 0.5) / 65536 - 0.5
    dev = 1 / np.sqrt(12)
    assert abs(u.mean()) < 6 * dev / np.sqrt(n)
    other = (orc.cache_bits(78, 64, 64, 64) + 0.5) / 65536 - 0.5
    flat = u.reshape(-1, 64)
    for p, q in ((u[..., :-1], u[..., 1:]), (u[..., :-2], u[..., 2:]), (flat[:-1], flat[1:]), (u, other)):
        assert abs((p * q).mean()) < 6 * dev * dev / np.sqrt(p.size)
    for bit in range(16):
        assert abs(((b >> bit) & 1).mean() - 0.5) < 6 * 0.5 / np.sqrt(n), bit


def test_cache_codes():
    h = np.array([[[1.0, -2.0, 0.3, 0.0], [0.0, 0.0, 0.0, 0.0]]])
    t, scale = orc.cache_code(h)
    assert np.array_equal(np.floor(t[0, 0]), [64, -127, 19, 0]) and scale[0, 0] == 2.0 / 127 and scale[0, 1] == 0
    means = np.mean([np.floor(orc.cache_code(h, seed=s)[0]).clip(-127, 127)[0, 0] for s in range(4000)], 0)
    assert np.all(np.abs(means - h[0, 0] * 63.5) < 6 * 0.5 / np.sqrt(4000))


def test_step_is_one_token_of_the_scan():
    import oracle
    rng = np.random.default_rng(5)
    B, D, N = 2, 3, 4
    u, z = (rng.standard_normal((B, 1, D)).astype(np.float32) for _ in range(2))
    Bm, Cm = (rng.standard_normal((B, 1, N)).astype(np.float32) for _ in range(2))
    delta = rng.uniform(0.01, 0.5, (B, 1, D)).astype(np.float32)
    A = -rng.uniform(0, 3, (D, N)).astype(np.float32)
    A[0, 0] = 0
    Ds = rng.standard_normal(D).astype(np.float32)
    y_ref, h_ref = oracle.fwd(u, delta, A, Bm, Cm, Ds, z)
    y, h = orc.step(np.zeros((B, D, N)), u[:, 0], delta[:, 0], A, Bm[:, 0], Cm[:, 0], Ds, z[:, 0])
    assert np.allclose(y, y_ref[:, 0], rtol=0, atol=1e-12) and np.allclose(h, h_ref, rtol=0, atol=1e-12)
