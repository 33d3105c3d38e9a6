"""The group norm's activation over its whole range, and its sums over many rows, on the GPU against 64 bits.

Where a group has no spread, the normalised value is zero and n the bias alone, so y = bias silu(z) is off by the activation's
own roundings: in fp32, in units of 2^-24 of it, 1 for its product with the bias, 1 for t s, 2 for the reciprocal and its step, 1
for 1 + e, 4 for e^-t (the instruction's 2^-23, its correction's rounding, and the rest of the exponent): 9.  The slope s (1 +
t (1 - s)) is off by as many of s (1 + |t| (1 - s)), and 2 for its sum.  s below 2^-126 is zero."""
import numpy as np
import pytest

from tests.test_norm_gpu import dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def act(t):
    """silu, its slope, and the slope's addends' magnitudes."""
    with np.errstate(over="ignore"):
        s, c = 1.0 / (1.0 + np.exp(-t)), 1.0 / (1.0 + np.exp(t))
    return t * s, s * (1.0 + t * c), s * (1.0 + np.abs(t) * c)


def points():
    rng = np.random.default_rng(0)
    edges = [0.0, -0.0, 1e-30, -1e-30, 88.0, -87.3, -88.8, 103.0, -110.0, 1e4, -1e4, 3e38, -3e38, -1.2784645]
    t = np.concatenate([rng.uniform(-100, 100, 3000), rng.uniform(-2, 2, 3000), edges])
    return np.resize(t, 6400).astype(np.float32)


@pytest.mark.parametrize("gate", [True, False])
def test_the_activation_in_fp32(gate):
    import selective_state_space_s6_amd as ss
    t = points().reshape(100, 64)
    T = t.astype(np.float64)
    a, slope, mag = act(T)
    x = dev(np.ones_like(t))
    if gate:
        bias = np.linspace(-3, 3, 64).astype(np.float32)
        y = host(ss.group_norm_fwd(x, None, dev(bias), dev(t), groups=4))
        with np.errstate(over="ignore"):
            big = np.abs(bias * a) < 3e38
        assert np.all(np.abs(y - bias * a)[big] <= (9 * U * np.abs(bias * a) + 2.0 ** -126 * np.abs(bias * T))[big])
        dy = np.random.default_rng(1).standard_normal(t.shape).astype(np.float32)
        d = ss.group_norm_bwd(x, None, dev(bias), dev(t), dy=dev(dy), groups=4)
        assert np.all(np.abs(host(d["dz"]) - dy * bias * slope) <= np.abs(dy * bias) * (12 * U * mag + 2.0 ** -126 * (1 + np.abs(T))))
    else:
        for row in t[:20]:
            y = host(ss.group_norm_fwd(x, None, dev(row), groups=4))
            a, _, _ = act(row.astype(np.float64))
            assert np.all(np.abs(y - a) <= 9 * U * np.abs(a) + 2.0 ** -126 * np.abs(row))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,groups", [(20000, 8, 2), (5000, 256, 2)])
def test_sums_of_one_sign(rows, C, groups, io):
    """dbias of dy = 1 + small: rows of one part are summed in fp32 one after the other, each rounding at most 2^-24 of the
    sum so far, the parts in 64 bits: the rows of a thread times 2^-24, and the activation's share."""
    import selective_state_space_s6_amd as ss
    rng = np.random.default_rng(2)
    x, dy = dev(rng.standard_normal((rows, C)), io), dev(1 + rng.uniform(0, 1, (rows, C)), io)
    w = dev(np.ones(C))
    d = ss.group_norm_bwd(x, w, dev(np.zeros(C)), dy=dy, groups=groups, activation="none")
    want = host(dy).sum(0)
    # (both sizes: workgroups of one part for 32 rows and fewer)
    assert np.all(np.abs(host(d["dbias"]) - want) <= 33 * U * want)
