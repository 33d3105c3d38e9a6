"""The 8-bit state cache and the decode steps on it, against their 64-bit statement.

A code is the floor of h * 127 / amax + u.  The kernels form that sum in fp32 (up to 128: half a
step is 2^-18) from a state of relative error e, so a code may differ by one from the floor of
the exact sum only where that sum is within 2^-17 + 127 e of a whole number; e is 2^-22 for
states given (the quotient and the product) and 4e-6 for states of a step (an exp2 whose
argument, up to about 10 here, was rounded; the ZOH coefficient; two products).  The scale is
off by e alone.  A step's state is the sum of what is kept and what comes in, each with that
relative error: where the two cancel, its error is e times the sum of their magnitudes, not
of the state itself."""
import numpy as np
import pytest

from oracle import recurrent as orc
from tests.test_gated_gpu import TOL, bf, close, dev, host

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def check_codes(q, scale, h, seed, e, what=""):
    """q, scale (host, [count, rows, row_len] and [count, rows]) against states h."""
    t, s = orc.cache_code(h, seed)
    margin = 2.0 ** -17 + 127 * e
    lo, hi = np.floor(t - margin).clip(-127, 127), np.floor(t + margin).clip(-127, 127)
    assert np.all((q >= lo) & (q <= hi)), (what, np.argwhere((q < lo) | (q > hi))[:4])
    assert np.all(np.abs(scale - s) <= (e + 2.0 ** -23) * s), what
    assert (lo != hi).mean() < 0.01 + 400 * e or h.size < 1000, what


SHAPES = [((3, 1), 3), ((5, 7), 4), ((130, 16), 3), ((33, 64), 2), ((2, 64, 64), 3), ((3, 64, 128), 2), ((1,), 2),
          ((63,), 3), ((64,), 2), ((1001,), 5), ((17, 4), 6), ((9, 33), 2), ((6, 12), 3), ((300, 8), 2)]


@pytest.mark.parametrize("seeded", [False, True])
@pytest.mark.parametrize("shape,count", SHAPES)
def test_write_and_read(shape, count, seeded):
    import selective_state_space_s6_amd as ss
    t = _torch()
    rng = np.random.default_rng(len(shape) + count)
    h = (rng.standard_normal((count,) + shape) * np.exp(rng.standard_normal((count,) + (1,) * len(shape)))).astype(np.float32)
    row_len = 64 if len(shape) == 1 else shape[-1]
    slots_n = 2 * count + 1
    q, scale = ss.state_cache(slots_n, *shape)
    assert not ss.state_cache_read(q, scale).any()
    q.fill_(99)
    scale.fill_(3.0)
    ids = rng.permutation(slots_n)[:count].astype(np.int32)
    seed = t.tensor([-(1 << 62) + 12345], dtype=t.int64, device="cuda") if seeded else None
    ss.state_cache_write(dev(h), q, scale, slots=dev(ids), seed=seed)
    Q, S = q.cpu().numpy(), scale.cpu().numpy().astype(np.float64)
    rest = np.setdiff1d(np.arange(slots_n), ids)
    assert np.all(Q[rest] == 99) and np.all(S[rest] == 3.0)
    flat = h.reshape(count, -1)
    rows = orc.as_rows(flat, row_len)
    codes = orc.as_rows(Q[ids].reshape(count, -1).astype(np.float64), row_len)
    if flat.shape[1] % row_len:                                 # what lies behind the last value is no state
        pad = rows.shape[1] * row_len - flat.shape[1]
        tt, _ = orc.cache_code(rows, int(seed) if seeded else None)
        codes.reshape(count, -1)[:, -pad:] = np.floor(tt).reshape(count, -1)[:, -pad:]
    check_codes(codes, S[ids], rows, int(seed) if seeded else None, 2.0 ** -22, str(shape))
    back = host(ss.state_cache_read(q, scale, slots=dev(ids)))
    exact = orc.as_rows(Q[ids].reshape(count, -1).astype(np.float64), row_len) * S[ids][..., None]
    exact = exact.reshape(count, -1)[:, :flat.shape[1]].reshape(h.shape)
    assert np.array_equal(back, exact.astype(np.float32).astype(np.float64))
    low = ss.state_cache_read(q, scale, slots=dev(ids), dtype=t.bfloat16)
    assert t.equal(low, t.from_numpy(exact.astype(np.float32)).cuda().to(t.bfloat16))
    step = np.repeat(S[ids][..., None], row_len, -1).reshape(count, -1)[:, :flat.shape[1]].reshape(h.shape)
    assert np.all(np.abs(back - h) <= step * ((1.0 if seeded else 0.5) + 1e-3))


def test_rows_that_hold_nothing_or_no_number():
    import selective_state_space_s6_amd as ss
    t = _torch()
    h = np.random.default_rng(0).standard_normal((1, 9, 16)).astype(np.float32)
    h[0, 0] = 0
    h[0, 1] = 1e-40
    h[0, 2] *= np.float32(2.0 ** -101 / np.abs(h[0, 2]).max())
    h[0, 3] *= np.float32(2.0 ** -99 / np.abs(h[0, 3]).max())
    h[0, 4, 5] = np.inf
    h[0, 5, 15] = -np.inf
    h[0, 6, 0] = np.nan
    h[0, 7] *= np.float32(3e38 / np.abs(h[0, 7]).max())
    h[0, 8] = -0.0
    for seed in (None, t.tensor([5], dtype=t.int64, device="cuda")):
        q, scale = ss.state_cache(1, 9, 16)
        ss.state_cache_write(dev(h), q, scale, seed=seed)
        back = host(ss.state_cache_read(q, scale))[0]
        assert not back[[0, 1, 2, 8]].any() and not scale[0, [0, 1, 2, 8]].any() and not q[0, [0, 1, 2, 8]].any()
        assert np.all(np.isnan(back[4:7]))
        for row in (3, 7):
            assert np.all(np.abs(back[row] - h[0, row].astype(np.float64)) <= np.abs(h[0, row]).max() / 127 * 1.001)


def test_ids_outside_the_cache():
    import selective_state_space_s6_amd as ss
    t = _torch()
    h = t.randn(5, 6, 16, device="cuda")
    q, scale = ss.state_cache(4, 6, 16)
    before = q.clone()
    ids = t.tensor([-1, 4, 2, -(1 << 31), (1 << 31) - 1], dtype=t.int32, device="cuda")
    ss.state_cache_write(h, q, scale, slots=ids)
    assert t.equal(q[[0, 1, 3]], before[[0, 1, 3]]) and q[2].any()
    back = ss.state_cache_read(q, scale, slots=ids)
    assert not back[[0, 1, 3, 4]].any() and back[2].any()
    twice = ss.state_cache_read(q, scale, slots=t.tensor([2, 2, 0], dtype=t.int32, device="cuda"))
    assert t.equal(twice[0], twice[1]) and t.equal(twice[0], back[2]) and not twice[2].any()


class Beams:
    """Random cached states, parents (one shared, one of them absent) and slots of their own."""

    def __init__(self, count, shape, seed, pad=True):
        rng = np.random.default_rng(seed)
        n = 2 * count + 3
        self.q = rng.integers(-127, 128, (n,) + shape).astype(np.int8)
        rows = int(np.prod(shape[:-1]))
        self.scale = np.exp(rng.standard_normal((n, rows)) - 4).astype(np.float32)
        perm = rng.permutation(n).astype(np.int32)
        self.read, self.write = perm[:count].copy(), perm[count:2 * count].copy()
        if count > 2:
            self.read[1] = self.read[0]
            self.read[2] = -1
        if count > 3 and pad:
            self.write[-1] = -1
            self.read[-2] = n                                    # not below slots: no slot either
        held = (self.read >= 0) & (self.read < n)
        self.h = self.q[self.read * held].reshape(count, rows, -1).astype(np.float64) * self.scale[self.read * held][..., None]
        self.h[~held] = 0
        self.rows, self.count = rows, count


def check_step(b, q, scale, y, y0, y_ref, h_ref, h_abs, io, seed, what):
    """New codes, scales and y of the written rows; all else as it was."""
    live = b.write >= 0
    Q, S = q.cpu().numpy(), scale.cpu().numpy().astype(np.float64)
    rest = np.setdiff1d(np.arange(len(Q)), b.write[live])
    assert np.array_equal(Q[rest], b.q[rest]) and np.array_equal(S[rest], b.scale[rest].astype(np.float64)), what
    t, s = orc.cache_code(h_ref.reshape(b.count, b.rows, -1), seed)
    e = 4e-6 * h_abs.reshape(b.count, b.rows, -1).max(-1)     # absolute, by rows
    margin = 2.0 ** -17 + np.where(s > 0, e / np.maximum(s, 1e-300), 0)[..., None]
    lo, hi = np.floor(t - margin).clip(-127, 127)[live], np.floor(t + margin).clip(-127, 127)[live]
    codes = Q[b.write[live]].reshape(lo.shape)
    assert np.all((codes >= lo) & (codes <= hi)), (what, np.argwhere((codes < lo) | (codes > hi))[:4])
    assert np.all(np.abs(S[b.write[live]] - s[live]) <= (e / 127 + 2.0 ** -23 * s)[live]), what
    y, y_ref = host(y).reshape(b.count, -1), y_ref.reshape(b.count, -1)
    close(y[live], y_ref[live], TOL[io], what + " y")
    assert np.array_equal(y[~live], y0.reshape(b.count, -1)[~live]), what


@pytest.mark.parametrize("seeded", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 4, 8, 12, 16, 20, 33, 48, 64])
@pytest.mark.parametrize("B,D", [(1, 1), (6, 37), (9, 260)])
def test_step_cached(B, D, N, io, seeded):
    import selective_state_space_s6_amd as ss
    t = _torch()
    rng = np.random.default_rng(N + D)
    b = Beams(B, (D, N), N)
    u, z = (bf(rng.standard_normal((B, D)), io) for _ in range(2))
    Bm, Cm = (bf(rng.standard_normal((B, N)), io) for _ in range(2))
    raw = bf(rng.standard_normal((B, D)) - 4, io)
    bias = rng.standard_normal(D).astype(np.float32)
    A = -(1.0 + np.arange(N, dtype=np.float32))[None].repeat(D, 0)
    A[0, 0] = 0.0
    Ds = rng.standard_normal(D).astype(np.float32)
    y0 = bf(rng.standard_normal((B, D)), io)
    opts = [dict(Dskip=Ds, z=z, softplus=True, bias=bias), dict(euler=True), dict(z=z, bias=np.abs(bias))]
    for n, o in enumerate(opts):
        delta = raw if o.get("softplus") else bf(np.exp(raw), io)
        y_ref, h_ref = orc.step(b.h.reshape(B, D, N), u, delta, A, Bm, Cm, **o)
        mag = {k: v for k, v in o.items() if k not in ("Dskip", "z")}
        h_abs = orc.step(np.abs(b.h).reshape(B, D, N), np.abs(u), delta, A, np.abs(Bm), Cm, **mag)[1]
        q, scale, y = dev(b.q), dev(b.scale), dev(y0, io)
        seed = (3 << 40) + 77 + n if seeded else None
        ss.selective_scan_step_cached(dev(u, io), dev(delta, io), dev(A), dev(Bm, io), dev(Cm, io), dev(o.get("Dskip")),
                                      None if "z" not in o else dev(z, io), y, q=q, scale=scale, read_slots=dev(b.read),
                                      write_slots=dev(b.write), delta_bias=dev(o.get("bias")),
                                      delta_softplus=o.get("softplus", False),
                                      discretization="euler" if o.get("euler") else "zoh",
                                      seed=None if seed is None else t.tensor([seed], dtype=t.int64, device="cuda"))
        check_step(b, q, scale, y, y0.astype(np.float64), y_ref, h_ref, h_abs, io, seed, "option %d" % n)


@pytest.mark.parametrize("seeded", [False, True])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (5, 3), (3, 24), (18, 5)])
def test_ssd_step_cached(B, H, N, seeded):
    import selective_state_space_s6_amd as ss
    t = _torch()
    rng = np.random.default_rng(N + H)
    b = Beams(B, (H, 64, N), H)
    x, z = (bf(rng.standard_normal((B, H, 64)), "bf16") for _ in range(2))
    Bm, Cm = (bf(rng.standard_normal((B, N)), "bf16") for _ in range(2))
    delta = bf(np.exp(rng.standard_normal((B, H)) - 4), "bf16")
    A = -rng.uniform(0.5, 16, H).astype(np.float32)
    A[0] = 0.0
    Ds = rng.standard_normal(H * 64).astype(np.float32)
    y0 = bf(rng.standard_normal((B, H, 64)), "bf16")
    for n, (euler, with_z) in enumerate([(False, True), (True, False)]):
        y_ref, h_ref = orc.step(b.h, x.reshape(B, -1), np.repeat(delta, 64, 1), np.repeat(A, 64)[:, None].repeat(N, 1), Bm, Cm,
                                Ds if with_z else None, z.reshape(B, -1) if with_z else None, euler=euler)
        h_abs = orc.step(np.abs(b.h), np.abs(x).reshape(B, -1), np.repeat(delta, 64, 1),
                         np.repeat(A, 64)[:, None].repeat(N, 1), np.abs(Bm), Cm, euler=euler)[1]
        q, scale, y = dev(b.q), dev(b.scale), dev(y0, "bf16")
        seed = 1000 + n if seeded else None
        ss.selective_scan_ssd_step_cached(dev(x, "bf16"), dev(delta, "bf16"), dev(A), dev(Bm, "bf16"), dev(Cm, "bf16"),
                                          dev(Ds) if with_z else None, dev(z, "bf16") if with_z else None, y, q=q, scale=scale,
                                          read_slots=dev(b.read), write_slots=dev(b.write),
                                          discretization="euler" if euler else "zoh",
                                          seed=None if seed is None else t.tensor([seed], dtype=t.int64, device="cuda"))
        check_step(b, q, scale, y, y0.astype(np.float64), y_ref, h_ref, h_abs, "bf16", seed, "option %d" % n)


def test_in_place_and_strided():
    """No ids: row b in slot b, in place; u, delta, B, C, z and y are blocks of wider rows."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N = 5, 70, 16
    rng = np.random.default_rng(2)
    b = Beams(B, (D, N), 3)
    A = -(1.0 + np.arange(N, dtype=np.float32))[None].repeat(D, 0)
    wide = {k: rng.standard_normal((B, w + 9)).astype(np.float32) for k, w in (("u", D), ("d", D), ("B", N), ("C", N), ("z", D))}
    wide["d"] = np.exp(wide["d"] - 4)
    v = {k: a[:, 3:3 + (N if k in "BC" else D)] for k, a in wide.items()}
    h = b.q[:B].astype(np.float64) * b.scale[:B].astype(np.float64)[..., None]
    y_ref, h_ref = orc.step(h, v["u"], v["d"], A, v["B"], v["C"], z=v["z"])
    h_abs = orc.step(np.abs(h), np.abs(v["u"]), v["d"], A, np.abs(v["B"]), v["C"])[1]
    g = {k: dev(a)[:, 3:3 + (N if k in "BC" else D)] for k, a in wide.items()}
    q, scale, out = dev(b.q), dev(b.scale), t.full((B, D + 4), 5.0, device="cuda")
    ss.selective_scan_step_cached(g["u"], g["d"], dev(A), g["B"], g["C"], None, g["z"], out[:, 1:1 + D], q=q, scale=scale)
    b.write = np.arange(B, dtype=np.int32)
    check_step(b, q, scale, out[:, 1:1 + D], np.zeros((B, D)), y_ref, h_ref, h_abs, "f32", None, "in place")
    assert t.all(out[:, 0] == 5) and t.all(out[:, 1 + D:] == 5)


def test_a_misaligned_cache():
    """A cache that starts at an odd byte of a larger buffer."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N = 4, 40, 16
    b = Beams(B, (D, N), 4)
    rng = np.random.default_rng(1)
    u, delta = rng.standard_normal((B, D)).astype(np.float32), np.full((B, D), 0.02, np.float32)
    Bm, Cm = (rng.standard_normal((B, N)).astype(np.float32) for _ in range(2))
    A = -np.ones((D, N), np.float32)
    y_ref, h_ref = orc.step(b.h.reshape(B, D, N), u, delta, A, Bm, Cm)
    h_abs = orc.step(np.abs(b.h).reshape(B, D, N), np.abs(u), delta, A, np.abs(Bm), Cm)[1]
    buf = t.zeros(b.q.size + 1, dtype=t.int8, device="cuda")
    q = buf[1:].view(b.q.shape)
    q.copy_(dev(b.q))
    scale, y = dev(b.scale), t.zeros(B, D, device="cuda")
    ss.selective_scan_step_cached(dev(u), dev(delta), dev(A), dev(Bm), dev(Cm), None, None, y, q=q, scale=scale,
                                  read_slots=dev(b.read), write_slots=dev(b.write))
    check_step(b, q, scale, y, np.zeros((B, D)), y_ref, h_ref, h_abs, "f32", None, "misaligned")
    back = ss.state_cache_read(q, scale)
    assert t.equal(back, q.float() * scale[..., None])
    h = t.randn(3, D, N, device="cuda")
    ss.state_cache_write(h, q, scale)
    other, oscale = ss.state_cache(3, D, N)
    ss.state_cache_write(h, other, oscale)
    assert t.equal(q[:3], other) and t.equal(scale[:3], oscale) and buf[0] == 0


def test_not_finite_states_in_a_step():
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N = 2, 5, 16
    q, scale = ss.state_cache(2, D, N)
    u = t.ones(B, D, device="cuda")
    u[0, 1] = float("inf")
    u[1, 2] = float("nan")
    one = t.ones(B, N, device="cuda")
    y = ss.selective_scan_step_cached(u, t.full((B, D), 0.1, device="cuda"), -t.ones(D, N, device="cuda"), one, one, q=q,
                                      scale=scale)
    back, bad = ss.state_cache_read(q, scale), t.zeros(B, D, dtype=t.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert t.equal(~t.isfinite(y), bad) and t.equal(t.isnan(back).all(-1), bad) and t.equal(t.isnan(back).any(-1), bad)


@pytest.mark.parametrize("N", [1, 3, 4, 12, 16, 20, 48])
@pytest.mark.parametrize("euler", [False, True])
def test_growing_states(N, euler):
    """Positive exponents from steps and rates of either sign; steps of size 200, at which a rate of
    one would overflow.  All states stay in range, whatever stands behind the last of them."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D = 2, 9
    rng = np.random.default_rng(N)
    b = Beams(B, (D, N), N)
    u, Bm, Cm = (rng.standard_normal(s).astype(np.float32) for s in ((B, D), (B, N), (B, N)))
    delta = np.array([-200.0, 200.0], np.float32)[:, None].repeat(D, 1)
    A = (rng.uniform(-0.01, 0.01, (D, N))).astype(np.float32)
    y_ref, h_ref = orc.step(b.h.reshape(B, D, N), u, delta, A, Bm, Cm, euler=euler)
    h_abs = orc.step(np.abs(b.h).reshape(B, D, N), np.abs(u), np.abs(delta), np.abs(A), np.abs(Bm), Cm, euler=euler)[1]
    q, scale, y = dev(b.q), dev(b.scale), t.zeros(B, D, device="cuda")
    ss.selective_scan_step_cached(dev(u), dev(delta), dev(A), dev(Bm), dev(Cm), None, None, y, q=q, scale=scale,
                                  read_slots=dev(b.read), write_slots=dev(b.write),
                                  discretization="euler" if euler else "zoh")
    check_step(b, q, scale, y, np.zeros((B, D)), y_ref, h_ref, h_abs, "f32", None, "N %d" % N)


def test_states_near_the_largest_number_are_kept():
    """2^127 down to 2^-98 through a step that changes nothing (no input, rate zero)."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    D, N = 226, 4
    h = (t.tensor([1.0, -0.5, 0.25, 0.75], device="cuda") * 2.0 ** t.arange(127.0, 127.0 - D, -1.0, device="cuda",
                                                                            dtype=t.float64)[:, None]).float()[None]
    q, scale = ss.state_cache(1, D, N)
    ss.state_cache_write(h, q, scale)
    zero, one = t.zeros(1, D, device="cuda"), t.ones(1, N, device="cuda")
    for _ in range(2):
        back = ss.state_cache_read(q, scale)
        assert t.all((back.double() - h.double()).abs() <= scale.double()[..., None] * 0.51) and t.all(scale > 0)
        ss.selective_scan_step_cached(zero, zero, t.zeros(D, N, device="cuda"), one, one, q=q, scale=scale)
    q, scale = ss.state_cache(1, 64, 64, 64)
    ss.state_cache_write((h[:, :64, :1, None] * t.ones(64, 64, device="cuda")).contiguous(), q, scale)
    kept = ss.state_cache_read(q, scale)
    bf = lambda *s: t.zeros(*s, dtype=t.bfloat16, device="cuda")                          # noqa: E731
    ss.selective_scan_ssd_step_cached(bf(1, 64, 64), bf(1, 64), t.zeros(64, device="cuda"), bf(1, 64), bf(1, 64), q=q, scale=scale)
    assert t.all((ss.state_cache_read(q, scale).double() - kept.double()).abs() <= kept.double().abs() * 2.0 ** -18)


def test_stochastic_rounding_lets_slow_decays_through():
    """200 tokens without input, decay 0.99 each, in 4096 rows.  Rounded to nearest, values under
    half the largest never move (each token's change is below half a code); with a seed the
    mean follows the decay.  A token adds at most half a scale of deviation to a value, so the
    mean of 4096 rows stays within six times 0.5 scale sqrt(200) / sqrt(4096) of it."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N, steps = 4, 1024, 4, 200
    h0 = t.tensor([1.0, 0.3, -0.2, 0.1], device="cuda").expand(B, D, N).contiguous()
    zero, one = t.zeros(B, D, device="cuda"), t.ones(B, N, device="cuda")
    dt, A = t.full((B, D), -float(np.log(0.99)), device="cuda"), -t.ones(D, N, device="cuda")
    got = {}
    for name in ("nearest", "seeded"):
        q, scale = ss.state_cache(B, D, N)
        seed = t.tensor([1], dtype=t.int64, device="cuda") if name == "seeded" else None
        ss.state_cache_write(h0, q, scale, seed=seed)
        for _ in range(steps):
            if seed is not None:
                seed.add_(1)
            ss.selective_scan_step_cached(zero, dt, A, one, one, q=q, scale=scale, seed=seed)
        got[name] = host(ss.state_cache_read(q, scale)).reshape(-1, N).mean(0)
    true = 0.99 ** steps * host(h0)[0, 0]
    bound = 6 * 0.5 * (1 / 127) * np.sqrt(steps) / np.sqrt(B * D)
    assert np.all(np.abs(got["seeded"] - true) <= bound), (got, true)


def test_captured_decoding_loop():
    """A step and the seed's increment in a graph; each replay is the eager call's."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N = 6, 200, 16
    gen = t.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: t.randn(*s, generator=gen, device="cuda")                           # noqa: E731
    u, delta, Bm, Cm, A = rnd(B, D), t.full((B, D), 0.05, device="cuda"), rnd(B, N), rnd(B, N), -t.ones(D, N, device="cuda")
    q, scale = ss.state_cache(B, D, N)
    seed, y = t.tensor([7], dtype=t.int64, device="cuda"), t.empty(B, D, device="cuda")

    def once():
        ss.selective_scan_step_cached(u, delta, A, Bm, Cm, None, None, y, q=q, scale=scale, seed=seed)
        seed.add_(1)

    once()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        once()
    for _ in range(5):
        u.copy_(rnd(B, D))
        before = (q.clone(), scale.clone(), seed.clone())
        graph.replay()
        t.cuda.synchronize()
        after = (q.clone(), scale.clone(), seed.clone(), y.clone())
        for a, b in zip((q, scale, seed), before):
            a.copy_(b)
        once()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(after, (q, scale, seed, y)))


def test_prefill_decode_and_prefill_again():
    """The operators as a server uses them: a prompt's scan leaves its state in a slot, two beams
    continue it on the cache, one is read back and continues as a prompt.  Against the same
    run on fp32 states: a stored state is off by at most one scale a value, and each later token
    multiplies what it carries by a decay below one."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    L, D, N, steps, more = 100, 96, 16, 3, 40
    gen = t.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: t.randn(*s, generator=gen, device="cuda")                           # noqa: E731
    u, Bm, Cm = rnd(1, L + steps + more, D), rnd(1, L + steps + more, N), rnd(1, L + steps + more, N)
    delta = t.rand(1, L + steps + more, D, generator=gen, device="cuda") * 0.1
    A = -(1.0 + t.arange(N, device="cuda", dtype=t.float32)).expand(D, N).contiguous()
    cut = lambda a, lo, hi: a[:, lo:hi].contiguous()                                     # noqa: E731
    y_ref, _ = ss.selective_scan_fwd(u, delta, A, Bm, Cm)
    _, last = ss.selective_scan_fwd(*(cut(a, 0, L) for a in (u, delta)), A, *(cut(a, 0, L) for a in (Bm, Cm)),
                                    return_last_state=True)
    q, scale = ss.state_cache(6, D, N)
    ids = lambda *v: t.tensor(v, dtype=t.int32, device="cuda")                           # noqa: E731
    seed = t.tensor([11], dtype=t.int64, device="cuda")
    ss.state_cache_write(last, q, scale, slots=ids(5), seed=seed)
    off = scale[5].clone()                                       # [D]: the largest error of a stored value
    sets = [(0, 1), (2, 3)]
    read = ids(5, 5)
    for n in range(steps):
        write = ids(*sets[n % 2])
        seed.add_(1)
        y = ss.selective_scan_step_cached(*(a[:, L + n].expand(2, -1) for a in (u, delta)), A,
                                          *(a[:, L + n].expand(2, -1) for a in (Bm, Cm)), q=q, scale=scale,
                                          read_slots=read, write_slots=write, seed=seed)
        bound = off * Cm[:, L + n].abs().sum() * 1.001 + 1e-4 * y_ref.abs().max()
        assert t.all((y - y_ref[:, L + n]).abs() <= bound)
        off = off + scale[sets[n % 2][1]].maximum(scale[sets[n % 2][0]])
        read = write
    state = ss.state_cache_read(q, scale, slots=read[1:])
    y, _ = ss.selective_scan_fwd(*(cut(a, L + steps, None) for a in (u, delta)), A,
                                 *(cut(a, L + steps, None) for a in (Bm, Cm)), initial_state=state)
    bound = off * Cm[:, L + steps:].abs().sum(-1, keepdim=True) * 1.001 + 1e-4 * y_ref.abs().max()
    assert t.all((y - y_ref[:, L + steps:]).abs() <= bound)


def test_gated_states_in_the_cache():
    """A gated layer's state parked between its prompt and its tokens: off by one scale at most."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, L, D = 3, 50, 150
    gen = t.Generator(device="cuda").manual_seed(4)
    x, r, g = (t.randn(B, L + 4, D, generator=gen, device="cuda") for _ in range(3))
    lam = t.linspace(-7, -3, D, device="cuda")
    y_ref, _ = ss.gated_scan_fwd(x, r, g, lam)
    _, last = ss.gated_scan_fwd(*(a[:, :L] for a in (x, r, g)), lam, return_last_state=True)
    q, scale = ss.state_cache(4, D)
    ids = t.tensor([3, 0, 2], dtype=t.int32, device="cuda")
    ss.state_cache_write(last, q, scale, slots=ids)
    state = ss.state_cache_read(q, scale, slots=ids)
    off = scale[ids.long()].repeat_interleave(64, 1)[:, :D] * 0.501
    assert t.all((state - last).abs() <= off)
    for n in range(4):
        y = ss.gated_scan_step(*(a[:, L + n] for a in (x, r, g)), lam, state=state)
        assert t.all((y - y_ref[:, L + n]).abs() <= off + 1e-4 * y_ref.abs().max())


def test_offsets_past_32_bits():
    """A cache of more than 2^32 codes."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    H, N, slots = 80, 128, 6700
    q, scale = ss.state_cache(slots, H, 64, N)
    assert q.numel() > 1 << 32
    h = t.randn(2, H, 64, N, device="cuda")
    ids = t.tensor([slots - 1, 0], dtype=t.int32, device="cuda")
    ss.state_cache_write(h, q, scale, slots=ids)
    back = ss.state_cache_read(q, scale, slots=ids)
    step = scale[ids.long()].reshape(2, H, 64, 1)
    assert t.all((back - h).abs() <= step * 0.501)
    B = 2
    gen = t.Generator(device="cuda").manual_seed(5)
    bfr = lambda *s: t.randn(*s, generator=gen, device="cuda").to(t.bfloat16)             # noqa: E731
    x, Bm, Cm = bfr(B, H, 64), bfr(B, N), bfr(B, N)
    delta = t.full((B, H), 0.02, device="cuda").to(t.bfloat16)
    A = -t.ones(H, device="cuda")
    y = ss.selective_scan_ssd_step_cached(x, delta, A, Bm, Cm, q=q, scale=scale, read_slots=ids,
                                          write_slots=t.tensor([slots - 2, 1], dtype=t.int32, device="cuda"))
    y_ref, _ = orc.step(host(back).reshape(B, -1, N), host(x).reshape(B, -1), np.repeat(host(delta), 64, 1),
                        np.repeat(host(A), 64)[:, None].repeat(N, 1), host(Bm), host(Cm))
    close(y, y_ref.reshape(B, H, 64), TOL["bf16"], "y")
