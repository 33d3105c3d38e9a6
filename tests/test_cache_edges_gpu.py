"""The state cache and the steps on it where large batches, held states and infinite numbers take
them.  Tolerances as in test_cache_gpu."""
import numpy as np
import pytest

from oracle import recurrent as orc
from tests.test_cache_gpu import Beams, _torch, check_step
from tests.test_gated_gpu import bf, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layer", ["s6", "s6 softplus", "ssd"])
def test_held_states_keep_their_codes(layer):
    """1500 tokens whose step size leaves the states as they are, a new seed each.  A state is then
    c s for its code c and scale s, off by half an ulp (2^-24) like the factor that takes it back to
    c: 127 (2^-24 + 2^-24) < 2^-16, within which a code is kept whatever is drawn.  The scale is
    127 s / 127 again, both rounded, and that is s but where 127 s lies halfway between two
    numbers (one scale in 128): it moves by an ulp in the first token and stays from there on."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    gen = t.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: t.randn(*s, generator=gen, device="cuda")                           # noqa: E731
    B, D, N = (2, 192, 128) if layer == "ssd" else (3, 512, 16)
    q, scale = ss.state_cache(B, D // 64, 64, N) if layer == "ssd" else ss.state_cache(B, D, N)
    h = rnd(*q.shape) * t.exp(rnd(*q.shape[:-1], 1))
    seed = t.tensor([1 << 40], dtype=t.int64, device="cuda")
    ss.state_cache_write(h, q, scale, seed=seed)
    written, first = (q.clone(), scale.clone()), None
    A = -1.0 - t.arange(N, device="cuda", dtype=t.float32).expand(D, N).contiguous()
    Bm, Cm, u = rnd(B, N), rnd(B, N), rnd(B, D)
    low = lambda a: a.to(t.bfloat16)                                                     # noqa: E731
    for n in range(1500):
        seed.add_(1)
        if layer == "ssd":
            ss.selective_scan_ssd_step_cached(low(u).view(B, D // 64, 64), low(t.zeros(B, D // 64, device="cuda")), A[0, :D // 64].contiguous(),
                                              low(Bm), low(Cm), q=q, scale=scale, seed=seed)
        elif layer == "s6":
            ss.selective_scan_step_cached(u, t.zeros_like(u), A, Bm, Cm, q=q, scale=scale, seed=seed)
        else:                                                    # softplus(-60) = 9e-27
            ss.selective_scan_step_cached(u, t.full_like(u, -60.0), A, Bm, Cm, q=q, scale=scale, seed=seed, delta_softplus=True)
        if n == 0:
            first = (q.clone(), scale.clone())
    assert t.equal(q, first[0]) and t.equal(scale, first[1])
    assert t.equal(first[0], written[0])
    moved = (first[1] != written[1])
    assert moved.float().mean() < 0.05 and t.all((first[1] - written[1]).abs() <= written[1] * 2.0 ** -23)


def test_stochastic_rounding_follows_where_rounding_to_nearest_stalls():
    """A row's largest value does not decay, so the codes keep their size; the others decay by 0.99 a
    token, less than half a code at first and so for ever when rounded to nearest.  Rounding
    changes a value by less than a scale s a token, with a variance of s^2 / 4 at most, which
    later tokens shrink: after many of them s^2 / 4 / (1 - 0.99^2) = (3.55 s)^2 for a value, and
    the mean of 65536 rows is within six of its deviations, 0.083 s, of the decay."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N, steps = 16, 4096, 4, 200
    h0 = t.tensor([1.0, 0.3, -0.2, 0.1], device="cuda").expand(B, D, N).contiguous()
    zero, one = t.zeros(B, D, device="cuda"), t.ones(B, N, device="cuda")
    rate = -float(np.log(0.99))
    dt, A = t.ones(B, D, device="cuda"), t.tensor([0.0, -rate, -rate, -rate], device="cuda").expand(D, N).contiguous()
    got = {}
    for name in ("nearest", "seeded"):
        q, scale = ss.state_cache(B, D, N)
        seed = t.tensor([1], dtype=t.int64, device="cuda") if name == "seeded" else None
        ss.state_cache_write(h0, q, scale, seed=seed)
        stored = ss.state_cache_read(q, scale)
        for _ in range(steps):
            if seed is not None:
                seed.add_(1)
            ss.selective_scan_step_cached(zero, dt, A, one, one, q=q, scale=scale, seed=seed)
        back = ss.state_cache_read(q, scale)
        if name == "nearest":
            assert t.equal(back, stored)
        assert t.all((back[..., 0] - 1).abs() <= 2.0 ** -20)
        got[name] = host(back).reshape(-1, N).mean(0)
    true = 0.99 ** (steps * (np.arange(N) > 0)) * host(h0)[0, 0]
    err = {k: np.abs(v - true)[1:] for k, v in got.items()}
    bound = 6 * 0.5 / 127 / np.sqrt(1 - 0.99 ** 2) / np.sqrt(B * D)
    print(err, bound)
    assert np.all(err["seeded"] <= bound) and np.all(err["nearest"] > 20 * bound)


@pytest.mark.parametrize("N", [5, 16, 20, 48])
def test_steps_too_large_for_a_product(N):
    """Zero-order hold of step sizes up to infinity: the coefficient is (e^(dt A) - 1) / A, -1 / A from
    where the exponential is nothing."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    sizes = np.array([np.inf, 3e38, 1e38, 1e30, 2.0 ** 21, 2.0 ** 20, 1e4, 0.01], np.float32)
    B, D = len(sizes), 40
    rng = np.random.default_rng(N)
    b = Beams(B, (D, N), N)
    u, Bm, Cm = (rng.standard_normal(s).astype(np.float32) for s in ((B, D), (B, N), (B, N)))
    A = (-np.exp(rng.uniform(-4, 4, (D, N)))).astype(np.float32)
    delta = sizes[:, None].repeat(D, 1)
    y_ref, h_ref = orc.step(b.h.reshape(B, D, N), u, delta, A, Bm, Cm)
    h_abs = orc.step(np.abs(b.h).reshape(B, D, N), np.abs(u), delta, A, np.abs(Bm), Cm)[1]
    for softplus in (False, True):
        q, scale, y = dev(b.q), dev(b.scale), t.zeros(B, D, device="cuda")
        raw = np.where(delta < 1, np.log(np.expm1(np.minimum(delta.astype(np.float64), 1))), delta).astype(np.float32)
        if softplus:
            y_ref, h_ref = orc.step(b.h.reshape(B, D, N), u, raw, A, Bm, Cm, softplus=True)
        ss.selective_scan_step_cached(dev(u), dev(raw if softplus else delta), dev(A), dev(Bm), dev(Cm), None, None, y, q=q,
                                      scale=scale, read_slots=dev(b.read), write_slots=dev(b.write), delta_softplus=softplus)
        check_step(b, q, scale, y, np.zeros((B, D)), y_ref, h_ref, h_abs, "f32", None, "softplus %d" % softplus)


def ssd_case(B, H, N, seeded, first=0, steps=None):
    """One scalar-decay step of B rows, codes from the `first`-th byte of a buffer on, against the statement."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    rng = np.random.default_rng(N + H + B)
    b = Beams(B, (H, 64, N), H)
    x, z, y0 = (bf(rng.standard_normal((B, H, 64)), "bf16") for _ in range(3))
    Bm, Cm = (bf(rng.standard_normal((B, N)), "bf16") for _ in range(2))
    delta = bf(np.exp(rng.standard_normal((B, H)) - 4), "bf16")
    if steps is not None:
        delta = bf(np.resize(steps, (B, H)), "bf16")
    A = -rng.uniform(0.5, 16, H).astype(np.float32)
    Ds = rng.standard_normal(H * 64).astype(np.float32)
    args = (np.repeat(delta, 64, 1), np.repeat(A, 64)[:, None].repeat(N, 1))
    y_ref, h_ref = orc.step(b.h, x.reshape(B, -1), *args, Bm, Cm, Ds, z.reshape(B, -1))
    h_abs = orc.step(np.abs(b.h), np.abs(x).reshape(B, -1), *args, np.abs(Bm), Cm)[1]
    buf = t.full((b.q.size + first + 64,), 77, dtype=t.int8, device="cuda")
    q = buf[first:first + b.q.size].view(b.q.shape)
    q.copy_(dev(b.q))
    scale, y = dev(b.scale), dev(y0, "bf16")
    seed = 1000 if seeded else None
    ss.selective_scan_ssd_step_cached(dev(x, "bf16"), dev(delta, "bf16"), dev(A), dev(Bm, "bf16"), dev(Cm, "bf16"), dev(Ds),
                                      dev(z, "bf16"), y, q=q, scale=scale, read_slots=dev(b.read), write_slots=dev(b.write),
                                      seed=None if seed is None else t.tensor([seed], dtype=t.int64, device="cuda"))
    check_step(b, q, scale, y, y0.astype(np.float64), y_ref, h_ref, h_abs, "bf16", seed, "%d rows, %d heads" % (B, H))
    assert t.all(buf[:first] == 77) and t.all(buf[first + b.q.size:] == 77)


@pytest.mark.parametrize("seeded", [False, True])
@pytest.mark.parametrize("B,H,N", [(64, 33, 64), (64, 65, 64), (64, 17, 128), (64, 33, 128)])
def test_ssd_step_of_large_batches(B, H, N, seeded):
    """Workgroups that walk 2, 4, 2 and 4 groups of rows; with 33 heads (64 states: 33 groups, 128: 66) and
    with 65 the last workgroup's walk ends behind the last row.  All slots but the written ones are
    compared, so nothing may be stored there."""
    ssd_case(B, H, N, seeded)


@pytest.mark.parametrize("seeded", [False, True])
@pytest.mark.parametrize("first", [1, 4, 8])
@pytest.mark.parametrize("B,H,N", [(3, 2, 64), (64, 33, 128)])
def test_ssd_step_on_a_misaligned_cache(B, H, N, first, seeded):
    ssd_case(B, H, N, seeded, first)


@pytest.mark.parametrize("N", [64, 128])
def test_ssd_steps_too_large_for_a_product(N):
    ssd_case(5, 7, N, True, steps=np.array([np.inf, 3e38, 1e30, 1e4, 0.01, 0.0], np.float32))


def test_a_step_size_for_all_rows_and_shared_inputs():
    """delta [D], and u, B and C of one row expanded over the batch: as written out."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D, N = 7, 70, 16
    gen = t.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: t.randn(*s, generator=gen, device="cuda")                           # noqa: E731
    u, Bm, Cm, delta, A = rnd(1, D), rnd(1, N), rnd(1, N), t.rand(D, generator=gen, device="cuda"), -t.ones(D, N, device="cuda")
    got = []
    for wide in (lambda a, n: a.expand(B, n), lambda a, n: a.expand(B, n).contiguous()):
        q, scale = ss.state_cache(B, D, N)
        ss.state_cache_write(t.arange(B * D * N, device="cuda", dtype=t.float32).view(B, D, N), q, scale)
        d = delta if not got else delta.expand(B, D).contiguous()
        y = ss.selective_scan_step_cached(wide(u, D), d, A, wide(Bm, N), wide(Cm, N), q=q, scale=scale)
        got.append((y, q, scale))
    assert all(t.equal(a, b) for a, b in zip(*got)) and got[0][0].unique(dim=0).shape[0] == B


def test_cached_layers_on_two_streams_and_in_a_graph():
    """Writing, both steps and reading in one graph, replayed on new inputs between eager calls, and as
    eager calls on two other streams at once (a cache of its own each)."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, H, N, D, M = 5, 6, 64, 384, 16
    gen = t.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: t.randn(*s, generator=gen, device="cuda")                           # noqa: E731
    low = lambda *s: rnd(*s).to(t.bfloat16)                                              # noqa: E731
    A, AH = -t.rand(D, M, generator=gen, device="cuda"), -t.rand(H, generator=gen, device="cuda")
    read = t.tensor([4, 3, -1, 4, 0], dtype=t.int32, device="cuda")
    write = t.tensor([5, 6, 7, -1, 8], dtype=t.int32, device="cuda")

    def inputs():
        return [rnd(B, D), 0.1 * t.rand(B, D, generator=gen, device="cuda"), rnd(B, M), rnd(B, M), low(B, H, 64),
                (0.1 * t.rand(B, H, generator=gen, device="cuda")).to(t.bfloat16), low(B, N), low(B, N), rnd(B, D, M), rnd(B, H, 64, N)]

    def caches():
        return ss.state_cache(9, D, M) + ss.state_cache(9, H, 64, N) + (t.ones(1, dtype=t.int64, device="cuda"), t.zeros(B, D, device="cuda"),
                                                                         t.zeros(B, H, 64, device="cuda", dtype=t.bfloat16))

    def once(v, c, stream=None):
        u, d, b1, c1, x, dh, b2, c2, s1, s2 = v
        q1, e1, q2, e2, seed, y1, y2 = c
        kw = dict(read_slots=read, write_slots=write, seed=seed, stream=stream)
        ss.state_cache_write(s1, q1, e1, seed=seed, stream=stream)
        ss.state_cache_write(s2, q2, e2, seed=seed, stream=stream)
        ss.selective_scan_step_cached(u, d, A, b1, c1, None, None, y1, q=q1, scale=e1, **kw)
        ss.selective_scan_ssd_step_cached(x, dh, AH, b2, c2, None, None, y2, q=q2, scale=e2, **kw)
        return [ss.state_cache_read(q1, e1, slots=write, stream=stream), ss.state_cache_read(q2, e2, slots=write, stream=stream), y1, y2]

    v, c = inputs(), caches()
    once(v, c)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out = once(v, c)
    for n in range(4):
        for a, b in zip(v, inputs()):
            a.copy_(b)
        c[4].fill_(n)
        graph.replay()
        t.cuda.synchronize()
        got = [a.clone() for a in out]
        assert all(t.equal(a, b) for a, b in zip(got, once(v, c))), n
    w, e, f = inputs(), caches(), caches()
    alone = [[a.clone() for a in once(i, k)] for i, k in ((v, e), (w, f))]
    one, two = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    for _ in range(3):
        both = [once(v, e, one), once(w, f, two.cuda_stream)]
        t.cuda.synchronize()
        assert all(t.equal(a, b) for p, r in zip(both, alone) for a, b in zip(p, r))
