"""The gradient of linear attention's decays on the GPU: its error at weak, strong and mixed decays, and what is not
finite in it.  Bounds in linear_bounds.py."""
import numpy as np
import pytest

from oracle import linear as orc
from tests import linear_bounds as bounds
from tests import test_linear_gpu as lin
from tests.test_oracle_linear_decay import with_decay

pytestmark = pytest.mark.gpu

dev, host = lin.dev, lin.host

#        one chunk; two; heads that share; segments and spans (a last one of one chunk, of one token); widths apart; sequences
#        that are not split
SIZES = [(2, 40, 2, 1, 24, 40), (1, 130, 2, 2, 16, 24), (2, 513, 4, 2, 64, 64), (1, 1500, 2, 1, 64, 130), (1, 577, 1, 1, 256, 256),
         (1, 330, 2, 1, 200, 20), (1, 330, 1, 1, 20, 200), (1, 700, 2, 2, 37, 83), (1, 500, 344, 344, 4, 4), (1, 520, 344, 172, 4, 5)]


def cast(i, io):
    return {k: lin.bf(v, io) if k in ("q", "k", "v", "do") else v for k, v in i.items()}


def check(got, i, size, io, S0, dlast, what, more=0.0):
    ref, bound = bounds.decay_bound(i, size, io, S0, dlast)
    bound = bound + more
    got = host(got)
    if i["g"].ndim == 1:
        ref, bound = ref.sum((0, 1)), bound.sum((0, 1))
        lin.near(got, ref, bound + 2.0 ** -24 * np.abs(ref), what)
        return
    lin.near(got, ref, bound, what)
    norm = bounds.norms(got - ref, ref)[np.abs(ref).max(1) > 1e-20]
    assert norm.size == 0 or norm.max() <= bounds.NORM, (what, norm.max())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["fixed", "token", "packed", "fast", -0.02, -2.0, -5.0, -10.0, -20.0, "mixed"])
@pytest.mark.parametrize("size", SIZES)
def test_weak_and_strong_decays(size, decay, io):
    i = cast(with_decay(size, decay, seed=sum(size)), io)
    for ends in (True, False):
        d = lin.backward(i, io, S0=ends, dlast=ends)
        check(d["dlog_decay"], i, size, io, ends, ends, "%s %s ends %s" % (size, decay, ends))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("S0,dlast", [(True, False), (False, True)])
@pytest.mark.parametrize("size", [(2, 40, 2, 1, 24, 40), (1, 600, 3, 1, 32, 16)])
def test_one_end(size, S0, dlast, io):
    for decay in ("token", "mixed"):
        i = cast(with_decay(size, decay, seed=5), io)
        check(lin.backward(i, io, S0=S0, dlast=dlast)["dlog_decay"], i, size, io, S0, dlast, decay)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "mixed", "packed"])
@pytest.mark.parametrize("size", [(1, 700, 4, 2, 64, 64), (1, 330, 2, 2, 128, 128), (3, 64, 2, 1, 40, 16), (1, 330, 2, 1, 20, 200)])
def test_other_gradients_are_the_same_without_it(size, decay, io):
    t = lin._torch()
    i = cast(with_decay(size, decay, seed=6), io)
    a, b = lin.backward(i, io), lin.backward(i, io, decay_grad=False)
    assert all(t.equal(a[k], b[k]) for k in ("dq", "dk", "dv", "dinitial_state"))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["v", "k", "q", "do", "q, then v", "do, then k", "v of a chunk's first", "do of a chunk's last"])
@pytest.mark.parametrize("size", [(1, 900, 2, 1, 64, 64), (2, 150, 2, 2, 32, 48), (1, 450, 344, 344, 4, 4), (1, 300, 1, 1, 20, 200)])
def test_what_is_not_finite(size, where, io):
    """dlog_decay_t has the keys and rows of v before t and the queries and rows of do from t on: with one that is not finite it
    is finite where its definition is, and what it is without the others."""
    B, L, H, Hk, K, V = size
    i = cast(with_decay(size, "token", seed=7), io)
    i["g"][:, 20] = i["g"][:, L - 10] = -np.inf
    at = {"v of a chunk's first": 128, "do of a chunk's last": 127}.get(where, 70)
    bad = {n: at for n in (("v",) if where[0] == "v" else ("do",) if where[:2] == "do" else (where[0],))}
    if "then" in where:
        bad[where[-1]] = at + 25
    clean = dict(i, **{n: i[n].copy() for n in bad})
    i = dict(i, **{n: i[n].copy() for n in bad})
    value = {"v": np.inf, "k": -np.inf, "q": np.nan, "do": np.inf}
    for n, t in bad.items():
        i[n][0, t] = value[n]
        clean[n][0, t] = 0.0
    got = host(lin.backward(i, io)["dlog_decay"])
    with np.errstate(invalid="ignore", over="ignore"):
        want = orc.linear_bwd(i["q"], i["k"], i["v"], i["g"], i["do"], i["scale"], i["S0"], i["dlast"])["dlog_decay"]
    fine = np.isfinite(want) | np.isinf(i["g"])               # (zero where the state starts anew)
    assert not fine.all()
    assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
    ref, bound = bounds.decay_bound(clean, size, io)
    # (spans with it have products of their own: what is finite has the bound of what passes it)
    lin.near(np.where(fine, got, 0.0), np.where(fine, ref, 0.0), bound, where)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("total", [-60.0, -95.0, -101.0])
def test_what_passes_a_whole_chunk_alone(total, io):
    """A chunk without keys and queries: what passes its tokens is the state before it, large, and the gradient behind it, by decays
    that add up to e^total.  A product of decays that fp32 holds as a subnormal number is off by half of 2^-149 at most,
    however small it is, and so is a second one that it meets (the chunk's and a token's): an addend by 2^-149 of what it is without
    decays."""
    size = (1, 192, 2, 2, 16, 24)
    i = cast(with_decay(size, "fixed", seed=9), io)
    for decay in ("even", "one"):
        g = np.full((1, 192, 2), -0.01, np.float32)
        g[:, 64:128] = total / 64 if decay == "even" else -0.01
        if decay == "one":
            g[:, 100] = total + 0.63
        j = dict(i, g=g, S0=(1e15 * i["S0"]).astype(np.float32), dlast=(1e15 * i["dlast"]).astype(np.float32))
        for n in ("q", "k"):
            j[n] = i[n].copy()
            j[n][:, 64:128] = 0.0
        without = bounds.parts(dict(bounds.absolute(j), g=np.zeros_like(g)), size, io)["dlog_decay"]
        check(lin.backward(j, io)["dlog_decay"], j, size, io, True, True, "%s %s" % (total, decay), 2.0 ** -149 * without)
        if decay == "one":
            # (the span has products of its own; in the other, what is 512 tokens behind has its share in the error: the bound's)
            got, ref = host(lin.backward(j, io)["dlog_decay"])[:, 70:120], bounds.parts(j, size, io)["dlog_decay"][:, 70:120]
            assert np.all(np.abs(got / ref - 1) < 1e-4), (got[0, 0], ref[0, 0])


def test_states_kept_far_apart():
    """64 rows of the same sequence, whose kept states take more than 2^31 values: every row's gradients are the first's."""
    import selective_state_space_s6_amd as ss
    t = lin._torch()
    B, L, H, K, V = 64, 4160, 32, 128, 128
    gen = t.Generator(device="cuda").manual_seed(1)
    new = lambda *s: t.randn(*s, device="cuda", generator=gen)                            # noqa: E731
    q, k, v, do = (new(1, L, H, 128).bfloat16().expand(B, L, H, 128) for _ in range(4))
    g = -0.1 * t.rand(1, L, H, device="cuda", generator=gen)
    g[:, 1000::1500] = -6.0                                   # (some spans have products of their own)
    g[:, 2000] = -float("inf")
    dlast = new(1, H, K, V).expand(B, H, K, V).contiguous()
    d = ss.linear_attention_bwd(q, k, v, g.expand(B, L, H), do=do, scale=K ** -0.5, dlast_state=dlast)
    for name in ("dlog_decay", "dq", "dk", "dv"):
        for row in (1, 31, 62, 63):
            assert t.equal(d[name][row], d[name][0]), (name, row)
    assert t.isfinite(d["dlog_decay"]).all() and (d["dlog_decay"][:, 2000] == 0).all()
    # and the first row's, alone in segments, up to rounding: 2^-8 of dq and dk, NORM of the decays'
    one = ss.linear_attention_bwd(q[:1], k[:1], v[:1], g, do=do[:1], scale=K ** -0.5, dlast_state=dlast[:1])
    a, b = host(d["dlog_decay"][:1]), host(one["dlog_decay"])
    assert bounds.norms(a - b, b).max() <= 2 * bounds.NORM


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name,at", [("k", 520), ("q", 500), ("k", 512), ("q", 511), ("v", 520), ("do", 500)])
@pytest.mark.parametrize("size", [(1, 800, 2, 2, 64, 48), (1, 700, 344, 344, 20, 4), (2, 1100, 2, 1, 128, 130)])
def test_one_channel_that_is_not_finite_beside_a_span_s_end(size, name, at, io):
    """Where the walks keep a state, a chunk of which one channel's wavefront alone is not finite: what the others keep is the
    state before the chunk."""
    B, L, H, Hk, K, V = size
    i = cast(with_decay(size, "token", seed=11), io)
    clean = dict(i, **{name: i[name].copy()})
    i = dict(i, **{name: i[name].copy()})
    i[name][0, at, 0, 3], clean[name][0, at, 0, 3] = np.inf, 0.0
    got = host(lin.backward(i, io)["dlog_decay"])
    with np.errstate(invalid="ignore", over="ignore"):
        fine = np.isfinite(orc.linear_bwd(i["q"], i["k"], i["v"], i["g"], i["do"], i["scale"], i["S0"], i["dlast"])["dlog_decay"])
    assert not fine.all() and np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
    ref, bound = bounds.decay_bound(clean, size, io)
    lin.near(np.where(fine, got, 0.0), np.where(fine, ref, 0.0), bound, name)
