"""What linear attention keeps of its sums, against its 64-bit statement: the bits of what meets the matrix
cores, and the range of the states.

Tolerances as in test_linear_gpu.py, where a pair or a state in two bf16 parts is off by at most 2^-17 of
itself: the first part leaves at most 2^-8 of its power of two, whose own rounding is 2^-9 of that."""
import numpy as np
import pytest

from oracle import linear as orc
from tests import test_linear_gpu as lin

pytestmark = pytest.mark.gpu

dev, host, inputs = lin.dev, lin.host, lin.inputs
TWO_PARTS = 2.0 ** -17


@pytest.mark.parametrize("decay", ["fixed", "token", "packed", "grow"])
@pytest.mark.parametrize("size", lin.SIZES + [(1, 1100, 4, 1, 64, 64), (2, 705, 4, 2, 128, 32), (1, 900, 2, 2, 16, 256)])
def test_bf16_results_are_rounded_once(size, decay):
    """2^-8 of the result, its own rounding, and 16 bits of what adds up to it: not 8 bits of each pair."""
    i = inputs(size, "bf16", seed=sum(size) + 2, decay=decay)
    n, _, out = lin.units(size, "bf16")
    args = lambda j: tuple(j[a] for a in "qkvg")                                          # noqa: E731
    a = lin.absolute(i)
    (ro, _), (mo, _) = (orc.linear_fwd(*args(j), i["scale"], j["S0"]) for j in (i, a))
    o, _ = lin.forward(i, "bf16")
    lin.near(o, ro, out * np.abs(ro) + (n + 2 * TWO_PARTS) * mo, "o")
    ref, mag = (orc.linear_bwd(*args(j), j["do"], i["scale"], j["S0"], j["dlast"]) for j in (i, a))
    for decay_grad in (True, False):
        d = lin.backward(i, "bf16", decay_grad=decay_grad)
        for k in ("dq", "dk", "dv"):
            more = size[2] // size[3] * 2.0 ** -24
            lin.near(d[k], ref[k], out * np.abs(ref[k]) + (n + more + 2 * TWO_PARTS) * mag[k], "%s, decay_grad %s" % (k, decay_grad))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("at", ["the chunk's last token", "the sequence's last token", "both directions"])
@pytest.mark.parametrize("size", [(1, 64, 2, 2, 16, 16), (2, 200, 2, 1, 64, 64), (1, 200, 2, 2, 128, 128), (1, 1500, 2, 1, 64, 130),
                                  (1, 200, 1, 1, 256, 256)])
def test_states_up_to_the_largest_value(size, at, io):
    """States of 3e34 and more behind tokens whose decays add up to 2^-14 and less: within fp32, and kept."""
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=41)
    i["g"] = np.full((B, L, H), -0.15, np.float32)
    token = L - 1 if at == "the sequence's last token" else 63
    i["k"][:, token, :, 3] = lin.bf(1.0e17, io)
    i["v"][:, token, :, 5] = lin.bf(3.0e17, io)
    if at == "both directions":
        i["q"][:, min(64, L - 1), :, 2] = lin.bf(1.0e17, io)
        i["do"][:, min(64, L - 1), :, 7] = lin.bf(3.0e17, io)
        if L == 64:
            i["k"][:, 63] = i["v"][:, 63] = 0.0                # (the two would meet beyond the largest value)
        i["S0"][:, :, 2, 7] = i["S0"][:, :, 3, 5] = 0.0
        i["k"][:, :, :, 2] = i["v"][:, :, :, 7] = 0.0
    o, last = lin.forward(i, io)
    lin.check_forward(i, size, io, o, last)
    if at == "both directions":
        lin.check_backward(i, size, io, lin.backward(i, io))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1500, 2, 1, 64, 64), (1, 1100, 1, 1, 128, 130)])
def test_segments_that_grow_beyond_the_range(size, io):
    """Decays of e per token over a segment and more: a state of zeros stays one, and what is finite behind it."""
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=43)
    i["g"][:, :400] = 1.0
    i["k"][:, :400] = 0.0
    o, last = lin.forward(i, io, S0=False)
    lin.check_forward(i, size, io, o, last, S0=False)
    i = inputs(size, io, seed=44)
    i["g"][:, -400:] = 1.0
    i["do"][:, -400:] = 0.0
    d = lin.backward(i, io, dlast=False)
    n, mixed, out = lin.units(size, io)
    ref, mag = (orc.linear_bwd(*(j[a] for a in ("q", "k", "v", "g", "do")), i["scale"], j["S0"]) for j in (i, lin.absolute(i)))
    for k in ("dk", "dv", "dinitial_state"):
        lin.near(d[k], ref[k], out * np.abs(ref[k]) + (mixed + H / Hk * 2.0 ** -24) * mag[k], k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 150, 2, 1, 64, 64), (1, 1500, 2, 1, 64, 64), (2, 200, 1, 1, 256, 200)])
def test_large_states_that_decay(size, io):
    """A state of 1e36 whose decays leave fp32 is nothing, in a chunk and over segments.  Without keys o is q S0 by a
    factor.  Where it is subnormal its roundings are half of 2^-149 each, however small it is: that of the decay since the
    chunk's start, which the scale multiplies, that of the two's product, and as much again for the chunks before: together
    2^-149 (1 + scale) of what q S0 sums up."""
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=45)
    i["k"][:] = 0.0
    i["g"][:] = -2.0
    i["S0"] = (1e36 * np.sign(i["S0"])).astype(np.float32)
    o, last = lin.forward(i, io)
    (ro, rl), (mo, ml) = (orc.linear_fwd(*(j[a] for a in "qkvg"), i["scale"], j["S0"]) for j in (i, lin.absolute(i)))
    n, _, out = lin.units(size, io)
    whole = np.repeat(np.abs(i["q"]).sum(-1), H // Hk, 2)[..., None] * 1e36
    lin.near(o, ro, out * np.abs(ro) + (n + 2.0 ** -17) * mo + 2.0 ** -149 * (1 + i["scale"]) * whole, "o")
    lin.near(last, rl, n * ml + 2.0 ** -149 * 1e36, "last_state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 450, 4, 2, 32, 48), (1, 1500, 2, 1, 64, 130), (1, 320, 300, 100, 20, 64)])
def test_chunks_behind_what_is_not_finite(size, io):
    """A value that is not finite ends with its document in the same chunk: from the next chunk on, which starts anew, the same
    bits as without it, walked by chunks and not token by token."""
    t = lin._torch()
    B, L, H, Hk, K, V = size
    i = inputs(size, io, seed=47)
    i["g"][:, 64] = i["g"][:, 70] = i["g"][:, 110] = i["g"][:, 128] = -np.inf
    (o, last), grads = lin.forward(i, io), lin.backward(i, io)
    for name in ("q", "k", "v", "do"):
        j = dict(i, **{name: i[name].copy()})
        j[name][0, 90] = np.inf
        (o2, last2), g2 = lin.forward(j, io), lin.backward(j, io)
        if name != "do":
            assert not t.isfinite(o2[0, 70:110]).all() and t.isfinite(o2[0, :70]).all() and t.isfinite(o2[0, 110:]).all()
        assert t.equal(o2[:, 128:], o[:, 128:]) and t.equal(last2, last) and t.equal(o2[:, :64], o[:, :64]), name
        for k in ("dq", "dk", "dv"):
            assert t.equal(g2[k][:, 128:], grads[k][:, 128:]) and t.equal(g2[k][:, :64], grads[k][:, :64]), (name, k)
        assert t.equal(g2["dinitial_state"], grads["dinitial_state"]), name


@pytest.mark.parametrize("log_decay", [-88.0, -103.2, -103.5, -103.9, -103.97, -103.98, -np.inf])
def test_a_step_keeps_an_infinite_state_as_the_walk_does(log_decay):
    """Decays down to 2^-150 keep an infinity, and hold what is finite to half of 2^-149 of it; below it the state starts anew."""
    import selective_state_space_s6_amd as ss
    t = lin._torch()
    ones = lambda *s: t.ones(*s, device="cuda")                                           # noqa: E731
    q, v, g = ones(1, 1, 4), ones(1, 1, 8), t.tensor([log_decay], device="cuda")
    for value in (np.inf, 1e38):
        state = t.full((1, 1, 4, 8), value, device="cuda")
        o2, last = ss.linear_attention_fwd(q[:, None], q[:, None], v[:, None], g, initial_state=state, return_last_state=True)
        o = ss.linear_attention_step(q, q, v, g, state=state)
        anew = log_decay * np.log2(np.e) < -150.0
        for got, each in ((o, 4.0), (o2, 4.0), (state, 1.0), (last, 1.0)):
            want = each * (1.0 + (0.0 if anew else np.exp(log_decay) * value))
            if np.isinf(want):
                assert t.isposinf(got).all()
            else:                                             # (2^-22 of the decay, and the sum's and o's roundings)
                assert np.all(np.abs(host(got) - want) <= want * 2.0 ** -20 + each * 2.0 ** -149 * value)
