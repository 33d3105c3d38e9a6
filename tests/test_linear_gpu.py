"""Linear attention on the GPU against its 64-bit statement.

Tolerances.  ``mag`` is the same formula on magnitudes: the sum of the absolute values of what an
element adds up.  In fp32 each addend passes at most K + V + 64 + L / 16 roundings of 2^-24 (the
contraction over the widths and over a chunk of 64 tokens, one product and sum a chunk) and a
handful for the decays (e^x is off by 2^-23 (1 + |x|), of which an addend keeps at most e^x: below 2^-22),
so it is off by at most n 2^-24 of it with n = K + V + L / 16 + 100.  bf16: the result is rounded, 2^-8 of
it, and the pairs of a chunk are, 2^-8 of mag; the state in two parts is 2^-17 of it off.  States and the
decays' gradient are fp32 in either case; the latter is what remains of the sum over all later tokens of
q . dq - k . dk, whose magnitudes its bound takes.  A product of decays below 2^-126 is not held to
these: each addend is then off by at most 2^-126 of what it is without decays, together by less than
2^-126 times L K V 5^3 (five deviations of each factor) = 1e-38 1500 256^2 125 < 1e-28."""
import numpy as np
import pytest

from oracle import linear as orc

pytestmark = pytest.mark.gpu

#          batch, L, H, Hk, K, V
SIZES = [(1, 1, 1, 1, 1, 1), (2, 2, 2, 1, 3, 5), (1, 63, 2, 2, 16, 16), (2, 64, 4, 2, 64, 64), (1, 65, 3, 3, 40, 72),
         (1, 130, 2, 1, 128, 128), (2, 200, 1, 1, 100, 50), (1, 257, 2, 2, 256, 200), (1, 100, 2, 1, 65, 129),
         (1, 1500, 1, 1, 64, 64), (1, 1100, 3, 1, 128, 64), (1, 600, 1, 1, 256, 256), (1, 700, 2, 2, 20, 130),
         (9, 5, 50, 25, 33, 64)]
UNDERFLOW = 1e-28
DECAYS = ["fixed", "token", "packed", "fast", "all", "grow"]


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
    """Values as the I/O type holds them."""
    t = _torch()
    a = np.asarray(a, np.float32)
    return t.from_numpy(a).to(t.bfloat16).float().numpy() if io == "bf16" else a


def inputs(size, io="f32", seed=0, decay="token"):
    B, L, H, Hk, K, V = size
    rng = np.random.default_rng(seed)
    i = {n: bf(rng.standard_normal((B, L, Hk, K)), io) for n in "qk"}
    i.update({n: bf(rng.standard_normal((B, L, H, V)), io) for n in ("v", "do")})
    fixed = np.log1p(-2.0 ** -rng.uniform(2, 9, H))
    g = {"fixed": lambda: fixed, "token": lambda: fixed * rng.uniform(0, 3, (B, L, H)),
         "packed": lambda: np.where(rng.random((B, L, 1)) < 0.05, -np.inf, fixed * rng.uniform(0, 3, (B, L, H))),
         "fast": lambda: -np.exp(rng.uniform(-3, 5.2, (B, L, H))), "all": lambda: np.full((B, L, H), -np.inf),
         "grow": lambda: rng.uniform(-0.05, 0.02, (B, L, H))}[decay]()
    i["g"] = np.asarray(g, np.float32)
    i["S0"], i["dlast"] = (rng.standard_normal((B, H, K, V)).astype(np.float32) for _ in range(2))
    i["scale"] = K ** -0.5
    return i


def near(got, ref, bound, what):
    got = host(got) if hasattr(got, "detach") else got
    assert got.shape == ref.shape, what
    if ref.size == 0:
        return
    assert np.all(np.isfinite(got)), what
    r = np.abs(got - ref) / (bound + UNDERFLOW)
    print("%s: %.3f of the bound" % (what, r.max()))
    assert r.max() <= 1.0, "%s: %.3g of the bound at %s" % (what, r.max(), np.unravel_index(r.argmax(), r.shape))


def units(size, io):
    B, L, H, Hk, K, V = size
    n = (K + V + L / 16 + 100) * 2.0 ** -24
    return n, (n + 2.0 ** -8 + 2.0 ** -17 if io == "bf16" else n), (2.0 ** -8 if io == "bf16" else 2.0 ** -24)


def absolute(i):
    return {k: (np.abs(v) if k in ("q", "k", "v", "do", "S0", "dlast") and v is not None else v) for k, v in i.items()}


def check_forward(i, size, io, o, last, S0=True, what=""):
    args = ("q", "k", "v", "g")
    run = lambda j: orc.linear_fwd(*(j[a] for a in args), i["scale"], j["S0"] if S0 else None)    # noqa: E731
    (ro, rl), (mo, ml) = run(i), run(absolute(i))
    n, mixed, out = units(size, io)
    near(o, ro, out * np.abs(ro) + mixed * mo, what + " o")
    if last is not None:
        near(last, rl, n * ml, what + " last_state")


def check_backward(i, size, io, d, S0=True, dlast=True, what=""):
    run = lambda j: orc.linear_bwd(j["q"], j["k"], j["v"], j["g"], j["do"], i["scale"],              # noqa: E731
                                   j["S0"] if S0 else None, j["dlast"] if dlast else None)
    ref, mag = run(i), run(absolute(i))
    n, mixed, out = units(size, io)
    share = size[2] // size[3]
    for k in ("dq", "dk", "dv"):
        more = share * 2.0 ** -24 if k != "dv" else 0.0
        near(d[k], ref[k], out * np.abs(ref[k]) + (mixed + more) * mag[k], what + " " + k)
    assert ("dinitial_state" in d) == S0
    if S0:
        near(d["dinitial_state"], ref["dinitial_state"], n * mag["dinitial_state"], what + " dinitial_state")
    if "dlog_decay" in d:
        B, L, H, Hk, K, V = size
        j = absolute(i)
        # each head's own |q| . |dq| + |k| . |dk|: the magnitudes of the heads that share a row, one by one
        one = orc.linear_bwd(np.repeat(j["q"], share, 2), np.repeat(j["k"], share, 2), j["v"], j["g"], j["do"], i["scale"],
                             j["S0"] if S0 else None, j["dlast"] if dlast else None)
        rows = (np.repeat(j["q"], share, 2) * one["dq"]).sum(-1) + (np.repeat(j["k"], share, 2) * one["dk"]).sum(-1)
        later = rows[:, ::-1].cumsum(1)[:, ::-1]
        _, lm = orc.linear_fwd(j["q"], j["k"], j["v"], j["g"], i["scale"], j["S0"] if S0 else None)
        ends = (lm * j["dlast"]).sum((-1, -2))[:, None] if dlast else 0.0
        r, m = ref["dlog_decay"], later + ends
        if i["g"].ndim == 1:
            r, m = r.sum((0, 1)), m.sum((0, 1))
        near(d["dlog_decay"], r, 2 * n * m, what + " dlog_decay")


def forward(i, io, S0=True, **kw):
    import selective_state_space_s6_amd as ss
    return ss.linear_attention_fwd(dev(i["q"], io), dev(i["k"], io), dev(i["v"], io), dev(i["g"]), scale=i["scale"],
                                   initial_state=dev(i["S0"]) if S0 else None, return_last_state=True, **kw)


def backward(i, io, S0=True, dlast=True, **kw):
    import selective_state_space_s6_amd as ss
    return ss.linear_attention_bwd(dev(i["q"], io), dev(i["k"], io), dev(i["v"], io), dev(i["g"]), do=dev(i["do"], io),
                                   scale=i["scale"], initial_state=dev(i["S0"]) if S0 else None,
                                   dlast_state=dev(i["dlast"]) if dlast else None, **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", DECAYS)
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, decay, io):
    i = inputs(size, io, seed=sum(size), decay=decay)
    o, last = forward(i, io)
    check_forward(i, size, io, o, last, what="%s %s" % (size, decay))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", DECAYS)
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, decay, io):
    i = inputs(size, io, seed=sum(size) + 1, decay=decay)
    d = backward(i, io)
    check_backward(i, size, io, d, what="%s %s" % (size, decay))
    if decay in ("packed", "all"):
        assert np.all(host(d["dlog_decay"])[np.isinf(i["g"])] == 0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 70, 2, 2, 24, 40), (1, 1100, 2, 1, 64, 128)])
def test_without_the_optional_arguments(size, io):
    i = inputs(size, io, seed=5)
    o, last = forward(i, io, S0=False)
    check_forward(i, size, io, o, last, S0=False)
    check_backward(i, size, io, backward(i, io, S0=False, dlast=False), S0=False, dlast=False)
    d = backward(i, io, S0=False, dlast=False, decay_grad=False)
    assert "dlog_decay" not in d and "dinitial_state" not in d
    check_backward(i, size, io, d, S0=False, dlast=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1, 1), (3, 1, 4, 2, 64, 64), (2, 1, 3, 3, 33, 50), (5, 1, 2, 1, 256, 256),
                                  (4, 1, 6, 2, 128, 20), (2, 1, 2, 2, 7, 129)])
@pytest.mark.parametrize("per_row", [False, True])
def test_step(size, io, per_row):
    import selective_state_space_s6_amd as ss
    B, _, H, Hk, K, V = size
    i = inputs(size, io, seed=sum(size), decay="packed" if per_row else "fixed")
    g = i["g"][:, 0] if per_row else i["g"]
    t = _torch()
    n, _, out = units(size, io)
    if per_row and B > 1:
        g[1] = -np.inf
    for slots in (False, True):
        states = np.random.default_rng(1).standard_normal((2 * B + 1 if slots else B, H, K, V)).astype(np.float32)
        read = np.arange(B)[::-1] if slots else np.arange(B)
        write = B + np.arange(B) if slots else np.arange(B)
        S = states[read]
        if slots:
            read = read.copy()
            read[0] = [-1, 2 * B + 1, -2 ** 31][B % 3]       # no slot: the zero state
            S[0] = 0
            if B > 2:
                write[2] = -1 if B % 2 else 2 * B + 1        # padding
                read[1] = read[2]
                S[1] = S[2]
        args = [x[:, 0] for x in (i["q"], i["k"], i["v"])]
        ro, rs = orc.linear_step(*args, g, S, i["scale"])
        mo, ms = orc.linear_step(*(np.abs(a) for a in args), g, np.abs(S), i["scale"])
        state, o = dev(states), t.full((B, H, V), 7.0, dtype=t.bfloat16 if io == "bf16" else t.float32, device="cuda")
        ids = dict(read_slots=t.tensor(read, dtype=t.int32).cuda(), write_slots=t.tensor(write, dtype=t.int32).cuda()) if slots else {}
        got = ss.linear_attention_step(*(dev(a, io) for a in args), dev(g), state=state, scale=i["scale"], o=o, **ids)
        assert got is o
        want, bound = states.astype(np.float64), np.zeros(states.shape)
        for b in range(B):
            if 0 <= write[b] < len(states):
                want[write[b]], bound[write[b]] = rs[b], n * ms[b]
            else:
                ro[b], mo[b] = 7.0, 0.0
        near(state, want, bound, "state")
        near(o, ro, out * np.abs(ro) + n * mo, "o")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_run_of_the_layer(io):
    """Prompt, norm and gate, then tokens one by one on the state it left: as the whole sequence; and the
    gradients of the whole as those of its parts chained."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, L, H, Hk, K, V = size = (2, 150, 4, 2, 32, 48)
    i = inputs(size, io, seed=3, decay="token")
    q, k, v, g = dev(i["q"], io), dev(i["k"], io), dev(i["v"], io), dev(i["g"])
    rng = np.random.default_rng(4)
    z = dev(rng.standard_normal((B, L, H * V)), io)
    w = dev(1 + 0.1 * rng.standard_normal(H * V))
    norm = dict(groups=H, weight=w)
    o, last = ss.linear_attention_fwd(q, k, v, g, scale=i["scale"], return_last_state=True)
    y = ss.group_norm_fwd(o.view(B, L, H * V), z=z, **norm)
    m = 90
    o1, state = ss.linear_attention_fwd(q[:, :m], k[:, :m], v[:, :m], g[:, :m], scale=i["scale"], return_last_state=True)
    ys = [ss.group_norm_fwd(o1.view(B, m, H * V), z=z[:, :m], **norm)]
    for s in range(m, L):
        o2 = ss.linear_attention_step(q[:, s], k[:, s], v[:, s], g[:, s], state=state, scale=i["scale"])
        ys.append(ss.group_norm_fwd(o2.view(B, H * V), z=z[:, s], **norm)[:, None])
    n, mixed, out = units(size, io)
    _, ml = orc.linear_fwd(*(absolute(i)[a] for a in "qkvg"), i["scale"])
    near(state, host(last), 2 * n * ml, "state")
    # o of the two is off by twice its bound at most; the norm makes (2 + |xh|) / std of that, |xh| below sqrt(48),
    # and the weight (below 1.5) and the gate (below 5) act on it
    ref = host(y)
    ro, _ = orc.linear_fwd(i["q"], i["k"], i["v"], i["g"], i["scale"])
    mo, _ = orc.linear_fwd(*(absolute(i)[a] for a in "qkvg"), i["scale"])
    std = ro.std(-1, keepdims=True)
    off = 2 * (out * np.abs(ro) + mixed * mo).max(-1, keepdims=True) / std * 9 * 5 * 1.5
    near(t.cat(ys, 1), ref, np.broadcast_to(off, ro.shape).reshape(ref.shape) + 2 * out * np.abs(ref), "y")
    dy = dev(rng.standard_normal((B, L, H * V)), io)
    d = ss.group_norm_bwd(o.view(B, L, H * V), z=z, dy=dy, **norm)
    grads = ss.linear_attention_bwd(q, k, v, g, do=d["dx"].view(B, L, H, V), scale=i["scale"])
    j = dict(i, do=host(d["dx"]).reshape(B, L, H, V))
    check_backward(j, size, io, grads, S0=False, dlast=False, what="chained")
