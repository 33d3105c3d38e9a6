"""The decays' gradient of linear attention by chunks, in 64 bits: against the product that defines it, and that the bound which the
GPU's is held to tells what is left out (CPU)."""
import numpy as np
import pytest

from oracle import linear as orc
from tests import linear_bounds as bounds
from tests.test_linear_gpu import inputs

SIZES = [(1, 130, 2, 1, 16, 24), (2, 200, 2, 2, 8, 8), (1, 600, 1, 1, 64, 64), (1, 333, 1, 1, 200, 20)]
DECAYS = ["fixed", "token", "packed", "fast", -0.02, -2.0, -10.0, -20.0, "mixed"]


def with_decay(size, decay, seed=0):
    B, L, H = size[:3]
    i = inputs(size, "f32", seed=seed, decay=decay if isinstance(decay, str) and decay != "mixed" else "token")
    if decay == "mixed":
        i["g"] = np.where(np.random.default_rng(seed).random((B, L, H)) < 0.1, -12.0, -0.02).astype(np.float32)
    elif not isinstance(decay, str):
        i["g"] = np.full((B, L, H), decay, np.float32)
    return i


@pytest.mark.parametrize("decay", DECAYS + ["all"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("ends", [True, False])
def test_by_chunks_as_defined(size, decay, ends):
    i = with_decay(size, decay)
    p = bounds.parts(i, size, "f32", ends, ends)
    want = orc.linear_bwd(i["q"], i["k"], i["v"], i["g"], i["do"], i["scale"], i["S0"] if ends else None,
                          i["dlast"] if ends else None)["dlog_decay"]
    mag = bounds.parts(bounds.absolute(i), size, "f32", ends, ends)["dlog_decay"]
    assert np.all(np.abs(p["dlog_decay"] - want) <= 1e-9 * mag)     # (exponents of some thousands in 64 bits)
    # what is beside a chunk, from chunk to chunk
    chunk, n = bounds.chunk_of("f32", size[4], size[5]), p["through"].shape[1]
    for c in range(n):
        r = slice(c * chunk, (c + 1) * chunk)
        assert np.allclose(p["beside"][:, c], p["through"][:, c] + p["y"][:, r].sum(1), rtol=1e-9, atol=1e-9 * np.abs(p["y"]).sum(1).max())


@pytest.mark.parametrize("decay", DECAYS)
@pytest.mark.parametrize("size", SIZES)
def test_the_bound_tells_what_is_left_out(size, decay):
    """One addend less, or the sums over all later tokens of q . dq - k . dk with these rounded to fp32, where decays are strong."""
    i = with_decay(size, decay, seed=3)
    ref, bound = bounds.decay_bound(i, size, "f32")
    p = bounds.parts(i, size, "f32")
    chunk, (B, L, H) = bounds.chunk_of("f32", size[4], size[5]), ref.shape
    tell = lambda d: max(np.max(np.abs(d) / (bound + 1e-28)), bounds.norms(d, ref).max() / bounds.NORM)      # noqa: E731
    start = np.broadcast_to(np.asarray(i["g"], np.float64), ref.shape) < -104.0
    per_token = lambda d: np.where(start, 0.0, d)                                          # noqa: E731
    # what one chunk hands to the tokens of another: the state before it, the gradient behind it, both
    for name, of in (("x", 1), ("y", 0)):
        d = np.zeros_like(ref)
        r = slice(of * chunk, (of + 1) * chunk)
        s = p[name][:, r]
        if name == "x":
            d[:, r] = s[:, ::-1].cumsum(1)[:, ::-1]
        else:
            d[:, 1:chunk] = s[:, :-1].cumsum(1)
        # (a token's y has the next chunk's decay too, and among fast ones the chunk may start anew)
        if decay != "fast" and (name == "x" or decay not in (-10.0, -20.0)):
            assert tell(per_token(d)) > 1, name
    d = np.zeros_like(ref)
    d[:, :chunk] = p["through"][:, :1]
    if decay == -0.02:                                        # (of stronger ones less passes a whole chunk)
        assert tell(d) > 1, "through"
    # a pair of neighbours
    d = np.zeros_like(ref)
    qh, kh = (np.repeat(i[n], H // size[3], 2) for n in "qk")
    g = np.broadcast_to(i["g"], ref.shape)
    one = i["scale"] * np.exp(g[:, 1:]) * (qh[:, 1:] * kh[:, :-1]).sum(-1) * (i["do"][:, 1:] * i["v"][:, :-1]).sum(-1)
    one[:, chunk - 1::chunk] = 0.0                            # (not of one chunk)
    at = np.unravel_index(np.abs(one / (bound[:, 1:] + 1e-28)).argmax(), one.shape)
    d[at[0], at[1] + 1, at[2]] = one[at]
    assert tell(per_token(d)) > 1, "pair"
    if decay in (-10.0, -20.0):
        b = orc.linear_bwd(np.repeat(i["q"], H // size[3], 2), np.repeat(i["k"], H // size[3], 2), i["v"], i["g"], i["do"], i["scale"],
                           i["S0"], i["dlast"])
        rows = (qh * b["dq"]).sum(-1).astype(np.float32).astype(np.float64) - (kh * b["dk"]).sum(-1).astype(np.float32)
        _, last = orc.linear_fwd(i["q"], i["k"], i["v"], i["g"], i["scale"], i["S0"])
        d = rows[:, ::-1].cumsum(1)[:, ::-1] + (last * i["dlast"]).sum((-1, -2))[:, None] - ref
        assert tell(per_token(d)) > 1, "sums over all later tokens"
