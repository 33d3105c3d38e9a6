"""The gated linear recurrence where workgroups take several chunks, where decays are strong and where
numbers are infinite.  Tolerances as in test_gated_gpu."""
import numpy as np
import pytest

from oracle import recurrent as orc
from tests.test_gated_gpu import (GTOL, TOL, _torch, backward, bf, check_backward, check_forward, close, dev, forward, host,
                                   inputs)

pytestmark = pytest.mark.gpu


def same_infinities(got, ref, tol, what, signs=True):
    """NaN nowhere, infinities (of the same sign) where the reference has them, the rest close to it."""
    got = host(got)
    assert not np.isnan(ref).any() and not np.isnan(got).any(), what
    assert np.array_equal(np.isinf(got), np.isinf(ref)), what
    if signs:
        assert np.array_equal(got == np.inf, ref == np.inf), what
    fine = np.isfinite(ref)
    close(np.where(fine, got, 0), np.where(fine, ref, 0), tol, what)


def bwd_by_sequences(i, cut):
    """The statement's gradients of rows that a reset at token `cut` (None: nowhere) parts, sequence by
    sequence: no infinity is multiplied by the reset's zero."""
    part = lambda lo, hi: [i[k][:, lo:hi] for k in ("x", "r", "g")] + [i["lam"], i["dy"][:, lo:hi]]       # noqa: E731
    if cut is None:
        return orc.gated_bwd(*part(0, None), h0=i["h0"], dlast=i["dlast"])
    one = orc.gated_bwd(*part(0, cut), h0=i["h0"])
    two = orc.gated_bwd(*part(cut, None), reset=i["reset"][:, cut:], dlast=i["dlast"])
    two["dr"][:, 0] = 0
    return dict({k: np.concatenate([one[k], two[k]], 1) for k in ("dx", "dr", "dg")}, dinitial_state=one["dinitial_state"])


@pytest.mark.filterwarnings("ignore::RuntimeWarning")
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 40, 70), (2, 700, 70), (2, 3001, 71)])
@pytest.mark.parametrize("cut", [False, True])
def test_an_infinity_stays_one(cut, size, io):
    """From the initial state, from an input and from gradients, through decays of which a run's product
    stays in fp32 (channels 3 and 7) and through ones of which it does not (2, 5)."""
    B, L, D = size
    i = inputs(B, L, D, io=io, seed=L)
    i["lam"][[2, 5]] = 2.0
    if cut:
        i["reset"] = np.arange(L)[None].repeat(B, 0) == L - 10
    i["h0"][0, 3], i["h0"][1, 2] = np.inf, -np.inf
    i["x"][1, L // 3, 5], i["x"][0, L // 3, 7] = np.inf, -np.inf
    got, last, marks = forward(i, io)
    y, l = orc.gated_fwd(i["x"], i["r"], i["g"], i["lam"], h0=i["h0"], reset=i["reset"])
    same_infinities(got, y, TOL[io], "y")
    same_infinities(last, l, TOL["f32"], "last_state")
    same_infinities(marks, np.concatenate([i["h0"].astype(np.float64)[:, None], y], 1)[:, :-1:64], TOL["f32"], "checkpoints")
    i["h0"], i["x"] = (np.where(np.isinf(i[k]), 1, i[k]).astype(np.float32) for k in ("h0", "x"))
    _, _, marks = forward(i, io)
    i["dlast"][0, 3], i["dlast"][1, 2] = np.inf, -np.inf
    i["dy"][1, L // 3, 5], i["dy"][0, L // 3, 7] = np.inf, -np.inf
    g = backward(i, io, marks=marks)
    ref = bwd_by_sequences(i, L - 10 if cut else None)
    same_infinities(g["dx"], ref["dx"], GTOL[io], "dx")
    same_infinities(g["dg"], ref["dg"], GTOL[io], "dg")
    same_infinities(g["dr"], ref["dr"], GTOL[io], "dr", signs=False)     # (a difference of like numbers)
    same_infinities(g["dinitial_state"], ref["dinitial_state"], GTOL["f32"], "dinitial_state")
    assert np.array_equal(np.flatnonzero(~np.isfinite(host(g["dlam"]))), [2, 3, 5, 7])


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("lam", [5.0, 30.0])
@pytest.mark.parametrize("size", [(1, 64, 4), (2, 700, 70)])
def test_nothing_is_left_of_a_large_state(size, lam, cut):
    """1e38 through decays of e^-40 and e^-240: from the eighth token on nothing of it is left (a product
    of decays held at the least number of fp32, 2^-149, leaves 1.4e-7)."""
    B, L, D = size
    i = inputs(B, L, D, seed=L)
    i["lam"][:], i["r"][:] = lam, 20.0
    i["h0"][:], i["dlast"][:] = 1e38, -1e38
    if cut:
        i["reset"] = np.arange(L)[None].repeat(B, 0) == L // 2
    y, last, marks = forward(i, "f32")
    y_ref, l_ref = orc.gated_fwd(i["x"], i["r"], i["g"], i["lam"], h0=i["h0"], reset=i["reset"])
    close(y[:, 8:], y_ref[:, 8:], TOL["f32"], "y")
    close(last, l_ref, TOL["f32"], "last_state")
    g = backward(i, "f32", marks=marks)
    ref = orc.gated_bwd(i["x"], i["r"], i["g"], i["lam"], i["dy"], h0=i["h0"], reset=i["reset"], dlast=i["dlast"])
    for k in ("dx", "dg"):
        close(g[k][:, :-8], ref[k][:, :-8], GTOL["f32"], k)


def test_one_token_of_a_time_major_buffer():
    """A token's rows with a token stride past 2^20, which one token does not use (the C entry points)."""
    import ctypes

    import selective_state_space_s6_amd as ss
    t = _torch()
    B, D = 512, 2560
    i = inputs(B, 1, D, seed=5)
    v = {k: dev(i[k]) for k in ("x", "r", "g", "lam", "h0", "dy", "dlast")}
    p, lib, s = (lambda a: a.data_ptr()), ss.lib(), t.cuda.current_stream().cuda_stream       # noqa: E731
    d = ss.GatedDims()
    lib.gated_scan_dims_init(ctypes.byref(d), 0, B, 1, D)
    d.x_sl = d.r_sl = d.g_sl = d.y_sl = B * D
    assert B * D > 1 << 20
    y, last, marks = t.empty_like(v["x"]), t.empty_like(v["h0"]), ss.gated_checkpoints(v["x"])
    assert lib.gated_scan_fwd(p(v["x"]), p(v["r"]), p(v["g"]), p(v["lam"]), None, p(y), p(v["h0"]), p(last), p(marks),
                              ctypes.byref(d), None, 0, s) == 0
    check_forward(i, "f32", (y, last, marks))
    g = {k: t.empty_like(v["x"]) for k in ("dx", "dr", "dg")}
    g.update(dlam=t.empty_like(v["lam"]), dinitial_state=t.empty_like(v["h0"]))
    assert lib.gated_scan_bwd(p(v["x"]), p(v["r"]), p(v["g"]), p(v["lam"]), None, p(v["h0"]), p(marks), p(v["dy"]), p(v["dlast"]),
                              *(p(g[k]) for k in ("dx", "dr", "dg", "dlam", "dinitial_state")), ctypes.byref(d), None, 0, s) == 0
    check_backward(i, "f32", g)
    d.reset_sb = -1
    state = v["h0"].clone()
    y.zero_()
    assert lib.gated_scan_step(p(v["x"]), p(v["r"]), p(v["g"]), p(v["lam"]), p(y), p(state), ctypes.byref(d), s) == 0
    check_forward(i, "f32", (y, state, None))


# Chunks of the forward (fp32, bf16) and of the backward pass: 525, 273 and 525; 1560, 780 and 1560; 516, 260
# and 516, where the 256 workgroups that are resident take a second, a third and more of them.
LARGE = [(3, 1537, 771), (6, 8300, 130), (4, 8193, 1)]


@pytest.mark.parametrize("reset", [None, "some"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", LARGE)
def test_workgroups_that_take_several_chunks(size, io, reset):
    i = inputs(*size, io=io, seed=sum(size), reset=reset)
    got = forward(i, io)
    check_forward(i, io, got, what=str(size))
    check_backward(i, io, backward(i, io, marks=got[2]), what=str(size))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_several_chunks_without_checkpoints(io):
    i = inputs(3, 1537, 770, io=io, seed=1, reset="some")
    check_backward(i, io, backward(i, io))


@pytest.mark.parametrize("reset", [None, "some"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 129, 65), (2, 1000, 70), (3, 257, 130), (3, 1537, 771)])
def test_decays_on_both_sides_of_the_series(size, io, reset):
    """log a between -17 and 0: tokens and channels of one wavefront on both sides of 1/8, from which on
    the decay comes from exp2.  Its argument, off by four ulp, leaves |y| 2^-21 of a, at most 2^-22.5
    of one; m and log a keep their relative errors, so the tolerances of the series hold."""
    i = inputs(*size, io=io, seed=sum(size) + 2, reset=reset)
    i["lam"] = np.random.default_rng(size[2]).uniform(-7, 2, size[2]).astype(np.float32)
    got = forward(i, io)
    check_forward(i, io, got, what=str(size))
    check_backward(i, io, backward(i, io, marks=got[2]), what=str(size))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_windows_of_one_buffer_and_shared_marks(io):
    """Rows that overlap (a window of D elements at every second one), a batch that shares r, and reset
    marks of one sequence expanded over the batch."""
    import selective_state_space_s6_amd as ss
    t = _torch()
    B, L, D = 3, 200, 37
    i = inputs(B, L, D, io=io, seed=6, reset="some")
    flat = dev(bf(np.random.default_rng(1).standard_normal(B * 3 * L + D), io), io)
    x = flat.as_strided((B, L, D), (3 * L, 2, 1))
    i["x"] = host(x)
    i["r"] = i["r"][:1].repeat(B, 0)
    i["reset"] = i["reset"][:1].repeat(B, 0)
    r, marks = dev(i["r"][:1], io).expand(B, L, D), dev(i["reset"][:1]).expand(B, L)
    g, dy = dev(i["g"], io), dev(i["dy"], io)
    y, last = ss.gated_scan_fwd(x, r, g, dev(i["lam"]), reset=marks, initial_state=dev(i["h0"]), return_last_state=True)
    check_forward(i, io, (y, last, None))
    check_backward(i, io, ss.gated_scan_bwd(x, r, g, dev(i["lam"]), dy=dy, reset=marks.to(t.uint8) * 3, initial_state=dev(i["h0"]),
                                            dlast_state=dev(i["dlast"])))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_captured_step(io):
    import selective_state_space_s6_amd as ss
    t = _torch()
    i = inputs(6, 1, 250, io=io, seed=3)
    v = {k: dev(i[k][:, 0], io) for k in ("x", "r", "g")}
    lam, state, y = dev(i["lam"]), dev(i["h0"]), t.zeros_like(v["x"])
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        ss.gated_scan_step(v["x"], v["r"], v["g"], lam, state=state, y=y)
    for seed in range(3, 7):
        i = inputs(6, 1, 250, io=io, seed=seed)
        for k in v:
            v[k].copy_(dev(i[k][:, 0], io))
        lam.copy_(dev(i["lam"]))
        state.copy_(dev(i["h0"]))
        graph.replay()
        t.cuda.synchronize()
        check_forward(i, io, (y[:, None], state, None))
