"""The gated linear recurrence where workgroups take several chunks, where decays are strong and where
numbers are infinite.  Tolerances as in test_gated_gpu."""
import numpy as np
import pytest

from oracle import recurrent as orc
from tests.test_gated_gpu import GTOL, TOL, backward, close, forward, inputs

pytestmark = pytest.mark.gpu


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
