"""The sizes that linear attention takes, as include/selscan.h gives them (no GPU: each call ends at the pointers'
alignment, which is looked at behind the sizes)."""
import pytest

import selective_state_space_s6_amd as ss
from tests.test_abi_linear import ODD, bwd, fwd, lin, step

UNSUPPORTED, ALIGN = -3, -4


@pytest.mark.parametrize("batch,H,K,V,takes", [
    (1 << 20, 1, 256, 64, True), (1 << 20, 1, 256, 256, False), (1 << 20, 1, 64, 256, False), (1 << 20, 3, 200, 1, True),
    (1 << 21, 1, 256, 65, False), ((1 << 22) - 1, 1, 256, 64, True), (1 << 22, 1, 1, 1, False), (1 << 11, 1 << 10, 256, 64, True)])
def test_workgroups_of_the_forward_and_the_step(batch, H, K, V, takes):
    """batch * nheads * ceil(dv / 64) below 2^22, whatever dk is."""
    want = ALIGN if takes else UNSUPPORTED
    for io in (ss.SELSCAN_F32, ss.SELSCAN_BF16):
        assert fwd(lin(io, batch, 5, H, H, K, V), q=ODD) == want
        assert step(lin(io, batch, 1, H, H, K, V), q=ODD, slots=batch) == want


@pytest.mark.parametrize("batch,H,K,V,takes", [
    (1 << 20, 1, 256, 64, False), (1 << 20, 1, 64, 256, False), (1 << 20, 1, 128, 192, True), (1 << 20, 1, 192, 64, True),
    ((1 << 22) - 1, 1, 64, 64, True), (1 << 22, 1, 1, 1, False)])
def test_workgroups_of_the_backward(batch, H, K, V, takes):
    """batch * nheads * ceil(max(dk, dv) / 64) below 2^22."""
    assert bwd(lin(ss.SELSCAN_F32, batch, 5, H, H, K, V), q=ODD) == (ALIGN if takes else UNSUPPORTED)


@pytest.mark.parametrize("io,batch,L,H,K,V,takes", [
    (ss.SELSCAN_BF16, 1 << 10, 1 << 21, 1, 64, 64, True), (ss.SELSCAN_BF16, 1 << 11, 1 << 21, 1, 64, 64, False),
    (ss.SELSCAN_BF16, 1 << 11, (1 << 21) - 512, 1, 64, 64, True), (ss.SELSCAN_BF16, 1 << 10, 1 << 21, 1, 65, 1, False), (ss.SELSCAN_BF16, 1365, 1 << 19, 1, 200, 1, True), (ss.SELSCAN_BF16, 1366, 1 << 19, 2, 200, 1, False),
    (ss.SELSCAN_BF16, 1 << 10, 1 << 21, 1, 200, 1, False), (ss.SELSCAN_F32, 1 << 8, 1 << 20, 1, 20, 129, True),
    (ss.SELSCAN_F32, 1 << 8, (1 << 21) + 1, 2, 20, 200, False)])
def test_spans_of_the_decays_gradient(io, batch, L, H, K, V, takes):
    """ceil(seqlen / 512) (fp32 wider than 128: 256) batch nheads ceil(max(dk, dv) / 64) below 2^23."""
    d = lin(io, batch, L, H, H, K, V)
    assert bwd(d, q=ODD) == ALIGN                             # without it
    assert bwd(d, q=ODD, dg=0x100000) == (ALIGN if takes else UNSUPPORTED)


@pytest.mark.parametrize("batch,L,takes", [(1 << 18, 1 << 30, True), (1 << 18, (1 << 30) + 1, False), ((1 << 22) - 1, (1 << 31) - 1, False)])
def test_workspaces_whose_size_has_64_bits(batch, L, takes):
    """batch * nheads * seqlen at most 2^48: 2 fp32 values of dk for each where heads share queries and keys."""
    import ctypes
    d = lin(ss.SELSCAN_BF16, batch, L, 1, 1, 256, 64)
    assert bwd(d, q=ODD) == (ALIGN if takes else UNSUPPORTED)
    e = lin(ss.SELSCAN_BF16, batch // 2, L, 2, 1, 256, 64)
    need = ss.lib().linear_attention_bwd_workspace_size(ctypes.byref(e), 0)
    assert need >= 2 * 4 * 256 * L * (batch // 2) * 2 if takes else need == 0
