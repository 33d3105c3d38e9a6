"""Refusals of the gated recurrence and of the state cache, before anything is enqueued (no GPU)."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import selective_state_space_s6_amd as ss

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 0x100000                                # never dereferenced
ODD = 0x100001
HALF = 0x100002


def gated(io=ss.SELSCAN_F32, batch=2, L=10, D=8, **kw):
    d = ss.GatedDims()
    ss.lib().gated_scan_dims_init(ctypes.byref(d), io, batch, L, D)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(d, x=F, r=F, g=F, lam=F, reset=None, y=F, h0=None, last=None, ckpt=None, ws=None, n=0):
    return ss.lib().gated_scan_fwd(x, r, g, lam, reset, y, h0, last, ckpt, ctypes.byref(d) if d else None, ws, n, None)


def bwd(d, x=F, r=F, g=F, lam=F, reset=None, h0=None, ckpt=F, dy=F, dlast=None, dx=F, dr=F, dg=F, dlam=F, dh0=None,
        ws=None, n=0):
    return ss.lib().gated_scan_bwd(x, r, g, lam, reset, h0, ckpt, dy, dlast, dx, dr, dg, dlam, dh0,
                                   ctypes.byref(d) if d else None, ws, n, None)


def step(d, x=F, r=F, g=F, lam=F, y=F, state=F):
    return ss.lib().gated_scan_step(x, r, g, lam, y, state, ctypes.byref(d) if d else None, None)


@pytest.mark.parametrize("cls,name", [(ss.GatedDims, "selscan_gated_dims"), (ss.CacheDims, "selscan_cache_dims")])
def test_struct_layouts(cls, name):
    fields = [f for f, _ in cls._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"selscan.h\"\nint main(void){printf(\"%%zu\\n\", sizeof(%s));\n" % name
    src += "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        vals = [int(v) for v in subprocess.check_output([exe]).split()]
    assert vals == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def test_gated_dims_init():
    d = gated(ss.SELSCAN_BF16, 3, 20, 6)
    assert (d.x_sb, d.x_sl, d.r_sb, d.g_sl, d.y_sb, d.y_sl, d.reset_sb) == (120, 6, 120, 6, 120, 6, 20)
    assert d.decay_c == 8.0 and d.abi_version == ss.SELSCAN_ABI_VERSION
    ss.lib().gated_scan_dims_init(None, 0, 1, 1, 1)


BAD_DIMS = [("batch", -1, -2), ("seqlen", -1, -2), ("dim", 0, -2), ("x_sb", -1, -2), ("x_sl", -1, -2), ("r_sl", -1, -2),
            ("g_sb", -5, -2), ("y_sl", -1, -2), ("reset_sb", -1, -2), ("decay_c", 0.0, -2), ("decay_c", -1.0, -2),
            ("decay_c", float("nan"), -2), ("decay_c", float("inf"), -2), ("io_dtype", 2, -3), ("io_dtype", -1, -3),
            ("abi_version", 1, -7), ("x_sl", (1 << 20) + 1, -3),
            ("g_sl", (1 << 20) + 1, -3), ("batch", 1 << 31, -3), ("seqlen", 1 << 41, -3)]


@pytest.mark.parametrize("field,value,status", BAD_DIMS)
def test_gated_dims_errors(field, value, status):
    d = gated(**{field: value})
    assert fwd(d) == status and bwd(d) == status and step(d) == status
    assert ss.lib().gated_scan_workspace_size(ctypes.byref(d)) == 0
    assert ss.lib().gated_scan_bwd_workspace_size(ctypes.byref(d), 0) == 0


def test_gated_output_rows_must_not_overlap():
    for d in (gated(y_sl=7), gated(y_sb=79)):
        assert fwd(d) == -3
        assert bwd(d, ws=F + 16, n=1 << 40) == -6        # dy is read: its rows may overlap
    assert step(gated(L=1, y_sb=7)) == -3


def test_gated_pointer_errors():
    d = gated()
    assert fwd(None) == bwd(None) == step(None) == -1
    for k in ("x", "r", "g", "lam", "y"):
        assert fwd(d, **{k: None}) == -1, k
    for k in ("x", "r", "g", "lam", "dy", "dx", "dr", "dg", "dlam"):
        assert bwd(d, **{k: None}) == -1, k
    one = gated(L=1)
    for k in ("x", "r", "g", "lam", "y", "state"):
        assert step(one, **{k: None}) == -1, k
    for k in ("x", "r", "g", "lam", "y", "h0", "last", "ckpt"):
        assert fwd(d, **{k: HALF}) == -4, k
    for k in ("x", "r", "g", "lam", "dy", "dx", "dr", "dg", "dlam", "h0", "ckpt", "dlast", "dh0"):
        assert bwd(d, **{k: HALF}) == -4, k
    for k in ("x", "r", "g", "lam", "y", "state"):
        assert step(one, **{k: HALF}) == -4, k
    half = gated(ss.SELSCAN_BF16)
    assert fwd(half, x=ODD) == -4 and bwd(half, dg=ODD) == -4
    assert step(d) == -2                                  # ten tokens are no step


def test_gated_workspace_errors():
    d = gated(L=5000, D=200)
    need = ss.lib().gated_scan_bwd_workspace_size(ctypes.byref(d), 1)
    more = ss.lib().gated_scan_bwd_workspace_size(ctypes.byref(d), 0)
    assert 0 < need < more and more >= need + 4 * 2 * 79 * 200
    assert bwd(d, ws=F, n=need - 1) == -6 and bwd(d, ws=F + 16, n=need) == -6
    assert bwd(d, ckpt=None, ws=F, n=need) == -6
    size = ss.lib().gated_scan_workspace_size(ctypes.byref(d))
    if size:
        assert fwd(d, ws=F, n=size - 1) == -6 and fwd(d, ws=F + 16, n=size) == -6


def test_gated_empty_batch_is_a_no_op():
    assert fwd(gated(batch=0), x=None, r=None, g=None, y=None) == 0
    assert step(gated(batch=0, L=1), x=None, r=None, g=None, y=None, state=None) == 0
    for d in (gated(batch=0), gated(L=0)):
        assert ss.lib().gated_scan_workspace_size(ctypes.byref(d)) == 0
        assert ss.lib().gated_scan_bwd_workspace_size(ctypes.byref(d), 0) == 0


def cache(slots=10, elems=128, row_len=16, **kw):
    return ss.CacheDims(abi_version=ss.SELSCAN_ABI_VERSION, slots=slots, elems=elems, row_len=row_len, **kw)


def cwrite(c, state=F, ids=None, count=4, q=F, scale=F, seed=None):
    return ss.lib().state_cache_write(state, ids, count, q, scale, seed, ctypes.byref(c) if c else None, None)


def cread(c, ids=None, count=4, q=F, scale=F, out=F, dtype=0):
    return ss.lib().state_cache_read(q, scale, ids, count, out, dtype, ctypes.byref(c) if c else None, None)


@pytest.mark.parametrize("field,value,status", [("slots", -1, -2), ("elems", 0, -2), ("row_len", 0, -2), ("row_len", 129, -3),
                                                ("elems", 1 << 31, -3), ("slots", 1 << 31, -3), ("abi_version", 3, -7),
                                                ("slots", 3, -2)])
def test_cache_dims_errors(field, value, status):
    c = cache()
    setattr(c, field, value)
    assert cwrite(c) == status and cread(c) == status


def test_cache_pointer_errors():
    c = cache()
    assert cwrite(None) == cread(None) == -1
    assert cwrite(c, state=None) == cwrite(c, q=None) == cwrite(c, scale=None) == -1
    assert cread(c, q=None) == cread(c, scale=None) == cread(c, out=None) == -1
    assert cwrite(c, state=HALF) == cwrite(c, scale=HALF) == cwrite(c, ids=HALF) == cwrite(c, seed=F + 4) == -4
    assert cread(c, scale=HALF) == cread(c, ids=HALF) == cread(c, out=HALF) == cread(c, out=ODD, dtype=1) == -4
    assert cread(c, dtype=2) == -3
    assert cwrite(c, count=-1) == cread(c, count=-1) == -2
    assert cwrite(c, count=11) == cread(c, count=11) == -2            # 0 .. 10 do not all exist
    assert cwrite(cache(elems=(1 << 31) - 1, row_len=1, slots=10), count=3) == -3
    assert cwrite(c, count=0, state=None) == 0 and cread(c, count=0, out=None) == 0
    assert cwrite(cache(slots=0), ids=F, q=None, scale=None) == 0     # no id names a slot


def s6(d, c, u=F, delta=F, bias=None, A=F, B=F, C=F, Ds=None, z=None, y=F, q=F, scale=F, rd=F, wr=F, seed=None):
    return ss.lib().selective_scan_step_cached(u, delta, bias, A, B, C, Ds, z, y, q, scale, rd, wr, seed,
                                               ctypes.byref(d) if d else None, ctypes.byref(c) if c else None, None)


def test_step_cached_errors():
    d, c = ss.dims_init(ss.SELSCAN_F32, 4, 1, 8, 16), cache()
    assert s6(None, c) == s6(d, None) == -1
    for k in ("u", "delta", "A", "B", "C", "y", "q", "scale"):
        assert s6(d, c, **{k: None}) == -1, k
    for k in ("u", "delta", "bias", "A", "B", "C", "Ds", "z", "y", "scale", "rd", "wr"):
        assert s6(d, c, **{k: HALF}) == -4, k
    assert s6(d, c, seed=F + 4) == -4
    assert s6(ss.dims_init(ss.SELSCAN_F32, 4, 2, 8, 16), c) == -2
    assert s6(d, cache(elems=112)) == -2 and s6(d, cache(row_len=8)) == -2
    assert s6(ss.dims_init(ss.SELSCAN_F32, 4, 1, 8, 16, time_invariant=True), c) == -3
    assert s6(ss.dims_init(ss.SELSCAN_F32, 11, 1, 8, 16), c, rd=None) == -2
    assert s6(ss.dims_init(ss.SELSCAN_F32, 11, 1, 8, 16), c, wr=None) == -2
    assert s6(ss.dims_init(ss.SELSCAN_F32, 0, 1, 8, 16), c, u=None, delta=None, B=None, C=None, y=None) == 0


def ssd(d, c, x=F, delta=F, A=F, B=F, C=F, Ds=None, z=None, y=F, q=F, scale=F, rd=F, wr=F, seed=None):
    return ss.lib().selective_scan_ssd_step_cached(x, delta, A, B, C, Ds, z, y, q, scale, rd, wr, seed,
                                                   ctypes.byref(d) if d else None, ctypes.byref(c) if c else None, None)


def test_ssd_step_cached_errors():
    d, c = ss.ssd_dims(4, 1, 3, 64, 128), cache(elems=3 * 64 * 128, row_len=128)
    assert ssd(None, c) == ssd(d, None) == -1
    for k in ("x", "delta", "A", "B", "C", "y", "q", "scale"):
        assert ssd(d, c, **{k: None}) == -1, k
    for k in ("x", "B", "C", "z", "y"):
        assert ssd(d, c, **{k: F + 8}) == -4, k
    for k in ("A", "Ds", "scale", "rd", "wr"):
        assert ssd(d, c, **{k: HALF}) == -4, k
    assert ssd(d, c, delta=ODD) == -4 and ssd(d, c, seed=F + 4) == -4
    assert ssd(ss.ssd_dims(4, 2, 3, 64, 128), c) == -2
    assert ssd(d, cache(elems=3 * 64 * 64, row_len=64)) == -2
    assert ssd(ss.ssd_dims(4, 1, 3, 32, 128), c) == -3
    assert ssd(ss.ssd_dims(11, 1, 3, 64, 128), c, wr=None) == -2
    assert ssd(ss.ssd_dims(0, 1, 3, 64, 128), c, x=None, delta=None, B=None, C=None, y=None) == 0


def test_the_binding_wants_gpu_tensors():
    import torch
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        ss.gated_scan_fwd(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError):
        ss.gated_scan_bwd(x, x, x, torch.zeros(8), dy=x)
    with pytest.raises(ValueError):
        ss.gated_scan_step(x[0], x[0], x[0], torch.zeros(8), state=x[0])
    with pytest.raises(ValueError):
        ss.gated_scan_fwd(x[0], x[0], x[0], torch.zeros(8))
    q, scale = ss.state_cache(2, 8, 16, device="cpu")
    assert q.shape == (2, 8, 16) and scale.shape == (2, 8)
    assert ss.state_cache(2, 130, device="cpu")[1].shape == (2, 3) and ss.state_cache(2, 3, 64, 128, device="cpu")[1].shape == (2, 192)
    with pytest.raises(ValueError):
        ss.state_cache_write(torch.zeros(2, 8, 16), q, scale)
    with pytest.raises(ValueError):
        ss.state_cache_read(q, scale)
    with pytest.raises(ValueError):
        ss.selective_scan_step_cached(x[0], x[0], torch.zeros(8, 16), x[0], x[0], q=q, scale=scale)
    with pytest.raises(ValueError):
        ss.selective_scan_ssd_step_cached(torch.zeros(1, 2, 64), x[0], x[0], x[0], x[0], q=q, scale=scale)


def test_gated_workspace_of_one_chunk_is_empty():
    for io, chunk in ((ss.SELSCAN_F32, 64), (ss.SELSCAN_BF16, 128)):
        size = lambda n: ss.lib().gated_scan_workspace_size(ctypes.byref(gated(io, L=n, D=200)))       # noqa: E731
        assert size(chunk) == 0 and size(chunk + 1) > 0


def test_one_launch_has_fewer_than_2_32_threads():
    assert fwd(gated(batch=1 << 23)) == step(gated(batch=1 << 22, L=1, D=129)) == -3
    c = cache(elems=1 << 20, row_len=64, slots=1 << 20)
    assert cwrite(c, count=1 << 12) == cread(c, count=1 << 12) == -3


def test_one_token_has_no_token_stride():
    far = dict(x_sl=(1 << 20) + 1, r_sl=1 << 40, g_sl=-1, y_sl=1 << 22)
    d = gated(batch=0, L=1, **far)
    assert fwd(d, x=None, r=None, g=None, y=None) == step(d, x=None, r=None, g=None, y=None, state=None) == 0
    assert step(gated(batch=0, L=1, reset_sb=-1), x=None, r=None, g=None, y=None, state=None) == 0
    d = gated(L=1, **far)
    assert fwd(d, x=None) == bwd(d, dx=None) == step(d, state=None) == -1       # on to the pointers
    assert fwd(gated(L=1, y_sb=7, **far)) == step(gated(L=1, y_sb=7, **far)) == -3
    assert fwd(gated(L=2, **far)) == bwd(gated(L=2, **far)) == -2


def test_the_ssd_step_does_not_look_at_path_and_segments():
    d, c = ss.ssd_dims(4, 1, 3, 64, 128), cache(elems=3 * 64 * 128, row_len=128)
    for d.path, d.segments in ((0, 2), (3, 2), (7, 0), (-1, -1)):
        assert ssd(d, c, x=None) == -1 and ssd(d, c, x=F + 8) == -4       # on to the pointers
