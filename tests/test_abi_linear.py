"""Refusals of linear attention and of the group norm, before anything is enqueued (no GPU)."""
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
INF, NAN = float("inf"), float("nan")


def lin(io=ss.SELSCAN_F32, batch=2, L=10, H=4, Hk=2, K=8, V=12, **kw):
    d = ss.LinattnDims()
    ss.lib().linear_attention_dims_init(ctypes.byref(d), io, batch, L, H, Hk, K, V)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def norm(io=ss.SELSCAN_F32, batch=2, L=10, C=24, groups=4, **kw):
    d = ss.NormDims()
    ss.lib().group_norm_dims_init(ctypes.byref(d), io, batch, L, C, groups)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def ref(d):
    return ctypes.byref(d) if d is not None else None


def fwd(d, q=F, k=F, v=F, g=F, o=F, s0=None, s1=None, ws=None, n=0):
    return ss.lib().linear_attention_fwd(q, k, v, g, o, s0, s1, ref(d), ws, n, None)


def bwd(d, q=F, k=F, v=F, g=F, s0=None, do=F, dlast=None, dq=F, dk=F, dv=F, dg=None, ds0=None, ws=None, n=0):
    return ss.lib().linear_attention_bwd(q, k, v, g, s0, do, dlast, dq, dk, dv, dg, ds0, ref(d), ws, n, None)


def step(d, q=F, k=F, v=F, g=F, o=F, state=F, slots=2, read=None, write=None):
    return ss.lib().linear_attention_step(q, k, v, g, o, state, slots, read, write, ref(d), None)


def nfwd(d, x=F, w=None, b=None, z=None, y=F):
    return ss.lib().group_norm_fwd(x, w, b, z, y, ref(d), None)


def nbwd(d, x=F, w=None, b=None, z=None, dy=F, dx=F, dw=None, db=None, dz=None, ws=None, n=0):
    return ss.lib().group_norm_bwd(x, w, b, z, dy, dx, dw, db, dz, ref(d), ws, n, None)


@pytest.mark.parametrize("cls,name", [(ss.LinattnDims, "selscan_linattn_dims"), (ss.NormDims, "selscan_norm_dims")])
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


def test_dims_init():
    d = lin(ss.SELSCAN_BF16, 3, 20, 6, 2, 5, 7)
    assert (d.q_sb, d.q_sl, d.q_sh, d.k_sb, d.v_sb, d.v_sl, d.v_sh) == (200, 10, 5, 200, 840, 42, 7)
    assert (d.o_sb, d.g_sb, d.g_sl, d.g_sh, d.decay_tokens, d.scale) == (840, 120, 6, 1, 1, 1.0)
    n = norm(ss.SELSCAN_BF16, 3, 5, 12, 4)
    assert (n.x_sb, n.x_sl, n.z_sb, n.y_sl, n.activation) == (60, 12, 60, 12, 1) and abs(n.eps - 1e-5) < 1e-12
    ss.lib().linear_attention_dims_init(None, 0, 1, 1, 1, 1, 1, 1)
    ss.lib().group_norm_dims_init(None, 0, 1, 1, 1, 1)


LIN_BAD = [("batch", -1, -2), ("seqlen", -1, -2), ("nheads", 0, -2), ("qk_heads", 0, -2), ("qk_heads", 3, -2), ("dk", 0, -2),
           ("dv", 0, -2), ("dk", 257, -3), ("dv", 257, -3), ("q_sb", -1, -2), ("k_sl", -1, -2), ("v_sh", -1, -2),
           ("o_sb", -1, -2), ("g_sl", -1, -2), ("scale", NAN, -2), ("scale", INF, -2), ("io_dtype", 2, -3),
           ("decay_tokens", 2, -3), ("abi_version", 1, -7), ("batch", 1 << 22, -3), ("nheads", 1 << 40, -3)]


@pytest.mark.parametrize("field,value,status", LIN_BAD)
def test_linear_dims_errors(field, value, status):
    for L in (10, 1):
        d = lin(L=L)
        setattr(d, field, value)
        assert fwd(d) == status and bwd(d) == status
        if L == 1:
            assert step(d) == status
        assert ss.lib().linear_attention_workspace_size(ref(d)) == 0
        assert ss.lib().linear_attention_bwd_workspace_size(ref(d), 1) == 0


@pytest.mark.parametrize("name", ["q_sl", "k_sl", "v_sl", "o_sl"])
def test_long_token_strides(name):
    assert fwd(lin(batch=1, **{name: (1 << 22) + 1})) == -3 and bwd(lin(batch=1, **{name: (1 << 22) + 1})) == -3
    assert bwd(lin(batch=1, L=1, **{name: 1 << 30}), ws=F + 16, n=1 << 40) == -6      # one token's is not looked at
    assert fwd(lin(L=1 << 31, batch=1)) == -3
    assert fwd(lin(batch=1, g_sl=(1 << 22) + 1)) == -3
    wide = lin(batch=1, L=3, H=1 << 16, Hk=1, K=8, V=128)                       # its gradients' rows are 2^23 apart
    assert bwd(wide, ws=F + 16, n=1 << 60) == -3


def test_linear_null_and_alignment():
    d = lin()
    for name in "qkvgo":
        assert fwd(d, **{name: None}) == -1 and fwd(d, **{name: ODD}) == -4
    for name in ("q", "k", "v", "g", "do", "dq", "dk", "dv"):
        assert bwd(d, **{name: None}) == -1 and bwd(d, **{name: ODD}) == -4
    for name in ("s0", "s1"):
        assert fwd(d, **{name: HALF}) == -4
    for name in ("s0", "dlast", "dg", "ds0"):
        assert bwd(d, **{name: HALF}) == -4
    assert fwd(lin(ss.SELSCAN_BF16), q=ODD) == -4
    d = lin(L=1)
    for name in "qkvgo":
        assert step(d, **{name: None}) == -1 and step(d, **{name: ODD}) == -4
    assert step(d, state=None) == -1 and step(d, state=HALF) == -4 and step(d, read=HALF) == -4 and step(d, write=HALF) == -4
    assert fwd(None) == -1 and bwd(None) == -1 and step(None) == -1


def test_step_sizes():
    assert step(lin(L=2)) == -2 and step(lin(L=0)) == -2 and step(lin(L=1), slots=-1) == -2
    assert step(lin(L=1), slots=1) == -2 and step(lin(L=1), slots=1, read=F) == -2      # 0, 1 must exist
    assert step(lin(L=1), slots=1 << 31) == -3
    assert step(lin(L=1), slots=0, read=F, write=F, state=None) == 0                    # every row is padding
    assert step(lin(L=1, batch=0), q=None, k=None, v=None, o=None, state=None) == 0


def test_output_rows_must_not_overlap():
    for d in (lin(o_sl=47), lin(o_sb=479), lin(o_sh=11), lin(o_sb=0), lin(o_sh=0), lin(o_sl=0)):
        assert fwd(d) == -3
        assert bwd(d, ws=F + 16, n=1 << 40) == -6        # do is read: its rows may overlap
    # any order of the axes is one: heads before tokens, tokens before batch rows; and rows with room between
    for d in (lin(o_sb=480, o_sh=120, o_sl=12), lin(o_sl=96, o_sb=48, o_sh=12), lin(o_sh=20, o_sl=80, o_sb=800)):
        assert fwd(d, q=None) == -1
    assert step(lin(L=1, o_sb=47)) == -3 and step(lin(L=1, o_sh=11)) == -3


def test_linear_workspace():
    few, many = lin(batch=1, L=5000), lin(batch=200, L=5000)
    need = ss.lib().linear_attention_workspace_size(ref(few))
    assert need > 0 and ss.lib().linear_attention_workspace_size(ref(many)) == 0
    assert fwd(few, ws=F, n=need - 1) == -6 and fwd(few, ws=F + 16, n=need) == -6
    plain, decay = (ss.lib().linear_attention_bwd_workspace_size(ref(few), i) for i in (0, 1))
    assert 0 < plain < decay
    assert bwd(few, ws=F, n=plain - 1) == -6 and bwd(few, dg=F, ws=F, n=plain) == -6
    assert ss.lib().linear_attention_workspace_size(ref(lin(L=0))) == 0
    assert ss.lib().linear_attention_workspace_size(None) == 0


def test_linear_empty_calls():
    none = dict(q=None, k=None, v=None, g=None)
    assert fwd(lin(batch=0), o=None, **none) == 0
    assert fwd(lin(L=0), o=None, **none) == 0                                  # nothing to hand back
    assert bwd(lin(L=0), do=None, dq=None, dk=None, dv=None, **none) == 0


NORM_BAD = [("batch", -1, -2), ("seqlen", -1, -2), ("dim", 0, -2), ("groups", 0, -2), ("groups", 5, -2), ("x_sb", -1, -2),
            ("z_sl", -1, -2), ("y_sb", -1, -2), ("eps", 0.0, -2), ("eps", NAN, -2), ("eps", INF, -2), ("eps", -1.0, -2),
            ("io_dtype", 7, -3), ("activation", 2, -3), ("abi_version", 3, -7), ("batch", 1 << 31, -3),
            ("seqlen", 1 << 31, -3)]


@pytest.mark.parametrize("field,value,status", NORM_BAD)
def test_norm_dims_errors(field, value, status):
    d = norm(**{field: value})
    assert nfwd(d) == status and nbwd(d) == status
    assert ss.lib().group_norm_bwd_workspace_size(ref(d)) == 0


def test_norm_sizes():
    assert nfwd(norm(C=8193, groups=1)) == -3 and nfwd(norm(C=1 << 21, groups=1 << 20)) == -3
    assert nfwd(norm(batch=1 << 20, L=1 << 11)) == -3                          # 2^31 rows
    assert nfwd(norm(batch=1 << 12, L=1 << 12, C=8192, groups=128)) == -3      # groups, and threads of a launch
    assert nfwd(norm(batch=1, L=1 << 24, C=8192, groups=1)) == -3


def test_norm_null_alignment_workspace():
    d = norm()
    assert nfwd(None) == -1 and nbwd(None) == -1
    for name in "xy":
        assert nfwd(d, **{name: None}) == -1 and nfwd(d, **{name: ODD}) == -4
    for name in ("x", "dy", "dx"):
        assert nbwd(d, **{name: None}) == -1 and nbwd(d, **{name: ODD}) == -4
    assert nfwd(d, z=ODD) == -4 and nfwd(d, w=HALF) == -4 and nfwd(d, b=HALF) == -4
    assert nbwd(d, z=F) == -1 and nbwd(d, z=F, dz=ODD) == -4 and nbwd(d, dw=HALF) == -4 and nbwd(d, db=HALF) == -4
    need = ss.lib().group_norm_bwd_workspace_size(ref(d))
    assert need > 0 and nbwd(d, dw=F, ws=F, n=need - 1) == -6 and nbwd(d, db=F, ws=F + 16, n=need) == -6
    for bad in (norm(y_sl=23), norm(y_sb=100), norm(y_sb=0)):
        assert nfwd(bad) == -3
    assert nfwd(norm(batch=0), x=None, y=None) == 0 and nfwd(norm(L=0), x=None, y=None) == 0
    assert nbwd(norm(L=0), x=None, dy=None, dx=None) == 0
