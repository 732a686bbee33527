"""Refusals of the served mixer's entry points (no GPU: nothing is launched), and how it splits sequences."""
import ctypes
import os

import pytest

import selective_state_space_50_amd as ssm

A0 = 1 << 40
STEP = 1 << 38


def P(i, off=0):
    return ctypes.c_void_p(A0 + i * STEP + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssm.so not built")
    return ssm.lib()


def shape(tokens=10, sequences=3, max_seqlen=0, H=4, P_=64, N=128, G=1, W=4, nslots=5, x_row=0, z_row=0, d_row=0, dt=1, res=0):
    return ctypes.byref(ssm.SsdConvShape(tokens, sequences, max_seqlen, H, P_, N, G, W, nslots, x_row, z_row, d_row, dt, res))


def fwd(lib, xbc=P(0), delta=P(1), A=P(2), w=P(3), bias=P(4), D=P(5), z=P(6), db=P(7), sp=1, off=P(8), slots=P(9), fresh=P(10),
        h=P(11), cs=P(12), y=P(13), ws=P(14), n=1 << 40, **kw):
    return lib.ssm_ssdconv_fwd(shape(**kw), xbc, delta, A, w, bias, D, z, db, sp, off, slots, fresh, h, cs, y, ws, n, None)


def upd(lib, xbc=P(0), delta=P(1), A=P(2), w=P(3), bias=P(4), D=P(5), z=P(6), db=P(7), sp=1, slots=P(9), h=P(11), cs=P(12), y=P(13),
        ws=P(14), n=1 << 40, tokens=3, **kw):
    return lib.ssm_ssdconv_update(shape(tokens=tokens, **kw), xbc, delta, A, w, bias, D, z, db, sp, slots, h, cs, y, ws, n, None)


@pytest.mark.parametrize("bad,status,text", [
    (dict(dt=2), 1, "dtype"), (dict(sequences=-1, tokens=-1), 1, "negative"), (dict(H=-4), 1, "negative"), (dict(nslots=-1), 1, "negative"),
    (dict(max_seqlen=-1), 1, "negative"), (dict(res=1), 1, "reserved"), (dict(P_=0), 1, "headdim"), (dict(N=0), 1, "dstate"),
    (dict(G=0), 1, "ngroups"), (dict(G=3), 1, "ngroups"), (dict(W=0), 1, "width"), (dict(W=5), 1, "width"),
    (dict(N=129), 2, "dstate"), (dict(sequences=65536, tokens=65536), 2, "too large"), (dict(H=65537), 2, "too large"),
    (dict(nslots=1 << 31), 2, "too large"), (dict(x_row=511), 1, "shorter"), (dict(z_row=255), 1, "shorter"),
    (dict(d_row=3), 1, "shorter"), (dict(x_row=1 << 50), 2, "too large"), (dict(sp=2), 1, "delta_softplus"),
])
def test_shape_refusals(lib, bad, status, text):
    for call in (fwd, upd):
        assert call(lib, **bad) == status
        assert text in lib.ssm_last_error().decode()


def test_more_refusals(lib):
    assert fwd(lib, tokens=(1 << 28) + 1) == 2
    assert fwd(lib, tokens=1 << 28, sequences=60000, H=4096) == 2 and b"too many" in lib.ssm_last_error()
    assert upd(lib, tokens=65000, sequences=65000, H=4096) == 2 and b"too many" in lib.ssm_last_error()
    assert upd(lib, tokens=4) == 1 and b"one token" in lib.ssm_last_error()
    assert lib.ssm_ssdconv_workspace_bytes(None) == 0 and b"NULL" in lib.ssm_last_error()
    names = (("xbc", "xbc"), ("delta", "delta"), ("A", "A"), ("w", "w"), ("h", "h"), ("conv_state", "cs"), ("y", "y"))
    for name, c in names:
        for call in (fwd, upd):
            assert call(lib, **{c: None}) == 1 and f"{name} is NULL".encode() in lib.ssm_last_error()
    assert fwd(lib, off=None) == 1 and b"offsets is NULL" in lib.ssm_last_error()
    for call in (fwd, upd):
        assert call(lib, xbc=P(0, 1)) == 1 and b"xbc is not aligned" in lib.ssm_last_error()
        assert call(lib, h=P(11, 2)) == 1 and b"h is not aligned" in lib.ssm_last_error()
        assert call(lib, ws=P(14, 8)) == 1 and b"workspace is not aligned" in lib.ssm_last_error()
        assert call(lib, y=P(0)) == 1 and b"output y overlaps xbc" in lib.ssm_last_error()
        assert call(lib, h=P(13, 256)) == 1 and b"overlaps" in lib.ssm_last_error()
        assert call(lib, cs=P(6)) == 1 and b"output conv_state overlaps z" in lib.ssm_last_error()
        assert call(lib, ws=P(12)) == 1 and b"overlaps" in lib.ssm_last_error()
        assert call(lib, ws=None, n=0) == 3 and call(lib, n=100) == 3
    assert fwd(lib, fresh=P(14, 5)) == 1 and b"workspace overlaps fresh" in lib.ssm_last_error()


@pytest.mark.parametrize("bad,text", [
    (dict(H=32769), "too large"), (dict(H=32768, P_=64, N=128, nslots=1 << 30), "slots of"),
    (dict(H=2048, P_=16, N=64, G=2048, W=4, nslots=3), None),
])
def test_size_limits(lib, bad, text):
    """As many heads as a launch's grid takes; a pool of more states than can be counted in bytes; in between, calls that are fine."""
    for call in (fwd, upd):
        if text is None:
            assert call(lib, n=100, **bad) == 3
        else:
            assert call(lib, **bad) == 2 and text in lib.ssm_last_error().decode()


def test_wide_rows(lib):
    """A prompt's rows reach 2^22 elements, single tokens' any distance."""
    assert fwd(lib, x_row=(1 << 22) + 1) == 2 and b"too large" in lib.ssm_last_error()
    assert fwd(lib, x_row=1 << 22, n=100) == 3
    assert upd(lib, x_row=(1 << 22) + 1, n=100) == 3
    # one chunk more than a launch has threads for
    assert ssm.ssdconv_workspace_bytes((1 << 28) - 64, 1, 1, 1, 1, max_seqlen=64) == 0


def test_nothing_to_do(lib):
    none = dict.fromkeys(("xbc", "delta", "A", "w", "bias", "D", "z", "db", "slots", "h", "cs", "y", "ws"))
    assert fwd(lib, sequences=0, tokens=0, off=None, fresh=None, n=0, **none) == 0
    assert upd(lib, sequences=0, tokens=0, n=0, **none) == 0
    assert fwd(lib, H=0, off=None, fresh=None, n=0, **none) == 0


def test_workspaces():
    assert ssm.ssdconv_workspace_bytes(3, 3, 4, 64, 128, update=True) == 3 * (256 + 256) * 4
    assert ssm.ssdconv_workspace_bytes(64, 1, 4, 64, 200) == 0
    def split(*a, **k):    # a workgroup's states in the workspace
        T, S, H, P_, N = a
        return ssm.ssdconv_workspace_bytes(*a, **k) - ssm.ssdconv_workspace_bytes(*a, **{**k, "max_seqlen": 64}) > H * P_ * N * 4
    assert split(32768, 1, 24, 64, 128)                                # few heads, one long prompt
    assert not split(16384, 4, 64, 64, 128, max_seqlen=4096)           # a workgroup for every CU as it is
    assert split(16384, 4, 64, 64, 128, max_seqlen=16384)              # (one of them may be long)
    assert not split(100, 2, 4, 64, 64)
    assert ssm.ssdconv_workspace_bytes(32768, 1, 24, 64, 128, dtype="f32") > ssm.ssdconv_workspace_bytes(32768, 1, 24, 64, 128)


def test_binding_refuses():
    import torch
    x = torch.zeros(3, 512 + 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssdconv_update(x, x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssdconv_fwd(x, x, x, x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="offsets"):
        ssm.ssdconv_fwd(x, x, x, x, x, x, torch.zeros(0, dtype=torch.int32))
