"""Refusals of the rotary and head norm entry points, and the frequencies (no GPU: nothing is launched)."""
import ctypes
import math
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


def shape(tokens=10, period=0, q_heads=4, k_heads=2, dim=64, rot=64, q_row=0, k_row=0, inter=0, dt=1):
    return ctypes.byref(ssm.RotaryShape(tokens, period, q_heads, k_heads, dim, rot, q_row, k_row, inter, dt))


def fwd(lib, s=None, q=P(0), k=P(1), pos=P(2), f=P(3), back=0, qo=P(4), ko=P(5), **kw):
    return lib.ssm_rotary_fwd(s or shape(**kw), q, k, pos, f, 1.0, back, qo, ko, None)


def nrm(lib, q=P(0), k=P(1), wq=P(6), wk=P(7), pos=P(2), f=P(3), eps=1e-6, qo=P(4), ko=P(5), **kw):
    return lib.ssm_qknorm_fwd(shape(**kw), q, k, wq, wk, pos, f, eps, 1.0, qo, ko, None)


def bwd(lib, q=P(0), k=P(1), wq=P(6), wk=P(7), pos=P(2), f=P(3), eps=1e-6, gq=P(8), gk=P(9), dq=P(4), dk=P(5), dwq=P(10),
        dwk=P(11), ws=P(12), n=1 << 30, **kw):
    return lib.ssm_qknorm_bwd(shape(**kw), q, k, wq, wk, pos, f, eps, 1.0, gq, gk, dq, dk, dwq, dwk, ws, n, None)


@pytest.mark.parametrize("bad,status,text", [
    (dict(dt=2), 1, "dtype"), (dict(inter=2), 1, "interleaved"), (dict(tokens=-1), 1, "negative"),
    (dict(q_heads=-1), 1, "negative"), (dict(period=-1), 1, "negative"), (dict(dim=0, rot=0), 1, "dim"),
    (dict(rot=63), 1, "rot"), (dict(rot=66), 1, "rot"), (dict(rot=-2), 1, "rot"), (dict(dim=258), 2, "dim"),
    (dict(q_heads=4096), 2, "heads"), (dict(tokens=(1 << 31) + 1), 2, "tokens"), (dict(q_row=255), 1, "q_row"),
    (dict(k_row=100), 1, "k_row"), (dict(q_row=1 << 48), 2, "too large"),
])
def test_shape_refusals(lib, bad, status, text):
    for call in (fwd, nrm, bwd):
        assert call(lib, **bad) == status
        assert text in lib.ssm_last_error().decode()


def test_pointer_refusals(lib):
    assert lib.ssm_rotary_fwd(None, P(0), P(1), P(2), P(3), 1.0, 0, P(4), P(5), None) == 1
    for name, c in (("q", "q"), ("k", "k"), ("positions", "pos"), ("freqs", "f"), ("q_out", "qo"), ("k_out", "ko")):
        for call in (fwd, nrm):
            assert call(lib, **{c: None}) == 1 and f"{name} is NULL".encode() in lib.ssm_last_error()
    for name, c in (("q", "q"), ("dq_out", "gq"), ("dk_out", "gk"), ("dq", "dq"), ("dk", "dk")):
        assert bwd(lib, **{c: None}) == 1 and f"{name} is NULL".encode() in lib.ssm_last_error()
    assert fwd(lib, back=2) == 1 and b"back" in lib.ssm_last_error()
    assert nrm(lib, eps=-1.0) == 1 and nrm(lib, eps=float("nan")) == 1 and b"eps" in lib.ssm_last_error()
    assert fwd(lib, q=P(0, 1)) == 1 and b"q is not aligned" in lib.ssm_last_error()
    assert fwd(lib, q=P(0, 2), dt=0) == 1 and b"q is not aligned" in lib.ssm_last_error()
    assert fwd(lib, f=P(3, 4)) == 1 and b"freqs is not aligned" in lib.ssm_last_error()
    assert fwd(lib, pos=P(2, 2)) == 1 and b"positions is not aligned" in lib.ssm_last_error()
    assert nrm(lib, wq=P(6, 2)) == 1 and b"wq is not aligned" in lib.ssm_last_error()
    assert fwd(lib, qo=P(0)) == 1 and b"overlaps" in lib.ssm_last_error()
    assert fwd(lib, ko=P(4, 10 * 4 * 64 * 2 - 2)) == 1 and b"overlaps" in lib.ssm_last_error()
    assert bwd(lib, dq=P(8)) == 1 and b"output dq overlaps dq_out" in lib.ssm_last_error()
    assert bwd(lib, dwk=P(10)) == 1 and b"overlaps" in lib.ssm_last_error()
    assert bwd(lib, ws=P(0)) == 1 and b"workspace overlaps" in lib.ssm_last_error()
    assert bwd(lib, ws=None, n=0) == 3 and bwd(lib, n=10 * 2 * 64 * 4 - 1) == 3


def test_nothing_to_do(lib):
    assert fwd(lib, tokens=0, q=None, k=None, pos=None, f=None, qo=None, ko=None) == 0
    assert fwd(lib, q_heads=0, k_heads=0, q=None, k=None, qo=None, ko=None) == 0
    assert bwd(lib, tokens=0, q=None, k=None, gq=None, gk=None, dq=None, dk=None, dwq=None, dwk=None, ws=None, n=0) == 0


def test_workspace(lib):
    assert ssm.qknorm_bwd_workspace_bytes(7, 64) == 7 * 2 * 64 * 4
    assert ssm.qknorm_bwd_workspace_bytes(1 << 20, 128) == 1024 * 2 * 128 * 4
    assert ssm.qknorm_bwd_workspace_bytes(7, 1000) == 0


def test_freqs():
    f, m = ssm.rotary_freqs(8, device="cpu")
    assert m == 1.0 and [round(v, 12) for v in f.tolist()] == [1.0, 0.1, 0.01, 0.001]
    assert ssm.rotary_freqs(8, scaling="linear", factor=4, device="cpu")[0].tolist() == (f / 4).tolist()
    g, _ = ssm.rotary_freqs(8, scaling="base", factor=4, device="cpu")
    assert g[0] == 1.0 and abs(g[-1] * 4 / f[-1] - 1) < 1e-12
    assert ssm.rotary_freqs(2, scaling="base", factor=4, device="cpu")[0].tolist() == [1.0]
    b, m = ssm.rotary_freqs(64, scaling="bands", factor=8, context=4096, device="cpu")
    f, _ = ssm.rotary_freqs(64, device="cpu")
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-15
    turns = 4096 * f / (2 * math.pi)
    assert (b == f)[turns >= 32].all() and (abs(b * 8 / f - 1) < 1e-12)[turns <= 1].all()
    assert ((b < f) & (b > f / 8))[(turns > 1) & (turns < 32)].all()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="x"), dict(rot=8, base=-1.0), dict(rot=8, factor=0.5),
                dict(rot=8, fast=1.0)):
        with pytest.raises(ValueError):
            ssm.rotary_freqs(**{"device": "cpu", **bad})


def test_binding_refuses_cpu_tensors():
    import torch
    q = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssm.rotary_fwd(q, None, torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="required"):
        ssm.rotary_fwd(q)
    with pytest.raises(ValueError, match="GPU"):
        ssm.qk_norm(q, q)
