"""Refusals of the group norm entry points (no GPU: nothing is launched)."""
import ctypes
import os

import pytest

import selective_state_space_50_amd as ssm

A0 = 1 << 40
STEP = 1 << 34


def P(i, off=0):
    return ctypes.c_void_p(A0 + i * STEP + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssm.so not built")
    return ssm.lib()


def fwd(lib, N=2, L=10, C=64, G=4, dt=1, x=P(0), w=P(1), b=P(2), z=P(3), eps=1e-5, silu=0, y=P(4), mean=P(5), rstd=P(6),
        ws=None, n=0):
    return lib.ssm_groupnorm_fwd(N, L, C, G, dt, x, w, b, z, eps, silu, y, mean, rstd, ws, n, None)


def bwd(lib, N=2, L=1, C=64, G=4, dt=1, x=P(0), z=P(3), silu=0, dy=P(4), mean=P(5), rstd=P(6), dx=P(7), dw=P(8), db=P(9),
        dz=P(10), ws=P(11), n=1 << 33):
    return lib.ssm_groupnorm_bwd(N, L, C, G, dt, x, P(1), P(2), z, silu, dy, mean, rstd, dx, dw, db, dz, ws, n, None)


@pytest.mark.parametrize("bad,status,text", [
    (dict(dt=3), 1, "dtype"), (dict(N=-1), 1, "negative"), (dict(C=-4), 1, "negative"), (dict(G=0), 1, "groups"),
    (dict(G=5), 1, "groups"), (dict(silu=2), 1, "silu"), (dict(N=1 << 31), 2, "too large"), (dict(C=1 << 30, G=1), 2, "too large"),
    (dict(L=1 << 40), 2, "too large"), (dict(N=70000, L=1 << 20), 2, "too many"),
])
def test_shape_refusals(lib, bad, status, text):
    assert fwd(lib, **bad) == status
    assert text in lib.ssm_last_error().decode()
    assert bwd(lib, **bad) == status


def test_pointer_refusals(lib):
    assert fwd(lib, eps=-1.0) == 1 and b"eps" in lib.ssm_last_error()
    assert fwd(lib, eps=float("nan")) == 1
    assert fwd(lib, x=None) == 1 and b"x is NULL" in lib.ssm_last_error()
    assert fwd(lib, y=None) == 1 and b"y is NULL" in lib.ssm_last_error()
    assert fwd(lib, w=P(1, 4)) == 1 and b"w is not 16-byte aligned" in lib.ssm_last_error()
    assert fwd(lib, y=P(0)) == 1 and b"output y overlaps x" in lib.ssm_last_error()
    assert fwd(lib, mean=P(6)) == 1 and b"overlaps" in lib.ssm_last_error()
    for name, i in (("dy", None), ("mean", None), ("rstd", None), ("dx", None), ("dz", None)):
        assert bwd(lib, **{name: i}) == 1 and f"{name} is NULL".encode() in lib.ssm_last_error()
    assert bwd(lib, dx=P(4)) == 1 and b"output dx overlaps dy" in lib.ssm_last_error()
    assert bwd(lib, dz=P(7)) == 1
    assert bwd(lib, ws=None, n=0) == 3


def test_workspace(lib):
    # a group of 1000 x 64 values: slabs; one of 10 x 16: a team's registers
    need = ssm.groupnorm_workspace_bytes(2, 1000, 256, 4, span="sequence")
    assert need > 0 and fwd(lib, L=1000, C=256) == 3 and fwd(lib, L=1000, C=256, ws=P(12), n=need - 1) == 3
    assert ssm.groupnorm_workspace_bytes(2, 10, 64, 4, span="sequence") == 0
    assert ssm.groupnorm_workspace_bytes(2, 1000, 256, 4) == 0
    assert ssm.groupnorm_workspace_bytes(2, 1000, 256, 4, backward=True) > 0


def test_empty_is_a_no_op(lib):
    assert fwd(lib, N=0, x=None, y=None) == 0 and fwd(lib, C=0, x=None, y=None) == 0


def test_binding_refuses(lib):
    import torch
    x = torch.zeros(2, 3, 8)
    for call in (lambda: ssm.groupnorm_fwd(x, 2), lambda: ssm.group_norm(x, 2), lambda: ssm.groupnorm_bwd(x, 2, dy=x)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
    with pytest.raises(ValueError, match="span"):
        ssm.groupnorm_fwd(x, 2, span="row")
    with pytest.raises(ValueError, match="activation"):
        ssm.groupnorm_fwd(x, 2, activation="relu")
    with pytest.raises(ValueError, match="x must be"):
        ssm.groupnorm_fwd(x[None], 2)


def test_blocks_of_one_launch(lib):
    """Groups just wider than half a workgroup take one each, and a launch has 65535 of them across."""
    assert fwd(lib, N=1, L=100, C=129 * 100000, G=100000) == 2 and b"too many" in lib.ssm_last_error()
    assert fwd(lib, N=1, L=100, C=129 * 65000, G=65000, x=None) == 1 and b"x is NULL" in lib.ssm_last_error()


@pytest.mark.parametrize("N,L,C,G", [(1 << 16, 1, 5120, 1), (70000, 4, 512, 32), (66000, 1, 515, 1), (65535, 1, 1 << 14, 1), (1 << 20, 2, 64, 64),
                                     (1 << 16, 1, 1 << 15, 1), (70000, 1000, 512, 32), (2, 100, 129 * 100000, 100000), (3, 1, (1 << 24) - 1, 1),
                                     (2, 2, (1 << 24) - 1, (1 << 24) - 1), (70000, 2, 1025, 1)])
@pytest.mark.parametrize("dt", [0, 1])
def test_the_backward_takes_what_the_forward_takes(lib, N, L, C, G, dt):
    """(x NULL: refused as a pointer where the shape is taken)"""
    status = fwd(lib, N=N, L=L, C=C, G=G, dt=dt, x=None)
    assert status in (1, 2)
    assert bwd(lib, N=N, L=L, C=C, G=G, dt=dt, x=None) == status, lib.ssm_last_error()


def test_the_backwards_workspace_does_not_grow_with_the_tokens(lib):
    for dtype in ("bf16", "f32"):
        one, two, many = (ssm.groupnorm_workspace_bytes(1, n, 8192, 1, dtype, backward=True) for n in (16384, 32768, 65535))
        assert one == two == many <= 64 << 20
    # sequences of a few positions, short of a launch's slabs and beyond
    assert ssm.groupnorm_workspace_bytes(60000, 2, 4096, 8, span="sequence", backward=True) <= 64 << 20
    assert 0 < ssm.groupnorm_workspace_bytes(70000, 4, 512, 32, span="sequence", backward=True) <= 64 << 20
