"""Refusals of the linear attention entry points (no GPU: nothing is launched)."""
import ctypes
import os

import pytest

import selective_state_space_50_amd as ssm

A0 = 1 << 40
STEP = 1 << 32   # fake device addresses 4 GiB apart; never dereferenced


def P(i, off=0):
    return ctypes.c_void_p(A0 + i * STEP + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("libssm.so not built")
    return ssm.lib()


def shape(batch=2, seqlen=100, nheads=4, q_heads=4, k_heads=4, v_heads=4, dk=64, dv=64, q_row=0, k_row=0, v_row=0,
          dtype=1, reserved=0):
    return ssm.LinAttnShape(batch, seqlen, nheads, q_heads, k_heads, v_heads, dk, dv, q_row, k_row, v_row, dtype, reserved)


def fwd(lib, s, q=P(0), y=P(5), h0=P(6), h_last=P(7), lengths=None, ws=None, ws_bytes=0, log_decay=P(3)):
    return lib.ssm_linattn_fwd(ctypes.byref(s) if s else None, q, P(1), P(2), log_decay, 1.0, lengths, h0, h_last, y, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("bad,status,text", [
    (dict(dtype=2), 1, "dtype"), (dict(reserved=1), 1, "reserved"), (dict(batch=-1), 1, "bad size"),
    (dict(dk=0), 1, "bad size"), (dict(dv=0), 1, "bad size"), (dict(dk=257), 2, "at most 256"),
    (dict(dv=300), 2, "at most 256"), (dict(q_heads=3), 1, "q_heads"), (dict(k_heads=0), 1, "k_heads"),
    (dict(v_heads=8), 1, "v_heads"), (dict(q_row=255), 1, "q_row"), (dict(v_row=-1), 1, "v_row"),
    (dict(batch=1 << 30), 2, "too large"), (dict(seqlen=1 << 50), 2, "too large"),
    (dict(k_row=(1 << 24) + 1), 2, "k_row"), (dict(nheads=1 << 17, q_heads=1, k_heads=1, v_heads=1), 2, "too large"),
])
def test_shape_refusals(lib, bad, status, text):
    s = shape(**bad)
    assert fwd(lib, s) == status
    assert text in lib.ssm_last_error().decode()
    assert lib.ssm_linattn_bwd(ctypes.byref(s), *[P(i) for i in range(4)], 1.0, None, *[P(i) for i in range(4, 12)],
                               P(12), 1 << 40, None) == status
    assert lib.ssm_linattn_workspace_bytes(ctypes.byref(s)) == 0
    assert lib.ssm_linattn_bwd_workspace_bytes(ctypes.byref(s), 1) == 0


def test_pointer_refusals(lib):
    assert fwd(lib, None) == 1 and b"shape" in lib.ssm_last_error()
    assert fwd(lib, shape(), q=None) == 1 and b"q is NULL" in lib.ssm_last_error()
    assert fwd(lib, shape(), y=None) == 1 and b"y is NULL" in lib.ssm_last_error()
    assert fwd(lib, shape(), log_decay=None) == 1 and b"log_decay" in lib.ssm_last_error()
    assert fwd(lib, shape(), q=P(0, 2)) == 1 and b"q is not 16-byte aligned" in lib.ssm_last_error()
    assert fwd(lib, shape(), lengths=P(8, 4)) == 1 and b"lengths" in lib.ssm_last_error()
    assert fwd(lib, shape(), y=P(1)) == 1 and b"output y overlaps k" in lib.ssm_last_error()
    assert fwd(lib, shape(), h_last=P(6)) == 1 and b"output h_last overlaps h0" in lib.ssm_last_error()
    # y over the last strided token of q
    wide = shape(q_row=1000)
    last = (2 * 100 - 1) * 1000 * 2
    assert fwd(lib, wide, y=P(0, last)) == 1 and b"output y overlaps q" in lib.ssm_last_error()


def test_workspace(lib):
    few = shape(batch=1, seqlen=8192, nheads=2, q_heads=2, k_heads=2, v_heads=2)
    need = lib.ssm_linattn_workspace_bytes(ctypes.byref(few))
    assert need > 0 and need % (2 * 64 * 64 * 4) == 0          # whole segment states
    assert fwd(lib, few) == 3 and b"workspace" in lib.ssm_last_error()
    assert fwd(lib, few, ws=P(9), ws_bytes=need - 1) == 3
    assert fwd(lib, few, ws=P(9, 8), ws_bytes=need) == 1        # alignment
    assert fwd(lib, few, ws=P(5), ws_bytes=need) == 1           # y in the workspace
    # enough heads to fill the chip: one segment, no workspace
    assert lib.ssm_linattn_workspace_bytes(ctypes.byref(shape(batch=4, seqlen=4096, nheads=64, q_heads=64, k_heads=64,
                                                              v_heads=64, dk=128))) == 0
    # rows shared by heads need their per-head gradients
    s1, s2 = shape(), shape(k_heads=1, v_heads=1)
    assert lib.ssm_linattn_bwd_workspace_bytes(ctypes.byref(s2), 0) >= \
        lib.ssm_linattn_bwd_workspace_bytes(ctypes.byref(s1), 0) + 2 * 100 * 4 * 64 * 4
    assert ssm.linattn_workspace_bytes(1, 8192, 2, 64, 64) == need
    assert ssm.linattn_bwd_workspace_bytes(1, 8192, 2, 64, 64) > 2 * need


def test_backward_and_update_refusals(lib):
    def bwd(s, dy=P(5), dq=P(7), dk=P(8), dv=P(9), da=P(10), dh0=P(11), ws=P(12), n=1 << 31):
        return lib.ssm_linattn_bwd(ctypes.byref(s), P(0), P(1), P(2), P(3), 1.0, None, P(4), dy, P(6), dq, dk, dv, da, dh0,
                                   ws, n, None)
    assert bwd(shape(), dy=None) == 1 and b"dy is NULL" in lib.ssm_last_error()
    assert bwd(shape(), dk=None) == 1 and b"dk is NULL" in lib.ssm_last_error()
    assert bwd(shape(), dq=P(0)) == 1 and b"output dq overlaps q" in lib.ssm_last_error()
    assert bwd(shape(), dh0=P(6)) == 1 and b"output dh0 overlaps dh_last" in lib.ssm_last_error()
    assert bwd(shape(), dv=P(8)) == 1
    assert bwd(shape(), ws=None, n=0) == 3

    def upd(s, h=P(4), y=P(5)):
        return lib.ssm_linattn_update(ctypes.byref(s), h, P(0), P(1), P(2), P(3), 1.0, y, None)
    assert upd(shape()) == 1 and b"seqlen" in lib.ssm_last_error()
    assert upd(shape(seqlen=1), h=None) == 1 and b"h is NULL" in lib.ssm_last_error()
    assert upd(shape(seqlen=1), y=P(4)) == 1 and b"overlaps" in lib.ssm_last_error()
    assert upd(shape(seqlen=1, dk=512)) == 2


def test_empty_batches_are_no_ops(lib):
    assert fwd(lib, shape(batch=0), q=None, y=None) == 0
    assert upd_empty(lib) == 0


def upd_empty(lib):
    return lib.ssm_linattn_update(ctypes.byref(shape(batch=0, seqlen=1)), None, None, None, None, None, 1.0, None, None)


def test_binding_refuses_cpu_and_mismatched_tensors(lib):
    import torch
    q = torch.zeros(1, 4, 2, 8)
    a = torch.zeros(2)
    for call in (lambda: ssm.linattn_fwd(q, q, q, a), lambda: ssm.linear_attention(q, q, q, a),
                 lambda: ssm.linattn_bwd(q, q, q, a, dy=q), lambda: ssm.linattn_update(torch.zeros(1, 2, 8, 8), q[:, 0], q[:, 0], q[:, 0], a)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
    with pytest.raises(ValueError, match="must be"):
        ssm.linattn_fwd(q[0], q, q, a)


def test_strided_rows():
    """The token stride of a slice of a joint projection, and layouts that have none."""
    import torch
    wide = torch.zeros(2, 5, 3 * 32)
    s = wide[..., 32:64].unflatten(-1, (4, 8))

    def rows(t, *tokens):
        return ssm._rows((t.shape, t.stride()), "k", tokens, 4, 8)
    assert rows(s, 2, 5) == 96
    assert rows(s[:, 0], 2) == 480
    assert rows(s[:1, :1], 1, 1) == 32
    assert rows(s[:0], 0, 5) == 32
    assert rows(s.contiguous(), 2, 5) == 32
    for bad in (s.transpose(2, 3).contiguous().transpose(2, 3), torch.zeros(2, 4, 5, 8).transpose(1, 2),
                torch.zeros(5, 2, 4, 8).transpose(0, 1), torch.zeros(1, 1, 4, 8).expand(2, 5, 4, 8)):
        with pytest.raises(ValueError, match="evenly spaced"):
            rows(bad, 2, 5)
    with pytest.raises(ValueError, match="shape"):
        rows(s, 2, 4)


def test_rows_of_one_launch(lib):
    """Batch rows times heads: a launch's threads are counted in 32 bits."""
    s = shape(batch=1 << 18, seqlen=1, nheads=8, q_heads=8, k_heads=8, v_heads=8, dk=1, dv=1)
    assert fwd(lib, s) == 2 and b"too large" in lib.ssm_last_error()
    s.batch = 1 << 17
    assert fwd(lib, s, q=None) == 1 and b"q is NULL" in lib.ssm_last_error()


def test_one_tokens_rows_may_lie_far_apart(lib):
    """Offsets within a chunk are 32-bit, but one token (of a prompt, or the update) has no second row there."""
    for far in (dict(q_row=1 << 25), dict(k_row=1 << 40), dict(v_row=(1 << 24) + 1)):
        s = shape(seqlen=1, **far)
        assert fwd(lib, s, q=None) == 1 and b"q is NULL" in lib.ssm_last_error()
        assert lib.ssm_linattn_update(ctypes.byref(s), None, P(0), P(1), P(2), P(3), 1.0, P(5), None) == 1
        assert b"h is NULL" in lib.ssm_last_error()
        s.seqlen = 2
        assert fwd(lib, s, q=None) == 2 and b"_row" in lib.ssm_last_error()
    # byte offsets stay within 64 bits
    assert fwd(lib, shape(seqlen=1, k_row=1 << 60), q=None) == 2 and b"k_row" in lib.ssm_last_error()
    assert fwd(lib, shape(batch=1 << 16, seqlen=1 << 20, nheads=1, q_heads=1, k_heads=1, v_heads=1, q_row=1 << 24), q=None) == 2


def test_workspaces_elsewhere_or_in_pieces_are_refused():
    """(a kernel would write them by their address)"""
    import torch
    gpu, cpu = torch.device("cuda", 0), torch.device("cpu")
    with pytest.raises(ValueError, match="workspace is on cpu"):
        ssm._workspace(torch.empty(1000, dtype=torch.uint8), 100, gpu)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1000), torch.empty(2000, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            ssm._workspace(bad, 100, cpu)
    enough = torch.empty(30, dtype=torch.float32)
    assert ssm._workspace(enough, 120, cpu) is enough and ssm._workspace(None, 0, cpu) is None
    assert ssm._workspace(enough, 121, cpu).numel() == 121


def test_a_stream_of_another_device_is_refused():
    """(the call would run on the tensors' device, but not on the stream)"""
    from types import SimpleNamespace

    import torch
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        ssm._elsewhere(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1), device_type="cuda"))


def test_the_cases_of_uneven_parts_have_them(tmp_path):
    """The planner cuts the segments of test_gpu_linattn's PARTS into parts, the last one shorter: forward and backward."""
    import subprocess

    from tests.test_gpu_linattn import PARTS
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "selective_state_space_50_amd", "csrc")
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(root, "include"), "-I", csrc,
                    os.path.join(root, "tests", "host", "linattn_plan.cpp"), os.path.join(csrc, "ssm_host.cpp"), "-o", exe], check=True)
    lines = "".join(" ".join(map(str, (*p[:8], 1 if p[8] == "bf16" else 0))) + "\n" for p in PARTS)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(PARTS)
    for line in out:
        x = list(map(int, line.split()))
        for nseg, seg_len, nsub, sub_len in (x[:4], x[4:8]):
            assert nseg > 1 and nsub > 1 and nsub * sub_len > seg_len, line
