"""Linear attention, the group norm and the state update as a layer uses them: a training step through autograd
from slices of one projection to the gated norm of every head, and the same layer token by token, eager and as a graph.

Every stage is checked with the tolerances of its own operator (test_gpu_linattn, test_gpu_groupnorm) against the
fp64 oracle on the stage's actual inputs, so no tolerance spans two roundings.
"""
import numpy as np
import pytest

import synth
from oracle.linattn_oracle import linattn, linattn_bwd
from oracle.norm_oracle import groupnorm, groupnorm_bwd
from tests import test_gpu_groupnorm as tn
from tests import test_gpu_linattn as ta
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_linattn import ssm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def norm_case(y, z, w, b, do=None):
    """fp64 rows of the norm's inputs."""
    r = lambda t: None if t is None else to_host(t).astype(np.float64).reshape(-1, 1, w.numel())  # noqa: E731
    return r(y), to_host(w).astype(np.float64), to_host(b).astype(np.float64), r(z), r(do)


@pytest.mark.parametrize("B,L,H,G,dk,dv,dt,lengths", [
    (2, 200, 4, 4, 32, 64, "bf16", None), (1, 1, 2, 1, 16, 16, "f32", None), (3, 77, 6, 2, 40, 24, "f32", [77, 0, 30]),
    (1, 900, 2, 2, 128, 128, "bf16", None)])
def test_training_step(ssm, B, L, H, G, dk, dv, dt, lengths):  # noqa: F811
    import torch
    c = ta.make(B, L, H, G, G, H, dk, dv, dt, seed=L)
    r = np.random.default_rng(1)
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    x = torch.cat([to_dev(c[n], dt).flatten(2) for n in ("q", "k", "v")], -1).requires_grad_()
    a = torch.from_numpy(c["a"]).cuda().requires_grad_()
    w, b = (torch.from_numpy(r.standard_normal(H * dv).astype(np.float32)).cuda().requires_grad_() for _ in range(2))
    z, do = (torch.from_numpy(r.standard_normal((B, L, H * dv)).astype(np.float32)).cuda().to(tdt) for _ in range(2))
    z.requires_grad_()
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q, k, v = (t.unflatten(-1, (-1, d)) for t, d in zip(x.split([G * dk, G * dk, H * dv], -1), (dk, dk, dv)))
    y = ssm.linear_attention(q, k, v, a, scale=0.3, lengths=n)
    y.retain_grad()
    o = ssm.group_norm(y.flatten(2), H, w, b, z)
    o.backward(do)
    torch.cuda.synchronize()
    (yr, _), (ya, _) = ta.both(linattn, c, ("q", "k", "v", "a", 0.3, None), lengths=lengths)
    ta.check(y.detach(), yr, ya, dt, c, "y")
    ys, ws, bs, zs, dos = norm_case(y.detach(), z.detach(), w.detach(), b.detach(), do)
    lim = tn.bounds(ys, H, ws, bs, zs, dos, False)
    tn.check(o.detach(), groupnorm(ys, H, ws, bs, zs, 1e-5, False), lim["y"], dt, "o")
    ref = groupnorm_bwd(ys, H, ws, bs, zs, dos, 1e-5, False)
    for name, t in (("dx", y.grad), ("dz", z.grad), ("dw", w.grad), ("dbias", b.grad)):
        tn.check(t, ref[name], lim[name], dt if name in ("dx", "dz") else "f32", name)
    c["dy"] = synth.store(to_host(y.grad).astype(np.float32), dt)   # (exact: its own type's values)
    ref, big = ta.both(linattn_bwd, c, ("q", "k", "v", "a", 0.3, None, "dy", None), lengths=lengths)
    got = dict(zip(("dq", "dk", "dv"), (t.unflatten(-1, (-1, d)) for t, d in
                                        zip(x.grad.split([G * dk, G * dk, H * dv], -1), (dk, dk, dv)))))
    for name in got:
        ta.check(got[name].contiguous(), ref[name], big[name], dt, c, name)
    ta.check(a.grad, ref["dlog_decay"], big["dlog_decay"], "f32", c, "dlog_decay")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_then_tokens(ssm, dt):  # noqa: F811
    """A prompt, then tokens one at a time: linear attention of the whole sequence, and its norm."""
    import torch
    B, L, P, H, dk, dv = 2, 70, 65, 4, 64, 32
    c = ta.make(B, L, H, H, 2, 2, dk, dv, dt, seed=9)
    q, k, v, a = ta.dev(c, "q", "k", "v", "a")
    w, b = (torch.randn(H * dv, device="cuda") for _ in range(2))
    z = torch.randn(B, L, H * dv, device="cuda").to(q.dtype)
    y, h = ssm.linattn_fwd(*(t[:, :P].contiguous() for t in (q, k, v)), a, return_last_state=True)
    h0 = h.clone()
    # the token's work, eager and as a graph over fixed buffers
    t1 = [t[:, P].contiguous() for t in (q, k, v, z)]

    def token():
        s = ssm.linattn_update(h, *t1[:3], a)
        return s, ssm.groupnorm_fwd(s.flatten(1), H, w, b, t1[3])

    eager = []
    for t in range(P, L):
        for buf, full in zip(t1, (q, k, v, z)):
            buf.copy_(full[:, t])
        eager.append([r.clone() for r in token()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = token()
    h.copy_(h0)
    for t in range(P, L):
        for buf, full in zip(t1, (q, k, v, z)):
            buf.copy_(full[:, t])
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(held, eager[t - P]):
            assert torch.equal(got, ref), t
    (yr, hr), (ya, ha) = ta.both(linattn, c, ("q", "k", "v", "a", dk ** -0.5, None))
    ta.check(torch.cat([y, torch.stack([e[0] for e in eager], 1)], 1), yr, ya, dt, c, "y")
    ta.check(h, hr, ha, "f32", c, "h")
    for t in range(P, L):
        ys, ws, bs, zs, _ = norm_case(eager[t - P][0], z[:, t].contiguous(), w, b)
        tn.check(eager[t - P][1], groupnorm(ys, H, ws, bs, zs, 1e-5, False), tn.bounds(ys, H, ws, bs, zs, np.zeros(1), False)["y"],
                 dt, "o")


def test_captured_training_step(ssm):  # noqa: F811
    """Forward and backward of the layer through autograd in one graph, replayed over new inputs between eager steps."""
    import torch
    B, L, H, d = 2, 300, 4, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    x, z, do = new(B, L, 3 * H * d).bfloat16(), new(B, L, H * d).bfloat16(), new(B, L, H * d).bfloat16()
    a, w, b = -new(H).abs(), new(H * d), new(H * d)

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, z, a, w, b)]
        q, k, v = (t.unflatten(-1, (H, d)) for t in leaves[0].chunk(3, -1))
        y = ssm.linear_attention(q, k, v, leaves[2])
        o = ssm.group_norm(y.flatten(2), H, leaves[3], leaves[4], leaves[1])
        return [o.detach(), *torch.autograd.grad(o, leaves, do)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        for t in (x, z, do, w, b):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
        ref = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, r) in enumerate(zip(held, ref)):
            assert torch.equal(t, r), i


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_outputs_joined_before_the_loss(ssm, dt):  # noqa: F811
    """Outputs joined along the batch: the second part's gradient is a part of the whole one and need not start on 16 bytes."""
    import torch
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    new = lambda *shape: torch.randn(*shape, device="cuda").to(tdt)  # noqa: E731
    q, k, v = (new(1, 17, 3, 33) for _ in range(3))
    a = -torch.rand(3, device="cuda")
    x, w = new(1, 17, 99), torch.randn(99, device="cuda")
    dt_, al, bl, cl = -torch.rand(99, 4, device="cuda"), new(1, 17, 99).abs(), new(1, 17, 4), torch.randn(99, 3, device="cuda")
    for f, args in ((lambda q, k, v, a: ssm.linear_attention(q, k, v, a), (q, k, v, a)),
                    (lambda x, w: ssm.group_norm(x, 3, w), (x, w)),
                    (lambda x, w: ssm.causal_conv1d(x, w), (x, cl)),
                    (lambda x, d, A, B: ssm.selective_scan(x, d, A, B, B), (x, al, dt_, bl))):
        one, two = ([t.clone().requires_grad_() for t in args] for _ in range(2))
        y1, y2 = f(*one), f(*two)
        dy = new(2, *y1.shape[1:])
        assert dy[1].data_ptr() % 16
        got = torch.autograd.grad(torch.cat([y1, y2]), [*one, *two], dy)
        ref = [*torch.autograd.grad(f(*one), one, dy[:1].clone()), *torch.autograd.grad(f(*two), two, dy[1:].clone())]
        for g, r in zip(got, ref):
            assert torch.equal(g, r)


def test_decays_and_lengths_of_a_larger_tensor(ssm):  # noqa: F811
    """One layer's row of [layers, 6] decays, and a batch's later lengths."""
    import torch
    decays = -torch.rand(3, 6, device="cuda")
    lengths = torch.tensor([3, 40, 17], dtype=torch.int32, device="cuda")
    q, k, v, dy = (torch.randn(2, 40, 6, 16, device="cuda").bfloat16() for _ in range(4))
    a, n = decays[1], lengths[1:]
    assert a.data_ptr() % 16 and n.data_ptr() % 16
    (y, h), (yr, hr) = (ssm.linattn_fwd(q, k, v, t, lengths=m, return_last_state=True) for t, m in ((a, n), (a.clone(), n.clone())))
    assert torch.equal(y, yr) and torch.equal(h, hr)
    g, r = (ssm.linattn_bwd(q, k, v, t, dy=dy, lengths=m) for t, m in ((a, n), (a.clone(), n.clone())))
    for name in r:
        assert torch.equal(g[name], r[name]), name
    h2 = h.clone()
    one = [t[:, 0].contiguous() for t in (q, k, v)]
    assert torch.equal(ssm.linattn_update(h, *one, a), ssm.linattn_update(h2, *one, a.clone())) and torch.equal(h, h2)
    # and through autograd, where the gradient is the whole tensor's
    whole = decays.clone().requires_grad_()
    (gw,) = torch.autograd.grad(ssm.linear_attention(q, k, v, whole[1], lengths=n), whole, dy)
    assert torch.equal(gw[1], r["dlog_decay"]) and not gw[0].any() and not gw[2].any()


def test_writes_are_seen_by_autograd(ssm):  # noqa: F811
    """A tensor that a backward has saved and a call then writes (a state advanced in place, a given output): the
    backward raises, as after torch's own in-place operations, and does not read the new values."""
    import torch
    new = lambda *shape: torch.randn(*shape, device="cuda")  # noqa: E731
    q, k, v, a, h = new(2, 9, 4, 16), new(2, 9, 4, 16), new(2, 9, 4, 16), -torch.rand(4, device="cuda"), new(2, 4, 16, 16)
    one = [t[:, 0].contiguous() for t in (q, k, v)]
    x, w, st = new(2, 9, 64), new(64, 4), new(2, 64, 3)
    d, A, B, hs = new(2, 9, 64).abs(), -torch.rand(64, 16, device="cuda"), new(2, 9, 16), new(2, 64, 16)
    x3 = new(2, 4, 16)
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    for what, forward, saved, write in (
            ("linattn_update's state", lambda: ssm.linear_attention(leaf(q), k, v, a, h), h, lambda: ssm.linattn_update(h, *one, a)),
            ("linattn_update's out", lambda: ssm.group_norm(x3, 4, leaf(x3[0, 0])), x3, lambda: ssm.linattn_update(h, *one, a, out=x3)),
            ("linattn_fwd's h_last", lambda: ssm.linear_attention(leaf(q), k, v, a, h), h,
             lambda: ssm.linattn_fwd(q, k, v, a, return_last_state=True, h_last=h)),
            ("linattn_fwd's out", lambda: ssm.linear_attention(leaf(q), k, v, a), v, lambda: ssm.linattn_fwd(q, k, q, a, out=v)),
            ("groupnorm_fwd's out", lambda: ssm.group_norm(x, 4, leaf(w[:, 0].contiguous())), x, lambda: ssm.groupnorm_fwd(d, 4, out=x)),
            ("conv1d_update's state", lambda: ssm.causal_conv1d(leaf(x), w, None, st), st, lambda: ssm.conv1d_update(st, x[:, 0].contiguous(), w)),
            ("conv1d_fwd's out", lambda: ssm.causal_conv1d(x, leaf(w)), x, lambda: ssm.conv1d_fwd(d, w, out=x)),
            ("state_update's state", lambda: ssm.selective_scan(leaf(x), d, A, B, B, h0=hs), hs,
             lambda: ssm.state_update(hs, x[:, 0].contiguous(), d[:, 0].contiguous(), A, B[:, 0].contiguous(), B[:, 0].contiguous())),
            ("scan_fwd's out", lambda: ssm.selective_scan(leaf(x), d, A, B, B), d, lambda: ssm.scan_fwd(x, d.clone(), A, B, B, out=d))):
        y = forward()
        before = saved._version
        write()
        assert saved._version > before, what
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_small_workspaces_are_replaced(ssm):  # noqa: F811
    """A workspace that is too small is left alone and another used; one on the host is refused."""
    import torch
    q, k, v = (torch.randn(1, 2000, 2, 64, device="cuda").bfloat16() for _ in range(3))
    a = -torch.rand(2, device="cuda")
    x, w = torch.randn(2, 3000, 64, device="cuda"), torch.randn(64, device="cuda")
    _, m, r = ssm.groupnorm_fwd(x, 2, w, span="sequence", return_stats=True)
    for need, call in ((ssm.linattn_workspace_bytes(1, 2000, 2, 64, 64), lambda ws: ssm.linattn_fwd(q, k, v, a, workspace=ws)),
                       (ssm.linattn_bwd_workspace_bytes(1, 2000, 2, 64, 64), lambda ws: ssm.linattn_bwd(q, k, v, a, dy=v, workspace=ws)["dq"]),
                       (ssm.groupnorm_workspace_bytes(2, 3000, 64, 2, "f32", "sequence"),
                        lambda ws: ssm.groupnorm_fwd(x, 2, w, span="sequence", workspace=ws)),
                       (ssm.groupnorm_workspace_bytes(2, 3000, 64, 2, "f32", "sequence", True),
                        lambda ws: ssm.groupnorm_bwd(x, 2, w, None, None, x, m, r, span="sequence", workspace=ws)["dx"])):
        ref = call(None)
        for size in (need, need - 1, 0):
            ws = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
            assert torch.equal(call(ws), ref)
            assert size == need or bool((ws == 7).all())
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call(torch.empty(need, dtype=torch.uint8))
