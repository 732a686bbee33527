"""The operators of a layer one after another, as a model runs them:

* a joint projection's slices through qk_norm (norms and rotary positions), linear_attention and group_norm, trained
  through autograd and generated token by token;
* a Mamba-2 layer's packed prompts through ssdconv_fwd and their next tokens through ssdconv_update, with the gated
  group norm behind both, the tokens as a graph whose slots move between replays.

Every stage is checked with its own operator's tolerances against the fp64 oracle on the stage's actual inputs, so no
tolerance spans two roundings.
"""
import numpy as np
import pytest

import synth
from oracle import rotary_oracle as ro
from oracle.linattn_oracle import linattn, linattn_bwd
from oracle.norm_oracle import groupnorm
from oracle.ssdconv_oracle import mixer
from tests import test_gpu_groupnorm as tn
from tests import test_gpu_linattn as ta
from tests import test_gpu_rotary as tr
from tests import test_gpu_ssdconv as ts
from tests.gpu_util import to_host
from tests.test_gpu_rotary import E, ssm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def stored(t, dt):
    """A tensor's own values in storage form (exact)."""
    return synth.store(to_host(t).astype(np.float32), dt)


def normed(c, x, wn, g=None):
    """qk_norm's output and bound, or its gradients and bounds, from 64-bit rows [tokens, heads, dim]."""
    u, r = ro.norm(x, wn, 1e-6)
    if g is None:
        return ro.turn(u, c["p"], c["f"]), 40 * E * ro.turn_size(u, c["f"])
    back, ga = ro.turn(g, c["p"], c["f"], back=True), ro.turn_size(g, c["f"])
    dx, dw = ro.norm_bwd(x, wn, back, 1e-6)
    e = ga * np.abs(wn)
    return (dx, 150 * E * r * (e + np.abs(x) * r * r * (e * np.abs(x)).mean(-1, keepdims=True)), dw,
            600 * E * (ga * np.abs(x) * r).reshape(-1, x.shape[-1]).sum(0))


@pytest.mark.parametrize("B,L,H,G,d,dt", [(2, 130, 4, 4, 64, "bf16"), (3, 40, 6, 2, 48, "f32"), (1, 1, 2, 1, 128, "bf16")])
def test_training_step(ssm, B, L, H, G, d, dt):  # noqa: F811
    import torch
    c = tr.make(B, L, H, G, d, d, dt, 31)
    x = torch.cat([c["q"].flatten(2), c["k"].flatten(2), torch.randn(B, L, G * d, device="cuda").to(c["q"].dtype)], -1).requires_grad_()
    q0, k0, v = (t.unflatten(-1, (-1, d)) for t in x.split([H * d, G * d, G * d], -1))
    wq, wk = (torch.from_numpy(c["w" + n]).cuda().requires_grad_() for n in ("q", "k"))
    a = torch.full((H,), -0.05, device="cuda", requires_grad=True)
    w, b = (torch.randn(H * d, device="cuda", requires_grad=True) for _ in range(2))
    z, do = (torch.randn(B, L, H * d, device="cuda").to(x.dtype) for _ in range(2))
    q, k = ssm.qk_norm(q0, k0, wq, wk, c["pos"], c["freqs"])
    y = ssm.linear_attention(q, k, v, a)
    for t in (q, k, y):
        t.retain_grad()
    o = ssm.group_norm(y.flatten(2), H, w, b, z)
    o.backward(do)
    torch.cuda.synchronize()
    for n, got, at in (("q", q, slice(0, H * d)), ("k", k, slice(H * d, (H + G) * d))):
        ref, lim = normed(c, c["x" + n], c["w" + n])
        tr.close(got.detach(), ref, lim, dt, n)
        dx, lx, dw, lw = normed(c, c["x" + n], c["w" + n], to_host(got.grad).reshape(c["x" + n].shape))
        tr.close(x.grad[..., at].contiguous(), dx, lx, dt, "d" + n)
        tr.close((wq if n == "q" else wk).grad, dw, lw, "f32", "dw" + n)
    lc = {"q": stored(q.detach(), dt), "k": stored(k.detach(), dt), "v": stored(v.detach(), dt), "a": np.full(H, -0.05, np.float32),
          "dy": stored(y.grad, dt), "dt": dt}
    (yr, _), (ya, _) = ta.both(linattn, lc, ("q", "k", "v", "a", d ** -0.5, None))
    ta.check(y.detach(), yr, ya, dt, lc, "y")
    ref, big = ta.both(linattn_bwd, lc, ("q", "k", "v", "a", d ** -0.5, None, "dy", None))
    ta.check(q.grad, ref["dq"], big["dq"], dt, lc, "dq'")
    ta.check(k.grad, ref["dk"], big["dk"], dt, lc, "dk'")
    ta.check(x.grad[..., (H + G) * d:].unflatten(-1, (G, d)).contiguous(), ref["dv"], big["dv"], dt, lc, "dv")
    ta.check(a.grad, ref["dlog_decay"], big["dlog_decay"], "f32", lc, "dlog_decay")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_then_tokens(ssm, dt):  # noqa: F811
    """Tokens one by one at their positions: the rows of the whole sequence's norm and turn, and its attention."""
    import torch
    B, L, P, H, d = 2, 70, 61, 4, 64
    c = tr.make(B, L, H, H, d, d // 2, dt, 32, far=5000)
    w = [torch.from_numpy(c["w" + n]).cuda() for n in ("q", "k")]
    a = torch.linspace(-0.3, -0.01, H, device="cuda")
    v = torch.randn(B, L, H, d, device="cuda").to(c["q"].dtype)
    q, k = ssm.qknorm_fwd(c["q"], c["k"], *w, c["pos"], c["freqs"])
    y, h = ssm.linattn_fwd(q[:, :P].contiguous(), k[:, :P].contiguous(), v[:, :P].contiguous(), a, return_last_state=True)
    out = [y]
    for t in range(P, L):
        qt, kt = ssm.qknorm_fwd(c["q"][:, t], c["k"][:, t], *w, c["pos"][:, t].contiguous(), c["freqs"])
        assert torch.equal(qt, q[:, t]) and torch.equal(kt, k[:, t])
        out.append(ssm.linattn_update(h, qt, kt, v[:, t], a).unsqueeze(1))
    lc = {"q": stored(q, dt), "k": stored(k, dt), "v": stored(v, dt), "a": a.cpu().numpy(), "dt": dt}
    (yr, hr), (ya, ha) = ta.both(linattn, lc, ("q", "k", "v", "a", d ** -0.5, None))
    ta.check(torch.cat(out, 1), yr, ya, dt, lc, "y")
    ta.check(h, hr, ha, "f32", lc, "h")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_served_mamba2_layer(ssm, dt):  # noqa: F811
    """Two batches of uneven prompts into one pool, one of them continuing slots of the other, then tokens of four
    sequences through a graph; the gated norm behind each."""
    import torch
    H, P, N, G, steps = 4, 64, 64, 2, 5
    lens, slots = [100, 7, 64], [5, 2, 0]
    c, dev = ts.make(lens + [steps] * 4, H, P, N, G, 4, dt, 33, slots=slots + [5, 2, 1, 0], pool=7)
    w, b = torch.randn(H * P, device="cuda"), torch.randn(H * P, device="cuda")
    zg = torch.randn(sum(lens) + 4 * steps, H * P, device="cuda").to(dev["xbc"].dtype)
    T = sum(lens)
    first = dict(dev, offsets=dev["offsets"][:4].contiguous(), slots=dev["slots"][:3].contiguous())
    y = torch.empty(T + 4 * steps, H, P, dtype=zg.dtype, device="cuda")
    ts.call(ssm, c, first, out=y, hint=False)
    # the tokens of sequence i lie in rows T + steps i ..: slot 1 starts from what its pool holds
    hold = {n: (None if dev[n] is None else dev[n][[T + steps * i for i in range(4)]].clone()) for n in ("xbc", "delta", "z")}
    gate = zg[:4].clone()
    moved = dict(dev, slots=torch.zeros(4, dtype=torch.int32, device="cuda"), **hold)

    def token():
        s = ts.step(ssm, c, moved, slice(None))
        return s, ssm.groupnorm_fwd(s.flatten(1), H, w, b, gate)
    keep = {n: dev[n].clone() for n in ("h", "conv_state")}
    with torch.cuda.stream(torch.cuda.Stream()):
        token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, o = token()
    for n in keep:
        dev[n].copy_(keep[n])
    real = torch.tensor([5, 2, 1, 0], dtype=torch.int32, device="cuda")
    for t in range(steps):
        order = torch.randperm(4, device="cuda")
        rows = T + steps * order + t
        for n in hold:
            if hold[n] is not None:
                moved[n].copy_(dev[n][rows])
        moved["slots"].copy_(real[order])
        gate.copy_(zg[rows])
        graph.replay()
        torch.cuda.synchronize()
        y[rows] = s
        ref = groupnorm(to_host(s).astype(np.float64).reshape(4, 1, H * P), H, to_host(w), to_host(b), to_host(gate).reshape(4, 1, H * P), 1e-5, False)
        ys, zs = (to_host(v).astype(np.float64).reshape(4, 1, H * P) for v in (s, gate))
        lim = tn.bounds(ys, H, to_host(w).astype(np.float64), to_host(b).astype(np.float64), zs, np.zeros(1), False)["y"]
        tn.check(o, ref, lim, dt, "o")
    # (the oracle takes the prompts first, then every sequence's tokens from its slot)
    ts.check(c, dev, y, mixer(c), 1000 * E, 1200 * E)
