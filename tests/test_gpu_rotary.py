"""GPU parity of rotary positions and head norms (forward and gradients) with the fp64 oracle.

Tolerance, per value:  |gpu - oracle| <= u |oracle| + c A, with u half a step of the output's type (bf16 2^-8, fp32
2^-24) and A the value's terms in absolute values:
 * forward, c = 40 * 2^-24: an angle is cut to a part of a turn in 64 bits and rounded to 32 (2^-26 of a turn: 2.6 * 2^-24
   rad), cosine and sine are 2 ulp off and scaled once (5), two products and a sum (3); normed: squares in lanes and a tree (22
   roundings of positive terms, half of that under the root), rsq and mean (4), two products (2): 29;
 * dx, c = 150 * 2^-24: g as above (11), e (1), its sum with x (24, a product more each), rstd three times (45), two
   products and a difference of terms that A adds up (6): 87, and as much again for e's own error inside that sum;
 * dw, c = 600 * 2^-24: rows of a lane one after another (under 300 here), teams (256), workgroups (under 64) and g xh.
"""
import numpy as np
import pytest

import synth
from oracle import rotary_oracle as ro
from tests.gpu_util import to_dev, to_host

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": E}


@pytest.fixture(scope="module")
def ssm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_50_amd as m
    m.lib()
    return m


def values(a, dt):
    """(storage form, the same values in 64 bits)"""
    st = synth.store(np.asarray(a, np.float32), dt)
    return st, to_host(to_dev(st, dt)) if dt == "bf16" else np.asarray(st, np.float64)


def make(B, L, hq, hk, d, rot, dt, seed, far=100, single=False):
    """q and k as parts of one wider projection, weights, positions, gradients: on the GPU, and in 64 bits."""
    import torch
    r = np.random.default_rng(seed)
    proj, val = values(r.standard_normal((B, L, (hq + 2 * hk) * d)), dt)
    dev = to_dev(proj, dt).view(B, L, hq + 2 * hk, d)
    val = val.reshape(B * L, hq + 2 * hk, d)
    c = {"q": dev[:, :, :hq], "k": dev[:, :, hq:hq + hk], "xq": val[:, :hq], "xk": val[:, hq:hq + hk]}
    p = (r.integers(0, far, (B, 1)) + np.arange(L)).astype(np.int32)
    c["pos"], c["p"] = torch.from_numpy(p).cuda(), p.reshape(-1)
    c["f"] = 10000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))
    c["freqs"] = torch.from_numpy(c["f"]).cuda()
    for n, h in (("q", hq), ("k", hk)):
        c["w" + n] = (1.0 + 0.3 * r.standard_normal(d)).astype(np.float32)
        st, c["g" + n] = values(r.standard_normal((B, L, h, d)), dt)
        c["d" + n] = to_dev(st, dt)
        c["g" + n] = c["g" + n].reshape(B * L, h, d)
    if single:
        c = {n: t[:, 0] if n in ("q", "k", "dq", "dk") else t for n, t in c.items()}
        c["pos"] = c["pos"][:, 0].contiguous()
    return c


def close(got, ref, lim, dt, what):
    g = to_host(got).reshape(ref.shape)
    assert np.isfinite(g).all(), what
    worst = float((np.abs(g - ref) / (HALF[dt] * np.abs(ref) + lim + 1e-35)).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"


def w_dev(w):
    import torch
    return torch.from_numpy(w).cuda()


# B, L, q heads, k heads, dim, rot, interleaved, dtype
CASES = [
    (1, 1, 16, 16, 64, 64, False, "bf16"),      # 16-byte loads
    (3, 77, 8, 2, 128, 128, False, "bf16"),
    (2, 50, 4, 4, 128, 128, True, "bf16"),
    (2, 33, 3, 1, 256, 64, False, "bf16"),      # half a wave to a row, a part of it turns
    (2, 33, 6, 3, 80, 32, True, "bf16"),
    (3, 21, 5, 5, 72, 24, False, "bf16"),       # 8-byte loads
    (3, 21, 5, 1, 40, 40, True, "bf16"),
    (2, 19, 3, 2, 33, 16, False, "bf16"),       # single elements, an odd column
    (2, 19, 3, 2, 33, 32, True, "bf16"),
    (2, 19, 2, 1, 255, 254, False, "bf16"),     # single elements, two units a lane
    (2, 19, 2, 1, 255, 30, True, "bf16"),
    (1, 5, 1, 1, 1, 0, False, "bf16"),          # nothing turns
    (1, 9, 1, 1, 2, 2, True, "bf16"),
    (2, 41, 6, 2, 64, 64, False, "f32"),
    (2, 41, 6, 2, 72, 40, True, "f32"),
    (2, 41, 6, 2, 256, 256, False, "f32"),
    (3, 10, 9, 3, 36, 36, False, "f32"),        # single elements
    (3, 10, 9, 3, 130, 66, True, "f32"),
    (2, 2100, 3, 1, 32, 32, False, "bf16"),     # several tokens a workgroup, several turns
    (2, 2100, 70, 2, 16, 16, True, "f32"),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_turn(ssm, case):
    B, L, hq, hk, d, rot, inter, dt = case
    if rot == 0:
        return
    c = make(B, L, hq, hk, d, rot, dt, 1)
    how = {"layout": "interleaved" if inter else "half", "magnitude": 1.25}
    q, k = ssm.rotary_fwd(c["q"], c["k"], c["pos"], c["freqs"], **how)
    dq, dk = ssm.rotary_bwd(c["dq"], c["dk"], c["pos"], c["freqs"], **how)
    for n, got, back, x in (("q", q, False, "xq"), ("k", k, False, "xk"), ("dq", dq, True, "gq"), ("dk", dk, True, "gk")):
        ref = ro.turn(c[x], c["p"], c["f"], inter, 1.25, back)
        close(got, ref, 40 * E * ro.turn_size(c[x], c["f"], inter, 1.25), dt, n)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_norm_and_gradients(ssm, case):
    B, L, hq, hk, d, rot, inter, dt = case
    c = make(B, L, hq, hk, d, rot, dt, 2)
    eps, mag = 1e-3, 0.75
    how = {"eps": eps, "layout": "interleaved" if inter else "half", "magnitude": mag}
    pos, freqs = (c["pos"], c["freqs"]) if rot else (None, None)
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    q, k = ssm.qknorm_fwd(c["q"], c["k"], *w, pos, freqs, **how)
    g = ssm.qknorm_bwd(c["q"], c["k"], *w, pos, freqs, c["dq"], c["dk"], **how)
    for n, got in (("q", q), ("k", k)):
        x, wn = c["x" + n], c["w" + n]
        u, r = ro.norm(x, wn, eps)
        close(got, ro.turn(u, c["p"], c["f"], inter, mag), 40 * E * ro.turn_size(u, c["f"], inter, mag), dt, n)
        back = ro.turn(c["g" + n], c["p"], c["f"], inter, mag, True)
        dx, dw = ro.norm_bwd(x, wn, back, eps)
        ga = ro.turn_size(c["g" + n], c["f"], inter, mag)
        e = ga * np.abs(wn)
        close(g["d" + n], dx, 150 * E * r * (e + np.abs(x) * r * r * (e * np.abs(x)).mean(-1, keepdims=True)), dt, "d" + n)
        close(g["dw" + n], dw, 600 * E * (ga * np.abs(x) * r).reshape(-1, d).sum(0), "f32", "dw" + n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_single_tokens_without_k_or_weights(ssm, dt):
    c = make(37, 1, 6, 3, 64, 32, dt, 3, far=1 << 20, single=True)
    q = ssm.qknorm_fwd(c["q"], None, None, None, c["pos"], c["freqs"], eps=0.0)
    u, _ = ro.norm(c["xq"], None, 0.0)
    close(q, ro.turn(u, c["p"], c["f"]), 40 * E * ro.turn_size(u, c["f"]), dt, "q")
    q = ssm.rotary_fwd(c["q"], None, c["pos"], c["freqs"])
    close(q, ro.turn(c["xq"], c["p"], c["f"]), 40 * E * ro.turn_size(c["xq"], c["f"]), dt, "q")
    g = ssm.qknorm_bwd(c["q"], None, w_dev(c["wq"]), None, c["pos"], c["freqs"], c["dq"], need_dw=False)
    assert g["dk"] is None and g["dwq"] is None and g["dwk"] is None


def test_far_and_negative_positions(ssm):
    """Angles at the ends of the positions' range: 32-bit products would be whole turns off."""
    import torch
    c = make(1, 6, 2, 1, 64, 64, "f32", 4)
    p = np.array([0, -1, 1048575, 2 ** 31 - 1, -2 ** 31, 123456789], np.int32)
    q, k = ssm.rotary_fwd(c["q"], c["k"], torch.from_numpy(p[None]).cuda(), c["freqs"])
    # (the oracle's angle, in the longest float there is, is off by 2^31 2^-53 at most: 2^-22, and the kernel's too)
    lim = (40 * E + 2.0 ** -20) * ro.turn_size(c["xq"], c["f"])
    close(q, ro.turn(c["xq"], p, c["f"]), lim, "f32", "q")


def test_positions_shared_by_rows(ssm):
    import torch
    c = make(4, 9, 2, 2, 32, 32, "bf16", 5)
    p = torch.arange(9, dtype=torch.int32, device="cuda") * 3
    q, k = ssm.rotary_fwd(c["q"], c["k"], p, c["freqs"])
    q2, k2 = ssm.rotary_fwd(c["q"], c["k"], p.repeat(4, 1), c["freqs"])
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_rows_off_their_alignment(ssm, dt, off):
    """Slices that start and stride off 16 bytes take narrower loads, to the same values."""
    import torch
    c = make(2, 17, 4, 2, 64, 32, dt, 6)
    wide = torch.zeros(2, 17, 6 * 64 + off, dtype=c["q"].dtype, device="cuda")
    wide[..., off:off + 256], wide[..., off + 256:off + 384] = c["q"].flatten(2), c["k"].flatten(2)
    q, k = wide[..., off:off + 256].view(2, 17, 4, 64) if off == 0 else wide[..., off:off + 256].unflatten(-1, (4, 64)), \
        wide[..., off + 256:off + 384].unflatten(-1, (2, 64))
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    a = ssm.rotary_fwd(c["q"], c["k"], c["pos"], c["freqs"])
    b = ssm.rotary_fwd(q, k, c["pos"], c["freqs"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    n = ssm.qknorm_fwd(q, k, *w, c["pos"], c["freqs"])
    for name, got in (("q", n[0]), ("k", n[1])):
        u, _ = ro.norm(c["x" + name], c["w" + name])
        close(got, ro.turn(u, c["p"], c["f"]), 40 * E * ro.turn_size(u, c["f"]), dt, name)
    g = ssm.qknorm_bwd(q, k, *w, c["pos"], c["freqs"], c["dq"], c["dk"])
    dx, _ = ro.norm_bwd(c["xq"], c["wq"], ro.turn(c["gq"], c["p"], c["f"], back=True))
    r = ro.norm(c["xq"])[1]
    e = ro.turn_size(c["gq"], c["f"]) * np.abs(c["wq"])
    close(g["dq"], dx, 150 * E * r * (e + np.abs(c["xq"]) * r * r * (e * np.abs(c["xq"])).mean(-1, keepdims=True)), dt, "dq")


def test_nan_and_infinity_stay_in_their_head(ssm):
    import torch
    c = make(2, 11, 4, 2, 64, 32, "f32", 7)
    q = c["q"].clone()
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    clean = ssm.qknorm_fwd(q, c["k"], *w, c["pos"], c["freqs"])[0]
    q[1, 3, 2, 5], q[0, 4, 0, 60] = float("nan"), float("inf")
    got = ssm.qknorm_fwd(q, c["k"], *w, c["pos"], c["freqs"])[0]
    assert torch.isnan(got[1, 3, 2]).all()
    same = torch.ones(2, 11, 4, dtype=torch.bool, device="cuda")
    same[1, 3, 2] = same[0, 4, 0] = False
    assert torch.equal(got[same], clean[same])
    turned = ssm.rotary_fwd(q, c["k"], c["pos"], c["freqs"])[0]
    assert torch.isinf(turned[0, 4, 0, 60]) and torch.isfinite(turned[0, 4, 0, :60]).all()
    assert torch.isnan(turned[1, 3, 2]).sum() == 2 and torch.isfinite(turned[1, 3, :2]).all()


@pytest.mark.parametrize("scale", [1e-15, 1e15])
def test_gradients_of_tiny_and_huge_rows(ssm, scale):
    """rstd reaches 1e15 without eps: its cube would be infinite."""
    c = make(2, 11, 4, 2, 64, 32, "f32", 9)
    q = (c["q"] * scale).contiguous()
    x = to_host(q).reshape(22, 4, 64)
    g = ssm.qknorm_bwd(q, None, w_dev(c["wq"]), None, c["pos"], c["freqs"], c["dq"], eps=0.0)
    _, r = ro.norm(x, c["wq"], 0.0)
    dx, dw = ro.norm_bwd(x, c["wq"], ro.turn(c["gq"], c["p"], c["f"], back=True), 0.0)
    ga = ro.turn_size(c["gq"], c["f"])
    e = ga * np.abs(c["wq"])
    close(g["dq"], dx, 150 * E * r * (e + np.abs(x) * r * r * (e * np.abs(x)).mean(-1, keepdims=True)), "f32", "dq")
    close(g["dwq"], dw, 600 * E * (ga * np.abs(x) * r).reshape(-1, 64).sum(0), "f32", "dwq")


def test_as_many_heads_as_there_can_be(ssm):
    """4096 heads of a token, of which a turn of a workgroup takes one; and one head over many tokens."""
    for B, L, hq, hk, d in ((1, 3, 4000, 96, 16), (1, 70001, 1, 1, 16)):
        c = make(B, L, hq, hk, d, d, "bf16", 11)
        w = [w_dev(c["wq"]), w_dev(c["wk"])]
        q, k = ssm.qknorm_fwd(c["q"], c["k"], *w, c["pos"], c["freqs"])
        g = ssm.qknorm_bwd(c["q"], c["k"], *w, c["pos"], c["freqs"], c["dq"], c["dk"])
        for n, got in (("q", q), ("k", k)):
            u, r = ro.norm(c["x" + n], c["w" + n])
            close(got, ro.turn(u, c["p"], c["f"]), 40 * E * ro.turn_size(u, c["f"]), "bf16", n)
            dx, dw = ro.norm_bwd(c["x" + n], c["w" + n], ro.turn(c["g" + n], c["p"], c["f"], back=True))
            ga = ro.turn_size(c["g" + n], c["f"])
            e = ga * np.abs(c["w" + n])
            x = np.abs(c["x" + n])
            close(g["d" + n], dx, 150 * E * r * (e + x * r * r * (e * x).mean(-1, keepdims=True)), "bf16", "d" + n)
            close(g["dw" + n], dw, 600 * E * (ga * x * r).reshape(-1, d).sum(0), "f32", "dw" + n)


def test_empty_and_deterministic(ssm):
    import torch
    c = make(2, 1500, 9, 3, 64, 64, "bf16", 8)
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    a, b = (ssm.qknorm_bwd(c["q"], c["k"], *w, c["pos"], c["freqs"], c["dq"], c["dk"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    e = c["q"][:, :0]
    q, k = ssm.rotary_fwd(e, c["k"][:, :0], c["pos"][:, :0].contiguous(), c["freqs"])
    assert q.shape == (2, 0, 9, 64) and k.shape == (2, 0, 3, 64)
    g = ssm.qknorm_bwd(e, c["k"][:, :0], *w, c["pos"][:, :0].contiguous(), c["freqs"], c["dq"][:, :0].contiguous(), c["dk"][:, :0].contiguous())
    assert not g["dwq"].any() and not g["dwk"].any()


def test_autograd(ssm):
    """The autograd forms give the entry points' gradients; an output that nothing is made of counts as zero."""
    import torch
    c = make(2, 13, 4, 2, 64, 32, "f32", 9)
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    ref = ssm.qknorm_bwd(c["q"], c["k"], *w, c["pos"], c["freqs"], c["dq"], c["dk"])
    leaves = [c["q"].detach().requires_grad_(), c["k"].detach().requires_grad_(), w[0].requires_grad_(), w[1].requires_grad_()]
    q, k = ssm.qk_norm(*leaves, c["pos"], c["freqs"])
    got = torch.autograd.grad([q, k], leaves, [c["dq"], c["dk"]])
    assert all(torch.equal(x, ref[n]) for x, n in zip(got, ("dq", "dk", "dwq", "dwk")))
    q, k = ssm.qk_norm(*leaves, c["pos"], c["freqs"])
    got = torch.autograd.grad(k, leaves, c["dk"])
    assert torch.equal(got[1], ref["dk"]) and torch.equal(got[3], ref["dwk"]) and not got[0].any() and not got[2].any()
    q, k = ssm.rotary(leaves[0], leaves[1], c["pos"], c["freqs"])
    got = torch.autograd.grad([q, k], leaves[:2], [c["dq"].transpose(1, 2).contiguous().transpose(1, 2), c["dk"]])
    both = ssm.rotary_bwd(c["dq"], c["dk"], c["pos"], c["freqs"])
    assert torch.equal(got[0], both[0]) and torch.equal(got[1], both[1])
    q = ssm.rotary(leaves[0], None, c["pos"], c["freqs"])
    assert torch.equal(torch.autograd.grad(q, leaves[0], c["dq"])[0], both[0])


def test_refusals(ssm):
    import torch
    c = make(2, 5, 4, 2, 32, 32, "bf16", 10)
    ok = (c["q"], c["k"], c["pos"], c["freqs"])
    for bad, err in (((c["q"], c["k"].float(), *ok[2:]), TypeError), ((c["q"], c["k"], c["pos"].long(), ok[3]), TypeError),
                     ((c["q"], c["k"], c["pos"][:1], ok[3]), ValueError), ((*ok[:3], c["freqs"].float()), TypeError),
                     ((*ok[:3], torch.zeros(17, dtype=torch.float64, device="cuda")), ValueError),
                     ((c["q"].transpose(2, 3), c["k"], *ok[2:]), ValueError), ((c["q"][0], c["k"], *ok[2:]), ValueError),
                     ((c["q"], c["k"], c["pos"].cpu(), ok[3]), ValueError)):
        with pytest.raises(err):
            ssm.rotary_fwd(*bad)
    with pytest.raises(ValueError):
        ssm.rotary_fwd(*ok, layout="other")
    with pytest.raises(ValueError):
        ssm.rotary_fwd(*ok, out=torch.empty_like(c["q"]))
    with pytest.raises(TypeError):
        ssm.rotary_fwd(c["q"].half(), None, *ok[2:])
    with pytest.raises(ValueError):
        ssm.qknorm_fwd(c["q"], c["k"], torch.ones(31, device="cuda"))
    with pytest.raises(ValueError):
        ssm.qknorm_bwd(c["q"], c["k"], dq_out=c["dq"])
    out = (torch.empty(2, 5, 4, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 5, 2, 32, dtype=torch.bfloat16, device="cuda"))
    v = out[0]._version
    assert ssm.rotary_fwd(*ok, out=out)[0] is out[0] and out[0]._version > v


def test_streams_and_graphs(ssm):
    """Two streams at once, and a captured training step replayed with new inputs between eager work."""
    import torch
    c = make(2, 700, 8, 4, 64, 64, "bf16", 11)
    w = [w_dev(c["wq"]), w_dev(c["wk"])]
    call = lambda s=None: ssm.qknorm_bwd(c["q"], c["k"], *w, c["pos"], c["freqs"], c["dq"], c["dk"], stream=s)  # noqa: E731
    ref = call()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [call(s) for _ in range(3) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(ref[n], g[n]) for g in got for n in ref)
    x = {n: c[n].clone() for n in ("q", "k", "dq", "dk")}
    step = lambda: (ssm.qknorm_fwd(x["q"], x["k"], *w, c["pos"], c["freqs"]),  # noqa: E731
                    ssm.qknorm_bwd(x["q"], x["k"], *w, c["pos"], c["freqs"], x["dq"], x["dk"]))
    with torch.cuda.stream(side[0]):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = step()
    for i in range(3):
        for n in x:
            x[n].copy_(c[n] * (1.0 + i))
        graph.replay()
        torch.cuda.synchronize()
        y, g = step()
        assert all(torch.equal(a, b) for a, b in zip(out, y)) and all(torch.equal(grads[n], g[n]) for n in g)


def test_strides_past_32_bits(ssm):
    """Tokens further apart than 2^31 elements in all."""
    import torch
    row = (1 << 24) + 8
    big = torch.empty(140 * row, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((140, 2, 64), (row, 64, 1))
    q.copy_(torch.randn(140, 2, 64, device="cuda"))
    p = torch.arange(140, dtype=torch.int32, device="cuda")
    f = ssm.rotary_freqs(64)[0]
    assert torch.equal(ssm.rotary_fwd(q, None, p, f), ssm.rotary_fwd(q.contiguous(), None, p, f))
    del big, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("norm", [False, True])
def test_angles_next_to_a_quarter_turn(ssm, norm):
    """A part of a turn is not cut to 32 bits: next to the zeros of cosine and sine, by less than half a 32-bit step of the part, they
    are as good as their own digits.  Relative to such a value of size t <= 2 pi 2^-27: the 32-bit remainder and its product
    with 2 pi 3 * 2^-24, the fused product with a sine or cosine of 2 ulp 4 * 2^-24, t^2 / 6 nothing; the norm 7 more: 14."""
    import torch
    near = np.repeat([0.25, 0.5, 0.75, 1.0], 4) + np.tile([2.0 ** -27, -2.0 ** -28, 2.0 ** -31, -2.0 ** -33], 4)
    f = 2 * np.pi * near
    q = torch.zeros(1, 1, 1, 32, device="cuda")
    q[..., :16] = 1.0
    pos, freqs = torch.ones(1, 1, dtype=torch.int32, device="cuda"), torch.from_numpy(f).cuda()
    if norm:
        y = ssm.qknorm_fwd(q, None, None, None, pos, freqs, eps=0.0)
    else:
        y = ssm.rotary_fwd(q, None, pos, freqs)
    y = to_host(y).reshape(2, 16) / (np.sqrt(2.0) if norm else 1.0)
    # (the frequency's own rounding to 64 bits is 2^-53 of it, 2^-18 of the smallest distance: what the 64-bit formula gives for it)
    ref = np.stack([np.cos(f), np.sin(f)])
    small = np.abs(ref) < 1e-6
    assert small.sum() == 16
    # (the kernel's product with 1 / (2 pi) rounds once more in 64 bits: 2^-53 of a turn, 2 pi 2^-53 rad, against 2 pi 2^-33)
    assert (np.abs(y - ref)[small] <= (14 * E + 2.0 ** -18) * np.abs(ref)[small]).all()
    assert (np.abs(y - ref)[~small] <= 14 * E).all()


@pytest.mark.parametrize("where", ["tokens", "heads"])
def test_sums_of_dw_are_joined_in_64_bits(ssm, where):
    """2^25 + 1 - 2^25, each term of another workgroup (one token each) or another team (a head each), whichever two are added first."""
    import itertools
    import torch
    n, d = 3, 16
    for order in itertools.permutations([2.0 ** 25, 1.0, -2.0 ** 25]):
        q = torch.ones(1, n if where == "tokens" else 1, 1 if where == "tokens" else n, d, device="cuda")
        dq = torch.tensor(order, device="cuda").view(q.shape[:-1])[..., None].expand(q.shape).contiguous()
        w = torch.ones(d, device="cuda")
        g = ssm.qknorm_bwd(q, None, w, None, dq_out=dq, eps=0.0)     # (xh is x: its mean square is one)
        assert torch.equal(g["dwq"], w), order
