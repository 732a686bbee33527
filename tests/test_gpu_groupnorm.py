"""GPU parity of the group norm (forward and gradients) with the fp64 oracle.

Tolerance, per value:  |gpu - oracle| <= u |oracle| + c K A, with
 * u half a step of the output's type (bf16 2^-8, fp32 2^-24);
 * A the output's formula over absolute values (sums of |terms|);
 * c = 600 * 2^-24: sums of a group in lanes, then trees (at most 200 additions in a row), and 8 ulp
   each for exp2, rcp, sqrt and the division, with exp2's argument rounded (|u| up to 40);
 * K = 1 + max |x| rstd over the group (+ |w|): an error of the mean moves xh by that much.
"""
import numpy as np
import pytest

import synth
from oracle.norm_oracle import groupnorm, groupnorm_bwd, parts, sigmoid
from tests.gpu_util import to_dev, to_host

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def ssm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_50_amd as m
    m.lib()
    return m


def make(B, L, C, dt, seed, affine, gate):
    r = np.random.default_rng(seed)
    st = lambda a: synth.store(np.asarray(a, np.float32), dt)  # noqa: E731
    c = {"x": st(r.standard_normal((B, L, C)) + 3.0 * r.standard_normal(C)), "dy": st(r.standard_normal((B, L, C)))}
    c["z"] = st(2.0 * r.standard_normal((B, L, C))) if gate else None
    c["w"] = (1.0 + 0.3 * r.standard_normal(C)).astype(np.float32) if affine else None
    c["b"] = (0.3 * r.standard_normal(C)).astype(np.float32) if affine else None
    return c


def rows(a, span):
    return None if a is None else (a.reshape(-1, 1, a.shape[-1]) if span == "token" else a)


def bounds(x, G, w, b, z, dy, silu, eps=EPS):
    """c K A for y and every gradient."""
    xh, rstd, u, a, gate = parts(x, G, w, b, z, eps, silu)
    N, L, C = xh.shape
    grp = lambda t: t.reshape(N, L, G, C // G)  # noqa: E731
    wa = np.ones(C) if w is None else np.abs(np.asarray(w, np.float64))
    ba = np.zeros(C) if b is None else np.abs(np.asarray(b, np.float64))
    K = (1.0 + np.abs(grp(np.asarray(x, np.float64))).max((1, 3), keepdims=True) * rstd) * np.ones((N, L, G, C // G))
    K = K.reshape(N, L, C)
    gate = np.abs(gate) + np.zeros_like(xh)
    c = 600 * 2.0 ** -24
    # |silu'| and |silu''| are below 1.1 and 0.51, and silu(u) below |u|
    uu = np.abs(xh) * wa + ba
    out = {"y": c * K * gate * 1.1 * (uu + wa)}
    ge = np.abs(dy) * gate * 1.1 * (1.0 + uu + wa)              # |g|, its slope in u taken in
    e = grp(ge * wa * K)
    n = grp(np.abs(xh) + 1.0)
    out["dx"] = c * (rstd * (e + e.mean((1, 3), keepdims=True) * n + n * (e * n).mean((1, 3), keepdims=True) * grp(K))).reshape(N, L, C)
    out["dw"] = c * (ge * K * (np.abs(xh) + 1.0)).sum((0, 1))
    out["dbias"] = c * (ge * K).sum((0, 1))
    if z is not None:
        zz = np.asarray(z, np.float64)
        out["dz"] = c * K * np.abs(dy) * 1.1 * (uu + wa) * (1.0 + np.abs(zz)) * np.maximum(sigmoid(zz), 1e-6)
    return out


def check(got, ref, lim, dt, what):
    g = to_host(got).reshape(ref.shape)
    assert np.isfinite(g).all(), what
    tol = (2.0 ** -8 if dt == "bf16" else 2.0 ** -24) * np.abs(ref) + lim + 1e-30
    worst = float((np.abs(g - ref) / tol).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"


# B, L, C, G, span, silu, gate, affine, dtype
CASES = [
    (1, 1, 1, 1, "token", False, False, False, "f32"),
    (2, 3, 8, 8, "token", False, False, True, "bf16"),       # groups of one channel
    (1, 1, 1024, 16, "token", False, True, True, "bf16"),
    (3, 5, 64, 1, "token", True, False, True, "f32"),
    (2, 7, 36, 3, "token", False, True, True, "bf16"),       # 12 channels: single elements
    (2, 9, 330, 10, "token", True, True, True, "f32"),
    (4, 33, 96, 4, "token", False, True, False, "bf16"),     # 24 channels: teams with idle lanes
    (2, 17, 512, 1, "token", False, True, True, "bf16"),     # one wave a group
    (2, 70, 1536, 1, "token", True, False, True, "bf16"),
    (1, 40, 5000, 1, "token", False, False, True, "f32"),    # a workgroup a group; the backward in slabs
    (1, 3, 20000, 1, "token", True, True, True, "bf16"),     # beyond a workgroup's registers
    (1, 3, 9001, 1, "token", False, False, True, "f32"),
    (2, 50, 64, 8, "sequence", True, False, True, "bf16"),
    (2, 1, 48, 6, "sequence", False, True, True, "f32"),
    (3, 1001, 330, 10, "sequence", True, False, True, "f32"),
    (2, 4000, 512, 32, "sequence", True, False, True, "bf16"),
    (1, 700, 4096, 2, "sequence", False, True, False, "bf16"),
    (5, 257, 99, 3, "sequence", False, True, True, "bf16"),
    (1, 20000, 8, 1, "sequence", True, False, True, "f32"),
    (2, 3000, 300, 1, "sequence", False, False, True, "f32"),
]


@pytest.mark.parametrize("B,L,C,G,span,silu,gate,affine,dt", CASES)
def test_parity(ssm, B, L, C, G, span, silu, gate, affine, dt):
    import torch
    c = make(B, L, C, dt, L + C + G, affine, gate)
    x, z, dy = (to_dev(c[n], dt) for n in ("x", "z", "dy"))
    w, b = (None if c[n] is None else torch.from_numpy(c[n]).cuda() for n in ("w", "b"))
    act = "silu" if silu else "none"
    y, mean, rstd = ssm.groupnorm_fwd(x, G, w, b, z, span=span, activation=act, eps=EPS, return_stats=True)
    g = ssm.groupnorm_bwd(x, G, w, b, z, dy, mean, rstd, span=span, activation=act)
    torch.cuda.synchronize()
    xs, zs, dys = (None if c[n] is None else rows(synth.to_f64(c[n], dt), span) for n in ("x", "z", "dy"))
    lim = bounds(xs, G, c["w"], c["b"], zs, dys, silu)
    check(y, groupnorm(xs, G, c["w"], c["b"], zs, EPS, silu), lim["y"], dt, "y")
    assert torch.equal(ssm.groupnorm_fwd(x, G, w, b, z, span=span, activation=act, eps=EPS), y)
    r = groupnorm_bwd(xs, G, c["w"], c["b"], zs, dys, EPS, silu)
    check(g["dx"], r["dx"], lim["dx"], dt, "dx")
    if affine:
        check(g["dw"], r["dw"], lim["dw"], "f32", "dw")
        check(g["dbias"], r["dbias"], lim["dbias"], "f32", "dbias")
    else:
        assert g["dw"] is None and g["dbias"] is None
    if gate:
        check(g["dz"], r["dz"], lim["dz"], dt, "dz")
    again = ssm.groupnorm_bwd(x, G, w, b, z, dy, mean, rstd, span=span, activation=act)
    for n in g:
        assert g[n] is None or torch.equal(g[n], again[n]), n


@pytest.mark.parametrize("L,span", [(1, "token"), (3000, "sequence")])
def test_offsets_and_constants(ssm, L, span):
    """A far outlier first, a large common offset, and constant groups (variance 0)."""
    import torch
    r = np.random.default_rng(1)
    x = r.standard_normal((2, L, 64)).astype(np.float32)
    x[0, 0, 0] = 1e4
    x[1] += 1000.0
    x[1, :, 32:] = 7.0
    y = ssm.groupnorm_fwd(torch.from_numpy(x).cuda(), 2, span=span)
    ref = groupnorm(rows(x.astype(np.float64), span), 2, eps=EPS)
    lim = bounds(rows(x.astype(np.float64), span), 2, None, None, None, np.zeros(1), False)["y"]
    check(y, ref, lim, "f32", "y")
    assert not to_host(y)[1, :, 32:].any()


def test_nan_stays_in_its_group(ssm):
    import torch
    for L, span in ((6, "token"), (2000, "sequence")):
        x = torch.randn(3, L, 64, device="cuda")
        y = ssm.groupnorm_fwd(x, 4, span=span)
        x2 = x.clone()
        x2[1, 2, 20] = float("nan")
        y2 = ssm.groupnorm_fwd(x2, 4, span=span)
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[1, (2 if span == "token" else slice(None)), 16:32] = True
        assert torch.isnan(y2[hit]).all() and torch.equal(y2[~hit], y[~hit])


def test_two_dimensions_and_refusals(ssm):
    import torch
    x = torch.randn(5, 96, device="cuda").bfloat16()
    assert torch.equal(ssm.groupnorm_fwd(x, 6), ssm.groupnorm_fwd(x[:, None], 6)[:, 0])
    for bad in (lambda: ssm.groupnorm_fwd(x.t(), 5), lambda: ssm.groupnorm_fwd(x, 6, w=torch.ones(95, device="cuda")),
                lambda: ssm.groupnorm_fwd(x, 6, out=torch.empty(5, 97, device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssm.groupnorm_fwd(x, 6, z=x.float()), lambda: ssm.groupnorm_fwd(x.half(), 6)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ssm.SSMError, match="divide"):
        ssm.groupnorm_fwd(x, 7)
    assert ssm.groupnorm_fwd(x[:0], 6).shape == (0, 96)


def test_autograd_and_differences(ssm):
    import torch
    for span in ("token", "sequence"):
        x, z, dy = (torch.randn(2, 40, 48, device="cuda") for _ in range(3))
        w, b = torch.randn(48, device="cuda"), torch.randn(48, device="cuda")
        leaves = [t.clone().requires_grad_() for t in (x, w, b, z)]
        y = ssm.group_norm(leaves[0], 3, *leaves[1:], span=span, activation="silu")
        got = torch.autograd.grad(y, leaves, dy.transpose(0, 1).contiguous().transpose(0, 1))
        _, mean, rstd = ssm.groupnorm_fwd(x, 3, w, b, z, span=span, activation="silu", return_stats=True)
        ref = ssm.groupnorm_bwd(x, 3, w, b, z, dy, mean, rstd, span=span, activation="silu")
        for g, n in zip(got, ("dx", "dw", "dbias", "dz")):
            assert torch.equal(g, ref[n]), n
        f = lambda t: (ssm.groupnorm_fwd(*t[:1], 3, *t[1:], span=span, activation="silu") * dy).double().sum()  # noqa: E731
        for i, g in enumerate(got):
            d = torch.randn_like(leaves[i])
            at = lambda e: [t + e * d if j == i else t for j, t in enumerate((x, w, b, z))]  # noqa: E731
            num, want = float(f(at(1e-2)) - f(at(-1e-2))) / 2e-2, float((g * d).double().sum())
            # e^2 f'''/6: 1e-4 of a sum of 3840 terms of size 1 (about 60 rms each way), and fp32 roundings over 2e-2
            assert abs(num - want) <= 0.02 * abs(want) + 0.5, (span, i)


def test_captured_and_other_stream(ssm):
    import torch
    x, z, dy = (torch.randn(4, 1500, 64, device="cuda").bfloat16() for _ in range(3))
    w, b = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")

    def work():
        out = []
        for span in ("token", "sequence"):
            y, m, r = ssm.groupnorm_fwd(x, 4, w, b, z, span=span, return_stats=True)
            out += [y, m, r, *ssm.groupnorm_bwd(x, 4, w, b, z, dy, m, r, span=span).values()]
        return out

    ref = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = ssm.groupnorm_fwd(x, 4, w, b, z, span="sequence", stream=side)
    side.synchronize()
    assert torch.equal(y, ssm.groupnorm_fwd(x, 4, w, b, z, span="sequence"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        dy.copy_(torch.randn_like(x))
        ref = [t.clone() for t in work()]
        torch.cuda.synchronize()
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for j, (t, r) in enumerate(zip(held, ref)):
            assert torch.equal(t, r), (i, j)


def test_more_threads_than_32_bits_count(ssm):
    """2^26 + 64 groups of 33 channels, a wave each: the last rows are those of a small call."""
    import torch
    rows, G = (1 << 20) + 1, 64
    x = torch.empty(rows, 33 * G, device="cuda", dtype=torch.bfloat16)
    x.view(-1)[-20 * 33 * G:] = torch.randn(20 * 33 * G, device="cuda").bfloat16()
    x[:-20] = x[-1]
    y, mean, rstd = ssm.groupnorm_fwd(x, G, return_stats=True)
    ref = ssm.groupnorm_fwd(x[-20:].clone(), G, return_stats=True)
    for a, b in zip((y, mean, rstd), ref):
        assert torch.equal(a[-20:], b) and torch.equal(a[:1000], b[-1:].expand(1000, -1))


# Wide tokens and short sequences: the backward walks each group
WALKED = [
    (2, 150, 5000, 1, "token", True, True, True, "f32"),
    (1, 300, 8192, 1, "token", False, True, True, "bf16"),
    (1, 70, 9001, 1, "token", False, False, True, "f32"),     # single elements
    (2, 40, 1040, 2, "token", False, True, False, "bf16"),
    (2, 40, 1030, 2, "token", True, True, True, "bf16"),      # 515 channels: single elements
    (300, 2, 96, 4, "sequence", True, False, True, "f32"),
    (33, 4, 330, 10, "sequence", False, True, True, "f32"),
    (9, 3, 4096, 2, "sequence", True, True, True, "bf16"),
    (5, 2, 20000, 1, "sequence", False, True, True, "bf16"),
    (70000, 4, 16, 2, "sequence", True, True, True, "bf16"),  # more rows than a launch has slabs for
    (66000, 5, 12, 3, "sequence", False, True, True, "f32"),
    (2, 1, 70000, 1, "token", False, False, True, "bf16"),
]


@pytest.mark.parametrize("B,L,C,G,span,silu,gate,affine,dt", WALKED)
def test_parity_walked(ssm, B, L, C, G, span, silu, gate, affine, dt):
    test_parity(ssm, B, L, C, G, span, silu, gate, affine, dt)


def test_more_wide_tokens_than_65535(ssm):
    """66000 tokens of 515 channels (more than a team's registers hold in the backward): the last tokens' dx and dz
    are those of a small call, dw and dbias those of the formula in 64 bits."""
    import torch
    N, C = 66000, 515
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, z, dy = (torch.randn(N, C, device="cuda", generator=gen).bfloat16() for _ in range(3))
    w, b = (torch.randn(C, device="cuda", generator=gen) for _ in range(2))
    _, mean, rstd = ssm.groupnorm_fwd(x, 1, w, b, z, return_stats=True)
    g = ssm.groupnorm_bwd(x, 1, w, b, z, dy, mean, rstd)
    tail = [t[-8:].clone() for t in (x, z, dy, mean, rstd)]
    ref = ssm.groupnorm_bwd(tail[0], 1, w, b, tail[1], tail[2], tail[3], tail[4])
    for n in ("dx", "dz"):
        assert torch.equal(g[n][-8:], ref[n]), n
    xd, zd = x.double(), z.double()
    xh = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
    e = dy.double() * zd * torch.sigmoid(zd)
    for got, term in ((g["dw"], e * xh), (g["dbias"], e)):
        # rows in slabs of at most 300 additions in a row and trees: 600 * 2^-24 of the sum of |terms|, as above
        assert bool(((got.double() - term.sum(0)).abs() <= 600 * 2.0 ** -24 * term.abs().sum(0)).all())


def test_wide_tokens_train(ssm):
    """The layer norm of wide tokens, through autograd."""
    import torch
    x = torch.randn(3, 50, 6000, device="cuda", requires_grad=True)
    w = torch.randn(6000, device="cuda", requires_grad=True)
    dy = torch.randn(3, 50, 6000, device="cuda")
    got = torch.autograd.grad(ssm.group_norm(x, 1, w), (x, w), dy)
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ref = torch.autograd.grad(torch.nn.functional.layer_norm(xd, (6000,), wd, None, 1e-5), (xd, wd), dy.double())
    for g, r in zip(got, ref):
        # 600 * 2^-24 of terms of size |x| |w| |dy|, at most 6^3, and of 150 such terms' sum in dw (root mean square 20)
        assert float((g.double() - r).abs().max()) <= 600 * 2.0 ** -24 * 6.0 ** 3


def test_walked_backward_captured_and_on_two_streams(ssm):
    """Wide tokens and short sequences in a graph, replayed over new inputs between eager calls; and two calls at once."""
    import torch
    x, z, dy = (torch.randn(6, 3, 9000, device="cuda").bfloat16() for _ in range(3))
    w, b = torch.randn(9000, device="cuda"), torch.randn(9000, device="cuda")

    def work(stream=None):
        out = []
        for span in ("token", "sequence"):
            _, m, r = ssm.groupnorm_fwd(x, 2, w, b, z, span=span, return_stats=True, stream=stream)
            out += ssm.groupnorm_bwd(x, 2, w, b, z, dy, m, r, span=span, stream=stream).values()
        return out

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        for t in (x, z, dy):
            t.copy_(torch.randn(t.shape, device="cuda"))
        ref = [t.clone() for t in work()]
        torch.cuda.synchronize()
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for j, (t, r) in enumerate(zip(held, ref)):
            assert torch.equal(t, r), (i, j)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [work(s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        for t, r in zip(g, ref):
            assert torch.equal(t, r)


def test_statistics_of_no_values(ssm):
    """A sequence of no positions has statistics of no values: zeros, not what the memory held."""
    import torch
    torch.full((12,), 7.0, device="cuda")   # (its memory is the allocator's next choice)
    x = torch.empty(3, 0, 16, device="cuda")
    y, mean, rstd = ssm.groupnorm_fwd(x, 4, span="sequence", return_stats=True)
    assert y.shape == (3, 0, 16) and mean.shape == rstd.shape == (3, 4) and not mean.any() and not rstd.any()
    g = ssm.groupnorm_bwd(x, 4, torch.ones(16, device="cuda"), None, None, x, mean, rstd, span="sequence")
    assert g["dx"].shape == x.shape and not g["dw"].any()
