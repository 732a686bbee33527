"""GPU parity of the served Mamba-2 mixer (packed prompts, single tokens) with the fp64 oracle.

Tolerance, per value:  |gpu - oracle| <= u |oracle| + c A, with u half a step of the output's type (bf16 2^-8, fp32 2^-24)
and A the oracle's bound (the formulas over absolute values, half the decays' exponents):
 * convolution and silu, 10 * 2^-24 for each of x, B and C; dt 5 (softplus) twice (in the decay, times 1.3, and in front);
   decays 2 ulp each, three factors, scans of 32; D, gate and roundings of factors 10: 80 in all;
 * a product of three-part factors leaves out less than 3 * 2^-24, two of them one after another in y: 6;
 * sums: at most 12 matrix instructions one after another a chunk for the state and 24 + 12 for y, each adding 32 terms and
   the sum before (33 roundings at worst; all relative to the absolute sum): the state of n chunks 12 * 33 n / 8 (no
   chunk's terms go through more than one chain of 12, and the sum of 32 inside an instruction keeps at least three bits
   more than its output), y on top 36 * 33 / 8;
 so c = (90 + 50 n + 150) 2^-24 for n chunks. bf16 y: factors of two parts are 2^-17 off and lo * lo is left out (2^-18): two
 products, 8 * 2^-17 more. Single tokens: one step of it without products of parts, c = 240 * 2^-24.
"""
import numpy as np
import pytest

import synth
from oracle.ssdconv_oracle import mixer
from tests.gpu_util import to_dev, to_host

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def ssm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_50_amd as m
    m.lib()
    return m


def make(lens, H, P, N, G, W, dt, seed, *, gate=True, softplus=True, D=True, bias=True, slots=None, fresh=None, behind=0, lead=0,
         joint=True, A=None, pool=None):
    """A case on the GPU ("dev") and in 64 bits."""
    import torch
    r = np.random.default_rng(seed)
    T, C, S = lead + sum(lens) + behind, H * P + 2 * G * N, len(lens)
    inner = H * P if gate else 0
    f32 = lambda a: np.asarray(a, np.float32)  # noqa: E731

    def stored(a):
        st = synth.store(f32(a), dt)
        d = to_dev(st, dt)
        return d, to_host(d)
    proj = r.standard_normal((T, inner + C + H))
    if not softplus:
        proj[:, inner + C:] = 0.1 * r.random((T, H))
    d, v = stored(proj)
    pool = S + 2 if pool is None else pool
    c = {"z": v[:, :inner].reshape(T, H, P) if gate else None, "xbc": v[:, inner:inner + C], "delta": v[:, inner + C:]}
    dev = {"z": d[:, :inner].view(T, H, P) if gate else None, "xbc": d[:, inner:inner + C], "delta": d[:, inner + C:]}
    if not joint:
        dev = {n: None if t is None else t.contiguous() for n, t in dev.items()}
    small = {"A": -np.exp(r.uniform(0, np.log(16), H)) if A is None else A, "D": 1 + 0.1 * r.standard_normal(H) if D else None,
             "delta_bias": np.log(np.expm1(np.exp(r.uniform(np.log(1e-3), np.log(1e-1), H)))) if softplus else None,
             "w": 0.5 * r.standard_normal((C, W)), "bias": 0.1 * r.standard_normal(C) if bias else None,
             "h": r.standard_normal((pool, H, P, N))}
    for n, a in small.items():
        c[n] = None if a is None else f32(a).astype(np.float64)
        dev[n] = None if a is None else torch.from_numpy(f32(a)).cuda()
    dev["conv_state"], c["conv_state"] = stored(r.standard_normal((pool, C, W - 1)))
    c["offsets"] = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    c["slots"] = (np.arange(S) if slots is None else np.asarray(slots)).astype(np.int64)
    c["fresh"] = np.zeros(S, bool) if fresh is None else np.asarray(fresh, bool)
    dev["offsets"] = torch.from_numpy(c["offsets"].astype(np.int32)).cuda()
    dev["slots"] = None if slots is None else torch.from_numpy(c["slots"].astype(np.int32)).cuda()
    dev["fresh"] = None if fresh is None else torch.from_numpy(c["fresh"]).cuda()
    c.update(G=G, softplus=softplus, dt=dt, longest=max(lens) if lens else 0)
    return c, dev


def call(ssm, c, dev, out=None, hint=True, **kw):
    return ssm.ssdconv_fwd(dev["xbc"], dev["delta"], dev["A"], dev["w"], dev["h"], dev["conv_state"], dev["offsets"], dev["slots"],
                           bias=dev["bias"], D=dev["D"], z=dev["z"], delta_bias=dev["delta_bias"], delta_softplus=c["softplus"],
                           fresh=dev["fresh"], max_seqlen=c["longest"] if hint else None, out=out, **kw)


def step(ssm, c, dev, rows, **kw):
    at = lambda n: None if dev[n] is None else dev[n][rows]  # noqa: E731
    return ssm.ssdconv_update(at("xbc"), at("delta"), dev["A"], dev["w"], dev["h"], dev["conv_state"], dev["slots"], bias=dev["bias"],
                              D=dev["D"], z=at("z"), delta_bias=dev["delta_bias"], delta_softplus=c["softplus"], **kw)


def close(got, ref, lim, half, what):
    g = to_host(got).reshape(ref.shape)
    ok = ~np.isnan(ref)
    assert np.isfinite(g[ok]).all(), what
    worst = float((np.abs(g - ref) / (half * np.abs(ref) + lim + 1e-30))[ok].max()) if ok.any() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"
    return worst


def check(c, dev, y, ref, c_h, c_y):
    bf = c["dt"] == "bf16"
    a = close(y, ref["y"], (c_y + (8 * 2.0 ** -17 if bf else 0.0)) * ref["y_hat"], 2.0 ** -8 if bf else E, "y")
    b = close(dev["h"], ref["h"], c_h * ref["h_hat"], E, "h")
    np.testing.assert_array_equal(to_host(dev["conv_state"]), ref["conv_state"])
    return a, b


def prompt(ssm, *args, **kw):
    c, dev = make(*args, **kw)
    ref = mixer(c)
    y = call(ssm, c, dev)
    n = (c["longest"] + 63) // 64
    check(c, dev, y, ref, (90 + 50 * n) * E, (240 + 50 * n) * E)
    return c, dev, y, ref


# lengths, H, P, N, G, W, dtype
CASES = [
    ([1], 1, 64, 128, 1, 4, "bf16"),
    ([1, 2, 3, 4, 5], 2, 64, 64, 1, 4, "bf16"),           # shorter than the filter
    ([63, 64, 65, 128, 129], 2, 64, 128, 1, 4, "bf16"),   # around a chunk
    ([17, 0, 200, 0, 1], 3, 64, 64, 1, 4, "bf16"),        # sequences without tokens
    ([300, 20], 4, 64, 128, 2, 4, "bf16"),                # two groups
    ([90, 33], 4, 48, 96, 1, 3, "bf16"),
    ([70], 3, 33, 20, 3, 2, "bf16"),                      # nothing a multiple of anything
    ([100, 30], 2, 80, 100, 1, 4, "bf16"),                # a second, partial block of channels
    ([66], 1, 130, 16, 1, 4, "bf16"),
    ([66, 10], 2, 16, 1, 1, 1, "bf16"),                   # no filter state, one state
    ([5, 70], 2, 1, 128, 2, 4, "bf16"),
    ([63, 64, 65, 1], 2, 64, 128, 1, 4, "f32"),
    ([150, 2], 4, 48, 96, 2, 3, "f32"),
    ([70, 3], 3, 33, 20, 3, 2, "f32"),
    ([130, 40], 2, 80, 64, 1, 1, "f32"),
    ([40] * 70, 1, 16, 16, 1, 4, "f32"),                  # more sequences than a wave has lanes
]
IDS = ["-".join(str(v).replace(" ", "") for v in c)[:60] for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_prompts(ssm, case):
    prompt(ssm, *case, 1)


@pytest.mark.parametrize("case", CASES[2:9:2] + CASES[12:14], ids=IDS[2:9:2] + IDS[12:14])
def test_options(ssm, case):
    """No gate, no softplus, no D, no biases; contiguous tensors."""
    prompt(ssm, *case, 2, gate=False, softplus=False, D=False, bias=False, joint=False)
    prompt(ssm, *case, 3, gate=True, softplus=False, D=False, bias=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slots_and_fresh(ssm, dt):
    """Any order of slots; slots outside the pool; fresh sequences, whose slots may hold anything; others left alone."""
    import torch
    lens, slots, fresh = [70, 5, 130, 0, 9, 0], [6, -1, 0, 3, 99, 5], [1, 0, 0, 1, 1, 0]
    c, dev = make(lens, 2, 64, 64, 1, 4, dt, 4, slots=slots, fresh=fresh)
    ref = mixer(c)
    for n in ("h", "conv_state"):
        dev[n][6], dev[n][3] = float("nan"), float("inf")
    y = call(ssm, c, dev)
    check(c, dev, y, ref, 250 * E, 400 * E)
    assert not dev["h"][3].any() and not dev["conv_state"][3].any()
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_no_sequence_stay(ssm, dt):
    import torch
    c, dev = make([30, 100], 2, 48, 64, 1, 4, dt, 5, behind=9, lead=7)
    out = torch.full((146, 2, 48), 7.0, dtype=dev["xbc"].dtype, device="cuda")
    bad = torch.cat([torch.arange(7), torch.arange(137, 146)]).cuda()
    for n in ("xbc", "delta", "z"):
        dev[n][bad] = float("nan")
    ref = mixer(c)
    y = call(ssm, c, dev, out=out)
    assert y is out and (y[bad] == 7.0).all()
    check(c, dev, y, ref, 250 * E, 400 * E)


SPLIT = [([2000], 2, 64, 128, 1, 4, "bf16"), ([1500, 40, 0, 700], 2, 64, 64, 2, 4, "bf16"), ([1990], 1, 80, 96, 1, 3, "f32"),
         ([0, 1203, 1], 2, 33, 16, 1, 4, "f32"), ([1500], 2, 64, 128, 1, 1, "bf16")]


@pytest.mark.parametrize("case", SPLIT, ids=[str(i) for i in range(len(SPLIT))])
def test_segments(ssm, case):
    """Few heads over long sequences: segments side by side give the oracle's values, and keep the states of others."""
    lens, H, P, N, G, W, dt = case
    T = sum(lens)
    b = lambda m: ssm.ssdconv_workspace_bytes(T, len(lens), H, P, N, G, W, dt, max_seqlen=m)  # noqa: E731
    assert b(max(lens)) > b(64)     # (the segments' states)
    prompt(ssm, *case, 6)
    prompt(ssm, *case, 7, fresh=[1] * len(lens), slots=list(range(len(lens)))[::-1])
    c, dev = make(*case, 8)
    ref = mixer(c)
    check(c, dev, call(ssm, c, dev, hint=False), ref, (90 + 50 * 32) * E, (240 + 50 * 32) * E)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cut", [1, 2, 64, 100])
def test_resume_and_tokens(ssm, dt, cut):
    """A prompt in two calls, and its last tokens one by one, against the oracle's single pass."""
    import torch
    c, dev = make([130, 130], 3, 64, 96, 1, 4, dt, 9, slots=[2, 0])
    ref = mixer(c)
    first = torch.tensor([0, cut, 130, 130 + cut], dtype=torch.int32, device="cuda")
    y = torch.zeros(260, 3, 64, dtype=dev["xbc"].dtype, device="cuda")
    # (sequences 0 .. cut and 130 .. 130 + cut; what lies between them, as a sequence of its own, is not kept)
    part = dict(dev, offsets=first, slots=torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda"))
    call(ssm, c, part, out=y, hint=False)
    at = max(cut + 3, 66)
    for i in range(cut, at):
        y[[i, 130 + i]] = step(ssm, c, dev, torch.tensor([i, 130 + i], device="cuda"))
    rest = torch.tensor([at, 130, 130 + at, 260], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(y)
    call(ssm, c, dict(part, offsets=rest), out=out, hint=False)
    y[at:130], y[130 + at:] = out[at:130], out[130 + at:]
    check(c, dev, y, ref, 1200 * E, 1400 * E)


TOKENS = [(1, 24, 64, 128, 1, 4, "bf16"), (3, 4, 64, 64, 2, 4, "bf16"), (5, 3, 33, 20, 3, 2, "bf16"), (2, 2, 80, 100, 1, 3, "f32"),
          (7, 2, 130, 33, 1, 4, "f32"), (2, 3, 1, 1, 1, 1, "f32"), (70, 8, 64, 127, 2, 4, "bf16"), (300, 2, 16, 128, 1, 4, "f32")]


@pytest.mark.parametrize("case", TOKENS, ids=["-".join(map(str, t)) for t in TOKENS])
def test_one_token(ssm, case):
    S = case[0]
    r = np.random.default_rng(10)
    slots = r.permutation(S + 2)[:S]
    slots[S // 2] = -1 if S > 1 else slots[0]
    c, dev = make([1] * S, *case[1:], 11, slots=slots)
    ref = mixer(c)
    y = step(ssm, c, dev, slice(None))
    check(c, dev, y, ref, 240 * E, 240 * E)
    c, dev = make([1] * S, *case[1:], 12, gate=False, softplus=False, D=False, bias=False, joint=False, pool=S)
    ref = mixer(c)
    check(c, dev, step(ssm, c, dev, slice(None)), ref, 240 * E, 240 * E)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strong_and_absent_decay(ssm, dt):
    """A = 0 (a running sum), and decays that leave nothing of the token before."""
    prompt(ssm, [200, 64], 3, 64, 64, 1, 4, dt, 13, A=np.array([0.0, -1e-3, -4000.0]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("seq", [[200, 90], [1300, 90]])
def test_nan_and_infinity(ssm, dt, seq):
    """One of x reaches its own channel from its token on; one of B, its group's heads; never an earlier token or another
    sequence (a masked score times it would)."""
    import torch
    c, dev = make(seq, 4, 64, 64, 2, 4, dt, 14)
    clean_dev = dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
    clean = call(ssm, c, clean_dev)
    for value in (float("nan"), float("inf")):
        bad = dict(dev, xbc=dev["xbc"].clone(), h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
        bad["xbc"][70, 64 + 5] = value          # head 1, channel 5
        y = call(ssm, c, bad)
        nan = torch.isnan(y.float())
        assert nan[71:seq[0], 1, 5].all() and torch.isnan(bad["h"][0, 1, 5]).all()
        nan[70:seq[0], 1, 5] = False
        assert not nan.any()
        same = torch.ones_like(nan)
        same[70:seq[0], 1, 5] = False
        assert torch.equal(y[same], clean[same])
        bad = dict(dev, xbc=dev["xbc"].clone(), h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
        bad["xbc"][70, 256 + 64 + 9] = value    # B of group 1
        y = call(ssm, c, bad)
        keep = torch.ones_like(nan)
        keep[70:seq[0], 2:] = False
        assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(bad["h"][0, 2:, :, 9]).any()
        assert torch.equal(bad["h"][1], clean_dev["h"][1])


def test_deterministic_and_streams(ssm):
    """Two streams at once, each with its own pool, bit for bit the same; a given workspace; another seed's in between."""
    import torch
    c, dev = make([500, 3, 1400], 2, 64, 128, 1, 4, "bf16", 15)
    pools = [dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone()) for _ in range(5)]
    ref = call(ssm, c, pools[0])
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [call(ssm, c, p, stream=side[i % 2]) for i, p in enumerate(pools[1:])]
    torch.cuda.synchronize()
    for y, p in zip(got, pools[1:]):
        assert torch.equal(y, ref) and torch.equal(p["h"], pools[0]["h"]) and torch.equal(p["conv_state"], pools[0]["conv_state"])
    ws = torch.full((ssm.ssdconv_workspace_bytes(1903, 3, 2, 64, 128, max_seqlen=1400),), 255, dtype=torch.uint8, device="cuda")
    p = dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
    assert torch.equal(call(ssm, c, p, workspace=ws), ref)    # (whatever the workspace held)


@pytest.mark.parametrize("seq", [[100, 30, 64], [1500, 30, 64]])
def test_graphs(ssm, seq):
    """A prompt and three tokens captured; replays with other inputs, lengths and slots, eager work between them."""
    import torch
    c, dev = make(seq, 2, 64, 64, 1, 4, "bf16", 16, slots=[0, 1, 2], fresh=[1, 0, 0])
    live = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in dev.items()}
    rows = torch.arange(3, device="cuda")

    def run(d):
        y = call(ssm, c, d)
        return [y] + [step(ssm, c, d, slice(3 * i, 3 * i + 3)) for i in range(3)]
    with torch.cuda.stream(torch.cuda.Stream()):
        run({n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in dev.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live)
    T = sum(seq)
    for i in range(3):
        c2, other = make(seq, 2, 64, 64, 1, 4, "bf16", 20 + i, slots=[(0, 1, 2), (3, 4, 0), (2, -1, 1)][i], fresh=[i == 1, 0, 1])
        ends = [[0, seq[0], seq[0] + seq[1], T], [5, 5, 60, T], [0, T - 80, T - 80, T - 3]][i]
        other["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        for n, t in live.items():
            if isinstance(t, torch.Tensor):
                t.copy_(other[n])
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref = run(other)
        lo, hi = ends[0], ends[-1]
        assert torch.equal(out[0][lo:hi], ref[0][lo:hi]) and all(torch.equal(a, b) for a, b in zip(out[1:], ref[1:]))
        assert torch.equal(live["h"], other["h"]) and torch.equal(live["conv_state"], other["conv_state"])


def test_offsets_out_of_range(ssm):
    """Offsets below zero, behind the last row or decreasing are cut: nothing outside is read or written."""
    import torch
    c, dev = make([20, 30, 14], 2, 32, 16, 1, 4, "f32", 17)
    for ends in ([-5, 20, 50, 1000], [0, 50, 20, 64], [64, 64, 64, 64], [70, 80, 90, 100], [-9, -8, -7, -6]):
        d = dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone(), offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"))
        out = torch.full((64, 2, 32), 3.0, device="cuda")
        call(ssm, c, d, out=out, hint=False)
        cut = np.clip(ends, 0, 64)
        if (np.diff(ends) >= 0).all():
            ref = mixer(dict(c, offsets=cut))
            check(c, d, out, ref, 150 * E, 300 * E)
            inside = np.zeros(64, bool)
            inside[cut[0]:cut[-1]] = True
            assert (out[torch.from_numpy(~inside).cuda()] == 3.0).all()
        assert torch.equal(d["h"][3:], dev["h"][3:])


@pytest.mark.parametrize("hint", [None, 64])
def test_decreasing_offsets_stay_inside(ssm, hint):
    """Offsets that fall by many chunks: what y and the states then are is not said, but nothing else is written."""
    import torch
    c, dev = make([500, 700, 400, 400], 2, 32, 16, 1, 4, "bf16", 23)
    T = 2000
    for ends in ([0, 1900, 0, 64, 2000], [2000, 1000, 500, 100, 0], [1500, 0, 1999, 0, 2000], [0, 2000, 10, 20, 30]):
        room = torch.full((6000, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")
        pool = torch.full((18, 2, 32, 16), 5.0, device="cuda")
        conv = torch.full((18, 96, 3), 7.0, dtype=torch.bfloat16, device="cuda")
        d = dict(dev, h=pool[6:12], conv_state=conv[6:12], offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"))
        c["longest"] = hint
        call(ssm, c, d, out=room[2000:4000], hint=hint is not None)
        assert (room[:2000] == 3.0).all() and (room[4000:] == 3.0).all(), ends
        assert (pool[:6] == 5.0).all() and (pool[10:] == 5.0).all(), ends
        assert (conv[:6] == 7.0).all() and (conv[10:] == 7.0).all(), ends


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slots_past_32_bits(ssm, dt):
    """A pool of more than 2^31 states: the last slots give what a small pool's give, to the bit."""
    import torch
    lens, H, P, N = [70, 1, 200], 64, 64, 128
    c, dev = make(lens, H, P, N, 1, 4, dt, 24, slots=[2, 0, 1], pool=3)
    many = (1 << 31) // (H * P * N) + 8
    h = torch.zeros(many, H, P, N, device="cuda")
    conv = torch.zeros(many, *dev["conv_state"].shape[1:], dtype=dev["conv_state"].dtype, device="cuda")
    h[-3:], conv[-3:] = dev["h"], dev["conv_state"]
    big = dict(dev, h=h, conv_state=conv, slots=dev["slots"] + (many - 3))
    y, yb = call(ssm, c, dev), call(ssm, c, big)
    t, tb = step(ssm, c, dev, slice(0, 3)), step(ssm, c, big, slice(0, 3))
    assert torch.equal(y, yb) and torch.equal(t, tb)
    assert torch.equal(h[-3:], dev["h"]) and torch.equal(conv[-3:], dev["conv_state"])
    assert not h[:-3].any() and not conv[:-3].any()


def test_rows_past_32_bits(ssm):
    """Rows of a very wide projection: 2^21 elements apart, the last ones behind 2^31."""
    import torch
    c, dev = make([1000, 80], 2, 32, 16, 1, 4, "bf16", 25, joint=False)
    T, C = dev["xbc"].shape
    wide = torch.empty(T, 1 << 21, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:5 + C], wide[:, 200:264], wide[:, 300:302] = dev["xbc"], dev["z"].flatten(1), dev["delta"]
    far = dict(dev, xbc=wide[:, 5:5 + C], z=wide[:, 200:264].unflatten(1, (2, 32)), delta=wide[:, 300:302],
               h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
    assert torch.equal(call(ssm, c, dev), call(ssm, c, far))
    assert torch.equal(dev["h"], far["h"]) and torch.equal(dev["conv_state"], far["conv_state"])


def test_as_many_sequences_as_there_can_be(ssm):
    """65535 sequences of one token; some of them against the oracle, which the single-token call meets too."""
    import torch
    S = 65535
    c, dev = make([1] * S, 1, 8, 4, 1, 4, "f32", 26, pool=S)
    pick = np.concatenate([np.arange(5), np.random.default_rng(1).integers(5, S, 40), [S - 2, S - 1]])
    sub = dict(c, offsets=np.arange(len(pick) + 1), slots=np.arange(len(pick)), fresh=np.zeros(len(pick), bool),
               **{n: c[n][pick] for n in ("xbc", "delta", "z", "h", "conv_state")})
    ref = mixer(sub)
    at = torch.from_numpy(pick).cuda()
    tok = dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone())
    for d, y, n in ((dev, call(ssm, c, dev), 1), (tok, step(ssm, c, tok, slice(None)), 0)):
        got = dict(d, h=d["h"][at], conv_state=d["conv_state"][at])
        check(c, got, y[at], ref, (90 + 50 * n) * E, (240 + 50 * n) * E)


def test_wide_heads_and_many_groups(ssm):
    """A head of many blocks of channels, and a group for every head."""
    prompt(ssm, [70, 9], 1, 1000, 40, 1, 4, "bf16", 27)
    prompt(ssm, [70, 9], 40, 8, 8, 40, 4, "bf16", 28)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_gate_and_outputs_off_16_bytes(ssm, dt, off):
    """z and y at any element, whole pieces of 16 bytes or not: the same values to the bit, and nothing beside them."""
    import torch
    for P in (64, 48, 36):
        c, dev = make([100, 31], 2, P, 64, 1, 4, dt, 29, joint=False)
        T = 131
        start = {n: dev[n].clone() for n in ("h", "conv_state")}
        y = call(ssm, c, dev)
        wide = torch.zeros(T, 2 * P + 9, dtype=y.dtype, device="cuda")
        wide[:, off:off + 2 * P] = dev["z"].flatten(1)
        room = torch.full((T * 2 * P + 16,), 3.0, dtype=y.dtype, device="cuda")
        out = room[off:off + T * 2 * P].view(T, 2, P)
        far = dict(dev, z=wide[:, off:off + 2 * P].unflatten(1, (2, P)), **start)
        call(ssm, c, far, out=out)
        assert torch.equal(out, y) and torch.equal(far["h"], dev["h"])
        assert (room[:off] == 3.0).all() and (room[off + T * 2 * P:] == 3.0).all()


def test_refusals(ssm):
    import torch
    c, dev = make([20, 30], 2, 32, 16, 1, 4, "bf16", 18)
    for n, t in (("delta", dev["delta"].float()), ("z", dev["z"][:, :1]), ("A", dev["A"][:1]), ("w", dev["w"].bfloat16()),
                 ("h", dev["h"].bfloat16()), ("h", dev["h"].transpose(0, 1)), ("conv_state", dev["conv_state"].float()),
                 ("conv_state", None), ("offsets", dev["offsets"].long()), ("slots", torch.zeros(3, dtype=torch.int32, device="cuda")),
                 ("fresh", torch.zeros(2, dtype=torch.int32, device="cuda")), ("xbc", dev["xbc"][:, :-1]), ("xbc", dev["xbc"].half()),
                 ("xbc", dev["xbc"].t().contiguous().t()), ("offsets", dev["offsets"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(ssm, c, dict(dev, **{n: t}))
    h = torch.zeros(4, 2, 32, 129, device="cuda")
    with pytest.raises(ssm.SSMError):
        ssm.ssdconv_fwd(torch.zeros(5, 64 + 258, device="cuda"), torch.zeros(5, 2, device="cuda"), dev["A"], torch.zeros(322, 4, device="cuda"),
                        h, torch.zeros(4, 322, 3, device="cuda"), dev["offsets"])
    v = dev["h"]._version
    call(ssm, c, dev)
    assert dev["h"]._version > v


def test_empty(ssm):
    import torch
    c, dev = make([0, 0], 2, 32, 16, 1, 4, "bf16", 19, fresh=[1, 0])
    h = dev["h"].clone()
    assert call(ssm, c, dev).shape == (0, 2, 32)
    assert not dev["h"][0].any() and torch.equal(dev["h"][1:], h[1:])
    none = dict(dev, offsets=dev["offsets"][:1], slots=None, fresh=None)
    assert call(ssm, c, none).shape == (0, 2, 32)
    assert step(ssm, c, dev, slice(0, 0)).shape == (0, 2, 32)


def test_benchmark_size(ssm):
    """64 heads of the multi-head scan's benchmark size: every value finite, sampled heads against the oracle."""
    import torch
    c, dev = make([700, 650], 64, 64, 128, 1, 4, "bf16", 21)
    heads = [0, 17, 63]
    ref_c = dict(c)
    P = 64
    ch = np.concatenate([np.arange(h * P, h * P + P) for h in heads] + [np.arange(64 * P, 64 * P + 256)])
    for n, f in (("xbc", lambda a: a[:, ch]), ("delta", lambda a: a[:, heads]), ("z", lambda a: a[:, heads]), ("A", lambda a: a[heads]),
                 ("D", lambda a: a[heads]), ("delta_bias", lambda a: a[heads]), ("w", lambda a: a[ch]), ("bias", lambda a: a[ch]),
                 ("h", lambda a: a[:, heads]), ("conv_state", lambda a: a[:, ch])):
        ref_c[n] = f(c[n])
    ref = mixer(ref_c)
    y = call(ssm, c, dev)
    assert torch.isfinite(y.float()).all() and torch.isfinite(dev["h"]).all()
    got = dict(dev, h=dev["h"][:, heads], conv_state=dev["conv_state"][:, torch.from_numpy(ch).cuda()])
    check(c, got, y[:, heads], ref, (90 + 50 * 11) * E, (240 + 50 * 11) * E)
