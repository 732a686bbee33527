"""Where the served Mamba-2 mixer's numbers could lose digits, against the fp64 oracle."""
import numpy as np
import pytest

from oracle.ssdconv_oracle import mixer
from tests.gpu_util import to_host
from tests.test_gpu_ssdconv import E, call, check, make, ssm, step  # noqa: F401  (ssm: the fixture)

pytestmark = pytest.mark.gpu


def pulse(dt, reset, at, L=130):
    """Three heads whose tokens' outputs are single products: a large step at token `at`, then small ones; x is zero but at
    token at + 1, B and C are 1.5 all along, one state, the filter a single column of one."""
    import torch
    P = 8
    c, dev = make([L], 3, P, 1, 1, 1, dt, 30, gate=False, softplus=False, D=False, bias=False, joint=False, fresh=[1],
                  A=np.array([-16.0, -4.0, -1.0]))
    r = np.random.default_rng(31)
    xbc, delta = np.zeros((L, 3 * P + 2), np.float32), (0.005 + 0.01 * r.random((L, 3))).astype(np.float32)
    xbc[at + 1, :3 * P] = 1.0 + r.random(3 * P)
    xbc[:, 3 * P:] = 1.5
    delta[at] = reset
    for n, a in (("xbc", xbc), ("delta", delta)):
        dev[n] = torch.from_numpy(a).cuda().to(dev[n].dtype)
        c[n] = dev[n].double().cpu().numpy()
    c["w"], dev["w"] = np.ones_like(c["w"]), torch.ones_like(dev["w"])
    return c, dev


@pytest.mark.parametrize("at", [0, 5, 30, 31, 40, 62, 63])
@pytest.mark.parametrize("dt,reset", [("f32", 20.0), ("f32", 100.0), ("f32", 4000.0), ("bf16", 4000.0), ("bf16", 30000.0)])
def test_decays_behind_a_large_step(ssm, dt, reset, at):  # noqa: F811
    """A step that leaves nothing of what was before must not touch the decays between the tokens behind it.

    One product a token, so the error is relative to the value: silu of x, B and C 6 * 2^-24 each; a product of three-part
    factors leaves out 3 * 2^-24 and rounds 3 times, C B and then with x (or the state): 12 and 3; the decay's up to
    three factors and the step in front 2 each: 8; a sum over 32 tokens or a chunk's chain 10: 51, taken as 60; and the exponent X
    from the pulse on, relative to itself a half step for each of the difference (or the sum) and the exponential's argument, twice
    behind a half or a chunk: 4 X.  bf16: half a step of the output; lo of the sums is half a bf16 step off, at a sum of 16 *
    30000 * 1.4427 < 2^20 that is 2^(20 - 24 - 1 - 8) twice, times log 2: less than 2^-12."""
    c, dev = pulse(dt, reset, at)
    ref = mixer(c)["y"]
    y = call(ssm, c, dev)
    X = -np.cumsum(np.where(np.arange(130)[:, None] > at + 1, c["delta"] * c["A"], 0.0), 0)[:, :, None]
    tol = (60 + 4 * X) * E
    if dt == "bf16":
        tol = tol + 2.0 ** -8 + 2.0 ** -12
    worst = (np.abs(to_host(y).reshape(ref.shape) - ref) / (tol * np.abs(ref) + 1e-30)).max()
    assert worst <= 1.0, f"{worst:.3g} of the tolerance"


@pytest.mark.parametrize("reset", [20.0, 400.0])
def test_prompt_and_tokens_behind_a_large_step(ssm, reset):  # noqa: F811
    """The same tokens one by one: both forms lie within the tolerance above of the oracle, so they are twice it apart at most."""
    import torch
    c, dev = pulse("f32", reset, 3, L=64)
    y = call(ssm, c, dict(dev, h=dev["h"].clone(), conv_state=dev["conv_state"].clone()))
    dev["h"].zero_()
    t = torch.cat([step(ssm, c, dev, slice(i, i + 1)) for i in range(64)])
    X = -np.cumsum(np.where(np.arange(64)[:, None] > 4, c["delta"] * c["A"], 0.0), 0)[:, :, None]
    a, b = to_host(y).reshape(64, 3, -1), to_host(t).reshape(64, 3, -1)
    # (the token form multiplies a decay and rounds the state once a token: 3 * 2^-24 more for each of 60)
    assert (np.abs(a - b) <= (2 * (60 + 4 * X) + 180) * E * np.abs(b) + 1e-30).all()


@pytest.mark.parametrize("at", [0, 20, 40, 70])
@pytest.mark.parametrize("which", ["x", "B", "C", "state"])
def test_bf16_outputs_round_the_whole_factor(ssm, which, at):  # noqa: F811
    """1 + 2^-8 + 2^-20 lies just above the middle of two bf16 values: y is the upper one only if no bit of the fp32 factor it comes
    from was dropped before a product.  Token 0's x and B reach the output of token `at` in its own half, from the first
    half, and through the state; without decay, and by values of 64, which silu leaves as they are (1 + e^-64 is 1)."""
    import torch
    f = 1.0 + 2.0 ** -8 + 2.0 ** -20
    H, P, N, L = 1, 16, 16, 80
    C = H * P + 2 * N
    dev = {"xbc": torch.zeros(L, C, dtype=torch.bfloat16), "delta": torch.zeros(L, H, dtype=torch.bfloat16), "A": torch.zeros(H),
           "w": torch.ones(C, 1), "h": torch.zeros(1, H, P, N), "conv_state": torch.zeros(1, C, 0, dtype=torch.bfloat16),
           "offsets": torch.tensor([0, L], dtype=torch.int32)}
    dev["xbc"][at, P + N + 3] = 64.0            # C
    if which == "state":
        dev["h"][0, 0, 5, 3] = f
    else:
        dev["xbc"][0, 5] = dev["xbc"][0, P + 3] = 64.0
        dev["delta"][0] = 1.0
        dev["w"][{"x": 5, "B": P + 3, "C": P + N + 3}[which]] = f
    y = ssm.ssdconv_fwd(**{n: t.cuda() for n, t in dev.items()}).float()
    # every product and sum here is exact in 24 bits: one rounding, to bf16
    assert float(y[at, 0, 5]) == (64.0 if which == "state" else 64.0 ** 3) * (1.0 + 2.0 ** -7)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("seq", [[200, 90], [1300, 90]])
def test_nan_from_its_own_token_on(ssm, dt, seq):  # noqa: F811
    """A NaN or infinity of x at the first and last token of chunks and halves, in every wave's share of a chunk, at a segment's border
    and at the sequence's last token: its channel's outputs are NaN from that very token on, every other output keeps its bits."""
    import torch
    c, dev = make(seq, 4, 64, 64, 2, 4, dt, 14)
    start = {n: dev[n].clone() for n in ("h", "conv_state")}
    again = lambda **kw: dict(dev, **{n: t.clone() for n, t in start.items()}, **kw)  # noqa: E731
    clean_dev = again()
    clean = call(ssm, c, clean_dev)
    for k, row in enumerate([0, 9, 18, 27, 31, 32, 45, 54, 63, 64, 70, 127, 128, seq[0] - 2, seq[0] - 1]):
        head, p = k % 4, (5 + 19 * k) % 64
        for value in (float("nan"), float("inf"), -float("inf")):
            xbc = dev["xbc"].clone()
            xbc[row, 64 * head + p] = value
            bad = again(xbc=xbc)
            y = call(ssm, c, bad)
            hit = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
            hit[row:seq[0], head, p] = True
            assert torch.equal(torch.isnan(y.float()), hit), (row, value)
            assert torch.equal(y[~hit], clean[~hit]), (row, value)
            gone = torch.zeros(bad["h"].shape, dtype=torch.bool, device="cuda")
            gone[0, head, p] = True
            assert torch.equal(torch.isnan(bad["h"]), gone) and torch.equal(bad["h"][~gone], clean_dev["h"][~gone]), (row, value)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L", [4, 68, 1284])
def test_rows_behind_the_end_are_not_convolved(ssm, dt, L):  # noqa: F811
    """Large finite values of x whose convolutions are finite at every token, but not at the rows behind the last one that its chunk
    has room for: 2e38, 2e38 with -2e38 in front of them, or the last row once more.  Outputs and states as the oracle's."""
    import torch
    c, dev = make([L], 2, 64, 64, 1, 4, dt, 32, gate=False, softplus=False, D=False, bias=False, joint=False, fresh=[1])
    c["w"][64 + 7], dev["w"][64 + 7] = 1.0, 1.0
    v = torch.tensor([-2e38, 0.0, 2e38, 2e38], dtype=dev["xbc"].dtype)
    dev["xbc"][-4:, 64 + 7], c["xbc"][-4:, 64 + 7] = v.cuda(), v.double().numpy()
    if L > 4:
        dev["xbc"][-8:-4, 64 + 7], c["xbc"][-8:-4, 64 + 7] = 0.0, 0.0
    ref = mixer(c)
    n = (L + 63) // 64
    check(c, dev, call(ssm, c, dev), ref, (90 + 50 * n) * E, (240 + 50 * n) * E)
