"""Pins of the fp64 linear attention oracle: the masked-product form, the SSD scan it is a
special case of, and central differences for its gradients."""
import numpy as np
import pytest

from oracle.linattn_oracle import linattn, linattn_bwd


def _case(B=2, L=9, H=4, hq=2, hk=4, hv=1, dk=3, dv=5, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, L, hq, dk)), k=r.standard_normal((B, L, hk, dk)), v=r.standard_normal((B, L, hv, dv)),
                a=-r.random(H), h0=r.standard_normal((B, H, dk, dv))), r


def test_matches_the_masked_product_form():
    c, _ = _case()
    B, L, H = 2, 9, 4
    y, h = linattn(c["q"], c["k"], c["v"], c["a"], 0.7)
    i = np.arange(L)
    for b in range(B):
        for hd in range(H):
            q, k, v = c["q"][b, :, hd // 2], c["k"][b, :, hd], c["v"][b, :, 0]
            D = np.where(i[:, None] >= i, np.exp(c["a"][hd] * (i[:, None] - i)), 0.0)
            np.testing.assert_allclose(y[b, :, hd], 0.7 * ((q @ k.T) * D) @ v, rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(h[b, hd], (k * np.exp(c["a"][hd] * (L - 1 - i))[:, None]).T @ v, rtol=1e-12, atol=1e-13)


def test_is_the_ssd_scan_with_a_step_of_one():
    from oracle.ssd_oracle import ssd
    r = np.random.default_rng(4)
    B, L, H, P, N = 2, 7, 3, 4, 5
    x, Bm, Cm = r.standard_normal((B, L, H, P)), r.standard_normal((B, L, N)), r.standard_normal((B, L, N))
    a, h0 = -r.random(H), r.standard_normal((B, H, P, N))
    y, h = linattn(Cm[:, :, None], Bm[:, :, None], x, a, 1.0, h0.transpose(0, 1, 3, 2))
    ys, hs = ssd(x, np.ones((B, L, H)), a, Bm, Cm, h0=h0)
    np.testing.assert_allclose(y, ys, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(h.transpose(0, 1, 3, 2), hs, rtol=1e-12, atol=1e-12)


def test_lengths_cut_every_row():
    c, r = _case()
    y, h = linattn(c["q"], c["k"], c["v"], c["a"], 1.0, c["h0"], [4, 0])
    y4, h4 = linattn(c["q"][:1, :4], c["k"][:1, :4], c["v"][:1, :4], c["a"], 1.0, c["h0"][:1])
    assert np.array_equal(y[0, :4], y4[0]) and np.array_equal(h[0], h4[0])
    assert not y[0, 4:].any() and not y[1].any() and np.array_equal(h[1], c["h0"][1])


@pytest.mark.parametrize("lengths", [None, [6, 9]])
def test_gradients_against_central_differences(lengths):
    c, r = _case(seed=3)
    dy, dh = r.standard_normal((2, 9, 4, 5)), r.standard_normal((2, 4, 3, 5))

    def loss(**k):
        x = {**c, **k}
        y, h = linattn(x["q"], x["k"], x["v"], x["a"], 0.6, x["h0"], lengths)
        return (y * dy).sum() + (h * dh).sum()

    g = linattn_bwd(c["q"], c["k"], c["v"], c["a"], 0.6, c["h0"], dy, dh, lengths)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("a", "dlog_decay"), ("h0", "dh0")):
        d = r.standard_normal(c[name].shape)
        e = 1e-6
        num = (loss(**{name: c[name] + e * d}) - loss(**{name: c[name] - e * d})) / (2 * e)
        # central differences: error e^2 f'''/6 (about 1e-11 here) plus 2^-52 |f| / e
        assert abs(num - (g[grad] * d).sum()) <= 1e-7 * max(1.0, abs(num)), name
