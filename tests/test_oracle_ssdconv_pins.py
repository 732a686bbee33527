"""The served mixer's oracle, pinned to the pinned convolution and multi-head scan oracles and to splits."""
import numpy as np
import pytest

from oracle import conv_oracle, ssd_oracle
from oracle.ssdconv_oracle import mixer


def case(lens, H=4, P=3, N=5, G=2, W=4, seed=0, softplus=True, gate=True, slots=None, fresh=None, behind=0):
    r = np.random.default_rng(seed)
    T, C, S = sum(lens) + behind, H * P + 2 * G * N, len(lens)
    return {"xbc": r.standard_normal((T, C)), "delta": r.standard_normal((T, H)) if softplus else 0.1 * r.random((T, H)),
            "z": r.standard_normal((T, H, P)) if gate else None, "A": -np.exp(r.standard_normal(H)), "D": r.standard_normal(H),
            "delta_bias": r.standard_normal(H) if softplus else None, "w": r.standard_normal((C, W)), "bias": r.standard_normal(C),
            "h": r.standard_normal((S + 2, H, P, N)), "conv_state": r.standard_normal((S + 2, C, W - 1)),
            "offsets": np.concatenate([[0], np.cumsum(lens)]), "slots": np.arange(S) if slots is None else np.array(slots),
            "fresh": np.zeros(S, bool) if fresh is None else np.array(fresh), "G": G, "softplus": softplus}


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("W", [1, 3, 4])
def test_is_the_convolution_and_the_scan(G, W):
    c = case([7, 4], G=G, W=W, slots=[1, 0], fresh=[False, True])
    got = mixer(c)
    H, P, N = 4, 3, 5
    for s, (a, b) in enumerate(((0, 7), (7, 11))):
        slot = c["slots"][s]
        st = c["conv_state"][slot][None] * (not c["fresh"][s])
        v, end = conv_oracle.conv1d(c["xbc"][None, a:b], c["w"], c["bias"], st, True)
        x, B, C = np.split(v[0], [H * P, H * P + G * N], axis=1)
        h0 = c["h"][slot][None] * (not c["fresh"][s])
        L = b - a
        for g in range(G):
            hs = slice(g * (H // G), (g + 1) * (H // G))
            y, hl = ssd_oracle.ssd(x.reshape(1, L, H, P)[:, :, hs], c["delta"][None, a:b, hs], c["A"][hs],
                                   B.reshape(1, L, G, N)[:, :, g], C.reshape(1, L, G, N)[:, :, g], c["D"][hs],
                                   c["z"][None, a:b, hs], h0[:, hs], delta_softplus=True, delta_bias=c["delta_bias"][hs])
            np.testing.assert_allclose(got["y"][a:b, hs], y[0], rtol=1e-11, atol=1e-12)
            np.testing.assert_allclose(got["h"][slot, hs], hl[0], rtol=1e-11, atol=1e-12)
        np.testing.assert_array_equal(got["conv_state"][slot], end[0])


@pytest.mark.parametrize("cut", [0, 1, 2, 5, 9])
def test_split_and_resume(cut):
    c = case([9])
    whole = mixer(c)
    one = dict(c, offsets=np.array([0, cut]))
    first = mixer(one)
    two = dict(c, offsets=np.array([cut, 9]), h=first["h"], conv_state=first["conv_state"])
    second = mixer(two)
    y = np.concatenate([first["y"][:cut], second["y"][cut:9]])
    np.testing.assert_array_equal(y, whole["y"])
    for n in ("h", "conv_state"):
        np.testing.assert_array_equal(second[n], whole[n])


def test_sequences_do_not_meet():
    c = case([5, 0, 6], slots=[2, 0, -1], behind=2)
    got = mixer(c)
    alone = mixer(dict(c, offsets=np.array([5, 11]), slots=np.array([-1]), fresh=np.array([False])))
    np.testing.assert_array_equal(got["y"][5:11], alone["y"][5:11])
    assert np.isnan(got["y"][11:]).all()
    for n in ("h", "conv_state"):
        np.testing.assert_array_equal(got[n][[0, 1, 3, 4]], np.asarray(c[n])[[0, 1, 3, 4]])   # (no tokens: as it was)


def test_bounds_hold_what_they_bound():
    c = case([40])
    got = mixer(c)
    assert (np.abs(got["y"]) <= got["y_hat"] + 1e-12).all() and (np.abs(got["h"]) <= got["h_hat"] + 1e-12).all()
