"""Pins of the fp64 group norm oracle: known values, and central differences for its gradients."""
import numpy as np
import pytest

from oracle.norm_oracle import groupnorm, groupnorm_bwd


def test_normed_groups_have_mean_zero_and_variance_one():
    r = np.random.default_rng(0)
    x = 3.0 + 2.0 * r.standard_normal((2, 5, 12))
    y = groupnorm(x, 3, eps=0.0).reshape(2, 5, 3, 4)
    np.testing.assert_allclose(y.mean((1, 3)), 0.0, atol=1e-14)
    np.testing.assert_allclose((y ** 2).mean((1, 3)), 1.0, rtol=1e-13)
    # two values: -1 and 1; a shift and a scale of x change nothing
    np.testing.assert_allclose(groupnorm(np.array([[[1.0, 5.0]]]), 1, eps=0.0), [[[-1.0, 1.0]]], rtol=1e-15)
    np.testing.assert_allclose(groupnorm(7.0 * x - 1.0, 3, eps=0.0), groupnorm(x, 3, eps=0.0), rtol=1e-11, atol=1e-12)


def test_torch_agrees():
    import torch
    r = np.random.default_rng(1)
    x, w, b = r.standard_normal((2, 7, 12)), r.standard_normal(12), r.standard_normal(12)
    t = torch.nn.functional.group_norm(torch.from_numpy(x).transpose(1, 2), 4, torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(groupnorm(x, 4, w, b), t.transpose(1, 2).numpy(), rtol=1e-12, atol=1e-13)
    t = torch.nn.functional.silu(t).transpose(1, 2).numpy()
    z = r.standard_normal(x.shape)
    np.testing.assert_allclose(groupnorm(x, 4, w, b, z, silu=True), t * z / (1 + np.exp(-z)), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_gradients_against_central_differences(silu, gate):
    r = np.random.default_rng(2)
    c = dict(x=r.standard_normal((2, 3, 8)), w=r.standard_normal(8), b=r.standard_normal(8))
    if gate:
        c["z"] = r.standard_normal((2, 3, 8))
    dy = r.standard_normal((2, 3, 8))
    g = groupnorm_bwd(c["x"], 2, c["w"], c["b"], c.get("z"), dy, silu=silu)
    for name, grad in (("x", "dx"), ("w", "dw"), ("b", "dbias"), ("z", "dz")):
        if name not in c:
            continue
        d, e = r.standard_normal(c[name].shape), 1e-6
        f = lambda s: (groupnorm(**{**c, name: c[name] + s * e * d}, groups=2, silu=silu) * dy).sum()  # noqa: E731
        num = (f(1) - f(-1)) / (2 * e)
        # error e^2 f'''/6 plus 2^-52 |f| / e
        assert abs(num - (g[grad] * d).sum()) <= 1e-7 * max(1.0, abs(num)), name
