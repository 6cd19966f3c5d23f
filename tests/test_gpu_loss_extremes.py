"""Tokens far from the reference or from the policy that sampled them: log-ratios so large that the exponential
over- or underflows, or that are infinite (a token of probability 0 under one of the models)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


def dev(*x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("n", [1, 5000, 70000])
@pytest.mark.parametrize("ref,grad,kl", [(INF, -1.0, INF), (1e30, -1.0, 1e30), (1e20, -1.0, 1e20), (800.0, -1.0, 797.0),
                                         (40.0, np.expm1(-38.0), np.expm1(-38.0) + 38.0), (-1e30, INF, INF)])
def test_gradient_of_the_divergence(qoh, n, ref, grad, kl):
    """d/dce of exp(d) - 1 - d is exp(d) - 1, -1 for a reference that rules the token out (d = ce - ref = 2 - ref)."""
    ce = torch.full((n,), 2.0, device="cuda")
    zero = torch.zeros_like(ce)
    loss, g, stats = qoh.policy_loss(ce, ce, zero, ce_ref=zero + ref, kl_coef=0.5, reduction="sum")
    want = torch.full_like(ce, 0.5 * grad)
    assert torch.allclose(g, want, rtol=2.0 ** -23, atol=0), g[:3]
    for got, value in ((loss, 0.5 * kl * n), (stats[2], kl)):
        assert torch.allclose(got, dev(value)[0], rtol=2.0 ** -22, atol=0), (float(got), value)


def test_a_token_of_probability_zero(qoh):
    """ce = infinity: the reference's ratio exp(d) is infinite, and so are the divergence and its gradient, not NaN."""
    loss, g, stats = qoh.policy_loss(dev(INF, 1.0), dev(1.0, 1.0), dev(1.0, 1.0), ce_ref=dev(2.0, 1.0), kl_coef=0.5, reduction="sum")
    assert loss == INF and g[0] == INF and g[1] == 1.0
    assert stats[0] == 0 and stats[1] == INF and stats[2] == INF
    # (and the divergence from the policy that sampled a token it gives probability 0)
    _, g, stats = qoh.policy_loss(dev(1.0, 1.0), dev(INF, 1.0), dev(1.0, 1.0), reduction="sum")
    assert g[0] == 0 and g[1] == 1.0 and stats[0] == 0.5 and stats[1] == INF


@pytest.mark.parametrize("reduction", ["tokens", "sequences", "sum"])
def test_no_advantage_no_loss(qoh, reduction):
    """An advantage of 0 (a group whose rewards are all equal) has no part in the loss, however large the ratio."""
    ce, old = dev(0.0, 0.0, 5.0, 1.0), dev(800.0, 3.4e38, 2.0, 1.0)
    loss, g, _ = qoh.policy_loss(ce, old, torch.zeros_like(ce), reduction=reduction)
    assert loss == 0 and not g.any()
    # (a NaN that counts is not hidden)
    loss, g, _ = qoh.policy_loss(dev(float("nan"), 1.0), dev(1.0, 1.0), dev(0.0, 0.0), reduction=reduction)
    assert torch.isnan(loss) and torch.isnan(g[0])
