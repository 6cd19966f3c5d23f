"""Refusals of the learning entry points, on the host before any CUDA call, and
the oracle's own gradients against differences.  No GPU."""
import ctypes

import numpy as np
import pytest

import archead_inputs as gen
import oracle


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


P = 4096   # an aligned address that is never dereferenced: the checks fail first


def _policy(qoh, ptrs=None, T=8, S=2, ws=1 << 20, **kw):
    o = dict(clip_low=0.2, clip_high=0.2, kl_coef=0.0, scale=1.0, reduction=0, advantage_per=0)
    o.update(kw)
    a = dict(ce=P, old=P, adv=P, ref=None, mask=None, cu=P, loss=P, grad=P, stats=P, ws=P)
    a.update(ptrs or {})
    opts = qoh.ArcheadPolicyOptions(*o.values())
    return qoh._lib.archead_policy_loss(a["ce"], a["old"], a["adv"], a["ref"], a["mask"], a["cu"], T, S,
                                        ctypes.byref(opts), a["loss"], a["grad"], a["stats"], a["ws"], ws, None)


def _preference(qoh, ptrs=None, T=8, N=2, ws=1 << 20, **kw):
    o = dict(beta=0.1, margin=0.0, label_smoothing=0.0, scale=1.0, kind=0, average=0)
    o.update(kw)
    a = dict(ce=P, ref=None, mask=None, cu=P, loss=P, grad=P, rewards=P, ws=P)
    a.update(ptrs or {})
    opts = qoh.ArcheadPreferenceOptions(*o.values())
    return qoh._lib.archead_preference_loss(a["ce"], a["ref"], a["mask"], a["cu"], T, N, ctypes.byref(opts), a["loss"],
                                            a["grad"], a["rewards"], a["ws"], ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ptrs=dict(ce=None)), "EINVAL"), (dict(ptrs=dict(old=None)), "EINVAL"), (dict(ptrs=dict(adv=None)), "EINVAL"),
    (dict(ptrs=dict(loss=None)), "EINVAL"), (dict(ptrs=dict(grad=None)), "EINVAL"), (dict(ptrs=dict(stats=None)), "EINVAL"),
    (dict(ptrs=dict(ws=None)), "EINVAL"), (dict(ptrs=dict(cu=None)), "EINVAL"), (dict(T=-1), "EINVAL"),
    (dict(T=(1 << 20) + 1), "EINVAL"), (dict(S=-1), "EINVAL"), (dict(clip_low=-0.1), "EINVAL"), (dict(clip_low=1.1), "EINVAL"),
    (dict(clip_low=float("nan")), "EINVAL"), (dict(clip_high=-1.0), "EINVAL"), (dict(kl_coef=float("inf")), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(reduction=3), "EINVAL"), (dict(reduction=-1), "EINVAL"),
    (dict(advantage_per=2), "EINVAL"), (dict(ptrs=dict(ce=P + 2)), "EALIGN"), (dict(ptrs=dict(ws=P + 64)), "EALIGN"),
    (dict(ptrs=dict(cu=P + 1)), "EALIGN"), (dict(ws=100), "ENOMEM")])
def test_policy_loss_refuses(qoh, kw, status):
    assert _policy(qoh, **kw) == getattr(qoh, "ARCHEAD_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(ptrs=dict(ce=None)), "EINVAL"), (dict(ptrs=dict(cu=None)), "EINVAL"), (dict(ptrs=dict(rewards=None)), "EINVAL"),
    (dict(ptrs=dict(loss=None)), "EINVAL"), (dict(ptrs=dict(grad=None)), "EINVAL"), (dict(ptrs=dict(ws=None)), "EINVAL"),
    (dict(T=-1), "EINVAL"), (dict(N=-1), "EINVAL"), (dict(beta=0.0), "EINVAL"), (dict(beta=float("inf")), "EINVAL"),
    (dict(margin=float("nan")), "EINVAL"), (dict(kind=3), "EINVAL"), (dict(label_smoothing=0.6), "EINVAL"),
    (dict(label_smoothing=0.1, kind=1), "EINVAL"), (dict(margin=0.5, kind=2), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(ptrs=dict(ref=P + 2)), "EALIGN"), (dict(ptrs=dict(ws=P + 128)), "EALIGN"), (dict(ws=100), "ENOMEM")])
def test_preference_loss_refuses(qoh, kw, status):
    assert _preference(qoh, **kw) == getattr(qoh, "ARCHEAD_" + status)


def test_workspace_sizes(qoh):
    lib = qoh._lib
    assert lib.archead_loss_workspace_bytes(-1) == 0 and lib.archead_loss_workspace_bytes(0) > 0
    assert lib.archead_loss_workspace_bytes(1000) > lib.archead_loss_workspace_bytes(10)
    assert lib.archead_grad_workspace_bytes(None, 4) == 0
    assert lib.archead_grad_hidden(None, P, 4, P, P, P, P, 0, P, 1 << 30, None) == qoh.ARCHEAD_EINVAL


def test_oracle_head_gradient_is_the_derivative():
    shape = (200, 64, 16, 8, 16, 64)
    comps = gen.random_components(gen.HeadShape(*shape), 1)
    bits, targets = gen.random_hidden(64, 5, 2, 200)
    W, absW = oracle.dense_rows(comps, 16, 64)
    assert np.allclose(W, oracle.w_hat_rows(comps, 16, 64, np.arange(200)), rtol=0, atol=1e-12) and np.all(absW >= np.abs(W) - 1e-12)
    h = oracle.hidden_f64(bits)
    g = np.array([1.0, -2.0, 0.0, 0.5, 3.0])

    def loss(x):
        return float(g @ oracle.lse_argmax_ce(x @ W.T, targets)[2])

    dh, _ = oracle.ce_gradient(W, h, oracle.lse_argmax_ce(h @ W.T)[0], targets, g)
    assert not dh[2].any()
    rng = np.random.default_rng(3)
    for _ in range(5):
        v = 1e-4 * rng.standard_normal(h.shape)
        assert abs((loss(h + v) - loss(h - v)) / 2 - np.sum(dh * v)) <= 1e-9


@pytest.mark.parametrize("reduction", ["tokens", "sequences", "sum"])
@pytest.mark.parametrize("per", ["token", "sequence"])
def test_oracle_policy_gradient_is_the_derivative(reduction, per):
    rng = np.random.default_rng(4)
    cu = [1, 4, 4, 9, 12]
    ce, old, ref = (rng.random(14) * 2 for _ in range(3))
    mask = rng.random(14) < 0.7
    adv = rng.standard_normal(14 if per == "token" else 4)
    kw = dict(mask=mask, ref=ref, kl_coef=0.3, reduction=reduction, advantage_per=per, scale=1.5)
    _, g, _ = oracle.policy_loss(ce, old, adv, cu, **kw)
    for t in range(14):
        e = np.zeros(14)
        e[t] = 1e-6
        d = (oracle.policy_loss(ce + e, old, adv, cu, **kw)[0] - oracle.policy_loss(ce - e, old, adv, cu, **kw)[0]) / 2e-6
        assert abs(d - g[t]) < 1e-7


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_oracle_preference_gradient_is_the_derivative(kind, average):
    rng = np.random.default_rng(5)
    cu = [0, 3, 5, 5, 9]
    ce, ref = rng.random(10) * 2, rng.random(10) * 2
    mask = rng.random(10) < 0.8
    kw = dict(mask=mask, ref=ref, beta=0.4, kind=kind, average=average, scale=0.7)
    if kind == "sigmoid":
        kw.update(label_smoothing=0.2, margin=0.1)
    _, g, _ = oracle.preference_loss(ce, cu, **kw)
    for t in range(10):
        e = np.zeros(10)
        e[t] = 1e-6
        d = (oracle.preference_loss(ce + e, cu, **kw)[0] - oracle.preference_loss(ce - e, cu, **kw)[0]) / 2e-6
        assert abs(d - g[t]) < 1e-7
