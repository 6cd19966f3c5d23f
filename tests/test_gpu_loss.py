"""The policy and preference losses on the GPU against the float64 oracle.

The kernels work in fp64 from the same fp32 inputs and round each output to
fp32 once (per-sequence factors too), so an output is within 4 * 2^-24 of the
oracle's value, relative, plus 2^-40 of the size of the terms that are added up:
the exponential is good to 2^-41 of its value, and a sum over up to 2^20 tokens
is at most 1100 additions long in any chain (2^-42 of the sum of magnitudes)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
EPS = 4 * 2.0 ** -24


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


def close(got, want, size, what):
    got = got.double().cpu().numpy()
    d = np.abs(got - want)
    bound = EPS * np.abs(want) + 2.0 ** -40 * size + 1e-300
    assert np.all(d <= bound), f"{what}: off by {np.max(d / bound):.3g} x the bound"


def tokens(lengths, seed, tail=0, head=0, spread=0.2):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[head], head + np.cumsum(lengths)]).astype(np.int32)
    T = int(cu[-1]) + tail
    ce = rng.lognormal(-0.5, 1.0, T).astype(np.float32)
    old = np.maximum(ce + spread * rng.standard_normal(T), 0).astype(np.float32)
    ref = np.maximum(ce + spread * rng.standard_normal(T), 0).astype(np.float32)
    mask = rng.random(T) < 0.6
    return rng, cu, T, ce, old, ref, mask


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def shifted(x, n=1):
    """The same values at an address that is n elements off a 16-byte boundary."""
    if x is None:
        return None
    b = torch.empty(x.shape[0] + n, dtype=x.dtype, device="cuda")
    b[n:] = x
    return b[n:]


LENGTHS = {
    "one token": [1],
    "one sequence": [77],
    "single tokens": [1] * 300,
    "empty ones": [0, 5, 0, 0, 130, 0, 1, 0],
    "all empty": [0, 0, 0, 0],
    "ragged": [3, 128, 127, 129, 4000, 1, 0, 2, 513, 256],
    "long": [70000, 3, 40000, 0],
    "many short": list(np.random.default_rng(1).integers(0, 9, 6000)),
}


@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("reduction,per", [("tokens", "token"), ("sequences", "sequence"), ("sum", "sequence"),
                                           ("sequences", "token")])
@pytest.mark.parametrize("masked,with_ref,off", [(False, False, 0), (True, True, 1), (True, False, 0)])
def test_policy_loss_matches_the_oracle(qoh, name, reduction, per, masked, with_ref, off):
    lengths = LENGTHS[name]
    rng, cu, T, ce, old, ref, mask = tokens(lengths, 7, tail=5, head=3 if masked else 0)
    adv = rng.standard_normal(T if per == "token" else len(lengths)).astype(np.float32)
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.04, reduction=reduction, advantage_per=per, scale=0.5)
    m, r = (mask if masked else None), (ref if with_ref else None)
    args = [dev(x) for x in (ce, old, adv)]
    opt = dict(mask=dev(m), ce_ref=dev(r))
    if off:
        args, opt = [shifted(x) for x in args], {k: shifted(v) for k, v in opt.items()}
    loss, grad, stats = qoh.policy_loss(*args, dev(cu), **opt, **kw)
    want = oracle.policy_loss(ce, old, adv, cu, m, r, **kw)
    size = np.abs(adv).max() * 3 if reduction != "sum" else T * np.abs(adv).max() * 3
    close(loss, want[0], size, "loss")
    close(grad, want[1], np.abs(want[1]).max(), "gradient")
    close(stats, want[2], 1, "stats")


def test_policy_loss_without_offsets_is_one_sequence(qoh):
    rng, cu, T, ce, old, ref, mask = tokens([1000], 8)
    adv = rng.standard_normal(T).astype(np.float32)
    a = qoh.policy_loss(dev(ce), dev(old), dev(adv))
    b = qoh.policy_loss(dev(ce), dev(old), dev(adv), dev(cu))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_policy_loss_borders_masked_values_and_extremes(qoh):
    """At a border the ratio counts as inside; what the mask leaves out may be
    NaN or infinite; a token of probability 0 has ratio 0; a huge ratio is
    clipped (A > 0) or infinite (A < 0); a small divergence keeps its digits."""
    ce = np.array([1, 1, np.nan, np.inf, np.inf, 0, 0, 1], np.float32)
    old = np.array([1, 1, 1, np.nan, 2, 800, 800, 1], np.float32)
    adv = np.array([1, -1, 3, np.inf, 1, 1, -1, 2], np.float32)
    mask = np.array([1, 1, 0, 0, 1, 1, 1, 1], bool)
    loss, grad, stats = qoh.policy_loss(dev(ce), dev(old), dev(adv), mask=dev(mask), clip_low=0.0, clip_high=0.0,
                                        reduction="sum")
    g = grad.cpu().numpy()
    assert g[2] == 0 and g[3] == 0 and g[4] == 0 and g[5] == 0 and np.isneginf(g[6]) and g[7] == 2
    assert g[0] == 1 and g[1] == -1
    assert torch.isposinf(loss)
    ce = np.full(50, 1.0, np.float32)
    ref = np.float32(1.0) + np.arange(-25, 25, dtype=np.float32) * np.float32(2.0 ** -20)
    _, grad, stats = qoh.policy_loss(dev(ce), dev(ce), dev(np.zeros(50, np.float32)), ce_ref=dev(ref), kl_coef=1.0)
    d = 1.0 - ref.astype(np.float64)
    close(stats[2], np.mean(d * d / 2 + d ** 3 / 6), 0, "divergence")
    close(grad, np.expm1(d) / 50, 0, "gradient")


def test_policy_gradient_is_the_derivative(qoh):
    """Central differences of the kernel's own loss (sum reduction; fp32 loss)."""
    rng, cu, T, ce, old, ref, mask = tokens([40, 0, 25], 9, spread=0.05)
    adv = np.ones(T, np.float32)
    kw = dict(mask=dev(mask), ce_ref=dev(ref), kl_coef=0.5, reduction="sequences", clip_low=0.9, clip_high=9.0)
    _, grad, _ = qoh.policy_loss(dev(ce), dev(old), dev(adv), dev(cu), **kw)
    step, v = 2.0 ** -7, rng.standard_normal(T).astype(np.float32)
    up = qoh.policy_loss(dev(ce + step * v), dev(old), dev(adv), dev(cu), **kw)[0]
    down = qoh.policy_loss(dev(ce - step * v), dev(old), dev(adv), dev(cu), **kw)[0]
    slope = float(up.double() - down.double()) / (2 * step)
    # third derivatives are below 3; rounding of the two losses and of the arguments below 2^-21
    bound = step ** 2 * np.mean(np.abs(v) ** 3) * 3 + 2.0 ** -21 / step
    assert abs(slope - float((grad.double().cpu() @ torch.from_numpy(v).double()))) <= bound


PAIRS = {
    "one pair": [5, 9],
    "single tokens": [1] * 400,
    "empty ones": [0, 3, 7, 200, 0, 0],
    "ragged": [128, 1, 0, 700, 129, 127, 4096, 5, 6, 2],
    "long": [60000, 3, 2, 30001],
    "many short": list(np.random.default_rng(2).integers(0, 6, 8000)),
}


@pytest.mark.parametrize("name", list(PAIRS))
@pytest.mark.parametrize("kind,extra", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.1, margin=0.3)),
                                        ("hinge", dict(margin=-0.2)), ("squared", {})])
@pytest.mark.parametrize("average,masked,with_ref,off", [(False, False, True, 0), (True, True, True, 1),
                                                         (False, True, False, 0)])
def test_preference_loss_matches_the_oracle(qoh, name, kind, extra, average, masked, with_ref, off):
    rng, cu, T, ce, _, ref, mask = tokens(PAIRS[name], 17, tail=3, head=2 if masked else 0)
    m, r = (mask if masked else None), (ref if with_ref else None)
    kw = dict(beta=0.1, kind=kind, average=average, scale=2.0, **extra)
    t = [dev(x) for x in (ce, m, r)]
    if off:
        t = [shifted(x) for x in t]
    loss, grad, rewards = qoh.preference_loss(t[0], dev(cu), mask=t[1], ce_ref=t[2], **kw)
    want = oracle.preference_loss(ce, cu, m, r, **kw)
    # sums of `terms`; the squared loss has a slope of up to `steep` in them
    N, terms, steep = want[2].shape[1], np.abs(ce).sum(), 2 * (np.abs(want[2]).max() / 0.1 * 2 + 5)
    close(rewards, want[2], 0.1 * terms, "rewards")
    close(loss, want[0], 2 * terms * (steep if kind == "squared" else 0.1), "loss")
    close(grad, want[1], 2 * terms * (2 if kind == "squared" else 0.01) / N + np.abs(want[1]).max(), "gradient")


def test_preference_loss_extremes(qoh):
    """Margins far out keep finite losses and full-precision slopes; a response
    of probability 0 loses outright; masked NaNs have no part; no pairs at all."""
    ce = np.array([500, 1, 1, 500, 1, np.nan, np.inf, 1], np.float32)
    cu = np.array([0, 1, 2, 4, 5, 6, 8], np.int32)   # chosen: [0:1] [1:2] [2:4]; rejected: [4:5] [5:6] [6:8]
    mask = np.array([1, 1, 1, 1, 1, 0, 1, 1], bool)
    loss, grad, rewards = qoh.preference_loss(dev(ce), dev(cu), mask=dev(mask), beta=1.0)
    g, r = grad.cpu().numpy(), rewards.cpu().numpy()
    assert r[0, 0] == -500 and r[1, 0] == -1 and r[1, 1] == 0 and np.isneginf(r[1, 2])
    assert abs(float(loss) - (499 + np.log1p(np.exp(1)) + 0) / 3) < 1e-4
    assert abs(g[0] - 1 / 3) < 1e-6 and abs(g[4] + 1 / 3) < 1e-6 and g[5] == 0 and g[2] == 0 and g[6] == 0
    loss, grad, rewards = qoh.preference_loss(dev(ce), dev(np.zeros(1, np.int32)))
    assert float(loss) == 0 and not grad.any() and rewards.shape == (2, 0)


def test_losses_of_no_tokens(qoh):
    none = torch.empty(0, device="cuda")
    loss, grad, stats = qoh.policy_loss(none, none, none)
    assert float(loss) == 0 and grad.shape == (0,) and not stats.any()
    loss, grad, rewards = qoh.preference_loss(none, torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert abs(float(loss) - np.log(2)) < 1e-6 and not rewards.any()


def test_offsets_outside_the_tokens_touch_nothing_else(qoh):
    """Offsets that are not what they should be give no access outside the arrays:
    the neighbours of the gradient stay as they were."""
    import ctypes
    lib, T = qoh._lib, 300
    ce = torch.rand(T, device="cuda")
    cu = torch.tensor([5, -7, 900, 20, 20, 2 ** 31 - 1, 100], dtype=torch.int32, device="cuda")
    buf = torch.full((T + 64,), 7.0, device="cuda")
    few = torch.empty(16, device="cuda")
    ws = torch.full((lib.archead_loss_workspace_bytes(6) + 256,), 255, dtype=torch.uint8, device="cuda")
    n = lib.archead_loss_workspace_bytes(6)
    for fn, opts, extra in ((lib.archead_policy_loss, qoh.ArcheadPolicyOptions(0.2, 0.2, 0.0, 1.0, 1, 0), True),
                            (lib.archead_preference_loss, qoh.ArcheadPreferenceOptions(0.1, 0, 0, 1.0, 0, 0), False)):
        p = ce.data_ptr()
        args = ([p, p, p, None, None, cu.data_ptr(), T, 6] if extra else [p, None, None, cu.data_ptr(), T, 3])
        rc = fn(*args, ctypes.byref(opts), few.data_ptr(), buf.data_ptr() + 128, few.data_ptr() + 4, ws.data_ptr(), n, None)
        torch.cuda.synchronize()
        assert rc == 0 and torch.all(buf[:32] == 7) and torch.all(buf[32 + T:] == 7) and torch.all(ws[n:] == 255)


@pytest.mark.parametrize("lengths", [[90, 3, 0, 1000], [900, 3000, 0, 10000], [30000, 70000, 1, 55000]])
def test_losses_on_another_stream_and_in_a_graph(qoh, lengths):
    """Two captured graphs and eager calls side by side give the same bits, and a
    replay reads the inputs as they are then (one block, a cluster, a grid)."""
    rng, cu, T, ce, old, ref, mask = tokens(lengths, 21)
    ce_d, old_d, ref_d, mask_d, cu_d = (dev(x) for x in (ce, old, ref, mask, cu))
    adv = dev(rng.standard_normal(4).astype(np.float32))

    def policy():
        return qoh.policy_loss(ce_d, old_d, adv, cu_d, mask=mask_d, ce_ref=ref_d, kl_coef=0.1, advantage_per="sequence",
                               reduction="sequences")

    def preference():
        return qoh.preference_loss(ce_d, cu_d, mask=mask_d, ce_ref=ref_d)

    want = policy() + preference()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = policy() + preference()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for f in (policy, preference):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    ce_d.mul_(1.01)
    want = policy() + preference()
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, graphs[0][1] + graphs[1][1]))


def test_largest_batch(qoh):
    """2^20 tokens, the library's limit: against the formula in fp64 on the device."""
    T = 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(5)
    ce = torch.rand(T, generator=gen, device="cuda") * 3
    old = ce + 0.1 * torch.randn(T, generator=gen, device="cuda")
    adv = torch.randn(T, generator=gen, device="cuda")
    loss, grad, stats = qoh.policy_loss(ce, old, adv)
    D = old.double() - ce.double()
    r, A = D.exp(), adv.double()
    plain, clipped = -A * r, -A * r.clamp(0.8, 1.2)
    close(loss, float(torch.maximum(plain, clipped).mean()), 5, "loss")
    close(grad, torch.where(clipped > plain, 0.0, A * r / T).cpu().numpy(), 0, "gradient")
    with pytest.raises(qoh.ArcheadError):
        qoh.policy_loss(*(torch.zeros(T + 1, device="cuda"),) * 3)


def test_refusals(qoh):
    z, zi = torch.zeros(8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [lambda: qoh.policy_loss(z.double(), z, z), lambda: qoh.policy_loss(z, z[:4], z),
           lambda: qoh.policy_loss(z, z, z, zi, advantage_per="sequence"), lambda: qoh.policy_loss(z.cpu(), z, z),
           lambda: qoh.policy_loss(z, z, z, mask=z), lambda: qoh.policy_loss(z, z, z, reduction="mean"),
           lambda: qoh.policy_loss(z, z, z, zi.float()), lambda: qoh.policy_loss(z.view(2, 4), z, z),
           lambda: qoh.preference_loss(z, zi[:2]), lambda: qoh.preference_loss(z, zi, kind="ipo"),
           lambda: qoh.preference_loss(z, zi, ce_ref=z[:3])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    worse = [lambda: qoh.policy_loss(z, z, z, clip_low=1.5), lambda: qoh.policy_loss(z, z, z, clip_high=-0.1),
             lambda: qoh.policy_loss(z, z, z, kl_coef=float("nan")), lambda: qoh.preference_loss(z, zi, beta=0.0),
             lambda: qoh.preference_loss(z, zi, label_smoothing=0.7), lambda: qoh.preference_loss(z, zi, kind="hinge", label_smoothing=0.1),
             lambda: qoh.preference_loss(z, zi, kind="squared", margin=1.0)]
    for f in worse:
        with pytest.raises(qoh.ArcheadError):
            f()
