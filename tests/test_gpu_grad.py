"""The gradient through the packed head on the GPU against the float64 oracle.

Bound of an entry of dh[t] = g[t] sum_v G[t,v] W[v,:], from the roundings the
kernels make (u = 2^-11, half a step of fp16): the entries of W, the stored G,
the low-rank columns of G W and the rows of R and B are each rounded once, so
the products are off by at most 4 u of sum_v |G| |W| (entrywise absolute sums of
the three branches); G's fp16 subnormals add 2^-40 per row of the vocabulary;
the recomputed logits are off by at most the forward's tolerance tau each, which
with the normalisation moves a probability by at most e^(2 tau) - 1; the fp32 accumulation adds one rounding
(2^-23) per 16 rows of the vocabulary; the result is rounded to bf16 (2^-8)."""
import math

import numpy as np
import pytest
import torch

import archead_inputs as gen
import oracle

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


class Case:
    """A head, hidden states, targets, lse and gradients, with the oracle's answer and its bound."""

    def __init__(self, qoh, shape, T, scale=2.0, seed=0):
        V, d = shape[:2]
        self.shape, self.T = shape, T
        self.comps = gen.random_components(gen.HeadShape(*shape), seed + 1)
        bits, self.targets = gen.random_hidden(d, T, seed + 2, V)
        self.bits = gen.f32_to_bf16_bits(gen.bf16_bits_to_f32(bits) * scale)
        self.W, self.absW = oracle.dense_rows(self.comps, shape[4], shape[5])
        self.h = oracle.hidden_f64(self.bits)
        self.y = self.h @ self.W.T
        self.lse = oracle.lse_argmax_ce(self.y)[0]
        rng = np.random.default_rng(seed + 3)
        self.g = rng.standard_normal(T).astype(np.float32)
        self.g[rng.random(T) < 0.2] = 0.0
        self.head = qoh.PackedHead(*shape, self.comps)
        self.hidden = torch.from_numpy(self.bits.view(np.int16)).cuda().view(torch.bfloat16)
        self.args = [self.hidden, torch.from_numpy(self.targets).cuda(),
                     torch.from_numpy(self.lse.astype(np.float32)).cuda(), torch.from_numpy(self.g).cuda()]

    def expected(self):
        dh, G = oracle.ce_gradient(self.W, self.h, self.lse, self.targets, self.g)
        tau = oracle.tolerance(self.bits, np.abs(self.W).max(axis=1)) + 2.0 ** -23 * (1 + np.abs(self.lse))[:, None]
        p = np.exp(self.y - self.lse[:, None])
        V = self.W.shape[0]
        slack = np.abs(G) * (4.1 * 2.0 ** -11 + V / 16 * 2.0 ** -23) + p * np.expm1(2 * tau) + 2.0 ** -40
        return dh, np.abs(self.g)[:, None] * (slack @ self.absW)

    def check(self, got, rounding):
        dh, bound = self.expected()
        got = got.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        assert not got[self.g == 0].any()
        d = np.abs(got - dh)
        bound = bound * (1 + rounding) + rounding * np.abs(dh) + 1e-30
        worst = np.unravel_index(np.argmax(d / bound), d.shape)
        assert np.all(d <= bound), f"off by {(d / bound)[worst]:.3g} x the bound at {worst}: {got[worst]} {dh[worst]}"
        live = self.g != 0
        if live.any():   # far inside the bound as a whole: half a bf16 step and the independent fp16 roundings
            rel = np.linalg.norm(d[live]) / np.linalg.norm(dh[live])
            assert rel <= rounding + 4 * 2.0 ** -11 + np.expm1(2 * tolerance_of(self)), rel


def tolerance_of(case):
    return float(oracle.tolerance(case.bits, np.abs(case.W).max(axis=1)).max())


SHAPES = [
    (1000, 256, 32, 8, 64, 64),       # ragged vocabulary tail, both low-rank branches
    (17, 320, 100, 3, 64, 10),        # less than a tile of rows; scales of B in groups of 10
    (300, 64, 0, 0, 16, 1),           # no low-rank branch, smallest hidden size
    (2050, 128, 0, 64, 32, 64),       # correction only
    (4099, 512, 96, 0, 128, 512),     # core only
    (33000, 192, 64, 16, 64, 192),    # more than two vocabulary chunks
    (16400, 128, 64, 40, 16, 32),     # a last chunk of a few rows; groups of 16 and of 32
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 130, 300])
def test_gradient_matches_the_oracle(qoh, shape, T):
    c = Case(qoh, shape, T, seed=T)
    c.check(c.head.grad_hidden(*c.args), 2.0 ** -8)
    c.check(c.head.grad_hidden(*c.args, out_dtype=torch.float32), 2.0 ** -24)


@pytest.mark.parametrize("scale", [2.0 ** -60, 0.25, 16.0])
def test_peaked_and_flat_distributions(qoh, scale):
    """Logits near zero (uniform probabilities of a large vocabulary) up to ones that leave one row all the mass."""
    c = Case(qoh, (33000, 192, 64, 16, 64, 192), 40, scale=scale, seed=50)
    # half of the targets are the likeliest row: G there is a small difference
    c.targets[::2] = c.y.argmax(axis=1)[::2]
    c.args[1] = torch.from_numpy(c.targets).cuda()
    c.check(c.head.grad_hidden(*c.args, out_dtype=torch.float32), 2.0 ** -24)


def test_more_tokens_than_one_pass(qoh):
    c = Case(qoh, (300, 64, 16, 8, 16, 64), 4096 + 77, seed=60)
    c.check(c.head.grad_hidden(*c.args), 2.0 ** -8)


@pytest.mark.parametrize("shape,T", [((65531, 1024, 0, 0, 16, 128), 777), ((151936, 4096, 512, 64, 128, 128), 70),
                                     ((151936, 4096, 512, 64, 128, 128), 1100), ((262144, 2560, 384, 64, 128, 128), 16)])
def test_full_size_heads(qoh, shape, T):
    """Against the formula in fp64 on the device; relative error of each token's row in the 2-norm: independent fp16
    roundings (at most 4 * 2^-11, each) and half a bf16 step."""
    V, d, r_c, r_r, g, g_B = shape
    comps = gen.random_components(gen.HeadShape(*shape), 3)
    head = qoh.PackedHead(*shape, comps)
    rnd = torch.Generator(device="cuda").manual_seed(4)
    h = (torch.randn(T, d, generator=rnd, device="cuda") * (60.0 / math.sqrt(d))).bfloat16()
    targets = torch.randint(0, V, (T,), generator=rnd, device="cuda", dtype=torch.int32)
    grad = torch.randn(T, generator=rnd, device="cuda")

    def real(codes, scales, group=None):
        x = torch.from_numpy(codes).cuda().double()
        s = torch.from_numpy(scales.view(np.float16)).cuda().double()
        return x * (s[:, None] if group is None else s.repeat_interleave(group, 1))

    R, B = real(comps["R"], comps["s_R"]), real(comps["B"], comps["s_B"], g_B)

    def rows(a, b):
        return (real(comps["q"][a:b], comps["s_res"][a:b], g) + real(comps["L"][a:b], comps["s_L"][a:b]) @ R
                + real(comps["A"][a:b], comps["s_A"][a:b]) @ B)

    blocks = [(a, min(V, a + 32768)) for a in range(0, V, 32768)]
    lse = torch.logsumexp(torch.cat([h.double() @ rows(a, b).T for a, b in blocks], 1), 1)
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for a, b in blocks:
        w = rows(a, b)
        G = torch.exp(h.double() @ w.T - lse[:, None])
        at = torch.nonzero((targets >= a) & (targets < b))[:, 0]
        G[at, targets[at].long() - a] -= 1
        want += G @ w
    want *= grad.double()[:, None]
    got = head.grad_hidden(h, targets, lse.float(), grad)
    rel = (got.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(rel.max()) <= 2.0 ** -8 + 4 * 2.0 ** -11, float(rel.max())


def test_tokens_without_a_gradient_hold_anything(qoh):
    """A token with g = 0 gets zeros whatever its target, lse and hidden state are, and leaves the others' bits alone."""
    for T in (6, 40):
        c = Case(qoh, SHAPES[0], T, seed=70)
        c.g[:] = np.where(np.arange(T) % 3 == 1, 0.0, 1.0)
        hidden, targets, lse, g = c.args
        g = torch.from_numpy(c.g).cuda()
        want = c.head.grad_hidden(hidden, targets, lse, g)
        hidden, targets, lse = hidden.clone(), targets.clone(), lse.clone()
        hidden[1::3], targets[1::3], lse[1::3] = NAN, -100, NAN
        ws = torch.full((c.head.grad_workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")
        got = c.head.grad_hidden(hidden, targets, lse, g, workspace=ws)
        assert torch.equal(got, want) and not got[1::3].any()
        assert c.head.status(ws) == 0
        targets[3] = c.shape[0]
        got = c.head.grad_hidden(hidden, targets, lse, g, workspace=ws)
        assert torch.isnan(got[3]).all() and torch.equal(got[:3], want[:3]) and torch.equal(got[4:], want[4:])
        assert c.head.status(ws) == qoh.STATUS_BAD_TARGET


def test_vocabulary_shards_add_up(qoh):
    shape = (3000, 256, 64, 16, 64, 64)
    c = Case(qoh, shape, 33, seed=80)
    total = torch.zeros(33, 256, device="cuda")
    for v0, v1 in ((0, 1024), (1024, 1040), (1040, 3000)):
        shard = qoh.PackedHead(v1 - v0, *shape[1:], qoh.shard_components(c.comps, v0, v1))
        shard.set_vocab_shard(v0, shape[0])
        total += shard.grad_hidden(*c.args, out_dtype=torch.float32)
    c.check(total, 4 * 2.0 ** -24)


def test_same_bits_on_any_stream_and_in_graphs(qoh):
    """Eager calls on two streams at once, two captured graphs, and a replay on changed inputs."""
    for T in (5, 50):
        a, b = Case(qoh, SHAPES[5], T, seed=90), Case(qoh, SHAPES[0], T, seed=91)
        want = [x.head.grad_hidden(*x.args) for x in (a, b)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(4)]
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x = (a, b)[i % 2]
                got.append(x.head.grad_hidden(*x.args))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
        graphs = []
        for x in (a, b):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = x.head.grad_hidden(*x.args)
            graphs.append((g, out))
        a.args[3].mul_(2.0)
        for _ in range(2):
            for g, _ in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], want[0] * 2) and torch.equal(graphs[1][1], want[1])


@pytest.mark.parametrize("T", [7, 60])
def test_a_training_step_follows_the_loss(qoh, T):
    """lse_argmax -> loss -> grad_hidden: the gradient of each loss along random directions against central differences
    of the whole loss in float64 (oracle), within the entrywise bound summed along the direction."""
    shape = (1500, 256, 64, 16, 64, 64)
    c = Case(qoh, shape, T, scale=4.0, seed=100 + T)
    head, hidden = c.head, c.hidden
    lse, _, ce = head.lse_argmax(hidden, c.args[1])
    rng = np.random.default_rng(5)
    cu = np.array([0, T // 3, T // 2, T - 1, T], np.int32)
    old, ref = ((ce.cpu().numpy() + 0.05 * rng.standard_normal(T)).astype(np.float32) for _ in range(2))
    adv = rng.standard_normal(4).astype(np.float32)
    mask = np.arange(T) % 5 != 2
    dev = [torch.from_numpy(x).cuda() for x in (old, adv, cu, mask, ref)]

    def by_oracle(h, kind):
        ce64 = oracle.lse_argmax_ce(h @ c.W.T, c.targets)[2]
        if kind == "policy":
            return oracle.policy_loss(ce64, old, adv, cu, mask, ref, kl_coef=0.3, reduction="sequences",
                                      advantage_per="sequence", clip_low=0.9, clip_high=5.0)[0]
        return oracle.preference_loss(ce64, cu, mask, ref, beta=0.5)[0]

    for kind in ("policy", "preference"):
        if kind == "policy":
            _, g, _ = qoh.policy_loss(ce, dev[0], dev[1], dev[2], mask=dev[3], ce_ref=dev[4], kl_coef=0.3,
                                      reduction="sequences", advantage_per="sequence", clip_low=0.9, clip_high=5.0)
        else:
            _, g, _ = qoh.preference_loss(ce, dev[2], mask=dev[3], ce_ref=dev[4], beta=0.5)
        dh = head.grad_hidden(hidden, c.args[1], lse, g, out_dtype=torch.float32).double().cpu().numpy()
        c.g = g.cpu().numpy()
        dh64, bound = c.expected()
        # the loss's own gradients start from ce, off by up to twice the forward's tolerance
        tau = 2 * tolerance_of(c)
        for _ in range(4):
            v = rng.standard_normal(c.h.shape)
            v *= 1e-4 / np.linalg.norm(v)
            slope = (by_oracle(c.h + v, kind) - by_oracle(c.h - v, kind)) / 2
            slack = np.sum(np.abs(v) * (bound + np.abs(dh64) * 2.0 ** -23)) + 2 * tau * np.sum(np.abs(v * dh64)) + 1e-12
            assert abs(np.sum(v * dh) - slope) <= slack


def test_refusals(qoh):
    c = Case(qoh, SHAPES[0], 4, seed=110)
    h, t, lse, g = c.args
    bad = [(h[:, :128], t, lse, g), (h.float(), t, lse, g), (h, t[:3], lse, g), (h, t, lse[:3], g), (h, t, lse, g.double()),
           (h.cpu(), t, lse, g), (h, t, lse.cpu(), g)]
    for args in bad:
        with pytest.raises(ValueError):
            c.head.grad_hidden(*args)
    with pytest.raises(ValueError):
        c.head.grad_hidden(*c.args, out_dtype=torch.float16)
    with pytest.raises(qoh.ArcheadError):
        c.head.grad_hidden(h[:0], t[:0], lse[:0], g[:0])
    with pytest.raises(qoh.ArcheadError):
        c.head.grad_hidden(*c.args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[4], SHAPES[5]])
def test_many_tokens(qoh, shape):
    """From 1024 tokens on z comes from fp16 rows of R and B: their rounding reaches the logits as well, by at most
    2^-11 of sum |h| |R| |L| per logit, which is added to the forward's tolerance (two branches, on both sides of the
    normalisation)."""
    c = Case(qoh, shape, 1030, seed=90)
    comps = c.comps

    def real(codes, scales, group=None):
        s = scales.view(np.float16).astype(np.float64)
        return np.abs(codes * (s[:, None] if group is None else np.repeat(s, group, axis=1)))

    low = real(comps["L"], comps["s_L"]) @ real(comps["R"], comps["s_R"])
    low += real(comps["A"], comps["s_A"]) @ real(comps["B"], comps["s_B"], shape[5])
    dz = 2.0 ** -11 * (np.abs(c.h) @ low.T)                  # [T, V]
    dh, bound = c.expected()
    p = np.exp(c.y - c.lse[:, None])
    bound = bound + np.abs(c.g)[:, None] * ((p * np.expm1(2 * dz.max(axis=1))[:, None]) @ c.absW)
    got = c.head.grad_hidden(*c.args).double().cpu().numpy()
    bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dh) + 1e-30
    assert not got[c.g == 0].any()
    assert np.all(np.abs(got - dh) <= bound), (np.abs(got - dh) / bound).max()


@pytest.mark.parametrize("shape,T", [(SHAPES[0], 1100), (SHAPES[5], 300), (SHAPES[6], 300)])
def test_many_tokens_without_a_gradient_hold_anything(qoh, shape, T):
    c = Case(qoh, shape, T, seed=95)
    hidden, targets, lse, _ = c.args
    g = torch.where(torch.arange(T, device="cuda") % 3 == 1, 0.0, 1.0)
    want = c.head.grad_hidden(hidden, targets, lse, g)
    hidden, targets, lse = hidden.clone(), targets.clone(), lse.clone()
    hidden[1::3], targets[1::3], lse[1::3] = NAN, -100, NAN
    hidden[4] = float("inf")
    ws = torch.full((c.head.grad_workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")
    got = c.head.grad_hidden(hidden, targets, lse, g, workspace=ws)
    assert torch.equal(got, want) and not got[1::3].any()
    assert c.head.status(ws) == 0


def test_chunks_and_passes_together(qoh):
    """Two passes over the tokens of a head of two chunks of rows, against each token alone in a small call."""
    shape, T = (70001, 128, 64, 16, 64, 64), 4096 + 300
    comps = gen.random_components(gen.HeadShape(*shape), 97)
    head = qoh.PackedHead(*shape, comps)
    rnd = torch.Generator(device="cuda").manual_seed(98)
    h = torch.randn(T, shape[1], generator=rnd, device="cuda").bfloat16()
    targets = torch.randint(0, shape[0], (T,), generator=rnd, device="cuda", dtype=torch.int32)
    targets[-1] = shape[0] - 1
    grad = torch.randn(T, generator=rnd, device="cuda")
    lse = torch.cat([head.lse_argmax(h[i:i + 512])[0] for i in range(0, T, 512)])
    got = head.grad_hidden(h, targets, lse, grad, out_dtype=torch.float32).double()
    for i in (0, 100, 4000, 4095, 4096, T - 100):
        few = head.grad_hidden(h[i:i + 100], targets[i:i + 100].contiguous(), lse[i:i + 100].contiguous(),
                               grad[i:i + 100].contiguous(), out_dtype=torch.float32).double()
        part = got[i:i + 100]
        # independent fp16 roundings on both sides (at most 4 * 2^-11, each)
        rel = (part - few).norm(dim=1) / few.norm(dim=1)
        assert float(rel.max()) <= 8 * 2.0 ** -11, (i, float(rel.max()))


@pytest.mark.parametrize("shape", [(700, 640, 600, 70, 64, 64), (700, 640, 400, 700, 64, 20)])
@pytest.mark.parametrize("T", [1, 3, 4, 7])
def test_few_tokens_of_many_low_rank_rows(qoh, shape, T):
    """More low-rank rows than the last product of a few tokens keeps in shared memory at a time."""
    c = Case(qoh, shape, T, seed=100 + T)
    c.check(c.head.grad_hidden(*c.args), 2.0 ** -8)
    c.check(c.head.grad_hidden(*c.args, out_dtype=torch.float32), 2.0 ** -24)


def test_many_tokens_on_streams_and_in_graphs(qoh):
    """Two calls of the many-token path at once, and each captured and replayed, with the bits of a call alone."""
    a, b = Case(qoh, SHAPES[0], 1100, seed=110), Case(qoh, SHAPES[6], 300, seed=111)
    want = [x.head.grad_hidden(*x.args) for x in (a, b)]
    torch.cuda.synchronize()
    got = []
    for i in range(4):
        with torch.cuda.stream(torch.cuda.Stream()):
            x = (a, b)[i % 2]
            got.append(x.head.grad_hidden(*x.args))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.head.grad_hidden(*x.args)
        graphs.append((g, out))
    a.args[3].mul_(2.0)
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want[0] * 2) and torch.equal(graphs[1][1], want[1])
