"""The gradient on a vocabulary shard: probabilities exp(y - lse) with the lse as it is given, so what the recomputed
logits are off by reaches the result, with nothing to normalise it."""
import numpy as np
import pytest
import torch

import archead_inputs as gen
import oracle
from test_gpu_grad_confident import SHAPE, Sure

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


def fp16(x):
    return np.asarray(x, np.float64).astype(np.float16).view(np.uint16)


def awkward_head(V, d, r_c, r_r, g_B, seed):
    """Logits of 30 to 40 from the low-rank branches alone.  Rows of R and B alternate codes 127 and 1 under a scale of
    1088 units: 127 * 1088 lies halfway between two fp16 values, every time on the same side, while the sums over h and
    the entries of L and A times their scales are fp16 values."""
    rng = np.random.default_rng(seed)
    c = gen.random_components(gen.HeadShape(V, d, r_c, r_r, 64, g_B), seed)
    c["q"] = np.zeros_like(c["q"])
    for rows, scale in (("R", "s_R"), ("B", "s_B")):
        c[rows] = np.where(np.arange(d) % 2 == 0, 127, 1).astype(np.int8) * np.ones((c[rows].shape[0], 1), np.int8)
        c[scale] = fp16(np.full(c[scale].shape, 1088 / 1024 * 2.0 ** -14))
    c["L"] = rng.integers(10, 16, c["L"].shape).astype(np.int8)
    c["s_L"] = fp16(np.full(V, 2.0 ** -5 if r_r == 0 else 2.0 ** -6))
    c["A"] = rng.integers(80, 128, c["A"].shape).astype(np.int8)
    c["s_A"] = fp16(np.full(V, 2.0 ** -8 if r_c == 0 else 2.0 ** -9))
    return c


@pytest.mark.parametrize("r_c,r_r", [(64, 0), (0, 64), (64, 64)])
@pytest.mark.parametrize("T,g_B", [(4, 64), (40, 64), (300, 64), (1100, 64), (5, 32), (40, 32)])
def test_logits_of_a_shard_are_the_forwards(qoh, T, g_B, r_c, r_r):
    """z and the rows are exact here, so a logit of up to 60 is off by the fp32 sums (of at most 2 * 64 products in one
    accumulator: 60 * 2^-24 * 128 at the very most, 2^-11) and lse by its rounding (2^-19): probabilities move by at
    most 2^-10.  G, the low-rank dX and the rows of the last product round to fp16 (2^-11 each)."""
    V, d = 600, 256
    comps = awkward_head(V, d, r_c, r_r, g_B, 5)
    head = qoh.PackedHead(V, d, r_c, r_r, 64, g_B, comps)
    head.set_vocab_shard(0, V + 1000)
    W, absW = oracle.dense_rows(comps, 64, g_B)
    rng = np.random.default_rng(6)
    h = np.where(np.arange(T) % 2 == 0, 1.0, 1.5)[:, None] * np.ones((1, d))
    bits = gen.f32_to_bf16_bits(h.astype(np.float32))
    y = h @ W.T
    lse = (oracle.lse_argmax_ce(y)[0] + 0.1).astype(np.float32)   # (the other shards hold a tenth of the mass)
    targets = rng.integers(0, V + 1000, T).astype(np.int32)
    g = rng.choice([-1.0, 0.5, 2.0], T).astype(np.float32)
    p = np.exp(y - lse.astype(np.float64)[:, None])
    G = p.copy()
    for t in np.nonzero(targets < V)[0]:
        G[t, targets[t]] -= 1.0
    assert 25 < y.min() and y.max() < 60
    want = g[:, None] * (G @ W)
    bound = np.abs(g)[:, None] * ((3 * 2.0 ** -11 + 2.0 ** -10) * (p @ absW) + 2.0 ** -10 * (np.abs(G) @ absW))
    got = head.grad_hidden(torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), torch.from_numpy(targets).cuda(),
                           torch.from_numpy(lse).cuda(), torch.from_numpy(g).cuda(), out_dtype=torch.float32)
    worst = np.abs(got.double().cpu().numpy() - want) / bound
    assert np.all(worst <= 1), worst.max()


@pytest.mark.parametrize("g_B", [64, 32])
@pytest.mark.parametrize("T", [1, 4, 40, 130, 300, 1100])
def test_sure_tokens_on_shards(qoh, T, g_B):
    """With the lse that the shards' forwards give, merged.  The rows of sure tokens (see test_gpu_grad_confident) get the
    target's coefficient from exp(y - lse) - 1, which is as exact as y and lse agree: both are sums of the same products in
    fp32, so off by lse's roundings (2^-22 (1 + |lse|)) and by those of K / 16 partial sums on either side, which are
    independent: four standard deviations at most, of sqrt(K / 16) 2^-24 times sum |W| |h| each."""
    shape = SHAPE[:5] + (g_B,)
    comps = gen.random_components(gen.HeadShape(*shape), 31)
    c = Sure(comps, T, 80 + T, shape)
    h, targets, _, g = c.args()
    shards = []
    for v0, v1 in ((0, 1008), (1008, 2000)):
        s = qoh.PackedHead(v1 - v0, *shape[1:], qoh.shard_components(comps, v0, v1))
        s.set_vocab_shard(v0, shape[0])
        shards.append(s)
    lse, _, _ = qoh.merge_shards(torch.stack([s.shard_partials(h, targets) for s in shards]))
    got = sum(s.grad_hidden(h, targets, lse, g, out_dtype=torch.float32) for s in shards).double().cpu().numpy()
    products = np.einsum("ij,ij->i", np.abs(c.h), c.absW[c.targets])
    agree = 2.0 ** -22 * (1 + np.abs(c.lse)) + 4 * np.sqrt(2 * (shape[1] + 32 + 64) / 16) * 2.0 ** -24 * products
    rel = 5.1 * 2.0 ** -11 + shape[0] / 16 * 2.0 ** -23
    bound = ((rel + np.expm1(2 * c.tau))[:, None] * c.terms + c.least + 2.0 ** -22 * np.abs(c.dh)
             + (np.abs(c.g) * agree)[:, None] * c.absW[c.targets])
    worst = (np.abs(got - c.dh) / bound).max(axis=1)
    assert np.all(worst <= 1), (worst.max(), c.left[worst.argmax()])
