"""Tokens that the head is sure of, and an lse that is not the head's own: the
gradient g (softmax - onehot) W of a whole head depends on lse only through its
own normalisation, and no term of it may be lost against 1.

With p the softmax, q = 1 - p[target] and |W| the entrywise sums of the three
branches' absolute terms, the exact row is
  dh / g = sum_{v != target} p[v] (W[v] - W[target]),
so it is of size q.  Each rounding to fp16 (2^-11 relative: W~ entries, G, the
low-rank columns of dX, the rows of R and B) acts on a term of that sum, the
recomputed logits move p[v] / p[target] by at most e^(2 tau) - 1 (tau: the forward's
tolerance of the row's largest logit), sums are fp32 (2^-23 per 16 rows), and G's subnormals add
2^-40 per row of the vocabulary:
  |error| <= |g| ( (4.1 * 2^-11 + V / 16 * 2^-23 + e^(2 tau) - 1) sum p[v] (|W[v]| + |W[target]|)
                   + 2^-40 sum |W[v]| )."""
import numpy as np
import pytest
import torch

import archead_inputs as gen
import oracle

pytestmark = pytest.mark.gpu
SHAPE = (2000, 256, 32, 8, 64, 64)
LEFT = (1e-2, 1e-4, 1e-6, 0.5)          # about 1 - p[target] of tokens 0, 1, 2, 3, 4, ...


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


@pytest.fixture(scope="module")
def comps():
    return gen.random_components(gen.HeadShape(*SHAPE), 31)


class Sure:
    """Hidden states along one row of the head each, as long as leaves the other rows the mass asked for; the target is
    that row or (every fifth token) any."""

    def __init__(self, comps, T, seed, shape=SHAPE):
        V = shape[0]
        rng = np.random.default_rng(seed)
        self.W, self.absW = oracle.dense_rows(comps, shape[4], shape[5])
        unit = self.W / np.linalg.norm(self.W, axis=1, keepdims=True)
        along = unit @ self.W.T
        first = np.nonzero(np.diag(along) > 1.3 * np.sort(along - np.diag(np.diag(along)), axis=1)[:, -1])[0]
        self.targets = rng.choice(first, T).astype(np.int32)
        towards = unit[self.targets]
        slope = towards @ self.W.T                               # logits per unit of length
        own = slope[np.arange(T), self.targets]
        lo, hi = np.zeros(T), np.full(T, 1e4)
        want = np.array([LEFT[t % len(LEFT)] for t in range(T)])
        for _ in range(60):
            mid = (lo + hi) / 2
            e = np.exp(np.minimum(mid[:, None] * (slope - own[:, None]), 50))
            e[np.arange(T), self.targets] = 0
            rest = e.sum(axis=1)
            big = rest / (1 + rest) > want
            lo, hi = np.where(big, mid, lo), np.where(big, hi, mid)
        self.bits = gen.f32_to_bf16_bits((towards * hi[:, None]).astype(np.float32))
        self.h = oracle.hidden_f64(self.bits)
        self.targets[4::5] = rng.integers(0, V, self.targets[4::5].size)
        y = self.h @ self.W.T
        self.lse = oracle.lse_argmax_ce(y)[0]
        p = np.exp(y - self.lse[:, None])
        p[np.arange(T), self.targets] = 0
        self.g = rng.choice([-2.0, 0.7, 1.0], T).astype(np.float32)
        self.left = p.sum(axis=1)
        sure = np.arange(T) % 5 != 4
        assert np.all((self.left[sure] > want[sure] / 3) & (self.left[sure] < want[sure] * 3))
        own_row = self.W[self.targets]
        self.dh = self.g[:, None] * (p @ self.W - self.left[:, None] * own_row)
        self.terms = np.abs(self.g)[:, None] * (p @ self.absW + self.left[:, None] * self.absW[self.targets])
        self.least = np.abs(self.g)[:, None] * 2.0 ** -40 * self.absW.sum(axis=0)
        top = np.abs(self.W).max()
        self.tau = 2e-3 * np.linalg.norm(self.h, axis=1) * top

    def args(self, delta=0.0):
        return (torch.from_numpy(self.bits.view(np.int16)).cuda().view(torch.bfloat16), torch.from_numpy(self.targets).cuda(),
                torch.from_numpy((self.lse + delta).astype(np.float32)).cuda(), torch.from_numpy(self.g).cuda())


@pytest.mark.parametrize("T", [1, 4, 40, 300, 1100])
@pytest.mark.parametrize("delta", [0.0, 0.01, 0.1, -0.3])
def test_rows_of_sure_tokens(qoh, comps, T, delta):
    c = Sure(comps, T, 40 + T)
    head = qoh.PackedHead(*SHAPE, comps)
    got = head.grad_hidden(*c.args(delta), out_dtype=torch.float32).double().cpu().numpy()
    rel = 4.1 * 2.0 ** -11 + SHAPE[0] / 16 * 2.0 ** -23
    bound = (rel + np.expm1(2 * c.tau))[:, None] * c.terms + c.least + 2.0 ** -24 * np.abs(c.dh)
    worst = (np.abs(got - c.dh) / bound).max(axis=1)
    assert np.all(worst <= 1), (worst.max(), c.left[worst.argmax()])


@pytest.mark.parametrize("T", [4, 40, 300, 1100])
@pytest.mark.parametrize("delta", [0.01, 0.1, -0.3])
def test_lse_is_only_a_scale(qoh, comps, T, delta):
    """Both calls recompute the same logits, so what differs is how G and the low-rank dX round (2^-11 each, in each call)
    and the sums; the exponentials are good to 2^-19 (argument of up to 2^5, an ulp of 2^-23 each)."""
    c = Sure(comps, T, 60 + T)
    head = qoh.PackedHead(*SHAPE, comps)
    a, b = (head.grad_hidden(*c.args(x), out_dtype=torch.float32).double().cpu().numpy() for x in (0.0, delta))
    rel = 4 * 2.0 ** -11 + SHAPE[0] / 8 * 2.0 ** -23 + 2.0 ** -17
    bound = rel * np.exp(2 * c.tau)[:, None] * c.terms + 2 * c.least + 2.0 ** -23 * np.abs(c.dh)
    worst = (np.abs(a - b) / bound).max(axis=1)
    assert np.all(worst <= 1), (worst.max(), c.left[worst.argmax()])
