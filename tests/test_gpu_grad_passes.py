"""The gradient where a call takes several passes over the head, and on vocabulary shards at every kernel path."""
import numpy as np
import pytest
import torch

import archead_inputs as gen
from test_gpu_grad import Case

pytestmark = pytest.mark.gpu
# 16-bit rows of more than 320 MB: calls of 129 to 256 tokens take the few-token kernels twice
LARGE = (41001, 4096, 40, 8, 128, 128)


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


@pytest.fixture(scope="module")
def large(qoh):
    return qoh.PackedHead(*LARGE, gen.random_components(gen.HeadShape(*LARGE), 11))


@pytest.mark.parametrize("T", [129, 200, 255, 256])
def test_two_passes_of_the_few_token_kernels(qoh, large, T):
    """The bits of two calls of half the tokens each; a bad target in the second pass is reported and spoils its row alone."""
    V, d = LARGE[:2]
    rnd = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn(T, d, generator=rnd, device="cuda").bfloat16()
    targets = torch.randint(0, V, (T,), generator=rnd, device="cuda", dtype=torch.int32)
    g = torch.randn(T, generator=rnd, device="cuda")
    g[::7] = 0.0
    g[-2] = 1.0
    lse, _, _ = large.lse_argmax(h, targets)
    first = (T + 1) // 2
    halves = [large.grad_hidden(h[a:b], targets[a:b], lse[a:b], g[a:b]) for a, b in ((0, first), (first, T))]
    want = torch.cat(halves)
    assert large.grad_workspace_bytes(T) == large.grad_workspace_bytes(first)   # (it is two passes)
    ws = torch.full((large.grad_workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")
    got = large.grad_hidden(h, targets, lse, g, workspace=ws)
    assert torch.equal(got, want) and not got[::7].any() and large.status(ws) == 0
    targets[-2] = V
    got = large.grad_hidden(h, targets, lse, g, workspace=ws)
    assert torch.isnan(got[-2]).all() and torch.equal(got[:-2], want[:-2]) and torch.equal(got[-1], want[-1])
    assert large.status(ws) == qoh.STATUS_BAD_TARGET


def test_two_passes_against_fp64(large):
    """Each row's relative error in the 2-norm: independent fp16 roundings (at most 4 * 2^-11, each) and half a bf16 step."""
    V, d, r_c, r_r, g_s, g_B = LARGE
    comps = gen.random_components(gen.HeadShape(*LARGE), 11)

    def real(codes, scales, group=None):
        x = torch.from_numpy(codes).cuda().double()
        s = torch.from_numpy(scales.view(np.float16)).cuda().double()
        return x * (s[:, None] if group is None else s.repeat_interleave(group, 1))

    W = (real(comps["q"], comps["s_res"], g_s) + real(comps["L"], comps["s_L"]) @ real(comps["R"], comps["s_R"])
         + real(comps["A"], comps["s_A"]) @ real(comps["B"], comps["s_B"], g_B))
    T = 200
    rnd = torch.Generator(device="cuda").manual_seed(12)
    h = torch.randn(T, d, generator=rnd, device="cuda").bfloat16()
    targets = torch.randint(0, V, (T,), generator=rnd, device="cuda", dtype=torch.int32)
    g = torch.randn(T, generator=rnd, device="cuda")
    y = h.double() @ W.T
    lse = torch.logsumexp(y, 1)
    G = torch.exp(y - lse[:, None])
    G[torch.arange(T, device="cuda"), targets.long()] -= 1
    want = g.double()[:, None] * (G @ W)
    got = large.grad_hidden(h, targets, lse.float(), g).double()
    rel = (got - want).norm(dim=1) / want.norm(dim=1)
    assert float(rel.max()) <= 2.0 ** -8 + 4 * 2.0 ** -11, float(rel.max())


@pytest.mark.parametrize("shape", [(3000, 256, 64, 16, 64, 64), (3000, 320, 0, 20, 64, 10), (3000, 192, 70, 0, 16, 192)])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 40, 130, 300, 1100])
def test_shards_add_up_on_every_path(qoh, shape, T):
    c = Case(qoh, shape, T, seed=300 + T)
    total = torch.zeros(T, shape[1], device="cuda")
    for v0, v1 in ((0, 1008), (1008, 1024), (1024, 2992), (2992, 3000)):
        shard = qoh.PackedHead(v1 - v0, *shape[1:], qoh.shard_components(c.comps, v0, v1))
        shard.set_vocab_shard(v0, shape[0])
        ws = torch.full((shard.grad_workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")
        total += shard.grad_hidden(*c.args, out_dtype=torch.float32, workspace=ws)
        assert shard.status(ws) == 0
    c.check(total, 6 * 2.0 ** -24)
