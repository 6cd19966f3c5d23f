"""Hidden states, or column ranges of them, so small that the power of two that brings them to fp16 range is no float."""
import math

import numpy as np
import pytest
import torch

import archead_inputs as gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qoh():
    import quantized_output_head_b200 as m
    return m


@pytest.mark.parametrize("g_B", [64, 32])
@pytest.mark.parametrize("T", [4, 40, 300, 1100])
@pytest.mark.parametrize("e", [-112, -116, -124, -130])
def test_tiny_tokens_are_uniform(qoh, e, T, g_B):
    """Logits below 2^-80: every row has probability 1 / V, to 2^-21 (lse is rounded to fp32 at 7.6)."""
    shape = (2000, 256, 32, 8, 64, g_B)
    head = qoh.PackedHead(*shape, gen.random_components(gen.HeadShape(*shape), 1))
    rnd = torch.Generator(device="cuda").manual_seed(T)
    h = (torch.randn(T, 256, generator=rnd, device="cuda", dtype=torch.float64) * 2.0 ** e).bfloat16()
    h[:, ::3] = 0
    zero = torch.zeros_like(h)
    targets = torch.randint(0, 2000, (T,), generator=rnd, device="cuda", dtype=torch.int32)
    lse, _, ce = head.lse_argmax(h, targets)
    for x in (lse, ce):
        assert float((x.double() - math.log(2000)).abs().max()) <= 2.0 ** -21
    logits, _ = head.logits(h[:4].contiguous())
    assert float(logits.abs().max()) < 2.0 ** -80
    got, want = (head.grad_hidden(x, targets, lse, torch.ones(T, device="cuda"), out_dtype=torch.float32) for x in (h, zero))
    assert torch.allclose(got, want, rtol=2.0 ** -20, atol=float(want.abs().max()) * 2.0 ** -20)


@pytest.mark.parametrize("T", [1, 4, 8, 9, 40, 300])
@pytest.mark.parametrize("first,last", [(0, 256), (256, 512), (448, 512), (64, 1024)])
def test_a_range_of_tiny_columns_counts_as_zero(qoh, T, first, last):
    shape = (1500, 1024, 64, 16, 128, 64)
    head = qoh.PackedHead(*shape, gen.random_components(gen.HeadShape(*shape), 2))
    rnd = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn(T, 1024, generator=rnd, device="cuda", dtype=torch.float64)
    h[:, first:last] *= 2.0 ** -125
    h = h.bfloat16()
    h[:, first:last:5] = 0
    without = h.clone()
    without[:, first:last] = 0
    targets = torch.arange(T, device="cuda", dtype=torch.int32)
    a, b = (head.lse_argmax(x, targets) for x in (h, without))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    ga, gb = (head.grad_hidden(x, targets, a[0], torch.ones(T, device="cuda")) for x in (h, without))
    assert torch.equal(ga, gb)
