"""The step that README shows, from a model's hidden states to the gradients of its weights: the head's calls return plain
tensors, and hidden.backward(grad) takes them on into the model."""
import pytest
import torch

import archead_inputs as gen

pytestmark = pytest.mark.gpu
SHAPE = (1000, 256, 32, 8, 64, 64)


@pytest.mark.parametrize("T", [6, 50])
def test_gradients_reach_the_model_below(T):
    import quantized_output_head_b200 as qoh
    head = qoh.PackedHead(*SHAPE, gen.random_components(gen.HeadShape(*SHAPE), 1))
    rnd = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, 64, generator=rnd, device="cuda").bfloat16()
    w = torch.randn(256, 64, generator=rnd, device="cuda").bfloat16().requires_grad_(True)
    tokens = torch.randint(0, 1000, (T,), generator=rnd, device="cuda")
    cu = torch.tensor([0, 2, T], device="cuda", dtype=torch.int32)
    hidden = x @ w.T
    lse, _, ce = head.lse_argmax(hidden, tokens)
    adv = torch.tensor([1.0, -0.5], device="cuda")
    loss, g, stats = qoh.policy_loss(ce, ce + 0.02, adv, cu, ce_ref=ce * 1.01, kl_coef=0.04, advantage_per="sequence")
    grad = head.grad_hidden(hidden, tokens, lse, g)
    hidden.backward(grad)
    assert bool(torch.isfinite(loss)) and stats.shape == (3,)
    # the weights' gradient of the product below, in 64 bits; bf16 result of an fp32 sum over T tokens
    want = grad.double().T @ x.double()
    bound = 2.0 ** -8 * want.abs() + T * 2.0 ** -23 * (grad.double().abs().T @ x.double().abs()) + 1e-30
    assert bool(((w.grad.double() - want).abs() <= bound).all())
    loss, g, rewards = qoh.preference_loss(ce, torch.tensor([0, 2, T], device="cuda", dtype=torch.int32), beta=0.1)
    assert rewards.shape == (2, 1) and bool(torch.isfinite(head.grad_hidden(hidden, tokens, lse, g)).all())
