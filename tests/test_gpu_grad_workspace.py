"""The workspace of the gradient: the size asked for a token count is enough for it and no less is; it does not grow with
the count throughout, so one workspace for several counts takes the largest of their sizes."""
import pytest
import torch

import archead_inputs as gen

pytestmark = pytest.mark.gpu
SHAPE = (33000, 192, 64, 16, 64, 192)
COUNTS = [1, 2, 8, 9, 64, 128, 129, 300, 1023, 1024, 1100]


def test_workspace_sizes_of_several_counts():
    import quantized_output_head_b200 as qoh
    head = qoh.PackedHead(*SHAPE, gen.random_components(gen.HeadShape(*SHAPE), 3))
    sizes = [head.grad_workspace_bytes(T) for T in COUNTS]
    assert sizes != sorted(sizes)
    rnd = torch.Generator(device="cuda").manual_seed(4)
    shared = torch.full((max(sizes),), 255, dtype=torch.uint8, device="cuda")
    for T, size in zip(COUNTS, sizes):
        h = torch.randn(T, SHAPE[1], generator=rnd, device="cuda").bfloat16()
        t = torch.randint(0, SHAPE[0], (T,), generator=rnd, device="cuda", dtype=torch.int32)
        lse, _, _ = head.lse_argmax(h, t)
        g = torch.randn(T, generator=rnd, device="cuda")
        want = head.grad_hidden(h, t, lse, g)
        exact = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(head.grad_hidden(h, t, lse, g, workspace=exact[:size]), want)
        assert bool((exact[size:] == 255).all())   # nothing behind it is touched
        assert torch.equal(head.grad_hidden(h, t, lse, g, workspace=shared), want)
        assert head.status(shared) == 0
        with pytest.raises(qoh.ArcheadError):
            head.grad_hidden(h, t, lse, g, workspace=exact[:size - 256])
