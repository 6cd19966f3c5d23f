"""Hidden states are bf16: a tensor of another type is refused, its bits are not read as bf16.  No GPU."""
import pytest
import torch

import quantized_output_head_b200 as qoh

HEAD = qoh.PackedHead.__new__(qoh.PackedHead)   # (the checks come before the handle is used)
HEAD.d = HEAD.V = 64
CALLS = {
    "logits": lambda h: HEAD.logits(h),
    "lse_argmax": lambda h: HEAD.lse_argmax(h),
    "sample": lambda h: HEAD.sample(h, 1.0, 0),
    "sample_partials": lambda h: HEAD.sample_partials(h, 1.0, 0),
    "shard_partials": lambda h: HEAD.shard_partials(h),
    "grad_hidden": lambda h: HEAD.grad_hidden(h, torch.zeros(2, dtype=torch.int32), torch.zeros(2), torch.zeros(2)),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.float64, torch.int32, torch.int8])
def test_other_types_are_refused(name, dtype):
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        CALLS[name](torch.zeros(2, 64, dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int16, torch.uint16])
def test_bf16_and_its_bits_pass(dtype):
    with pytest.raises(ValueError, match="on the CUDA device"):   # (the next check)
        qoh._check_hidden(torch.zeros(2, 64, dtype=dtype), 64)
