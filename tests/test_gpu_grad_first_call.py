"""The first gradient of a process sets its kernels up, also where that call is being captured."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
import archead_inputs as gen
import quantized_output_head_b200 as qoh
T, g_B = {T}, {g_B}
shape = (1000, 256, 32, 8, 64, g_B)
head = qoh.PackedHead(*shape, gen.random_components(gen.HeadShape(*shape), 1))
rnd = torch.Generator(device="cuda").manual_seed(2)
h = torch.randn(T, 256, generator=rnd, device="cuda").bfloat16()
t = torch.randint(0, 1000, (T,), generator=rnd, device="cuda", dtype=torch.int32)
lse, _, _ = head.lse_argmax(h, t)
g = torch.randn(T, generator=rnd, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = head.grad_hidden(h, t, lse, g)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, head.grad_hidden(h, t, lse, g))
print("same")
"""


@pytest.mark.parametrize("T,g_B", [(5, 64), (40, 64), (300, 64), (40, 32)])
def test_first_call_in_a_capture(T, g_B):
    run = subprocess.run([sys.executable, "-c", PROGRAM.format(T=T, g_B=g_B)], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]
