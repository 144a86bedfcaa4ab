"""The attention block example: prompts, replayed single-token steps and the
gradients of a linear layer, against the same block in float32."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Each of the two products has two 8-bit factors, each element off by at most
# 2^-4 of itself; over a sum of independent terms the relative error of a
# result stays below sqrt(2) * 2^-4 (mean square of both factors), and the
# cached keys and values add one factor each.
BOUND = 2.0 * 2.0 ** -4


@pytest.mark.parametrize("hidden,q_heads,kv_heads,dim,prompts", [
    (512, 8, 2, 64, [70, 1, 33]), (1024, 8, 8, 128, [200]), (512, 4, 1, 256, [65, 64])])
def test_serving(ex, hidden, q_heads, kv_heads, dim, prompts):
    block = ex.AttentionBlock(hidden, q_heads, kv_heads, dim, pages=16, seed=3)
    inputs, outputs = ex.serve(block, prompts, 6, hidden)
    torch.cuda.synchronize()
    want = ex.reference(block, prompts, inputs)
    for t, (a, b) in enumerate(zip(outputs, want)):
        assert ex.relative(a, b) < BOUND, t


def test_training_products(ex):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = (torch.randn((384, 512), generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16)
    layer = ex.Linear8(w)
    x, dy = (torch.randn((256, n), generator=g, device="cuda").to(torch.bfloat16) for n in (512, 384))
    y, dx = ex.Linear8.forward(layer.plan(256), x), layer.backward(x, dy)
    layer.backward(x, dy)  # the weight's gradient accumulates
    torch.cuda.synchronize()
    assert ex.relative(y, x.float() @ w.float().t()) < BOUND
    assert ex.relative(dx, dy.float() @ w.float()) < BOUND
    assert ex.relative(layer.grad, 2 * dy.float().t() @ x.float()) < BOUND
