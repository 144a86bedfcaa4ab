"""The feed-forward block example: the operators of a block in a row, each on
what the one before it wrote, served from a replayed graph and trained."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_util as B
from conftest import ROOT
from fp8_fp4_tensor_amd import fq
from test_gpu_mx_edges import check, reference, values

pytestmark = pytest.mark.gpu

E4, E5, E2 = fq.FQ_E4M3, fq.FQ_E5M2, fq.FQ_E2M1
# half a step of an element, relative to it
STEP = {E4: 2.0 ** -4, E5: 2.0 ** -3, E2: 2.0 ** -2}


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("feed_forward_block", os.path.join(ROOT, "examples", "feed_forward_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def product_is_right(p, what):
    """A product of the example against the 64-bit one of the planes it read."""
    d = p.desc
    shaped = lambda q, r: (q.data.view(torch.uint8).view(r, -1), q.scale.view(torch.uint8).view(r, -1))
    a, b = values(*shaped(p.a, d.m), p.a.fmt), values(*shaped(p.b, d.n), p.b.fmt)
    check(p.out, reference(a, b), d.k, p.a.fmt, p.b.fmt, p.out.dtype == torch.bfloat16, what)


def random(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


@pytest.mark.parametrize("tokens", [1, 3, 16, 65, 300])
@pytest.mark.parametrize("fmt", [E4, E5, E2], ids=["e4m3", "e5m2", "e2m1"])
def test_forward(ex, fmt, tokens):
    hidden, inner = 512, 1312
    weights = ex.random_weights(hidden, inner, 1)
    plan = ex.FeedForward(*weights, fmt).plan(tokens)
    x, res = random((tokens, hidden), 2), random((tokens, hidden), 3, 2.0)
    y, h = plan.forward(x, res)
    torch.cuda.synchronize()
    product_is_right(plan.up, "up")
    product_is_right(plan.down, "down")
    assert torch.equal(h, (x.float() + res.float()).to(torch.bfloat16))
    # Four quantized factors stand on a result's path, each with elements off by STEP at most (E2M1's values next to
    # zero by a quarter of the block's largest); errors of independent elements add in squares, the gate's slope is below 1.1 and its
    # curvature turns an error of the gate into at most twice of it
    want = ex.reference(weights, x.double(), res.double())[0]
    assert ex.relative(y, want) < 2 * np.sqrt(4) * STEP[fmt]


@pytest.mark.parametrize("batch", [1, 4, 40])
@pytest.mark.parametrize("fmt", [E4, E2], ids=["e4m3", "e2m1"])
def test_serving(ex, fmt, batch):
    """Replayed steps give what eager ones do, bit for bit."""
    ff = ex.FeedForward(*ex.random_weights(768, 1024, 2), fmt)
    steps = ex.serve(ff, batch, 5)
    plan = ff.plan(batch)
    for x, res, y in steps:
        eager, _ = plan.forward(x, res)
        torch.cuda.synchronize()
        assert torch.equal(eager, y)


@pytest.mark.parametrize("tokens,hidden,inner,fmt,grad_fmt", [(64, 256, 416, E4, E4), (416, 512, 1312, E4, E5),
                                                              (1024, 1024, 2816, E4, E4), (96, 384, 512, E2, E4)])
def test_training(ex, tokens, hidden, inner, fmt, grad_fmt):
    weights = ex.random_weights(hidden, inner, 3)
    ff = ex.FeedForward(*weights, fmt, grad_fmt)
    plan = ff.plan(tokens, training=True)
    x, res, dy, dh = (random((tokens, hidden), s) for s in (4, 5, 6, 7))
    y, h = plan.forward(x, res)
    dx = plan.backward(dy, dh)
    torch.cuda.synchronize()
    for name in ("up", "down", "d_act", "dw_out", "d_norm", "dw_in"):
        product_is_right(getattr(plan, name), name)
    # the norm's gradients from the tensors they were given
    d64 = lambda t: t.double().cpu().numpy()
    wx, ww, bx, bw = B.norm_gradients(d64(h), d64(plan.rstd), d64(weights[0]), d64(plan.d_norm.out), d64(dh))
    assert np.all(np.abs(d64(dx) - wx) <= bx + B.HALF_BF16 * (np.abs(wx) + bx))
    assert np.all(np.abs(d64(ff.grad_norm) - ww) <= bw + B.HALF_F32 * np.abs(ww))
    # and all of it from the formulas: eight quantized factors at most on a path (as in test_forward)
    leaves = [t.double().requires_grad_() for t in (x, *weights)]
    yr, hr = ex.reference(leaves[1:], leaves[0], res.double())
    (yr * dy.double() + hr * dh.double()).sum().backward()
    bound = 2 * np.sqrt(4 * STEP[fmt] ** 2 + 4 * max(STEP[fmt], STEP[grad_fmt]) ** 2)
    for name, got, want in (("y", y, yr.detach()), ("dx", dx, leaves[0].grad), ("norm", ff.grad_norm, leaves[1].grad),
                            ("in", ff.grad_in, leaves[2].grad), ("out", ff.grad_out, leaves[3].grad)):
        assert ex.relative(got, want) < bound, name


def test_gradients_against_differences(ex):
    """The loss of the formulas along a direction of x and of each weight, against the block's gradients: a symmetric
    difference of the 64-bit loss, which the 8-bit gradients meet as far as they meet the formulas'."""
    tokens, hidden, inner = 128, 256, 384
    weights = ex.random_weights(hidden, inner, 5)
    ff = ex.FeedForward(*weights)
    plan = ff.plan(tokens, training=True)
    x, res, dy, dh = (random((tokens, hidden), s) for s in (14, 15, 16, 17))
    plan.forward(x, res)
    dx = plan.backward(dy, dh)
    torch.cuda.synchronize()

    def loss(at):
        y, h = ex.reference(at[1:], at[0], res.double())
        return (y * dy.double() + h * dh.double()).sum().item()

    start = [t.double() for t in (x, *weights)]
    for i, grad in enumerate((dx, ff.grad_norm, ff.grad_in, ff.grad_out)):
        e = grad.double() / grad.double().norm()  # along the gradient itself: its length is the slope
        t = 1e-4
        ends = [loss(start[:i] + [start[i] + s * t * e] + start[i + 1:]) for s in (1, -1)]
        slope, norm = (ends[0] - ends[1]) / (2 * t), grad.double().norm().item()
        # <g, g'> / |g'| differs from |g'| by at most |g - g'|, bounded as in test_training by 2 sqrt(8) 2^-4 |g|
        assert abs(slope - norm) <= 2 * np.sqrt(8) * 2.0 ** -4 * max(norm, abs(slope)), i


def test_training_step_in_a_graph(ex):
    """A captured forward and backward pass, replayed: the same outputs, and the weights' gradients once more each."""
    tokens, hidden, inner = 224, 512, 1024
    ff = ex.FeedForward(*ex.random_weights(hidden, inner, 6))
    plan = ff.plan(tokens, training=True)
    x, res, dy, dh = (random((tokens, hidden), s) for s in (24, 25, 26, 27))
    grads = (ff.grad_norm, ff.grad_in, ff.grad_out)
    y, _ = plan.forward(x, res)
    dx = plan.backward(dy, dh)
    torch.cuda.synchronize()
    want, once = (y.clone(), dx.clone()), [g.clone() for g in grads]
    for g in grads:
        g.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, res)
        plan.backward(dy, dh)
    total = [torch.zeros_like(g) for g in grads]
    for _ in range(3):
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for s, o in zip(total, once):
            s += o
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        assert all(torch.equal(g, s) for g, s in zip(grads, total))


def test_example_runs(ex):
    ex.main()
