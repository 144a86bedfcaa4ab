"""A feed-forward block whose weights, activations and gradients are microscaled.

    h = x + residual;  n = rmsnorm(h) * w_norm;  [gate | up] = n W_in^T
    y = (silu(gate) * up) W_out^T

with both products on MX planes: the norm and the gated activation write the
planes that the next product reads, rowwise for it and colwise for the weight's
gradient, and nothing is quantized in a pass of its own but the gradient that
comes in. Serving: prompts, then token by token in a replayed HIP graph.
Training: the block's forward and backward pass. Buffers are allocated once;
every tensor operation is one of the library's entry points.

    python examples/feed_forward_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from fp8_fp4_tensor_amd import fq

ROW, BOTH = fq.FQ_ROWWISE, fq.FQ_ROWWISE | fq.FQ_COLWISE


def mx_planes(rows: int, cols: int, fmt: int, outputs: int, device) -> fq.Planes:
    d = fq.desc(fq.FQ_MX, fq.FQ_IN_BF16, fmt, rows, cols, (1, 32), outputs)
    return fq.Planes(d, fq.alloc_quantized(d, device))


class Product:
    """A product of two planes with its buffers."""

    def __init__(self, a: fq.MxPlane, b: fq.MxPlane, m: int, n: int, k: int, out: torch.Tensor, accumulate=False):
        self.desc = fq.gemm_mx_desc(m, n, k, a.fmt, b.fmt, fq.in_dtype_of(out), accumulate)
        self.a, self.b, self.out, self.ws = a, b, out, fq.alloc_gemm_mx_workspace(self.desc, out.device)

    def __call__(self) -> torch.Tensor:
        fq.fq_gemm_mx(self.desc, self.a, self.b, self.out, self.ws)
        return self.out


class FeedForward:
    """w_norm [H] fp32, w_in [2F, H] and w_out [H, F] bf16, the products' weights held in both directions."""

    def __init__(self, w_norm, w_in, w_out, fmt=fq.FQ_E4M3, grad_fmt=fq.FQ_E4M3, eps=1e-6):
        self.fmt, self.grad_fmt, self.eps, self.w_norm = fmt, grad_fmt, eps, w_norm
        self.hidden, self.inner, self.device = w_out.shape[0], w_out.shape[1], w_norm.device
        self.weights = []
        for w in (w_in, w_out):
            d = fq.desc(fq.FQ_MX, fq.in_dtype_of(w), fmt, *w.shape, (1, 32), BOTH)
            q = fq.alloc_quantized(d, self.device)
            fq.fq_quantize(d, w, q)
            self.weights.append(q)
        f32 = lambda *s: torch.zeros(s, device=self.device)
        self.grad_norm, self.grad_in, self.grad_out = f32(self.hidden), f32(*w_in.shape), f32(*w_out.shape)

    def plan(self, tokens: int, training: bool = False):
        """Buffers of a pass over this many tokens (with training a multiple of 32)."""
        return Plan(self, tokens, training)


class Plan:
    def __init__(self, ff: FeedForward, tokens: int, training: bool):
        dev, H, F, T = ff.device, ff.hidden, ff.inner, tokens
        row, col = fq.MxPlane.rowwise, fq.MxPlane.colwise
        w_in, w_out = ff.weights
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)
        self.ff, self.training = ff, training
        self.norm = fq.rmsnorm_desc(T, H, eps=ff.eps)
        self.act = fq.swiglu_desc(T, F)
        self.h, self.rstd = bf(T, H), torch.empty(T, device=dev) if training else None
        outputs = BOTH if training else ROW
        self.n, self.a = mx_planes(T, H, ff.fmt, outputs, dev), mx_planes(T, F, ff.fmt, outputs, dev)
        self.up = Product(row(self.n.out, ff.fmt), row(w_in, ff.fmt), T, 2 * F, H, bf(T, 2 * F))
        self.down = Product(row(self.a.out, ff.fmt), row(w_out, ff.fmt), T, H, F, bf(T, H))
        if not training:
            return
        g = ff.grad_fmt
        self.dy, self.dx = mx_planes(T, H, g, BOTH, dev), mx_planes(T, 2 * F, g, BOTH, dev)
        self.dy_desc = fq.desc(fq.FQ_MX, fq.FQ_IN_BF16, g, T, H, (1, 32), BOTH)
        self.d_act = Product(row(self.dy.out, g), col(w_out, ff.fmt), T, F, H, bf(T, F))
        self.dw_out = Product(col(self.dy.out, g), col(self.a.out, ff.fmt), H, F, T, ff.grad_out, True)
        self.d_norm = Product(row(self.dx.out, g), col(w_in, ff.fmt), T, H, 2 * F, bf(T, H))
        self.dw_in = Product(col(self.dx.out, g), col(self.n.out, ff.fmt), 2 * F, H, T, ff.grad_in, True)
        self.norm_back = fq.rmsnorm_desc(T, H, eps=ff.eps, accumulate=True)
        self.ws, self.dh = fq.alloc_rmsnorm_workspace(self.norm_back, dev), bf(T, H)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(y, h), both [tokens, H] bf16 and written again by the next pass; h is the next residual."""
        fq.fq_rmsnorm(self.norm, x, self.ff.w_norm, residual, self.h, self.rstd, planes=self.n)
        fq.fq_swiglu(self.act, self.up(), planes=self.a)
        return self.down(), self.h

    def backward(self, dy: torch.Tensor, dh: torch.Tensor) -> torch.Tensor:
        """The gradient of x and of the residual alike, from those of y and of h; the weights' are added to the block's."""
        fq.fq_quantize(self.dy_desc, dy, self.dy.out)
        self.dw_out()
        fq.fq_swiglu_backward(self.act, self.up.out, self.d_act(), planes=self.dx)
        self.dw_in()
        fq.fq_rmsnorm_backward(self.norm_back, self.h, self.rstd, self.ff.w_norm, self.d_norm(), self.dh,
                               self.ff.grad_norm, dh, self.ws)
        return self.dh


def random_weights(hidden: int, inner: int, seed: int = 0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=device)
    return (1 + 0.2 * rn(hidden), (rn(2 * inner, hidden) * hidden ** -0.5).to(torch.bfloat16),
            (rn(hidden, inner) * inner ** -0.5).to(torch.bfloat16))


def reference(weights, x, residual, eps=1e-6, dtype=torch.float64):
    """(y, h) of the formulas, differentiable."""
    w_norm, w_in, w_out = (w.to(dtype) for w in weights)
    h = x + residual
    gate, up = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * w_norm @ w_in.t()).chunk(2, 1)
    return (torch.nn.functional.silu(gate) * up) @ w_out.t(), h


def serve(ff: FeedForward, batch: int, tokens: int, seed: int = 7):
    """`tokens` steps of `batch` rows in a replayed graph: (inputs, residuals, outputs)."""
    g = torch.Generator(device=ff.device)
    g.manual_seed(seed)
    rows = lambda: torch.randn((batch, ff.hidden), generator=g, device=ff.device).to(torch.bfloat16)
    plan, x, residual = ff.plan(batch), rows(), rows()
    plan.forward(x, residual)  # once outside the graph: the library's first launches
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = plan.forward(x, residual)
    steps = []
    for _ in range(tokens):
        x.copy_(rows())
        residual.copy_(rows())
        graph.replay()
        steps.append((x.clone(), residual.clone(), y.clone()))
    return steps


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def main():
    torch.cuda.set_device(0)
    hidden, inner, tokens = 1024, 2816, 512
    weights = random_weights(hidden, inner)
    for name, fmt in (("8-bit", fq.FQ_E4M3), ("4-bit", fq.FQ_E2M1)):
        steps = serve(FeedForward(*weights, fmt), 4, 6)
        got = torch.cat([y for _, _, y in steps])
        want = reference(weights, *(torch.cat([s[i] for s in steps]).double() for i in (0, 1)))[0]
        print(f"{name}, tokens of 4 sequences: relative difference from float64 {relative(got, want):.4f}")
    ff = FeedForward(*weights)
    x, res, dy, dh = (torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16) for _ in range(4))
    plan = ff.plan(tokens, training=True)
    y, h = plan.forward(x, res)
    dx = plan.backward(dy, dh)
    leaves = [t.double().requires_grad_() for t in (x, *weights)]
    yr, hr = reference(leaves[1:], leaves[0], res.double())
    (yr * dy + hr * dh).sum().backward()
    print(f"8-bit training: y {relative(y, yr.detach()):.4f}, dx {relative(dx, leaves[0].grad):.4f}, " + ", ".join(
        f"{n} {relative(a, b.grad):.4f}" for n, a, b in (("dw_norm", ff.grad_norm, leaves[1]), ("dW_in", ff.grad_in, leaves[2]),
                                                        ("dW_out", ff.grad_out, leaves[3]))))


if __name__ == "__main__":
    main()
