"""An attention block that keeps its weights, activations and cache in 8 bits.

Serving: the joint projection of queries, keys and values, the append of the
new keys and values to the paged cache, attention over the cache and the
output projection, for a batch of ragged prompts and then token by token in a
replayed HIP graph. Training: the three products of a linear layer. Every
tensor operation but the norm between blocks (left to the caller) is one of
the library's entry points; buffers are allocated once.

    python examples/attention_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from fp8_fp4_tensor_amd import fq

BOTH = fq.FQ_ROWWISE | fq.FQ_COLWISE


def quantize(x: torch.Tensor, block, outputs=fq.FQ_ROWWISE) -> fq.Quantized:
    d = fq.desc(fq.FQ_BLOCK_FP32, fq.in_dtype_of(x), fq.FQ_E4M3, *x.shape, block, outputs)
    q = fq.alloc_quantized(d, x.device)
    fq.fq_quantize(d, x, q)
    return q


class Linear8:
    """y = x W^T with W [out, in] held in 128x128 blocks, both ways round."""

    def __init__(self, weight: torch.Tensor):
        self.out_features, self.in_features = weight.shape
        self.weight = quantize(weight, (128, 128), BOTH)
        self.grad = torch.zeros(weight.shape, dtype=torch.float32, device=weight.device)

    def plan(self, tokens: int, device="cuda"):
        """Buffers of a forward pass over this many tokens."""
        x = fq.desc(fq.FQ_BLOCK_FP32, fq.FQ_IN_BF16, fq.FQ_E4M3, tokens, self.in_features, (1, 128))
        xq = fq.alloc_quantized(x, device)
        d = fq.gemm_desc(tokens, self.out_features, self.in_features)
        y = torch.empty((tokens, self.out_features), dtype=torch.bfloat16, device=device)
        return x, xq, d, fq.Plane.rowwise(xq), fq.Plane.rowwise(self.weight), y, fq.alloc_gemm_workspace(d, device)

    @staticmethod
    def forward(plan, x: torch.Tensor) -> torch.Tensor:
        desc, xq, d, a, b, y, ws = plan
        fq.fq_quantize(desc, x, xq)
        fq.fq_gemm(d, a, b, y, ws)
        return y

    def backward(self, x: torch.Tensor, dy: torch.Tensor) -> torch.Tensor:
        """dx, and the weight's gradient added to self.grad (tokens a multiple of 128)."""
        tokens = x.shape[0]
        g, xq = quantize(dy, (1, 128), BOTH), quantize(x, (1, 128), fq.FQ_COLWISE)
        d = fq.gemm_desc(tokens, self.in_features, self.out_features)
        dx = torch.empty_like(x)
        fq.fq_gemm(d, fq.Plane.rowwise(g), fq.Plane.colwise(self.weight), dx, fq.alloc_gemm_workspace(d, x.device))
        d = fq.gemm_desc(self.out_features, self.in_features, tokens, b_block_rows=1, out_dtype=fq.FQ_IN_F32,
                         accumulate=True)
        fq.fq_gemm(d, fq.Plane.colwise(g), fq.Plane.colwise(xq), self.grad, fq.alloc_gemm_workspace(d, x.device))
        return dx


class AttentionBlock:
    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, pages: int, page_tokens: int = 64,
                 seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(o, i):
            return (torch.randn((o, i), generator=g, device=device) * i ** -0.5).to(torch.bfloat16)

        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight(hidden, q_heads * head_dim)
        self.qkv, self.out = Linear8(self.w_qkv), Linear8(self.w_out)
        self.cache = fq.alloc_kv_cache(fq.FQ_E4M3, pages, kv_heads, head_dim, page_tokens, page_tokens, device)

    def plan(self, batch: fq.KvBatch, device="cuda"):
        """Buffers of a pass over this batch."""
        n = batch.total_q
        d = fq.attention_desc(self.q_heads)
        att = torch.empty((n, self.q_heads, self.head_dim), dtype=torch.bfloat16, device=device)
        return self.qkv.plan(n, device), self.out.plan(n, device), d, att, fq.alloc_attention_workspace(
            self.cache, batch, d, device)

    def forward(self, plan, batch: fq.KvBatch, x: torch.Tensor) -> torch.Tensor:
        """x [total_q, hidden] bf16 -> [total_q, hidden] bf16; the batch's lengths count the new tokens."""
        p_qkv, p_out, d, att, ws = plan
        n, hq, hk, dim = batch.total_q, self.q_heads, self.kv_heads, self.head_dim
        qkv = Linear8.forward(p_qkv, x)
        q, k, v = qkv.split([hq * dim, hk * dim, hk * dim], 1)
        fq.fq_kv_append(self.cache, batch, k.view(n, hk, dim), v.view(n, hk, dim))
        fq.fq_attention(self.cache, batch, d, q.view(n, hq, dim), att, None, ws)
        return Linear8.forward(p_out, att.view(n, hq * dim))


def serve(block: AttentionBlock, prompts, tokens: int, hidden: int, page_tokens: int = 64, device="cuda"):
    """Prompts of the given lengths, then `tokens` tokens of each sequence in a
    replayed graph. Returns (inputs, outputs), each [prompt rows, then steps of batch rows]."""
    batch, most = len(prompts), max(prompts) + tokens
    per = -(-most // page_tokens)
    table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per).flip(0).contiguous()
    lens = torch.tensor(prompts, dtype=torch.int32, device=device)
    starts = torch.tensor([sum(prompts[:i]) for i in range(batch + 1)], dtype=torch.int32, device=device)
    g = torch.Generator(device=device)
    g.manual_seed(7)

    def rows(n):
        return torch.randn((n, hidden), generator=g, device=device).to(torch.bfloat16)

    first = fq.KvBatch(table, lens, starts, sum(prompts), max(prompts), max(prompts))
    x = rows(sum(prompts))
    inputs, outputs = [x], [block.forward(block.plan(first, device), first, x).clone()]
    each = fq.KvBatch(table, lens, None, batch, 1, most)  # lens is updated in place: the graph reads it
    plan, x = block.plan(each, device), torch.empty((batch, hidden), dtype=torch.bfloat16, device=device)
    graph, y = None, None
    for _ in range(tokens):
        lens += 1
        x.copy_(rows(batch))
        inputs.append(x.clone())
        if graph is None:
            y = block.forward(plan, each, x)  # once outside the graph: the library's first launches
            outputs.append(y.clone())
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = block.forward(plan, each, x)
            continue
        graph.replay()
        outputs.append(y.clone())
    return inputs, outputs


def reference(block: AttentionBlock, prompts, inputs):
    """The same block in float32, without 8-bit data."""
    hq, hk, dim = block.q_heads, block.kv_heads, block.head_dim
    batch = len(prompts)
    at = [sum(prompts[:i]) for i in range(batch)]
    outs = [torch.empty_like(x, dtype=torch.float32) for x in inputs]
    for i in range(batch):
        mine = [inputs[0][at[i]:at[i] + prompts[i]]] + [x[i:i + 1] for x in inputs[1:]]
        x = torch.cat(mine).float()
        q, k, v = (x @ block.w_qkv.float().t()).split([hq * dim, hk * dim, hk * dim], 1)
        n = x.shape[0]
        q, k, v = (t.view(n, h, dim).transpose(0, 1) for t, h in ((q, hq), (k, hk), (v, hk)))
        k, v = (t.repeat_interleave(hq // hk, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2).contiguous()) * dim ** -0.5
        s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool, device=x.device), 1), float("-inf"))
        o = (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, hq * dim) @ block.w_out.float().t()
        outs[0][at[i]:at[i] + prompts[i]] = o[:prompts[i]]
        for t in range(1, len(inputs)):
            outs[t][i] = o[prompts[i] + t - 1]
    return outs


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def main():
    torch.cuda.set_device(0)
    hidden, q_heads, kv_heads, dim = 1024, 16, 4, 64
    prompts, tokens = [300, 17, 129], 12
    block = AttentionBlock(hidden, q_heads, kv_heads, dim, pages=20)
    inputs, outputs = serve(block, prompts, tokens, hidden)
    want = reference(block, prompts, inputs)
    print(f"prompts of {prompts}: relative difference from float32 {relative(outputs[0], want[0]):.4f}")
    print(f"{tokens} tokens each: {relative(torch.cat(outputs[1:]), torch.cat(want[1:])):.4f}")
    layer = Linear8(block.w_out)
    x, dy = (torch.randn((512, n), device="cuda").to(torch.bfloat16) for n in (layer.in_features, layer.out_features))
    y = Linear8.forward(layer.plan(512), x)
    dx = layer.backward(x, dy)
    w = block.w_out.float()
    print(f"linear layer: y {relative(y, x.float() @ w.t()):.4f}, dx {relative(dx, dy.float() @ w):.4f}, "
          f"dW {relative(layer.grad, dy.float().t() @ x.float()):.4f}")


if __name__ == "__main__":
    main()
