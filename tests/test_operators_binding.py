"""What the binding of the operators on 8-bit data refuses before the library
sees it, on the host (no GPU): the tensors are on the CPU, so no call here may
reach a launch."""
import pytest
import torch

from fp8_fp4_tensor_amd import fq


class Stream:
    cuda_stream = 0


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def cache(heads=2, dim=64, page=32, block=16, pages=2, fmt=fq.FQ_E4M3, dtype=torch.uint8):
    return fq.KvCache(fmt, block, z(pages, heads, page, dim, dtype=dtype), z(pages, heads, dim, page, dtype=dtype),
                      z(pages, heads, page // block), z(pages, heads, page // block))


def batch(rows, **kw):
    v = dict(page_table=z(rows, 2, dtype=torch.int32), seq_lens=z(rows, dtype=torch.int32), q_start=None,
             total_q=rows, max_q=1)
    v.update(kw)
    return fq.KvBatch(**v)


@pytest.mark.parametrize("rows", [2, 5])
def test_tokens_that_overlap_are_refused(rows):
    """A token stride below a token's own length, 0 among them: the library takes a stride of 0 for contiguous
    queries and would read rows behind the tensor's only one."""
    c, b, d = cache(), batch(rows), fq.attention_desc(4)
    out = z(rows, 4, 64, dtype=torch.bfloat16)
    one = z(1, 4, 64, dtype=torch.bfloat16)
    half = z(rows * 256, dtype=torch.bfloat16).as_strided((rows, 4, 64), (128, 64, 1))
    for q in (one.expand(rows, 4, 64), half):
        with pytest.raises(ValueError):
            fq.fq_attention(c, b, d, q, out, None, None, Stream)
        new = q[:, :2]
        with pytest.raises(ValueError):
            fq.fq_kv_append(c, b, new.expand(rows, 2, 64) if q.stride(0) == 0 else new.as_strided((rows, 2, 64), (64, 64, 1)),
                            z(rows, 2, 64, dtype=torch.bfloat16), Stream)
