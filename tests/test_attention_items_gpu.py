"""Batches in which a CTA goes through many short items: what its warps hand
one another must belong to the item at hand."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import DEV, Cache, check_attention, fill_normal, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,kv,n", [(128, 4, 100), (256, 4, 100), (256, 4, 128), (128, 2, 250), (256, 2, 250), (256, 1, 31)])
def test_short_prompts_with_queries_of_different_size(D, kv, n):
    """Items of one and two blocks of keys; queries grow and shrink by powers of
    two from item to item, the keys the other way."""
    seqs = [(n, n - i % 3) for i in range(150)]
    c = Cache(seqs, kv, D, 16, seed=n + D)
    fill_normal(c, 5)
    q = torch.randn(c.tokens, 2 * kv, D, generator=gen(3), device=DEV)
    size = torch.tensor([2.0 ** ((i * 7) % 13 - 10) for i in range(150)], device=DEV)
    q = (q * size.repeat_interleave(n)[:, None, None]).to(torch.bfloat16)
    for _ in range(5):
        out = ops.fp8_kv_attention(q, *c.args())
        assert ops.get_status() == 0
    check_attention(c, q, None, out, D ** -0.5, only=set(range(0, 150, 10)) | {149})


@pytest.mark.parametrize("single", [False, True])
@pytest.mark.parametrize("seqs", [[(64, 900)] + [(0, 70)] * 63, [(1, 900), (1, 0), (1, 129)], [(1, 300)], [(3, 130), (0, 5), (40, 700), (1, 64)]])
@pytest.mark.parametrize("D,heads", [(128, 4), (256, 12), (256, 40)])
def test_one_token_expected_or_not(D, heads, seqs, single):
    """A promise of single tokens changes which kernel runs, not what is right."""
    c = Cache(seqs, 2, D, 32, seed=heads)
    fill_normal(c, 4)
    q, gate = (torch.randn(c.tokens, heads, D, generator=gen(i), device=DEV).to(torch.bfloat16) for i in (1, 2))
    out = ops.fp8_kv_attention(q, *c.args(), gate=gate, single_tokens=single)
    assert ops.get_status() == 0
    check_attention(c, q, gate, out, D ** -0.5)
