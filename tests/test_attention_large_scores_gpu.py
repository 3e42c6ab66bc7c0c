"""Scores so large that the steps of fp32 are wider than the room above the
softmax's reference: results stay finite and weights still sum to one."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import DEV, Cache, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("size", [22, 23, 24, 25])
def test_scores_of_millions(D, new, size):
    """All values are 1, so a result is sum p' / sum p whatever the scores are:
    within 2^-7 of 1 (a probability's 8 bits, 2^-8 and a little, and the
    result's rounding).  Scores from 2^size on (log2 units) in small steps of
    their scale; blocks of keys differ by a few units, so that some lie just
    above the reference of the blocks before."""
    blocks, k = 1480, 64.0
    c = Cache([(new, 128 * blocks)], 1, D, 64, seed=D, k_scale=1.0, v_scale=1.0)
    keys = torch.full((128 * blocks, 1, D), k, device=DEV)
    keys[:, 0, D - 1] = torch.randint(0, 4, (blocks,), generator=gen(5), device=DEV).repeat_interleave(128) * 2.0
    c.fill(0, keys, torch.ones_like(keys))
    q = torch.full((new, 3, D), 240.0, device=DEV)
    q[:, :, D - 1] = 1.0
    q = q.to(torch.bfloat16)
    raw = 240 * k * (D - 1)
    for i in range(48):
        scale = 2.0 ** (size + i / 48) / raw
        out = ops.fp8_kv_attention(q, *c.args(), softmax_scale=scale / 1.4426950408889634).float()
        assert torch.isfinite(out).all() and float((out - 1).abs().max()) <= 2.0 ** -7, (i, float(out.min()), float(out.max()))
    assert ops.get_status() == 0
