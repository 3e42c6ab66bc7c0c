"""The sign of the tile kernel's errors: the roundings of single probabilities
point both ways, so results of many keys must not drift to one side."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import DEV, Cache, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("std", [0.3, 1.0])
def test_probabilities_have_no_bias(D, std):
    """Every key holds the same value, so a result is that value times sum p' /
    sum p, p' the rounded probabilities.  256 value scales over an octave and 8
    significands average the result's own rounding.

    Bound on the mean relative error: to nearest even, the two roundings of a
    probability have errors of at most 2^-11 and 2^-8 of it with mean 0 over an
    octave (the rests are spread evenly, and the ties split evenly); 8000 keys
    that count and 120 rows leave less than 2^-8 / (8000 * 120) ** 0.5 = 4e-6
    of their spread.  The results' rounding: 2048 values spread evenly over an
    octave, at most 2^-8 apart from one tie to the next, leave less than 2^-8 /
    2048 ** 0.5 = 9e-5 even if they were random; here they are a grid, whose
    mean is 1.4e-6.  1e-4 holds both; ties rounded up instead shift the mean
    by 2.8e-4."""
    n, T, steps = 24000, 30, 256
    c = Cache([(T, n)], 1, D, 64, seed=D)
    value = 1 + (torch.arange(D, device=DEV) % 8) / 8.0
    c.v_scale.fill_(1.0)
    c.fill(0, torch.randn(n, 1, D, generator=gen(7), device=DEV), value.expand(n, 1, D))
    q = (torch.randn(T, 4, D, generator=gen(8), device=DEV) * std).to(torch.bfloat16)
    mean = 0.0
    for i in range(steps):
        c.v_scale.fill_(2.0 ** ((i + 0.5) / steps))
        out = ops.fp8_kv_attention(q, *c.args())
        mean += float((out.double() / (value.double() * c.v_scale.double()) - 1).mean()) / steps
    assert ops.get_status() == 0
    assert abs(mean) < 1e-4, mean
