"""Arguments of the attention layer's calls that should be truth values, on the
CPU."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from test_attention_binding import CU, F, K, LENS, ONE, P, POS, Q, TABLE, rec  # noqa: F401 (rec: a fixture)

CACHE = (P, P, ONE, ONE, TABLE, CU, LENS)


class _Neither:
    def __bool__(self):
        raise RuntimeError("neither")


@pytest.mark.parametrize("value", [torch.ones(2), _Neither()])
@pytest.mark.parametrize("call", [
    lambda v: ops.qk_norm_rope(Q, None, POS, F, plus_one=v), lambda v: ops.fp8_kv_append(K, K, *CACHE, plus_one=v),
    lambda v: ops.fp8_kv_attention(Q, *CACHE, single_tokens=v)])
def test_neither_true_nor_false(rec, call, value):  # noqa: F811
    with pytest.raises(ValueError, match="true or false"):
        call(value)
    assert rec.calls == []


@pytest.mark.parametrize("value", [0, 1, None, "", "x", torch.ones(1)])
def test_any_truth_value_serves(rec, value):  # noqa: F811
    ops.qk_norm_rope(Q, None, POS, F, plus_one=value)
    assert rec.structs["nvfp4_qk_norm_rope"][4].flags == (8 if value is not None and bool(value) else 0)
    ops.fp8_kv_attention(Q, *CACHE, single_tokens=value)
    assert rec.structs["nvfp4_fp8_kv_attention"][5].flags == (16 if value is not None and bool(value) else 0)
