"""Outputs and workspaces that the attention layer's calls allocate when they
run on another stream than the current one."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import DEV, Cache, fill_normal, gen

pytestmark = pytest.mark.gpu


def _case(seed):
    c = Cache([(1, 3000), (60, 700), (1, 90)], 2, 256, 16, seed=seed)
    fill_normal(c, seed)
    return c, torch.randn(c.tokens, 12, 256, generator=gen(seed), device=DEV).to(torch.bfloat16)


@pytest.fixture
def made(monkeypatch):
    """Addresses of what the calls allocate, in order."""
    got, new = [], ops._new

    def record(*a):
        t = new(*a)
        got.append(t.data_ptr())
        return t
    monkeypatch.setattr(ops, "_new", record)
    return got


def test_memory_belongs_to_the_stream_that_writes_it(made):
    """What the current stream has just given back to the allocator may still
    be in use by its queued calls: a call on another stream must not get it."""
    c, q = _case(1)
    pos = torch.zeros(c.tokens, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    for call in (lambda **kw: ops.fp8_kv_attention(q, *c.args(), **kw), lambda **kw: ops.qk_norm_rope(q, q[:, :4], pos, **kw)):
        torch.cuda.synchronize()
        del made[:]
        call()
        torch.cuda.synchronize()
        first = set(made)
        del made[:]
        call(stream=side)
        torch.cuda.synchronize()
        assert len(made) == 2 and not first & set(made)


def test_a_call_beside_one_that_is_still_queued():
    """A call with its own workspace waits on the current stream while the next
    one, on another stream, has its turn; both are right."""
    (c0, q0), (c1, q1) = _case(2), _case(3)
    want = [ops.fp8_kv_attention(q, *c.args()).clone() for c, q in ((c0, q0), (c1, q1))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(5_000_000)  # a few milliseconds
        a = ops.fp8_kv_attention(q0, *c0.args())
        b = ops.fp8_kv_attention(q1, *c1.args(), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        del a, b
    assert ops.get_status() == 0


@pytest.mark.parametrize("stream", [7, "side"])
def test_something_else_than_a_stream(stream):
    c, q = _case(4)
    with pytest.raises(ValueError, match="stream"):
        ops.fp8_kv_attention(q, *c.args(), stream=stream)
