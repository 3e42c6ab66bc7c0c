"""Memory that the quantize, GEMM and FP8 cache calls allocate when they run on
another stream than the current one, and their results there."""
import types

import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from nvfp4_w4a4_quantized_act_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _calls():
    X = wl.activation_normal(130, 256, 0).to(DEV)
    W = wl.weight_normal(256, 256, 0.02, 1).to(DEV)
    w, wg = ops.quantize_weights(W, [(0, 96), (96, 256)]), ops.quantize_weights_gated(W)
    codes, sf, g = ops.quantize_act(X)
    scale = ops.fp8_kv_calibrate(X)
    return {
        "quantize_weights": lambda **kw: ops.quantize_weights(W, **kw),
        "quantize_weights_gated": lambda **kw: ops.quantize_weights_gated(W, **kw),
        "quantize_act": lambda **kw: ops.quantize_act(X, **kw),
        "gemm_prequant": lambda **kw: ops.gemm_prequant(codes, sf, g, 130, 256, w, **kw),
        "linear_fused": lambda **kw: ops.linear_fused(X, w, **kw),
        "linear": lambda **kw: ops.linear(X, w, **kw),
        "linear_fused_noalloc": lambda **kw: ops.linear_fused_noalloc(X, w, **kw),
        "swiglu_quantize": lambda **kw: ops.swiglu_quantize(X, **kw),
        "linear_swiglu": lambda **kw: ops.linear_swiglu(X, wg, **kw),
        # (h, ws): the first word of the workspace is max|h|, nothing else in it is defined
        "gemm_prequant_swiglu": lambda **kw: [t.view(-1)[:n] for t, n in zip(
            ops.gemm_prequant_swiglu(codes, sf, g, 130, 256, wg, **kw), (130 * 128, 4))],
        "fp8_kv_calibrate": lambda **kw: ops.fp8_kv_calibrate(X, **kw),
        "fp8_kv_quantize": lambda **kw: ops.fp8_kv_quantize(X, scale, **kw),
    }


def _tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for y in (x if isinstance(x, (tuple, list)) else [x.codes, x.sf, x.g_w]) for t in _tensors(y)]


def test_a_stream_of_another_library():
    """Whatever has the address of a CUDA stream serves as one."""
    calls, side = _calls(), torch.cuda.Stream()
    want = calls["linear_fused"]()
    torch.cuda.synchronize()
    got = calls["linear_fused"](stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for bad in (7, "x", types.SimpleNamespace(cuda_stream="x")):
        with pytest.raises(ValueError, match="stream"):
            calls["linear_fused"](stream=bad)


@pytest.mark.parametrize("name", sorted(["quantize_weights", "quantize_weights_gated", "quantize_act", "gemm_prequant", "linear_fused",
                                         "linear", "linear_fused_noalloc", "swiglu_quantize", "linear_swiglu",
                                         "gemm_prequant_swiglu", "fp8_kv_calibrate", "fp8_kv_quantize"]))
def test_another_stream(name, monkeypatch):
    """Same results, and nothing that the current stream has just given back."""
    call = _calls()[name]
    made, new = [], ops.torch.empty

    def record(*a, **kw):
        t = new(*a, **kw)
        made.append(t.data_ptr())
        return t
    side = torch.cuda.Stream()
    monkeypatch.setattr(ops.torch, "empty", record)
    want = [t.clone() for t in _tensors(call())]
    first = set(made)
    torch.cuda.synchronize()
    del made[:]
    got = _tensors(call(stream=side))
    torch.cuda.synchronize()
    assert made and not first & set(made)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert ops.get_status() == 0
