"""The smoke run goes through every operator of the attention layer."""
import pytest

import __graft_entry__ as entry
from nvfp4_w4a4_quantized_act_b200 import ops

pytestmark = pytest.mark.gpu


def test_smoke_runs_the_attention_layer(monkeypatch, capsys):
    called = []
    for name in ("qk_norm_rope", "fp8_kv_append", "fp8_kv_attention"):
        monkeypatch.setattr(ops, name, lambda *a, _f=getattr(ops, name), _n=name, **kw: called.append(_n) or _f(*a, **kw))
    entry.smoke()
    assert called == ["qk_norm_rope", "fp8_kv_append", "fp8_kv_attention"] * 2
    assert capsys.readouterr().out.startswith("smoke ok: ")
