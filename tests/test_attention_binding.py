"""Refusals of the attention layer's entry points, on the CPU: the C ABI's
status codes (nothing is launched, no pointer is followed) and the binding's
ValueErrors before the library is called."""
import ctypes
import types

import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import build as nbuild
from nvfp4_w4a4_quantized_act_b200 import ops

nbuild.build()

# The host structs of include/nvfp4.h.
class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int64)]


class KvPages(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_page_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KvBatch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("cu_tokens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("num_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class NormRope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("rotary_dim", ctypes.c_int32), ("eps", ctypes.c_float), ("flags", ctypes.c_uint)]


class AttentionOpts(ctypes.Structure):
    _fields_ = [("softmax_scale", ctypes.c_float), ("flags", ctypes.c_uint)]


FAKE = 1 << 20  # aligned, never dereferenced: checks fail first


def _heads(heads=4, data=FAKE, st=1024, sh=256):
    return Heads(data, st, sh, heads)


def _pages(**kw):
    v = dict(k_pages=FAKE, v_pages=FAKE, k_scale=FAKE, v_scale=FAKE, k_page_stride=16384, k_token_stride=1024,
             k_head_stride=256, v_page_stride=16384, v_token_stride=1024, v_head_stride=256, num_pages=8, page_size=16,
             kv_heads=4, head_dim=256)
    v.update(kw)
    return KvPages(**v)


def _batch(**kw):
    v = dict(page_table=FAKE, cu_tokens=FAKE, seq_lens=FAKE, table_stride=8, num_seqs=2, max_pages=8)
    v.update(kw)
    return KvBatch(**v)


def _nr(**kw):
    v = dict(q_weight=FAKE, k_weight=FAKE, inv_freq=FAKE, rotary_dim=64, eps=1e-6, flags=0)
    v.update(kw)
    return NormRope(**v)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def norm_rope(q=_heads(), k=_heads(), qo=_heads(), ko=_heads(), tokens=3, dim=256, pos=FAKE, nr=_nr()):
    return ops.lib().nvfp4_qk_norm_rope(_ref(q), _ref(k), _ref(qo), _ref(ko), tokens, dim, pos, _ref(nr), None)


def append(k=_heads(), v=_heads(), tokens=3, pages=_pages(), batch=_batch(), pos=None, nr=_nr()):
    return ops.lib().nvfp4_fp8_kv_append(_ref(k), _ref(v), tokens, _ref(pages), _ref(batch), pos, _ref(nr), None)


def attend(q=_heads(24), gate=None, out=_heads(24), tokens=3, pages=_pages(), batch=_batch(), scale=0.1, flags=0, amax=None,
           ws=FAKE, ws_bytes=1 << 30, opts=True):
    o = AttentionOpts(scale, flags) if opts else None
    return ops.lib().nvfp4_fp8_kv_attention(_ref(q), _ref(gate), _ref(out), tokens, _ref(pages), _ref(batch), _ref(o), amax,
                                            ws, ws_bytes, None)


INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 7

ABI = {
    "norm: no queries": (lambda: norm_rope(q=None), INVALID),
    "norm: null data": (lambda: norm_rope(q=_heads(data=None)), INVALID),
    "norm: no output": (lambda: norm_rope(qo=None), INVALID),
    "norm: keys without output": (lambda: norm_rope(ko=None), INVALID),
    "norm: output without keys": (lambda: norm_rope(k=None), INVALID),
    "norm: other heads": (lambda: norm_rope(qo=_heads(5)), INVALID),
    "norm: no positions": (lambda: norm_rope(pos=None), INVALID),
    "norm: tokens < 0": (lambda: norm_rope(tokens=-1), INVALID),
    "norm: tokens too many": (lambda: norm_rope(tokens=1 << 25), SHAPE),
    "norm: head_dim": (lambda: norm_rope(dim=192), SHAPE),
    "norm: no struct": (lambda: norm_rope(nr=None), INVALID),
    "norm: unknown flag": (lambda: norm_rope(nr=_nr(flags=1)), INVALID),
    "norm: eps < 0": (lambda: norm_rope(nr=_nr(eps=-1.0)), INVALID),
    "norm: eps nan": (lambda: norm_rope(nr=_nr(eps=float("nan"))), INVALID),
    "norm: rotary % 16": (lambda: norm_rope(nr=_nr(rotary_dim=24)), SHAPE),
    "norm: rotary > dim": (lambda: norm_rope(nr=_nr(rotary_dim=272)), SHAPE),
    "norm: rotary < 0": (lambda: norm_rope(nr=_nr(rotary_dim=-16)), INVALID),
    "norm: rotation without frequencies": (lambda: norm_rope(nr=_nr(inv_freq=None)), INVALID),
    "norm: data alignment": (lambda: norm_rope(q=_heads(data=FAKE + 8)), ALIGN),
    "norm: stride": (lambda: norm_rope(k=_heads(st=1028)), ALIGN),
    "norm: weight alignment": (lambda: norm_rope(nr=_nr(q_weight=FAKE + 2)), ALIGN),
    "norm: positions alignment": (lambda: norm_rope(pos=FAKE + 2), ALIGN),
    "norm: heads too many": (lambda: norm_rope(q=_heads(1025)), SHAPE),
    "append: heads": (lambda: append(k=_heads(3)), INVALID),
    "append: no cache": (lambda: ops.lib().nvfp4_fp8_kv_append(_ref(_heads()), _ref(_heads()), 3, None, _ref(_batch()),
                                                                None, _ref(_nr()), None), INVALID),
    "append: no batch": (lambda: append(batch=None), INVALID),
    "append: no norm struct": (lambda: append(nr=None), INVALID),
    "append: page size": (lambda: append(pages=_pages(page_size=48)), SHAPE),
    "append: page size 8": (lambda: append(pages=_pages(page_size=8)), SHAPE),
    "append: page size 512": (lambda: append(pages=_pages(page_size=512)), SHAPE),
    "append: head_dim": (lambda: append(pages=_pages(head_dim=64)), SHAPE),
    "append: no pages": (lambda: append(pages=_pages(num_pages=0)), INVALID),
    "append: null pages": (lambda: append(pages=_pages(v_pages=None)), INVALID),
    "append: null scale": (lambda: append(pages=_pages(k_scale=None)), INVALID),
    "append: page alignment": (lambda: append(pages=_pages(k_pages=FAKE + 8)), ALIGN),
    "append: stride % 16": (lambda: append(pages=_pages(k_token_stride=1032)), ALIGN),
    "append: strides do not nest": (lambda: append(pages=_pages(k_head_stride=272)), ALIGN),
    "append: rows overlap": (lambda: append(pages=_pages(v_head_stride=128)), INVALID),
    "append: table stride": (lambda: append(batch=_batch(table_stride=7)), INVALID),
    "append: null table": (lambda: append(batch=_batch(page_table=None)), INVALID),
    "append: null lengths": (lambda: append(batch=_batch(seq_lens=None)), INVALID),
    "append: offsets alignment": (lambda: append(batch=_batch(cu_tokens=FAKE + 1)), ALIGN),
    "append: positions past 32 bits": (lambda: append(batch=_batch(max_pages=1 << 28, table_stride=1 << 28)), SHAPE),
    "attend: group": (lambda: attend(q=_heads(22), out=_heads(22)), SHAPE),
    "attend: group too large": (lambda: attend(q=_heads(516), out=_heads(516)), SHAPE),
    "attend: output heads": (lambda: attend(out=_heads(20)), INVALID),
    "attend: gate heads": (lambda: attend(gate=_heads(20)), INVALID),
    "attend: gate alignment": (lambda: attend(gate=_heads(24, data=FAKE + 4)), ALIGN),
    "attend: no options": (lambda: attend(opts=False), INVALID),
    "attend: scale 0": (lambda: attend(scale=0.0), INVALID),
    "attend: scale < 0": (lambda: attend(scale=-0.1), INVALID),
    "attend: scale nan": (lambda: attend(scale=float("nan")), INVALID),
    "attend: scale inf": (lambda: attend(scale=float("inf")), INVALID),
    "attend: flag": (lambda: attend(flags=1), INVALID),
    "attend: no workspace": (lambda: attend(ws=None), WORKSPACE),
    "attend: small workspace": (lambda: attend(ws_bytes=16), WORKSPACE),
    "attend: workspace alignment": (lambda: attend(ws=FAKE + 8), ALIGN),
    "attend: amax alignment": (lambda: attend(amax=FAKE + 2), ALIGN),
    "attend: tokens < 0": (lambda: attend(tokens=-1), INVALID),
}


@pytest.mark.parametrize("case", sorted(ABI))
def test_abi_refuses(case):
    call, want = ABI[case]
    before = ops.launch_count()
    assert call() == want
    assert ops.launch_count() == before


def test_workspace_sizes():
    f = ops.fp8_kv_attention_workspace_bytes
    assert f(100, 24, 4, 256) > 0 and f(100, 8, 8, 128) > 0
    assert f(100, 24, 5, 256) == 0 and f(100, 24, 4, 64) == 0 and f(-1, 24, 4, 256) == 0 and f(100, 258, 2, 256) == 0


class _Recorder:
    """Stands in for the library: counts the calls and copies the host structs
    that each is given."""
    NAMES = ("nvfp4_qk_norm_rope", "nvfp4_fp8_kv_append", "nvfp4_fp8_kv_attention")
    STRUCTS = {
        "nvfp4_qk_norm_rope": ((0, Heads), (1, Heads), (2, Heads), (3, Heads), (7, NormRope)),
        "nvfp4_fp8_kv_append": ((0, Heads), (1, Heads), (3, KvPages), (4, KvBatch), (6, NormRope)),
        "nvfp4_fp8_kv_attention": ((0, Heads), (1, Heads), (2, Heads), (4, KvPages), (5, KvBatch),
                                   (6, AttentionOpts)),
    }

    def __init__(self):
        self.calls, self.args, self.structs, self.status = [], {}, {}, 0
        self.keep = [self._callback(n) for n in self.NAMES]

    def _callback(self, name):
        def call(*a):
            self.calls.append(name)
            self.args[name] = a
            self.structs[name] = [kind.from_buffer_copy(ctypes.string_at(a[i], ctypes.sizeof(kind))) if a[i] else None
                                  for i, kind in self.STRUCTS[name]]
            return self.status
        kinds = [t if t in (ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t) else ctypes.c_void_p
                 for t in getattr(ops.lib(), name).argtypes]
        return ctypes.CFUNCTYPE(ctypes.c_int, *kinds)(call)


@pytest.fixture
def rec():
    """The marshalling module bound to a recorder; CPU tensors stand in for
    device ones."""
    r, m = _Recorder(), ops._attention()

    def bind(fns, any_device):
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (*fns, ops.lib().nvfp4_fp8_kv_attention_workspace_bytes)), any_device)
    bind(r.keep, True)
    yield r
    bind([getattr(ops.lib(), n) for n in r.NAMES], False)


bf16, i32 = torch.bfloat16, torch.int32
Q, K = torch.zeros(3, 24, 256, dtype=bf16), torch.zeros(3, 4, 256, dtype=bf16)
P = torch.zeros(8, 16, 4, 256, dtype=torch.uint8)
ONE = torch.ones(1)
G = torch.zeros_like(Q)
TABLE, CU, LENS = torch.zeros(2, 4, dtype=i32), torch.tensor([0, 1, 3], dtype=i32), torch.tensor([5, 9], dtype=i32)
F, W = torch.ones(32), torch.ones(256, dtype=bf16)
POS = torch.zeros(3, dtype=i32)


def _cache(k=P, v=P, ks=ONE, vs=ONE, table=TABLE, cu=CU, lens=LENS):
    return k, v, ks, vs, table, cu, lens


GOOD = {
    "norm": lambda: ops.qk_norm_rope(Q, K, POS, F, W, W),
    "norm, no tokens": lambda: ops.qk_norm_rope(Q[:0], K[:0], POS, F, W, W),
    "attend, no tokens": lambda: ops.fp8_kv_attention(Q[:0], *_cache()),
    "norm, one side, no rotation": lambda: ops.qk_norm_rope(Q, None, None, None, W),
    "norm, heads first": lambda: ops.qk_norm_rope(Q, K, POS, F, q_out=torch.zeros(24, 3, 256, dtype=bf16).transpose(0, 1)),
    "append": lambda: ops.fp8_kv_append(K, K, *_cache(), inv_freq=F, k_weight=W, positions=POS),
    "append, plain": lambda: ops.fp8_kv_append(K, K, *_cache()),
    "attend": lambda: ops.fp8_kv_attention(Q, *_cache()),
    "attend, all": lambda: ops.fp8_kv_attention(Q, *_cache(), softmax_scale=0.1, gate=Q, out=torch.zeros_like(Q),
                                                out_amax=torch.zeros(1, dtype=i32)),
    "attend, heads-first pages": lambda: ops.fp8_kv_attention(Q, *_cache(
        k=torch.zeros(8, 4, 16, 256, dtype=torch.uint8).transpose(1, 2))),
    "attend, one page and one head": lambda: ops.fp8_kv_attention(
        Q, *_cache(k=P[:1, :, :1], v=P[:1, :, :1])),
}

BAD = {
    "norm: fp32": lambda: ops.qk_norm_rope(Q.float(), None, POS, F),
    "norm: 2-D": lambda: ops.qk_norm_rope(Q[0], None, POS, F),
    "norm: inner stride": lambda: ops.qk_norm_rope(torch.zeros(3, 256, 24, dtype=bf16).transpose(1, 2), None, POS, F),
    "norm: k of other tokens": lambda: ops.qk_norm_rope(Q, K[:2], POS, F),
    "norm: k of another head_dim": lambda: ops.qk_norm_rope(Q, torch.zeros(3, 4, 128, dtype=bf16), POS, F),
    "norm: output shape": lambda: ops.qk_norm_rope(Q, None, POS, F, q_out=torch.zeros(3, 23, 256, dtype=bf16)),
    "norm: output overlaps itself": lambda: ops.qk_norm_rope(Q, None, POS, F, q_out=torch.zeros(1, 24, 256, dtype=bf16).expand(3, 24, 256)),
    "norm: k_out without k": lambda: ops.qk_norm_rope(Q, None, POS, F, k_out=K),
    "norm: rotation without positions": lambda: ops.qk_norm_rope(Q, None, None, F),
    "norm: positions int64": lambda: ops.qk_norm_rope(Q, None, POS.long(), F),
    "norm: positions too short": lambda: ops.qk_norm_rope(Q, None, POS[:2], F),
    "norm: frequencies fp64": lambda: ops.qk_norm_rope(Q, None, POS, F.double()),
    "norm: frequencies strided": lambda: ops.qk_norm_rope(Q, None, POS, torch.ones(64)[::2]),
    "norm: weight length": lambda: ops.qk_norm_rope(Q, None, POS, F, W[:128]),
    "norm: weight dtype": lambda: ops.qk_norm_rope(Q, None, POS, F, W.float()),
    "append: v shape": lambda: ops.fp8_kv_append(K, K[:, :2], *_cache()),
    "append: heads of the pages": lambda: ops.fp8_kv_append(K[:, :2], K[:, :2], *_cache()),
    "append: pages bf16": lambda: ops.fp8_kv_append(K, K, *_cache(k=P.to(bf16))),
    "append: pages 3-D": lambda: ops.fp8_kv_append(K, K, *_cache(k=P[0])),
    "append: pages of other shapes": lambda: ops.fp8_kv_append(K, K, *_cache(v=P[:4])),
    "append: scale fp64": lambda: ops.fp8_kv_append(K, K, *_cache(ks=ONE.double())),
    "append: two scales": lambda: ops.fp8_kv_append(K, K, *_cache(vs=torch.ones(2))),
    "append: table int64": lambda: ops.fp8_kv_append(K, K, *_cache(table=TABLE.long())),
    "append: table transposed": lambda: ops.fp8_kv_append(K, K, *_cache(table=torch.zeros(4, 2, dtype=i32).t())),
    "append: too few offsets": lambda: ops.fp8_kv_append(K, K, *_cache(cu=CU[:2])),
    "append: too few lengths": lambda: ops.fp8_kv_append(K, K, *_cache(lens=LENS[:1])),
    "attend: head_dim": lambda: ops.fp8_kv_attention(torch.zeros(3, 24, 128, dtype=bf16), *_cache()),
    "attend: group": lambda: ops.fp8_kv_attention(Q[:, :22], *_cache()),
    "attend: gate shape": lambda: ops.fp8_kv_attention(Q, *_cache(), gate=Q[:2]),
    "attend: out dtype": lambda: ops.fp8_kv_attention(Q, *_cache(), out=Q.float()),
    "attend: out overlaps itself": lambda: ops.fp8_kv_attention(Q, *_cache(), out=torch.zeros(3, 1, 256, dtype=bf16).expand(3, 24, 256)),
    "attend: out is q": lambda: ops.fp8_kv_attention(Q, *_cache(), out=Q),
    "attend: out is the gate": lambda: ops.fp8_kv_attention(Q, *_cache(), gate=G, out=G),
    "attend: small workspace": lambda: ops.fp8_kv_attention(Q, *_cache(), ws=torch.zeros(16, dtype=torch.uint8)),
    "attend: strided workspace": lambda: ops.fp8_kv_attention(Q, *_cache(), ws=torch.zeros(1 << 27, dtype=torch.uint8)[::2]),
    "norm: not a tensor": lambda: ops.qk_norm_rope(Q, None, [0, 1, 2], F),
    "norm: eps not a number": lambda: ops.qk_norm_rope(Q, None, POS, F, eps="x"),
    "norm: not a stream": lambda: ops.qk_norm_rope(Q, None, POS, F, stream=7),
    "norm: a stream of nonsense": lambda: ops.qk_norm_rope(Q, None, POS, F, stream=types.SimpleNamespace(cuda_stream="x")),
    "norm: too many frequencies": lambda: ops.qk_norm_rope(Q, None, POS, torch.ones(1025)),
    "attend: pages not a tensor": lambda: ops.fp8_kv_attention(Q, None, *_cache()[1:], ws=torch.zeros(16)),
    "attend: no kv heads": lambda: ops.fp8_kv_attention(Q, *_cache(k=P[:, :, :0], v=P[:, :, :0])),
    "attend: amax too small": lambda: ops.fp8_kv_attention(Q, *_cache(), out_amax=torch.zeros(2, dtype=torch.uint8)),
}


def test_structs_hold_what_the_tensors_say(rec):
    """The host structs that a call packs, read back field by field."""
    seen = rec.structs

    def same(x, **want):
        for k, v in want.items():
            assert getattr(x, k) == (v if v != 0 or isinstance(v, float) or "stride" in k or k == "flags" else None), k
    ko, qo, g = K.clone(), Q.clone(), Q.clone()
    ops.qk_norm_rope(Q, K, POS, F, W, None, eps=0.25, plus_one=True, q_out=qo, k_out=ko)
    q, k, q2, k2, nr = seen["nvfp4_qk_norm_rope"]
    same(q, data=Q.data_ptr(), token_stride=24 * 256, head_stride=256, heads=24)
    same(k, data=K.data_ptr(), token_stride=4 * 256, head_stride=256, heads=4)
    same(q2, data=qo.data_ptr(), heads=24)
    same(k2, data=ko.data_ptr(), heads=4)
    same(nr, q_weight=W.data_ptr(), k_weight=0, inv_freq=F.data_ptr(), rotary_dim=64, eps=0.25, flags=8)
    kp, vp = P, torch.zeros(8, 4, 16, 256, dtype=torch.uint8).transpose(1, 2)
    two = torch.ones(1)
    pages = dict(k_pages=kp.data_ptr(), v_pages=vp.data_ptr(), k_scale=ONE.data_ptr(), v_scale=two.data_ptr(), k_page_stride=16384,
                 k_token_stride=1024, k_head_stride=256, v_page_stride=16384, v_token_stride=256, v_head_stride=4096, num_pages=8,
                 page_size=16, kv_heads=4, head_dim=256)
    batch = dict(page_table=TABLE.data_ptr(), cu_tokens=CU.data_ptr(), seq_lens=LENS.data_ptr(), table_stride=4, num_seqs=2, max_pages=4)
    ops.fp8_kv_append(K, ko, kp, vp, ONE, two, TABLE, CU, LENS, inv_freq=F, k_weight=W)
    k, v, pg, bt, nr = seen["nvfp4_fp8_kv_append"]
    same(k, data=K.data_ptr())
    same(v, data=ko.data_ptr())
    same(pg, **pages)
    same(bt, **batch)
    same(nr, q_weight=0, k_weight=W.data_ptr(), inv_freq=F.data_ptr(), rotary_dim=64, flags=0)
    ops.fp8_kv_attention(Q, kp, vp, ONE, two, TABLE, CU, LENS, softmax_scale=0.5, gate=g, out=qo)
    q, gt, o, pg, bt, op = seen["nvfp4_fp8_kv_attention"]
    same(q, data=Q.data_ptr())
    same(gt, data=g.data_ptr())
    same(o, data=qo.data_ptr())
    same(pg, **pages)
    same(bt, **batch)
    same(op, softmax_scale=0.5, flags=0)


def test_other_arguments_arrive(rec):
    amax, ws, stream = torch.zeros(1, dtype=i32), torch.zeros(1 << 27, dtype=torch.uint8), types.SimpleNamespace(cuda_stream=0x1230)
    ops.qk_norm_rope(Q, None, POS, F, stream=stream)
    a = rec.args["nvfp4_qk_norm_rope"]
    assert a[1] is None and a[3] is None and a[4:7] == (3, 256, POS.data_ptr()) and a[8] == 0x1230
    ops.fp8_kv_append(K, K, *_cache(), positions=POS, stream=stream)
    a = rec.args["nvfp4_fp8_kv_append"]
    assert a[2] == 3 and a[5] == POS.data_ptr() and a[7] == 0x1230
    ops.fp8_kv_append(K, K, *_cache())
    assert rec.args["nvfp4_fp8_kv_append"][5] is None
    ops.fp8_kv_attention(Q, *_cache(), out_amax=amax, ws=ws, stream=stream)
    a = rec.args["nvfp4_fp8_kv_attention"]
    assert a[1] is None and a[3] == 3 and a[7:] == (amax.data_ptr(), ws.data_ptr(), 1 << 27, 0x1230)
    assert rec.structs["nvfp4_fp8_kv_attention"][5].softmax_scale == 0.0625


def test_a_status_is_raised(rec):
    rec.status = 3
    for call in (lambda: ops.qk_norm_rope(Q, None, POS, F), lambda: ops.fp8_kv_append(K, K, *_cache()),
                 lambda: ops.fp8_kv_attention(Q, *_cache())):
        with pytest.raises(ops.Nvfp4Error) as e:
            call()
        assert e.value.code == 3


@pytest.mark.parametrize("case", sorted(GOOD))
def test_valid_calls_reach_the_library(rec, case):
    GOOD[case]()
    assert len(rec.calls) == 1


@pytest.mark.parametrize("case", sorted(BAD))
def test_malformed_arguments_raise_before_the_library(rec, case):
    with pytest.raises(ValueError):
        BAD[case]()
    assert rec.calls == []


@pytest.mark.parametrize("call", [lambda: ops.qk_norm_rope(Q, None, POS), lambda: ops.fp8_kv_append(K, K, *_cache()),
                                  lambda: ops.fp8_kv_attention(Q, *_cache())])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensors only"):
        call()
