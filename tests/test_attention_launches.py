"""What the attention layer's entry points launch, on the CPU: they are linked
with recorders in place of the CUDA runtime (tests/cuda/fake_runtime.cpp)."""
import ctypes
import os
import subprocess

import pytest

from nvfp4_w4a4_quantized_act_b200 import build as nbuild
from test_attention_binding import AttentionOpts, FAKE, Heads, KvBatch, KvPages

HERE = os.path.dirname(os.path.abspath(__file__))
ERR_CUDA = 4


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    if not os.path.exists(nbuild.NVCC):
        pytest.skip("nvcc not available")
    so = str(tmp_path_factory.mktemp("fake") / "libattention_fake.so")
    source = os.path.join(HERE, "cuda", "fake_runtime.cpp")
    r = subprocess.run([nbuild.NVCC, *nbuild.NVCC_FLAGS, "-cudart", "none", "-Xlinker", "-Bsymbolic", "-o", so, *nbuild.attention_sources(), source],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    L = ctypes.CDLL(so)
    L.fake_name.restype = ctypes.c_char_p
    L.nvfp4_fp8_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_fp8_kv_attention_workspace_bytes.argtypes = [ctypes.c_int64] * 4
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.nvfp4_fp8_kv_attention.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    return L


def attend(L, tokens, seqs, heads=24, kv=4, dim=256, refuse=-1):
    """(status, kernels launched, in order)."""
    L.fake_reset(refuse)
    page = 16
    q, o = (Heads(FAKE + (i << 40), heads * dim, dim, heads) for i in range(2))
    pages = KvPages(k_pages=FAKE, v_pages=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=64, page_size=page, kv_heads=kv, head_dim=dim,
                    k_page_stride=page * kv * dim, k_token_stride=kv * dim, k_head_stride=dim,
                    v_page_stride=page * kv * dim, v_token_stride=kv * dim, v_head_stride=dim)
    batch = KvBatch(FAKE, FAKE, FAKE, 64, seqs, 64)
    rc = L.nvfp4_fp8_kv_attention(ctypes.byref(q), None, ctypes.byref(o), tokens, ctypes.byref(pages), ctypes.byref(batch),
                                  ctypes.byref(AttentionOpts(0.1, 0)), None, FAKE + (2 << 40),
                                  L.nvfp4_fp8_kv_attention_workspace_bytes(tokens, heads, kv, dim), None)
    kinds = {"join": "join", "paged_attention_kernel": "tiles", "paged_decode_kernel": "single"}
    names = [L.fake_name(i).decode() for i in range(L.fake_launches())]
    return rc, [next(v for k, v in kinds.items() if k in n) for n in names]


@pytest.mark.parametrize("tokens,seqs", [(4000, 3), (70, 64), (1, 1)])
def test_a_refused_launch_is_the_last(fake, tokens, seqs):
    """The join reads what the kernels before it wrote to the workspace: after a
    launch that was refused that is anything, so nothing more may be launched,
    and the call says so.  The next call is not affected."""
    rc, names = attend(fake, tokens, seqs)
    assert rc == 0 and names[-1] == "join" and fake.fake_counted() == len(names)
    for k in range(len(names)):
        assert attend(fake, tokens, seqs, refuse=k) == (ERR_CUDA, names[:k + 1])
        assert fake.fake_counted() == k
        assert attend(fake, tokens, seqs) == (0, names)
