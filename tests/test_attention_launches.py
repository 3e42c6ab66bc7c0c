"""What the attention layer's entry points launch, on the CPU: they are linked
with recorders in place of the CUDA runtime (tests/cuda/fake_runtime.cpp)."""
import ctypes
import os
import subprocess

import pytest

from nvfp4_w4a4_quantized_act_b200 import build as nbuild
from test_attention_binding import AttentionOpts, FAKE, Heads, KvBatch, KvPages, NormRope

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
    L.nvfp4_qk_norm_rope.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp]
    return L


def attend(L, tokens, seqs, heads=24, kv=4, dim=256, refuse=-1, q=None, gate=None, out=None, amax=None, ws=FAKE + (2 << 40), flags=0,
           max_pages=64):
    """(status, kernels launched, in order)."""
    L.fake_reset(refuse)
    page = 16
    q, o = (x or Heads(FAKE + (i << 40), heads * dim, dim, heads) for i, x in enumerate((q, out)))
    pages = KvPages(k_pages=FAKE, v_pages=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=64, page_size=page, kv_heads=kv, head_dim=dim,
                    k_page_stride=page * kv * dim, k_token_stride=kv * dim, k_head_stride=dim,
                    v_page_stride=page * kv * dim, v_token_stride=kv * dim, v_head_stride=dim)
    batch = KvBatch(FAKE, FAKE, FAKE, max_pages, seqs, max_pages)
    rc = L.nvfp4_fp8_kv_attention(ctypes.byref(q), ctypes.byref(gate) if gate else None, ctypes.byref(o), tokens, ctypes.byref(pages),
                                  ctypes.byref(batch), ctypes.byref(AttentionOpts(0.1, flags)), amax, ws,
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


# Head rows in one buffer of 2^20 elements, by (first element, token stride, head stride, heads), 5 tokens of head_dim 128.
W = 4096


def _rows(first, st, sh, heads):
    return Heads(FAKE + 2 * first, st, sh, heads)


def _elements(x, tokens=5, dim=128):
    first = (x.data - FAKE) // 2
    return {first + t * x.token_stride + h * x.head_stride + d for t in range(tokens) for h in range(x.heads) for d in range(dim)}


LAYOUTS = [(0, W, 128, 4), (0, W, 256, 4), (128, W, 256, 4), (128, W, 128, 4), (512, W, 128, 4), (1024, W, 128, 4), (384, W, 512, 4),
           (0, W, 1024, 4), (64, W, 128, 4), (8, W, 256, 4), (136, W, 256, 4), (W, W, 128, 4), (5 * W, W, 128, 4), (4 * W, W, 256, 4),
           (4 * W + 128, W, 256, 4), (3968, W, 128, 4), (W - 64, W, 1024, 4), (0, 512, 128, 4), (2560, 512, 128, 4), (2552, 512, 128, 4),
           (0, 128, 640, 4), (128, 128, 640, 4), (128, 128, 768, 4), (0, 256, 2048, 4), (128, 256, 2048, 4), (512, W, -128, 4),
           (896, W, -128, 4), (17000, -W, 128, 4)]


@pytest.mark.parametrize("a", range(len(LAYOUTS)))
def test_outputs_that_overlap_are_refused(fake, a):
    """Element by element: an output that shares one with the queries, the gate
    or, for norm and rotation, with the keys or the other output is refused, one
    that only lies between them is not (with two token strides it may be)."""
    nr = NormRope(None, None, None, 0, 1e-6, 0)

    def norm(q, k, qo, ko):
        fake.fake_reset(-1)
        ref = [ctypes.byref(x) if x else None for x in (q, k, qo, ko)]
        return fake.nvfp4_qk_norm_rope(*ref, 5, 128, None, ctypes.byref(nr), None), fake.fake_launches()
    far = [_rows(1 << (24 + i), W, 128, 4) for i in range(3)]
    for b in range(len(LAYOUTS)):
        x, y = _rows(*LAYOUTS[a]), _rows(*LAYOUTS[b])
        meet = bool(_elements(x) & _elements(y))
        if x.token_stride != y.token_stride and not meet:
            ex, ey = _elements(x), _elements(y)
            if min(ex) <= max(ey) and min(ey) <= max(ex):
                continue  # may be refused
        for got in (attend(fake, 5, 1, 4, 4, 128, q=x, out=y), attend(fake, 5, 1, 4, 4, 128, q=far[0], gate=x, out=y)):
            assert (got[0] == 1 and not got[1]) if meet else got[0] == 0, (LAYOUTS[a], LAYOUTS[b])
        same = a == b
        assert norm(x, None, y, None) == ((1, 0) if meet and not same else (0, 1))
        assert norm(far[0], x, far[1], y) == ((1, 0) if meet and not same else (0, 1))
        for rc, n in (norm(far[0], far[1], x, y), norm(x, far[0], far[1], y), norm(far[0], x, y, far[1])):
            assert (rc, n) == ((1, 0) if meet else (0, 1)), (LAYOUTS[a], LAYOUTS[b])


def test_views_of_one_projection(fake):
    """Queries, gate and keys of one projection's output, in place and beside."""
    T, W, D = 300, 24 * 512 + 2 * 1024, 256
    q, gate, k = (Heads(FAKE + 2 * at, W, step, n) for at, step, n in ((0, 512, 24), (256, 512, 24), (24 * 512, 256, 4)))
    nr = NormRope(None, None, None, 0, 1e-6, 0)
    fake.fake_reset(-1)
    r = ctypes.byref
    assert fake.nvfp4_qk_norm_rope(r(q), r(k), r(q), r(k), T, D, None, r(nr), None) == 0
    assert attend(fake, T, 2, q=q, gate=gate)[0] == 0
    assert attend(fake, T, 2, q=q, gate=gate, out=q)[0] == 1
    assert attend(fake, T, 2, q=q, gate=gate, out=gate)[0] == 1
    assert attend(fake, T, 2, q=q, gate=gate, out=Heads(FAKE + 512, W, 512, 24))[0] == 1  # a head further
    assert attend(fake, T, 2, q=q, out=gate)[0] == 0                                     # its columns are free


def test_a_workspace_that_is_something_else(fake):
    """Scratch must not be the output, the inputs or the word of max|out|."""
    ws = FAKE + (2 << 40)
    size = fake.nvfp4_fp8_kv_attention_workspace_bytes(40, 24, 4, 256)
    assert attend(fake, 40, 1, amax=ws + size)[0] == 0 and attend(fake, 40, 1, amax=ws - 4)[0] == 0
    for amax in (ws, ws + size - 4):
        assert attend(fake, 40, 1, amax=amax) == (1, [])
    for which in ("q", "gate", "out"):
        assert attend(fake, 40, 1, **{which: Heads(ws - 16, 24 * 256, 256, 24)}) == (1, [])
        assert attend(fake, 40, 1, **{which: Heads(ws + size, 24 * 256, 256, 24)})[0] == 0


@pytest.mark.parametrize("tokens,seqs,heads,flags,want", [
    (64, 64, 24, 0, "tiles single join"),   # single tokens, or a chunk of 64 among sequences that stand still
    (2, 2, 24, 0, "tiles single join"),
    (67, 64, 24, 0, "tiles single join"),
    (20, 64, 24, 0, "tiles single join"),
    (4000, 93, 24, 0, "tiles single join"),
    (73, 64, 24, 0, "tiles join"),
    (1, 1, 24, 0, "single join"),           # nothing but a single token can be
    (1, 40, 24, 0, "single join"),
    (64, 64, 24, 16, "single join"),        # the caller's word
    (300, 64, 24, 16, "single join"),
    (64, 64, 36, 16, "tiles join"),         # more heads share a key than that kernel has rows
    (64, 64, 36, 0, "tiles join"),
])
def test_which_kernels_run(fake, tokens, seqs, heads, flags, want):
    assert attend(fake, tokens, seqs, heads=heads, flags=flags) == (0, want.split())


def test_other_flags_are_refused(fake):
    assert attend(fake, 4, 4, flags=8) == (1, []) and attend(fake, 4, 4, flags=17) == (1, [])


def test_sizes_whose_sums_leave_the_integers(fake):
    """A position rounded up to the end of a key block, and the block behind it,
    fit 32 bits; the cost of a batch, times the number of CTAs, fits 64 bits
    even if every sequence claimed every row and the longest length."""
    most = (2 ** 31 - 256) // 16
    assert attend(fake, 4, 2, max_pages=most)[0] == 0
    assert attend(fake, 4, 2, max_pages=most + 1) == (2, [])
    assert attend(fake, 1 << 16, 1 << 12, max_pages=1 << 16)[0] == 0      # 4096 sequences, 2^20 keys each
    assert attend(fake, 1 << 20, 1 << 20, max_pages=1 << 24) == (2, [])
