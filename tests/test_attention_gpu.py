"""Attention over the paged FP8 cache against a 64-bit reference, with bounds
derived from the operator's roundings: head layouts, page sizes and layouts,
lengths from none to long, ragged batches, rows that see nothing, stale NaN
codes beyond the sequences and NaN in keys out of sight, streams, graphs."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import DEV, E4M3, Cache, check_attention, fill_normal, gen

pytestmark = pytest.mark.gpu


def _queries(c, heads, seed, std=1.0):
    """Queries and gates as views of one projection's output."""
    qg = (torch.randn(c.tokens, heads, 2 * c.dim, generator=gen(seed), device=DEV) * std).to(torch.bfloat16)
    return qg[:, :, :c.dim], qg[:, :, c.dim:]


def _run(c, heads, seed=5, std=1.0, gated=True, scale=None, only=None, q=None, **kw):
    qq, gate = _queries(c, heads, seed, std)
    q = qq if q is None else q
    scale = c.dim ** -0.5 if scale is None else scale
    out = torch.full((c.tokens, heads, c.dim), 3.0, device=DEV).to(torch.bfloat16)
    before = out.clone()
    ops.fp8_kv_attention(q, *c.args(), softmax_scale=scale, gate=gate if gated else None, out=out, **kw)
    assert ops.get_status() == 0
    check_attention(c, q, gate if gated else None, out, scale, before, only)
    return out


LENGTHS = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n", LENGTHS)
def test_single_tokens(D, n):
    c = Cache([(1, n)], 2, D, 16, seed=n + D, tokens_pad=2)
    fill_normal(c, n)
    _run(c, 12)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,n", [(2, 2), (21, 21), (22, 22), (43, 300), (64, 127), (64, 128), (64, 129), (130, 130), (128, 640)])
def test_chunks(D, new, n):
    c = Cache([(new, n)], 2, D, 32, seed=n + new, tokens_pad=1)
    fill_normal(c, n)
    _run(c, 12)


@pytest.mark.parametrize("heads,kv,D", [(1, 1, 128), (4, 4, 256), (5, 1, 256), (14, 2, 128), (24, 4, 256), (48, 1, 128),
                                        (128, 1, 256), (254, 2, 128), (9, 3, 256), (33, 1, 128)])
def test_head_layouts(heads, kv, D):
    c = Cache([(1, 90), (9, 140), (2, 129)], kv, D, 16, seed=heads, tokens_pad=3)
    fill_normal(c, heads)
    _run(c, heads, gated=heads % 2 == 0)


@pytest.mark.parametrize("pad", [0, 3, 40])
@pytest.mark.parametrize("heads,kv,D", [(1, 1, 128), (8, 1, 128), (5, 1, 256), (16, 2, 256), (21, 3, 128), (7, 7, 256), (18, 2, 128)])
def test_decode_batches(heads, kv, D, pad):
    """One new token each, unpadded and padded; beside them a sequence with
    none and, where the batch has no more rows than sequences, one with two."""
    seqs = [(1, n) for n in (1, 31, 32, 33, 64, 127, 128, 129, 500, 1025, 0)] + [(0, 77)]
    if pad == 0:
        seqs.append((2, 70))
    c = Cache(seqs, kv, D, 32, seed=heads, tokens_pad=pad)
    fill_normal(c, heads)
    _run(c, heads)


RAGGED = [(3, 3), (0, 40), (1, 200), (70, 70), (0, 0), (5, 130), (1, 1), (17, 333), (1, 128), (2, 129)]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_pages(page, layout):
    c = Cache(RAGGED, 3, 128 if page == 32 else 256, page, seed=page, layout=layout, tokens_pad=7)
    fill_normal(c, page)
    _run(c, 6)


def test_keys_and_values_of_one_tensor():
    """K and V pages interleaved in one pool: pages [n, 2, size, heads, dim]."""
    c = Cache(RAGGED, 2, 128, 16, seed=3)
    pool = torch.zeros(c.n_pages, 2, 16, 2, 128, dtype=torch.uint8, device=DEV)
    pool[:, 0], pool[:, 1] = c.k_pages, c.v_pages
    c.k_pages, c.v_pages = pool[:, 0], pool[:, 1]
    fill_normal(c, 8)
    _run(c, 4)


@pytest.mark.parametrize("n_seqs", [33, 150, 700])
def test_many_sequences(n_seqs):
    seqs = [(1 if i % 5 else (i % 3) * 2, 1 + (i * 37) % 300) for i in range(n_seqs)]
    c = Cache(seqs, 2, 128, 32, seed=n_seqs, tokens_pad=9)
    fill_normal(c, 3)
    _run(c, 8, only=set(range(0, n_seqs, 7)) | set(range(n_seqs - 5, n_seqs)))


@pytest.mark.parametrize("D,kv,n_seqs", [(256, 4, 91), (256, 4, 100), (128, 8, 46), (128, 8, 47), (256, 1, 370)])
def test_single_tokens_beside_chunks(D, kv, n_seqs):
    """Around the number of sequences from which the single tokens of a mixed
    batch have a kernel of their own."""
    seqs = [(1, 1 + (i * 61) % 400) for i in range(n_seqs)]
    seqs[3], seqs[n_seqs // 2], seqs[-1] = (40, 390), (2, 2), (25, 130)
    c = Cache(seqs, kv, D, 16, seed=n_seqs, tokens_pad=11)
    fill_normal(c, 9)
    _run(c, 4 * kv, only=set(range(0, n_seqs, 9)) | {3, n_seqs // 2, n_seqs - 1})


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new", [1, 20, 40])
def test_sequences_that_stand_still(D, new):
    """Fewer rows than sequences: a chunk or single tokens among sequences
    without new tokens, in one kernel's hands or both's."""
    seqs = [(0, 50 + i) for i in range(40)]
    seqs[7], seqs[30] = (new, 700), (1, 300)
    c = Cache(seqs, 2, D, 32, seed=new)
    fill_normal(c, 5)
    _run(c, 12)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("seqs", [[(1, 90)], [(1, 6000)], [(130, 300), (1, 40)], [(60, 5000)]])
def test_gates_of_any_size(D, seqs):
    """Single tokens and tiles, of one CTA and joined: gates that close, that
    are infinite or no numbers."""
    c = Cache(seqs, 1, D, 32, seed=D)
    fill_normal(c, 2)
    q, gate = _queries(c, 6, 31)
    gate = gate * 4
    for i, x in enumerate([float("inf"), float("-inf"), float("nan"), 60.0, -60.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, 0.0, -0.0]):
        gate[..., i::41] = x
    out = torch.empty(c.tokens, 6, D, dtype=torch.bfloat16, device=DEV)
    ops.fp8_kv_attention(q, *c.args(), gate=gate, out=out)
    assert ops.get_status() == 0
    check_attention(c, q, gate, out, D ** -0.5)


@pytest.mark.parametrize("D", [128, 256])
def test_long_history(D):
    c = Cache([(1, 20011), (3, 9000)], 2, D, 64, seed=D)
    fill_normal(c, 4)
    _run(c, 12, std=2.0)


def test_long_chunk():
    c = Cache([(700, 1500), (1, 2000), (333, 333)], 1, 256, 64, seed=21)
    fill_normal(c, 6)
    _run(c, 6)


def test_rows_that_see_nothing():
    """Lengths below the new tokens: the first rows see no key and give zeros;
    a sequence of length 0 gives zeros alone."""
    c = Cache([(5, 2), (3, 0), (200, 100), (1, 0), (2, 40)], 2, 256, 16, seed=9)
    fill_normal(c, 2)
    out = _run(c, 12, gated=False)
    assert torch.all(out[:3] == 0) and torch.all(out[5:8] == 0) and torch.all(out[8:108] == 0)


def test_keys_out_of_sight_do_not_matter():
    """A NaN in a key or value reaches the rows that see it and no other, and in
    a value only its own dimension."""
    c = Cache([(60, 200), (1, 130)], 2, 256, 16, seed=13)
    fill_normal(c, 5)
    at = c.slots(0)
    c.k_pages[at[0][180], at[1][180], 0] = 0x7F
    c.v_pages[at[0][170], at[1][170], 1, 37] = 0xFF
    c.v_pages[at[0][199], at[1][199], 0, 255] = 0x7F
    out = _run(c, 4, gated=False)  # the reference places the NaN; the bounds hold elsewhere
    assert torch.isfinite(out[:30].float()).all() and torch.isfinite(out[60:].float()).all()


def test_single_token_with_nan_in_sight():
    """A single token sees every key: NaN in a key makes its heads NaN, in a
    value one dimension."""
    c = Cache([(1, 200), (1, 130), (1, 40)], 2, 256, 16, seed=15)
    fill_normal(c, 5)
    at = c.slots(0)
    c.k_pages[at[0][180], at[1][180], 0] = 0x7F
    at = c.slots(1)
    c.v_pages[at[0][129], at[1][129], 1, 37] = 0xFF
    out = _run(c, 4, gated=False)
    assert torch.isnan(out[0, :2].float()).all() and int(torch.isnan(out.float()).sum()) == 2 * 256 + 2


def test_queries_that_are_not_finite():
    c = Cache([(4, 40), (1, 300)], 1, 128, 16, seed=17)
    fill_normal(c, 5)
    q, _ = _queries(c, 3, 1)
    q = q.clone()
    q[1, 0, 5], q[2, 1, 6] = float("nan"), float("inf")
    out = torch.empty_like(q)
    ops.fp8_kv_attention(q, *c.args(), out=out)
    bad = torch.isnan(out).all(-1)
    assert bool(bad[1, 0]) and bool(bad[2, 1]) and int(torch.isnan(out).any(-1).sum()) == 2


@pytest.mark.parametrize("std,k_std", [(1e-3, 1.0), (8.0, 2.0), (40.0, 2.0)])
def test_flat_and_sharp_scores(std, k_std):
    c = Cache([(1, 3000), (40, 900)], 2, 256, 64, seed=19)
    fill_normal(c, 7, k_std=k_std)
    _run(c, 8, std=std)


def test_single_token_queries_that_are_not_finite():
    c = Cache([(1, 300), (1, 40)], 1, 128, 16, seed=18)
    fill_normal(c, 5)
    q, _ = _queries(c, 3, 1)
    q = q.clone()
    q[0, 0, 5], q[1, 2, 6] = float("nan"), float("-inf")
    out = ops.fp8_kv_attention(q, *c.args())
    bad = torch.isnan(out).all(-1)
    assert bool(bad[0, 0]) and bool(bad[1, 2]) and int(torch.isnan(out).any(-1).sum()) == 2


@pytest.mark.parametrize("place", [0, 5, 1500, 2999])
def test_one_key_far_above_the_others(place):
    """A sink: one key's score tens of units above the rest, anywhere in a long
    history; the others still count by their sum."""
    D = 256
    c = Cache([(1, 3000), (30, 3000)], 1, D, 64, seed=23)
    g = gen(place)
    lean = torch.randn(D, generator=g, device=DEV)
    for b in range(2):
        k = torch.randn(3000, 1, D, generator=g, device=DEV) * 0.4
        k[place, 0] = lean * 0.75
        c.fill(b, k, torch.randn(3000, 1, D, generator=g, device=DEV))
    q = (torch.randn(31, 6, D, generator=g, device=DEV) * 0.3 + lean).to(torch.bfloat16)
    _run(c, 6, q=q)


def test_scores_that_fall_and_rise():
    """Scores that drift by more than 2^40 between blocks of keys, both ways."""
    D = 128
    c = Cache([(2, 2000)], 1, D, 16, seed=29)
    lean = torch.zeros(D, device=DEV)
    lean[0] = 4.0
    t = torch.arange(2000, device=DEV)
    k = torch.randn(2000, 1, D, generator=gen(1), device=DEV) * 0.3
    k[:, 0] += torch.cos(t / 300.0)[:, None] * lean
    c.fill(0, k, torch.randn(2000, 1, D, generator=gen(2), device=DEV))
    q = (torch.randn(2, 4, D, generator=gen(3), device=DEV) * 0.3).to(torch.bfloat16)
    q[:, :, 0] = 130.0
    _run(c, 4, q=q)


def test_outlier_channels():
    c = Cache([(3, 500)], 2, 256, 16, seed=31)
    fill_normal(c, 3)
    q, _ = _queries(c, 4, 9)
    q = q.clone()
    q[:, :, ::50] *= 60
    _run(c, 4, q=q)


def test_amax_of_the_output():
    c = Cache([(5, 60), (1, 300)], 2, 128, 16, seed=37, tokens_pad=4)
    fill_normal(c, 3)
    amax = torch.full((64,), 0x7FFF, dtype=torch.int32, device=DEV)
    out = _run(c, 8, out_amax=amax)
    want = out[:c.total].abs().max().view(torch.int16)
    assert int(amax[0]) == int(want) and torch.all(amax[1:] == 0x7FFF)


def test_strided_output_and_repeated_calls():
    c = Cache(RAGGED, 2, 256, 16, seed=41, tokens_pad=2)
    fill_normal(c, 3)
    q, gate = _queries(c, 12, 4)
    want = ops.fp8_kv_attention(q, *c.args(), gate=gate)
    wide = torch.full((c.tokens, 12, 272), 5.0, device=DEV).to(torch.bfloat16)
    for _ in range(3):
        ops.fp8_kv_attention(q, *c.args(), gate=gate, out=wide[:, :, 8:264])
        assert torch.equal(wide[:c.total, :, 8:264], want[:c.total])
    assert torch.all(wide[:, :, :8] == 5) and torch.all(wide[:, :, 264:] == 5) and torch.all(wide[c.total:] == 5)


def test_workspace_holds_nothing():
    """The workspace is scratch: any content before, and exactly the size asked for."""
    c = Cache([(1, 4000), (40, 700)], 2, 256, 64, seed=43)
    fill_normal(c, 3)
    need = ops.fp8_kv_attention_workspace_bytes(c.tokens, 12, 2, 256)
    raw = torch.empty(need + 8192, dtype=torch.uint8, device=DEV)
    got = []
    for fill in (0, 0xFF, 0x7F):
        raw.fill_(fill)
        got.append(_run(c, 12, ws=raw[4096:4096 + need]))
        assert torch.all(raw[:4096] == fill) and torch.all(raw[4096 + need:] == fill)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_no_tokens_and_no_sequences():
    c = Cache([(1, 40)], 2, 128, 16, seed=47)
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert ops.fp8_kv_attention(none, *c.args()[:5], zero, c.lens).shape == none.shape
    q = torch.ones(3, 4, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 2.0)
    amax = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    ops.fp8_kv_attention(q, *c.args()[:4], c.table[:0], zero[:1], c.lens[:0], out=out, out_amax=amax)
    ops.fp8_kv_attention(q, *c.args()[:5], zero, c.lens, out=out)
    assert ops.get_status() == 0 and torch.all(out == 2) and int(amax) == 0


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
@pytest.mark.parametrize("which", [0, 1])
def test_invalid_scale(bad, which):
    c = Cache([(1, 300)], 2, 128, 16, seed=4)
    fill_normal(c, 3)
    (c.k_scale, c.v_scale)[which].fill_(bad)
    q, _ = _queries(c, 4, 4)
    out = torch.full((1, 4, 128), 3.0, device=DEV).to(torch.bfloat16)
    ops.fp8_kv_attention(q, *c.args(), out=out)
    assert ops.get_status() == 6 and ops.get_status() == 0
    assert torch.all(out == 3)


def test_bad_pages_lengths_and_offsets():
    c = Cache([(2, 20), (3, 400), (1, 50)], 2, 128, 16, seed=6)
    fill_normal(c, 1)
    q, _ = _queries(c, 8, 3)
    for broken in ("negative", "too large", "length", "offsets"):
        table, cu, lens = c.table.clone(), c.cu.clone(), c.lens.clone()
        if broken == "negative":
            table[1] = -1
        elif broken == "too large":
            table[1] = c.n_pages
        elif broken == "length":
            lens[1] = 1 << 30
        else:
            cu[3] = 1 << 20
        out = torch.zeros(c.tokens, 8, 128, device=DEV).to(torch.bfloat16)
        ops.fp8_kv_attention(q, *c.args()[:4], table, cu, lens, out=out)
        assert ops.get_status() == 1, broken
        check_attention(c, q, None, out, 128 ** -0.5, only={0} if broken == "offsets" else {0, 2})


def test_far_pages():
    """Pages behind 2^32 bytes of one pool."""
    c = Cache([(1, 500), (9, 200)], 4, 256, 128, seed=51)
    fill_normal(c, 1)
    n = (1 << 32) // (128 * 4 * 256) + c.n_pages
    for name in ("k_pages", "v_pages"):
        pool = torch.zeros(n, 128, 4, 256, dtype=torch.uint8, device=DEV)
        pool[n - c.n_pages:] = getattr(c, name)
        setattr(c, name, pool)
    c.table += n - c.n_pages
    c.n_pages = n
    _run(c, 24)


def test_other_stream():
    c = Cache(RAGGED, 2, 256, 16, seed=53)
    fill_normal(c, 2)
    q, gate = _queries(c, 12, 2)
    want = ops.fp8_kv_attention(q, *c.args(), gate=gate)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ops.fp8_kv_attention(q, *c.args(), gate=gate, stream=side)
    side.synchronize()
    assert torch.equal(got[:c.total], want[:c.total])


def test_calls_on_two_streams_at_once():
    c = [Cache([(1, 3000 + 500 * i), (50, 400)], 2, 256, 64, seed=60 + i) for i in range(2)]
    qs, want = [], []
    for x in c:
        fill_normal(x, 2)
        qs.append(_queries(x, 12, 2)[0])
        want.append(ops.fp8_kv_attention(qs[-1], *x.args()).clone())
    streams = [torch.cuda.Stream() for _ in c]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, q, s, o in zip(c, qs, streams, outs):
            with torch.cuda.stream(s):
                ops.fp8_kv_attention(q, *x.args(), out=o)
    torch.cuda.synchronize()
    assert ops.get_status() == 0
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_graphs_that_share_a_workspace():
    """Two captured graphs over one workspace, replayed in turn with lengths
    and pages that changed since the capture."""
    c = [Cache([(1, 900), (1, 2000)], 2, 256, 64, seed=70), Cache([(30, 500), (1, 1000)], 2, 256, 64, seed=71)]
    need = max(ops.fp8_kv_attention_workspace_bytes(x.tokens, 12, 2, 256) for x in c)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    qs, outs, graphs = [], [], []
    for x in c:
        fill_normal(x, 2)
        qs.append(_queries(x, 12, 2)[0])
        outs.append(torch.zeros(x.tokens, 12, 256, device=DEV).to(torch.bfloat16))
    for x, q, o in zip(c, qs, outs):
        ops.fp8_kv_attention(q, *x.args(), out=o, ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.fp8_kv_attention(q, *x.args(), out=o, ws=ws)
        graphs.append(g)
    for step in range(3):
        for i, x in enumerate(c):
            x.seqs = [(new, n - 100 * step) for new, n in x.seqs]
            x.lens.copy_(torch.tensor([n for _, n in x.seqs], dtype=torch.int32))
            x.k_pages.copy_(x.k_pages.roll(1, 0))
            x.v_pages.copy_(x.v_pages.roll(1, 0))
            x.table.copy_(torch.where(x.table < x.n_pages, (x.table + 1) % x.n_pages, x.table))
            graphs[i].replay()
            x.seqs = [tuple(s) for s in x.seqs]
        torch.cuda.synchronize()
        assert ops.get_status() == 0
        for x, q, o in zip(c, qs, outs):
            check_attention(x, q, None, o, 256 ** -0.5)
    del graphs


def test_attention_layer_end_to_end():
    """The operators as a layer runs them: fused q/k/v projection, head norm and
    rotation, append, attention with the gate and max|out|, quantization of the
    output by it, output projection; prefill in two chunks, then single tokens.
    Each step is held to its reference on the step's own input."""
    Hq, Hk, D, rot, K = 6, 2, 256, 64, 512
    from nvfp4_w4a4_quantized_act_b200 import workloads as wl
    segs = wl.segments_from_widths([Hq * 2 * D, Hk * D, Hk * D])
    w_qkv = ops.quantize_weights(wl.weight_normal(segs[-1][1], K, 0.05, 1).to(DEV), segs)
    w_o = ops.quantize_weights(wl.weight_normal(K, Hq * D, 0.02, 2).to(DEV))
    qn, kn = [(torch.randn(D, generator=gen(i), device=DEV) * 0.2).to(torch.bfloat16) for i in (1, 2)]
    f = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)
    c = Cache([(0, 300), (0, 200)], Hk, D, 32, seed=80)
    done = [0, 0]
    for news in ([150, 90], [140, 101], [1, 1], [1, 1]):
        T = sum(news)
        done = [a + b for a, b in zip(done, news)]
        c.seqs = list(zip(news, done))
        c.ends = [0, news[0], T]
        c.total = c.tokens = T
        c.cu.copy_(torch.tensor(c.ends, dtype=torch.int32))
        c.lens.copy_(torch.tensor(done, dtype=torch.int32))
        pos = torch.cat([c.positions(0), c.positions(1)]).to(torch.int32)
        x = wl.activation_normal(T, K, sum(done)).to(DEV)
        y = ops.linear_fused(x, w_qkv)
        qg = y[:, :Hq * 2 * D].view(T, Hq, 2 * D)
        k, v = (y[:, a:b].view(T, Hk, D) for a, b in segs[1:])
        q, _ = ops.qk_norm_rope(qg[:, :, :D], None, pos, f, qn, plus_one=True)
        ops.fp8_kv_append(k, v, *c.args(), inv_freq=f, k_weight=kn, plus_one=True)
        qws = torch.zeros(ops.quant_workspace_bytes(1), dtype=torch.uint8, device=DEV)
        o = ops.fp8_kv_attention(q, *c.args(), gate=qg[:, :, D:], out_amax=qws)
        codes, sf, g = ops.quantize_act(o.view(T, Hq * D), ws=qws, amax_given=True)
        ops.gemm_prequant(codes, sf, g, T, Hq * D, w_o)
        assert ops.get_status() == 0
        check_attention(c, q, qg[:, :, D:], o, D ** -0.5)
        codes2, sf2, g2 = ops.quantize_act(o.view(T, Hq * D))
        assert torch.equal(codes, codes2) and torch.equal(sf, sf2) and torch.equal(g, g2)
