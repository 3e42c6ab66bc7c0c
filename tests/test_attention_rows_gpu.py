"""Head norm with rotation, and the append to the paged FP8 cache, against
64-bit references: odd sizes, head layouts, strided views, far positions,
ragged batches, pages in both layouts, stale and unused slots untouched."""
import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import ops
from attention_testutil import (DEV, E4M3, E4M3_ABS, E4M3_REL, BF16, NORM_ROPE_U, Cache, check, gen, norm_rope_ref)

pytestmark = pytest.mark.gpu


def _freqs(rot):
    return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV) if rot else None


@pytest.mark.parametrize("T,Hq,Hk,D,rot,plus", [
    (1, 24, 4, 256, 64, True), (1, 1, 1, 128, 128, False), (7, 5, 1, 256, 256, False), (33, 15, 3, 128, 16, True),
    (130, 6, 2, 256, 96, False), (5, 3, 3, 128, 0, True), (4801, 3, 1, 128, 32, True), (4737, 2, 1, 256, 240, False)])
def test_norm_rope(T, Hq, Hk, D, rot, plus):
    g = gen(T + D + rot)
    y = (torch.randn(T, Hq * 2 * D + Hk * D + 16, generator=g, device=DEV) * 3).to(torch.bfloat16)
    y[::3, ::11] *= 20
    q = y[:, :Hq * 2 * D].view(T, Hq, 2 * D)[:, :, :D]
    k = y[:, Hq * 2 * D:Hq * 2 * D + Hk * D].view(T, Hk, D)
    wq, wk = [(torch.randn(D, generator=g, device=DEV) * 0.3 + (0 if plus else 1)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    f = _freqs(rot)
    qo, ko = ops.qk_norm_rope(q, k, pos, f, wq, wk, eps=1e-6, plus_one=plus)
    assert ops.get_status() == 0
    for x, w, o in ((q, wq, qo), (k, wk, ko)):
        ref, size = norm_rope_ref(x, w, pos, f, 1e-6, plus)
        check(o, ref, BF16 * ref.abs() + NORM_ROPE_U * size + 1e-37, f"T={T}")


@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1500, 24, 4, 256, 64), (2900, 17, 3, 128, 128), (700, 19, 2, 256, 96), (3100, 33, 1, 128, 16), (400, 9, 9, 256, 0)])
def test_norm_rope_with_several_heads_a_warp(T, Hq, Hk, D, rot):
    """Long batches: a warp takes up to 8 heads (16 of 128), the last fewer."""
    test_norm_rope(T, Hq, Hk, D, rot, T % 200 == 0)


def test_no_norm_and_one_side_only():
    g = gen(3)
    q = torch.randn(9, 4, 256, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.arange(9, device=DEV, dtype=torch.int32)
    qo, ko = ops.qk_norm_rope(q, None, pos, _freqs(64))
    assert ko is None
    ref, size = norm_rope_ref(q, None, pos, _freqs(64), 0.0, False)
    check(qo, ref, BF16 * ref.abs() + NORM_ROPE_U * size)
    # neither norm nor rotation: a copy of every bit
    qo, _ = ops.qk_norm_rope(q, None, None)
    assert torch.equal(qo, q)
    # the norm of one side alone
    w = torch.full((256,), 0.5, device=DEV).to(torch.bfloat16)
    qo, ko = ops.qk_norm_rope(q, q[:, :2], pos, None, None, w)
    assert torch.equal(qo, q)
    ref, size = norm_rope_ref(q[:, :2], w, pos, None, 1e-6, False)
    check(ko, ref, BF16 * ref.abs() + NORM_ROPE_U * size)


def test_extreme_rows_and_positions():
    """A zero row stays zero, a NaN row touches no other, rows near the ends of
    bf16's range keep their size, and the angle is right at 2^31 - 1 and below
    zero."""
    D = 256
    q = torch.randn(6, 2, D, generator=gen(5), device=DEV).to(torch.bfloat16)
    q[0, 0] = 0
    q[1, 1, 7] = float("nan")
    q[2] = q[2] * 1e18
    q[3] = q[3] * 1e-18
    w = torch.ones(D, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([0, 1, 2 ** 31 - 1, 131071, -5, -(2 ** 31)], dtype=torch.int32, device=DEV)
    f = _freqs(64)
    qo, _ = ops.qk_norm_rope(q, None, pos, f, w, eps=1e-6)
    ref, size = norm_rope_ref(q, w, pos, f, 1e-6, False)
    check(qo, ref, BF16 * ref.abs() + NORM_ROPE_U * size + 1e-37)
    assert torch.all(qo[0, 0] == 0)


def test_norm_rope_in_place_and_strided_output():
    g = gen(8)
    buf = torch.randn(40, 6, 128, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.ones(128, device=DEV).to(torch.bfloat16)
    pos = torch.arange(40, device=DEV, dtype=torch.int32)
    want, want_k = ops.qk_norm_rope(buf[:, :4], buf[:, 4:], pos, _freqs(128), w, w)
    wide = torch.full((6, 44, 144), 7.0, device=DEV).to(torch.bfloat16)  # heads first, padded rows
    out = wide[:4, :40, 8:136].transpose(0, 1)
    ops.qk_norm_rope(buf[:, :4], None, pos, _freqs(128), w, q_out=out)
    assert torch.equal(out, want)
    assert torch.all(wide[:, :, :8] == 7) and torch.all(wide[:, :, 136:] == 7) and torch.all(wide[4:] == 7)
    ops.qk_norm_rope(buf[:, :4], buf[:, 4:], pos, _freqs(128), w, w, q_out=buf[:, :4], k_out=buf[:, 4:])
    assert torch.equal(buf[:, :4], want) and torch.equal(buf[:, 4:], want_k)


def test_norm_rope_no_tokens():
    q = torch.empty(0, 4, 256, device=DEV, dtype=torch.bfloat16)
    qo, _ = ops.qk_norm_rope(q, None, torch.empty(0, dtype=torch.int32, device=DEV), _freqs(64))
    assert qo.shape == q.shape and ops.get_status() == 0


RAGGED = [(3, 3), (0, 40), (1, 200), (70, 70), (0, 0), (5, 130), (1, 1), (17, 33)]


@pytest.mark.parametrize("seqs,heads,D,page,rot,layout", [
    ([(1, 1)], 4, 256, 16, 64, "NHD"), (RAGGED, 4, 256, 16, 64, "NHD"), (RAGGED, 3, 128, 32, 128, "HND"),
    (RAGGED, 1, 256, 64, 0, "HND"), ([(4900, 5000)], 1, 128, 256, 32, "NHD"), ([(1, 77 + i) for i in range(70)], 2, 128, 128, 48, "NHD")])
def test_append(seqs, heads, D, page, rot, layout):
    c = Cache(seqs, heads, D, page, seed=len(seqs) + D + rot, layout=layout, tokens_pad=5)
    g = gen(11)
    kv = (torch.randn(c.tokens, 2 * heads * D + 8, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    k, v = kv[:, :heads * D].view(c.tokens, heads, D), kv[:, heads * D:2 * heads * D].view(c.tokens, heads, D)
    k[c.total:] = float("nan")  # rows of no sequence: never read into the cache
    w = (torch.randn(D, generator=g, device=DEV) * 0.2).to(torch.bfloat16)
    f = _freqs(rot)
    before = c.k_pages.clone(), c.v_pages.clone()
    ops.fp8_kv_append(k, v, *c.args(), inv_freq=f, k_weight=w, plus_one=True)
    assert ops.get_status() == 0
    touched = torch.zeros(c.k_pages.shape[:2], dtype=torch.bool, device=DEV)
    for b, (new, n) in enumerate(seqs):
        if not new:
            continue
        rows = slice(c.ends[b], c.ends[b + 1])
        pos = c.positions(b)
        at = c.table[b].long()[pos // page], pos % page
        touched[at] = True
        ref, size = norm_rope_ref(k[rows], w, pos, f, 1e-6, True)
        s = c.k_scale.double()
        y = (ref / s).clamp(-448, 448)
        check(c.k_pages[at].view(E4M3), y, E4M3_REL * y.abs() + E4M3_ABS + (1 + E4M3_REL) * NORM_ROPE_U * size / s, f"keys of {b}")
        codes = ops.fp8_kv_quantize(v[rows].reshape(new, -1), c.v_scale)
        assert torch.equal(c.v_pages[at].reshape(new, -1), codes)
    assert torch.equal(c.k_pages[~touched], before[0][~touched])
    assert torch.equal(c.v_pages[~touched], before[1][~touched])


@pytest.mark.parametrize("seqs,heads,D", [
    ([(1300, 1300), (900, 1000)], 6, 256), ([(1500, 1600), (0, 9), (1100, 1100)], 11, 128), ([(2500, 2500)], 5, 256)])
def test_append_with_several_heads_a_warp(seqs, heads, D):
    test_append(seqs, heads, D, 64, 64, "HND")


def test_append_positions_given_and_negative_cache_positions():
    """Rotation positions of the caller's; tokens before position 0 (a length
    shorter than the new tokens) are not cached."""
    c = Cache([(4, 20), (6, 2)], 2, 128, 16, seed=1)
    k = torch.randn(10, 2, 128, generator=gen(2), device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (10,), generator=gen(3), device=DEV, dtype=torch.int32)
    f = _freqs(64)
    before = c.k_pages.clone()
    ops.fp8_kv_append(k, k, *c.args(), inv_freq=f, positions=pos)
    assert ops.get_status() == 0
    ref, size = norm_rope_ref(k, None, pos, f, 0.0, False)
    s = c.k_scale.double()
    touched = torch.zeros(c.k_pages.shape[:2], dtype=torch.bool, device=DEV)
    for b, rows, p in ((0, slice(0, 4), c.positions(0)), (1, slice(8, 10), torch.arange(2, device=DEV))):
        at = c.table[b].long()[p // 16], p % 16
        touched[at] = True
        y = (ref[rows] / s).clamp(-448, 448)
        check(c.k_pages[at].view(E4M3), y, E4M3_REL * y.abs() + E4M3_ABS + (1 + E4M3_REL) * NORM_ROPE_U * size[rows] / s)
    assert torch.equal(c.k_pages[~touched], before[~touched])


def test_append_nan_and_saturation():
    c = Cache([(3, 3)], 1, 128, 16, seed=4)
    k = torch.zeros(3, 1, 128, device=DEV, dtype=torch.bfloat16)
    k[0, 0, 0], k[0, 0, 1], k[1, 0, 2], k[2, 0, 3] = float("nan"), float("inf"), -1e30, -0.0
    ops.fp8_kv_append(k, k, *c.args())
    got = c.k_pages[c.slots(0)].view(E4M3).float()[:, 0]
    assert torch.isnan(got[0, 0]) and got[0, 1] == 448 and got[1, 2] == -448
    assert int(c.k_pages[c.slots(0)][2, 0, 3]) == 0x80


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
@pytest.mark.parametrize("which", [0, 1])
def test_append_invalid_scale(bad, which):
    c = Cache([(3, 30)], 2, 128, 16, seed=4)
    (c.k_scale, c.v_scale)[which].fill_(bad)
    before = c.k_pages.clone(), c.v_pages.clone()
    k = torch.ones(3, 2, 128, device=DEV, dtype=torch.bfloat16)
    ops.fp8_kv_append(k, k, *c.args())
    assert ops.get_status() == 6 and ops.get_status() == 0
    assert torch.equal(c.k_pages, before[0]) and torch.equal(c.v_pages, before[1])


def test_append_bad_pages_lengths_and_offsets():
    """Table entries, lengths and offsets out of range touch no memory outside
    the pages, latch the status and leave the other sequences right."""
    c = Cache([(2, 20), (3, 40), (1, 5)], 2, 128, 16, seed=6)
    k = torch.randn(6, 2, 128, generator=gen(7), device=DEV).to(torch.bfloat16)
    want = c.k_pages.clone(), c.v_pages.clone()
    ops.fp8_kv_append(k, k, want[0], want[1], *c.args()[2:])
    assert ops.get_status() == 0
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
        kp, vp = c.k_pages.clone(), c.v_pages.clone()
        ops.fp8_kv_append(k, k, kp, vp, c.k_scale, c.v_scale, table, cu, lens)
        assert ops.get_status() == 1, broken
        at = c.slots(0)
        assert torch.equal(kp[at], want[0][at]) and torch.equal(vp[at], want[1][at]), broken


def test_append_far_pages():
    """Pages behind 2^32 bytes of one pool."""
    page, heads, D = 128, 4, 256
    n = (1 << 32) // (page * heads * D) + 4
    pool = torch.zeros(n, page, heads, D, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device=DEV)
    cu, lens = torch.tensor([0, 3], dtype=torch.int32, device=DEV), torch.tensor([130], dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    k = torch.full((3, heads, D), 2.0, device=DEV).to(torch.bfloat16)
    ops.fp8_kv_append(k, k, pool, pool, one, one, table, cu, lens)
    assert ops.get_status() == 0
    assert torch.all(pool[n - 1, 127] == 0x40) and torch.all(pool[n - 2, :2] == 0x40)
    assert int(pool[n - 1, :127].max()) == 0 and int(pool[n - 2, 2:].max()) == 0 and int(pool[: n - 2].max()) == 0
