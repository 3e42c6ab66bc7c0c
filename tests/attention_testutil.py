"""Inputs and 64-bit references of the attention layer's operators (head norm
and rotation, the paged FP8 cache, attention over it), with error bounds that
are derived from the roundings each operator makes."""
from __future__ import annotations

import math

import torch

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
U32 = 2.0 ** -24       # half a unit in the last place of fp32, relative
BF16 = 2.0 ** -8       # of bf16
E4M3_REL = 2.0 ** -4   # of E4M3
E4M3_ABS = 2.0 ** -10  # half of E4M3's smallest step


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def norm_rope_ref(x, w, pos, inv_freq, eps, plus_one):
    """(y, size) in 64 bits for x [tokens, heads, D]; size: |a| + |b| of the
    element's pair, the scale of its 32-bit errors."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (w.double() + (1.0 if plus_one else 0.0))
    size = y.abs()
    if inv_freq is not None:
        n = inv_freq.numel()
        ang = pos.double()[:, None, None] * inv_freq.double()
        a, b = y[..., :n].clone(), y[..., n:2 * n].clone()
        y[..., :n] = a * ang.cos() - b * ang.sin()
        y[..., n:2 * n] = b * ang.cos() + a * ang.sin()
        size[..., :n] = a.abs() + b.abs()
        size[..., n:2 * n] = size[..., :n]
    return y, size


# fp32 steps of norm and rotation: 8 fused terms and 5 shuffle sums under a
# square root (13 / 2), the mean, eps, root and quotient (4), two products,
# cos and sin (angle 2, function 2), two products and a sum: below 32 halves
NORM_ROPE_U = 32 * U32


class Cache:
    """A pool of pages with every slot filled with stale codes, NaN among them,
    and sequences whose pages lie at random places in it."""

    def __init__(self, seqs, heads, dim, page, seed, layout="NHD", k_scale=6.0 / 448, v_scale=5.0 / 448, tokens_pad=0,
                 spare=3):
        g = gen(seed)
        self.seqs, self.heads, self.dim, self.page = seqs, heads, dim, page
        used = [-(-max(n, 0) // page) for _, n in seqs]
        self.n_pages = sum(used) + spare
        shape = (self.n_pages, page, heads, dim) if layout == "NHD" else (self.n_pages, heads, page, dim)

        def pool():
            c = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            return c if layout == "NHD" else c.transpose(1, 2)
        self.k_pages, self.v_pages = pool(), pool()
        self.k_scale = torch.tensor([k_scale], device=DEV)
        self.v_scale = torch.tensor([v_scale], device=DEV)
        order = torch.randperm(self.n_pages, generator=g, device=DEV).to(torch.int32)
        wide = max(used + [1]) + 1
        # entries that no kernel may use: far out of range
        self.table = torch.full((max(len(seqs), 1), wide), 0x7FFFFFF0, dtype=torch.int32, device=DEV)[: len(seqs)]
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        ends = [0]
        for n, _ in seqs:
            ends.append(ends[-1] + n)
        self.total = ends[-1]
        self.tokens = self.total + tokens_pad
        self.ends = ends
        self.cu = torch.tensor(ends, dtype=torch.int32, device=DEV)
        self.lens = torch.tensor([n for _, n in seqs], dtype=torch.int32, device=DEV)

    def args(self):
        return self.k_pages, self.v_pages, self.k_scale, self.v_scale, self.table, self.cu, self.lens

    def slots(self, b, n=None):
        """(page, row) of positions 0 .. n-1 of sequence b."""
        p = torch.arange(self.seqs[b][1] if n is None else n, device=DEV)
        return self.table[b].long()[p // self.page], p % self.page

    def fill(self, b, k, v):
        """Codes of positions 0 .. of sequence b from real values [n, heads, dim]."""
        at = self.slots(b, k.shape[0])
        for pages, x, s in ((self.k_pages, k, self.k_scale), (self.v_pages, v, self.v_scale)):
            pages[at] = (x / s).clamp(-448, 448).to(E4M3).view(torch.uint8)

    def read(self, b):
        """Codes' values of sequence b in 64 bits, without the scales."""
        at = self.slots(b)
        return [p[at].view(E4M3).double() for p in (self.k_pages, self.v_pages)]

    def positions(self, b):
        new, n = self.seqs[b]
        return torch.arange(n - new, n, device=DEV)


def fill_normal(cache, seed, k_std=1.0, v_std=1.0):
    g = gen(seed)
    for b, (_, n) in enumerate(cache.seqs):
        if n > 0:
            cache.fill(b, torch.randn(n, cache.heads, cache.dim, generator=g, device=DEV) * k_std,
                       torch.randn(n, cache.heads, cache.dim, generator=g, device=DEV) * v_std)


def attention_ref(cache, b, q, gate, softmax_scale):
    """(out, tolerance) in 64 bits for sequence b's new rows q [new, heads, D].

    Tolerance, from the roundings the operator makes:
      bf16 of the result, half a step (BF16);
      each query as two E4M3 terms scaled so that the row's largest lies in
        [128, 256): off by half the smallest step, 2^-10 / 128 of the largest;
        32-bit sums of the scores: 2^-18 of the sum of magnitudes;
        both shift a score by e_s, every weight by a factor within e^(+-e_s),
        the quotient by 2 e_s of sum p |v|;
      each probability as two E4M3 terms of 8 bits together (2^-8 of it), and
        never finer than 2^-9 in units in which the 128 keys of its block, or
        the blocks before on average, sum to 32 at least: 2^-14 of the largest
        sum of a block so far;
      32-bit sums: 2^-18 of the sums of magnitudes."""
    new, n = cache.seqs[b]
    Hq = q.shape[1]
    G = Hq // cache.heads
    k, v = cache.read(b)
    f = softmax_scale * cache.k_scale.double()
    pos = cache.positions(b)
    seen = torch.arange(n, device=DEV)[None] <= pos[:, None]
    out = torch.zeros(new, Hq, cache.dim, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    if n == 0:
        return out, tol
    pad = (-n) % 128
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        qq = q[:, h].double()
        s = qq @ torch.nan_to_num(kk).t() * f
        s = torch.where(torch.isnan(kk).any(1)[None], math.nan, s)
        z = torch.where(seen, s, -math.inf)
        m = torch.nan_to_num(z, nan=math.inf).amax(1, keepdim=True)
        p = torch.exp(z - torch.where(torch.isinf(m) & (m < 0), 0.0, m))
        p = torch.where(seen, p, 0.0)
        l = p.sum(1, keepdim=True)
        vs = torch.nan_to_num(vv)
        o = p @ vs / l
        a = p @ vs.abs() / l
        # a NaN value in sight makes its dimension NaN
        o = torch.where((seen.double() @ torch.isnan(vv).double()) > 0, math.nan, o)
        block = torch.nn.functional.pad(p, (0, pad)).view(new, -1, 128).sum(-1)
        fine = block.cummax(1)[0].repeat_interleave(128, 1)[:, :n] * seen @ vs.abs() / l * 2.0 ** -14
        big, kabs = qq.abs().amax(1, keepdim=True), torch.nan_to_num(kk).abs()
        e_s = (f * (big * 2.0 ** -17 * kabs.sum(1)[None] + 2.0 ** -18 * (qq.abs() @ kabs.t()))) * seen
        e = 2 * e_s.amax(1, keepdim=True) + 2.0 ** -8 + 2.0 ** -18
        t = e * a + fine
        vsc = cache.v_scale.double()
        o, t = o * vsc, t * vsc
        if gate is not None:
            sg = torch.sigmoid(gate[:, h].double())
            o, t = o * sg, t * sg * (1 + 8 * U32) + 8 * U32 * (o * sg).abs()
        empty = (pos < 0)[:, None]
        out[:, h] = torch.where(empty, 0.0, o)
        tol[:, h] = torch.where(empty, 0.0, t + BF16 * (o.abs() + t) + 1e-37)
    return out, tol


def check(got, ref, tol, what=""):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN at other places"
    bad = ((got - ref).abs() > tol) & ~torch.isnan(ref)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: "
                             f"{float(got[i])!r} for {float(ref[i])!r}, bound {float(tol[i])!r}")


def check_attention(cache, q, gate, out, softmax_scale, before=None, only=None):
    """Every sequence's rows within their bounds; and all together within 2^-7
    in the 2-norm, twice what rounding to bf16 alone may be off: the bounds of
    single values allow for errors that all point one way."""
    off = size = 0.0
    for b, (new, _) in enumerate(cache.seqs):
        if new and (only is None or b in only):
            rows = slice(cache.ends[b], cache.ends[b + 1])
            ref, tol = attention_ref(cache, b, q[rows], None if gate is None else gate[rows], softmax_scale)
            check(out[rows], ref, tol, f"sequence {b} {cache.seqs[b]}")
            off += float(torch.nan_to_num(out[rows].double() - ref).square().sum())
            size += float(torch.nan_to_num(ref).square().sum())
    assert off <= 2.0 ** -14 * size, f"2-norm of the error {(off / size) ** 0.5:.2g} of the result's"
    if before is not None:  # rows of no sequence keep what they held
        assert torch.equal(out[cache.total:].view(torch.int16), before[cache.total:].view(torch.int16))
