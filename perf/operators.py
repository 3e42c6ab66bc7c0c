"""The attention layer's operators over a paged FP8 (E4M3) cache: their plain forms in torch, and the same calls through the library.

`run` computes one pass of a case, in 32 bits with elementary torch operations, or, with `own`, through
nvfp4_w4a4_quantized_act_b200.ops.  Three operators, in the order a layer runs them:

  norm_rope   RMS norm of every query and key head and the position rotation of their first `rot` dimensions
  append      keys normalised and rotated the same way, then keys and values rounded to E4M3 into the pages of their sequences
  attend      causal attention of the new tokens over the pages of their sequences (one new token each: decode), times sigmoid(gate)

Token j of a sequence with `new` new tokens and length `len` (new ones included) sits at position len - new + j.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0
PAD = 3  # rows behind the last sequence in the batched cases: a serving batch is padded to a captured size


# ------------------------------------------------------------------ cases

def listed():
    layer = {"q_heads": 24, "kv_heads": 4, "head_dim": 256, "rot": 64}  # the stack's attention layer
    return [
        # a decode step of one user: nothing but latency
        {"name": "norm_rope 1 token", "op": "norm_rope", "tokens": 1, **layer},
        # a prefill of the benchmark's length
        {"name": "norm_rope 8192 tokens", "op": "norm_rope", "tokens": 8192, **layer},
        # an odd number of tokens in a narrower layer, every dimension rotated
        {"name": "norm_rope 1337 tokens", "op": "norm_rope", "tokens": 1337, "q_heads": 16, "kv_heads": 2, "head_dim": 128, "rot": 128},
        # a decode step of 64 users at different positions
        {"name": "append 64 tokens", "op": "append", "batch": 64, "new": 1, "chunks": 0, "length": 8192, "page": 16, "mix": 1, **layer},
        # a whole prompt at once
        {"name": "append 8192 tokens", "op": "append", "batch": 1, "new": 8192, "chunks": 1, "length": 8192, "page": 64, "mix": 0, **layer},
        # prompts and single tokens together
        {"name": "append mixed", "op": "append", "batch": 19, "new": 601, "chunks": 5, "length": 2500, "page": 32, "mix": 2,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128},
        # the smallest attention: one user, one token, a short history
        {"name": "attend 1 x 777", "op": "attend", "batch": 1, "new": 1, "chunks": 0, "length": 777, "page": 16, "mix": 0, **layer},
        # a decode step of 64 users with histories of up to 8192 tokens
        {"name": "attend 64 x 8192", "op": "attend", "batch": 64, "new": 1, "chunks": 0, "length": 8192, "page": 64, "mix": 3, **layer},
        # two users with very long histories
        {"name": "attend 2 x 131072", "op": "attend", "batch": 2, "new": 1, "chunks": 0, "length": 131072, "page": 128, "mix": 0, **layer},
        # chunked prefill: the next chunk of four long prompts
        {"name": "attend chunks of 509", "op": "attend", "batch": 4, "new": 509, "chunks": 4, "length": 16384, "page": 32, "mix": 4, **layer},
        # a whole prompt of the benchmark's length
        {"name": "attend prompt of 8192", "op": "attend", "batch": 1, "new": 8192, "chunks": 1, "length": 8192, "page": 64, "mix": 0, **layer},
        # a chunk of one prompt beside the single tokens of 23 users, in a narrower layer
        {"name": "attend mixed", "op": "attend", "batch": 24, "new": 1000, "chunks": 1, "length": 4000, "page": 16, "mix": 5,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice([(24, 4, 256), (16, 2, 256), (14, 2, 256), (8, 8, 256), (32, 8, 128), (15, 3, 128), (16, 1, 128)])
    case = {"op": rng.choice(["norm_rope", "append", "attend", "attend"]), "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rot": rng.choice([32, 64, 96, 128])}
    if case["op"] == "norm_rope":
        return {**case, "tokens": _log_int(rng, 1, 8192)}
    case["page"] = rng.choice([16, 32, 64, 128])
    case["mix"] = rng.randrange(1, 1 << 20)
    case["batch"] = _log_int(rng, 1, 64)
    if rng.random() < 0.5:  # a decode step, or the few tokens of a speculative one
        case["new"] = rng.choice([1, 1, 1, 2, 4])
        case["chunks"] = case["batch"]
        case["length"] = _log_int(rng, 1, min(131072, 500_000 // case["batch"]))
    else:
        case["new"] = _log_int(rng, 2, 8192 // case["batch"])
        case["chunks"] = rng.randint(1, case["batch"])
        most = min(1_500_000_000 // (case["batch"] * q_heads * case["new"]),         # the plain form's matrix of scores is kept to 6 GB,
                   800_000_000_000 // (4 * head_dim * q_heads * case["new"] * case["batch"]),  # the work to the listed prompt's
                   500_000 // case["batch"])
        case["length"] = _log_int(rng, case["new"], max(case["new"], min(32768, most)))
    return case


def _lengths(case):
    """(new tokens, length) of every sequence: all alike for mix 0, else spread up to the case's with the first at the largest."""
    rng = random.Random(case["mix"])
    got = []
    for b in range(case["batch"]):
        length = case["length"] if b == 0 or case["mix"] == 0 else _log_int(rng, max(1, case["length"] // 8), case["length"])
        new = case["new"] if b < case["chunks"] else 1
        if b and case["mix"] and new > 8:
            new = rng.randint(new // 2, new)
        got.append((min(new, length), length))
    return got


# ------------------------------------------------------------------ inputs

def _freqs(rot):
    """The usual inverse frequencies of a long-context model."""
    return (1e7 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    s = {"op": case["op"], "eps": EPS, "inv_freq": _freqs(case["rot"])}
    if case["op"] == "norm_rope":
        T = case["tokens"]
        # the fused projection's output: query and gate of each head side by side, then the keys and values of the layer
        y = normal(T, Hq * 2 * D + 2 * Hk * D, std=0.7)
        y[:, ::97] *= 8.0  # channels that stand out
        y = y.to(torch.bfloat16)
        s["q"] = y[:, : Hq * 2 * D].view(T, Hq, 2 * D)[:, :, :D]
        s["k"] = y[:, Hq * 2 * D: Hq * 2 * D + Hk * D].view(T, Hk, D)
        s["q_weight"], s["k_weight"] = (normal(D, std=0.2).to(torch.bfloat16) for _ in range(2))  # norms around 1: w = 1 + weight
        first = int(torch.randint(0, 200_000, (1,), generator=g, device=DEV))
        s["positions"] = torch.arange(first, first + T, device=DEV, dtype=torch.int32)
        s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.zeros(T, Hk, D, dtype=torch.bfloat16, device=DEV)
        return s

    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    T, page = total + PAD, case["page"]
    used = [-(-length // page) for _, length in lens]
    n_pages = sum(used) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)  # pages lie anywhere in the pool
    table = torch.zeros(len(lens), max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at: at + n]
        at += n
    ends = [0]
    for n, _ in lens:
        ends.append(ends[-1] + n)
    s.update(total=total, new_max=max(n for n, _ in lens), len_max=max(length for _, length in lens), table=table,
             cu=torch.tensor(ends, dtype=torch.int32, device=DEV),
             lens=torch.tensor([length for _, length in lens], dtype=torch.int32, device=DEV),
             k_scale=torch.tensor([7.5 / E4M3_MAX], device=DEV), v_scale=torch.tensor([4.5 / E4M3_MAX], device=DEV))

    def codes(std):
        c = torch.empty(n_pages, page, Hk, D, dtype=torch.uint8, device=DEV)
        for i in range(0, n_pages, 4096):
            x = normal(min(4096, n_pages - i), page, Hk, D, std=std).clamp_(-E4M3_MAX, E4M3_MAX)
            c[i: i + 4096] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    s["k_pages"], s["v_pages"] = codes(E4M3_MAX / 7.5), codes(E4M3_MAX / 4.5)
    if case["op"] == "append":
        kv = normal(T, 2 * Hk * D, std=0.9).to(torch.bfloat16)
        s["k"], s["v"] = kv[:, : Hk * D].view(T, Hk, D), kv[:, Hk * D:].view(T, Hk, D)
        s["k_weight"] = normal(D, std=0.2).to(torch.bfloat16)
        return s
    # queries lean towards one direction, and the first key of every sequence lies along it: the sink that trained layers have
    lean = normal(Hk, 1, D)
    qg = normal(T, Hq, 2 * D)
    qg[:, :, :D] = 1.3 * qg[:, :, :D] + 0.5 * lean.expand(Hk, Hq // Hk, D).reshape(Hq, D)
    qg = qg.to(torch.bfloat16)
    s["q"], s["gate"] = qg[:, :, :D], qg[:, :, D:]
    sink = (lean[:, 0] * (E4M3_MAX / 7.5)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k_pages"][table[:, 0].long(), 0] = sink
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["ws"] = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)  # the scratch that a serving program keeps for all its layers
    return s


# ------------------------------------------------------------------ plain forms

def _norm(x, w, eps):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (1.0 + w.float())


def _rotate(y, positions, inv_freq):
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()  # far positions: the angle in 64 bits
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = y[..., :half], y[..., half: 2 * half]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., 2 * half:]], -1)


def _rows(s):
    """Sequence and index within it of every token that belongs to one."""
    t = torch.arange(s["total"], device=DEV)
    b = (t[:, None] >= s["cu"][1:].long()).sum(1)
    return b, t - s["cu"].long()[b]


def _codes(y, scale):
    return (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_norm_rope(s):
    s["q_out"][:] = _rotate(_norm(s["q"], s["q_weight"], s["eps"]), s["positions"], s["inv_freq"]).to(torch.bfloat16)
    s["k_out"][:] = _rotate(_norm(s["k"], s["k_weight"], s["eps"]), s["positions"], s["inv_freq"]).to(torch.bfloat16)
    return [s["q_out"], s["k_out"]]


def _plain_append(s):
    b, j = _rows(s)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = s["lens"].long()[b] - new[b] + j
    page = s["k_pages"].shape[1]
    at = s["table"][b, pos // page].long(), pos % page
    n = s["total"]
    s["k_pages"][at] = _codes(_rotate(_norm(s["k"][:n], s["k_weight"], s["eps"]), pos, s["inv_freq"]), s["k_scale"])
    s["v_pages"][at] = _codes(s["v"][:n].float(), s["v_scale"])
    return [s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn)]


def _plain_attend(s):
    T, Hq, D = s["q"].shape
    page, Hk = s["k_pages"].shape[1:3]
    B, n, P = s["lens"].numel(), s["new_max"], -(-s["len_max"] // page)
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(n, device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=T - 1)].float()                              # [B, n, Hq, D], padded
    q = q.view(B, n, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    ids = s["table"][:, :P].long()
    key = torch.arange(P * page, device=DEV)
    k = s["k_pages"][ids].view(torch.float8_e4m3fn).float().view(B, P * page, Hk, D).permute(0, 2, 3, 1) * s["k_scale"]
    score = torch.matmul(q, k) * s["scale"]
    del k
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i                                         # [B, n]
    hidden = key > pos[:, :, None]
    score.view(B, Hk, n, Hq // Hk, -1).masked_fill_(hidden[:, None, :, None], float("-inf"))
    score -= score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.exp_()
    v = s["v_pages"][ids].view(torch.float8_e4m3fn).float().view(B, P * page, Hk, D) * s["v_scale"]
    v = torch.where((key < lens[:, None])[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    o = o.view(B, Hk, n, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    m = s["total"]
    s["out"][:m] = (o[_rows(s)] * torch.sigmoid(s["gate"][:m].float())).to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------ the library's calls

def _own_norm_rope(s):
    from nvfp4_w4a4_quantized_act_b200 import ops
    return ops.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], eps=s["eps"], plus_one=True,
                            q_out=s["q_out"], k_out=s["k_out"])


def _own_append(s):
    from nvfp4_w4a4_quantized_act_b200 import ops
    ops.fp8_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["cu"], s["lens"],
                      inv_freq=s["inv_freq"], k_weight=s["k_weight"], eps=s["eps"], plus_one=True)
    return [s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn)]


def _own_attend(s):
    from nvfp4_w4a4_quantized_act_b200 import ops
    return ops.fp8_kv_attention(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["cu"], s["lens"],
                                softmax_scale=s["scale"], gate=s["gate"], out=s["out"], ws=s["ws"])


def run(state):
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "attend": _own_attend}[state["op"]](state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attend": _plain_attend}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    Hq, Hk, D, half = case["q_heads"], case["kv_heads"], case["head_dim"], case["rot"] // 2
    if case["op"] == "norm_rope":
        rows = case["tokens"] * (Hq + Hk)
        return {"bytes": rows * D * 4 + case["tokens"] * 4 + 4 * D + 4 * half, "flops": rows * (4 * D + 6 * half)}
    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    if case["op"] == "append":
        return {"bytes": total * Hk * D * 2 * 3 + total * 8, "flops": total * Hk * (6 * D + 6 * half)}
    pairs = sum(n * (length - n) + n * (n + 1) // 2 for n, length in lens)
    return {"bytes": sum(length for _, length in lens) * Hk * D * 2 + total * Hq * D * 6, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_head(x, w, pos, inv_freq, eps):
    """One head's rows [n, D]: norm, then each pair of the rotated dimensions as a complex number times e^(i pos f)."""
    x = x.double()
    y = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * (w.double() + 1)
    half = inv_freq.numel()
    turned = torch.complex(y[:, :half], y[:, half: 2 * half]) * torch.polar(
        torch.ones(1, dtype=torch.float64, device=DEV), torch.outer(pos.double(), inv_freq.double()))
    y[:, :half], y[:, half: 2 * half] = turned.real, turned.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hk = case["q_heads"], case["kv_heads"]
    if case["op"] == "norm_rope":
        q, k = s["q_out"].double(), s["k_out"].double()
        for h in range(Hq):
            q[:, h] = _exact_head(s["q"][:, h], s["q_weight"], s["positions"], s["inv_freq"], s["eps"])
        for h in range(Hk):
            k[:, h] = _exact_head(s["k"][:, h], s["k_weight"], s["positions"], s["inv_freq"], s["eps"])
        return [q, k]
    page = case["page"]
    cache = [s[x].view(torch.float8_e4m3fn).to(torch.float64) for x in ("k_pages", "v_pages")]
    out = s["out"].double() if case["op"] == "attend" else None
    t0 = 0
    for b, (n, length) in enumerate(_lengths(case)):
        ids = s["table"][b, : -(-length // page)].long()
        pos = torch.arange(length - n, length, device=DEV)
        rows = slice(t0, t0 + n)
        t0 += n
        for h in range(Hk):
            if out is None:
                x = _exact_head(s["k"][rows, h], s["k_weight"], pos, s["inv_freq"], s["eps"]) / s["k_scale"].double()
                cache[0][ids[pos // page], pos % page, h] = x.clamp(-E4M3_MAX, E4M3_MAX)
                cache[1][ids[pos // page], pos % page, h] = (s["v"][rows, h].double() / s["v_scale"].double()).clamp(-E4M3_MAX, E4M3_MAX)
                continue
            k, v = (c[ids, :, h].reshape(-1, case["head_dim"])[:length] * sc.double() for c, sc in zip(cache, (s["k_scale"], s["v_scale"])))
            for i in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                z = s["q"][rows, i].double() @ k.t() * s["scale"]
                z = torch.where(torch.arange(length, device=DEV) <= pos[:, None], z, -math.inf)
                out[rows, i] = torch.softmax(z, -1) @ v / (1 + torch.exp(-s["gate"][rows, i].double()))
    return cache if out is None else out
