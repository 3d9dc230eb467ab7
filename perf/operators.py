"""Cases of the decoder-layer operators beside the hybrid linears, with their plain torch forms.

    rope     rotary positions of the query and key heads (a slice of the fused q|k|v rows), and their gradient
    append   new keys and values into a paged 8-bit cache (e4m3, one power-of-two scale per page and
             head), keys rotated on the way
    attn     attention over that cache: single tokens, ragged batches, chunks of new tokens
    gemm4    matrix-vector products (1 to 16 tokens) with 4-bit weights and group scales

Head layouts are LLaMA-2-7B's (32 query and 32 key/value heads of 128), LLaMA-3-8B's (32 and 8 of 128)
and Qwen-2.5-0.5B's (14 and 2 of 64), linear shapes theirs too, the shapes of this repository's benchmark.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -100, 119  # exponents a cache scale may take
TABLE_POSITIONS = 131072


# ---------------------------------------------------------------- cases


def listed():
    return [
        # a decode step of 16 sequences at far positions: latency
        dict(name="rope decode 16", op="rope", tokens=16, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             backward=False, dtype="bf16"),
        # a prefill of 8192 tokens with 32 key heads
        dict(name="rope prefill 8192", op="rope", tokens=8192, heads=32, kv_heads=32, dim=128, rot=128,
             interleaved=False, backward=False, dtype="bf16"),
        # the gradient through a partial, interleaved rotation, an odd number of tokens, small heads
        dict(name="rope grad 4001 partial", op="rope", tokens=4001, heads=14, kv_heads=2, dim=64, rot=32,
             interleaved=True, backward=True, dtype="fp16"),
        # a decode step: one new token for each of 64 sequences
        dict(name="append decode 64", op="append", batch=64, new_min=1, new_max=1, past_min=1, past_max=3000,
             kv_heads=8, dim=128, rot=128, page=64, interleaved=False, dtype="bf16", mix=1),
        # ragged prompts of eight sequences behind what they hold already
        dict(name="append prompts 8", op="append", batch=8, new_min=301, new_max=2000, past_min=0, past_max=1000,
             kv_heads=32, dim=128, rot=128, page=64, interleaved=False, dtype="bf16", mix=2),
        # one short chat with 32 key/value heads: latency
        dict(name="attn 1 x 1500", op="attn", batch=1, q_min=1, q_max=1, kv_min=1500, kv_max=1500, heads=32,
             kv_heads=32, dim=128, page=16, causal=True, dtype="bf16", mix=3),
        # a serving batch of ragged lengths, one of its slots empty
        dict(name="attn 64 ragged", op="attn", batch=64, q_min=1, q_max=1, kv_min=0, kv_max=8000, heads=32,
             kv_heads=8, dim=128, page=64, causal=True, dtype="bf16", mix=4),
        # one long document
        dict(name="attn 1 x 131000", op="attn", batch=1, q_min=1, q_max=1, kv_min=131000, kv_max=131000, heads=32,
             kv_heads=8, dim=128, page=64, causal=True, dtype="bf16", mix=5),
        # chunks of new tokens behind long pasts
        dict(name="attn chunks 4", op="attn", batch=4, q_min=100, q_max=512, kv_min=1000, kv_max=8000, heads=32,
             kv_heads=8, dim=128, page=32, causal=True, dtype="fp16", mix=6),
        # one token through an attention projection
        dict(name="gemm4 4096x4096 m1", op="gemm4", tokens=1, n=4096, k=4096, group=128, dtype="bf16"),
        # 16 tokens through an MLP projection
        dict(name="gemm4 14336x4096 m16", op="gemm4", tokens=16, n=14336, k=4096, group=64, dtype="fp16"),
        # one token through a vocabulary head with fine groups
        dict(name="gemm4 128000x4096 m1", op="gemm4", tokens=1, n=128000, k=4096, group=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "gemm4"])
    heads, kv_heads, dim = rng.choice([(32, 32, 128), (32, 8, 128), (14, 2, 64)])
    dtype = rng.choice(["bf16", "fp16"])
    mix = rng.randrange(1 << 30)
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    backward=rng.random() < 0.4, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "append":
        batch = _log(rng, 1, 128)
        new_max = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 12000 // batch))
        return dict(op=op, batch=batch, new_min=min(new_max, rng.choice([0, 1, 1, new_max])), new_max=new_max,
                    past_min=0, past_max=_log(rng, 1, 3000), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 0]), page=rng.choice([16, 32, 64, 128]),
                    interleaved=rng.random() < 0.5, dtype=dtype, mix=mix)
    if op == "attn":
        batch = _log(rng, 1, 128)
        kv_max = _log(rng, 1, min(131000, 256000 * 8 * 128 // (kv_heads * dim * batch)))
        q_most = min(kv_max, 600, 5_000_000 * 32 * 128 // (heads * dim * batch * kv_max))
        q_max = rng.choice([1, 1, 1, _log(rng, 1, max(1, q_most))])
        return dict(op=op, batch=batch, q_min=rng.randint(1, q_max), q_max=q_max, kv_min=rng.randint(0, kv_max),
                    kv_max=kv_max, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    causal=rng.random() < 0.8, dtype=dtype, mix=mix)
    k = 32 * _log(rng, 4, 448)
    return dict(op=op, tokens=rng.randint(1, 16), n=_log(rng, 100, min(128000, 128000 * 4096 // k)), k=k,
                group=rng.choice([g for g in (32, 64, 128) if k % g == 0]), dtype=dtype)


def _lens(case):
    """Per-sequence lengths of a case: the same for every seed."""
    rng = random.Random(case["mix"])
    lo, hi = ("past", "new") if case["op"] == "append" else ("kv", "q")
    a = [rng.randint(case[lo + "_min"], case[lo + "_max"]) for _ in range(case["batch"])]
    b = [rng.randint(case[hi + "_min"], case[hi + "_max"]) for _ in range(case["batch"])]
    if case["op"] == "attn" and case["kv_min"] == 0:
        a[0] = 0  # an empty slot
    if not sum(b):
        b[0] = 1
    return a, b


def work(case):
    op = case["op"]
    if op == "gemm4":
        m, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k / 2 + 2 * n * k / case["group"] + 2 * m * (n + k), "flops": 2 * m * n * k}
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "rope":
        t, h = case["tokens"], case["heads"] + case["kv_heads"]
        return {"bytes": 2 * size * t * h * case["dim"] + t * (4 + 4 * case["rot"]), "flops": 3 * t * h * case["rot"]}
    past, other = _lens(case)
    d, hk = case["dim"], case["kv_heads"]
    if op == "append":
        t = sum(other)
        pages = sum((p + n - 1) // case["page"] - p // case["page"] + 1 for p, n in zip(past, other) if n)
        return {"bytes": 2 * t * hk * d * (size + 1) + 8 * pages * hk + 4 * t * case["rot"],
                "flops": t * hk * (3 * case["rot"] + 4 * d)}
    seen = sum(_pairs(kv, q, case["causal"]) for kv, q in zip(past, other))
    kv = sum(past)
    return {"bytes": 2 * kv * hk * d + 8 * hk * kv / case["page"] + sum(other) * case["heads"] * (2 * size * d + 4),
            "flops": 4 * seen * case["heads"] * d}


def _pairs(kv, q, causal):
    return sum(max(0, kv - q + i + 1) for i in range(q)) if causal else kv * q


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 1)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rope_table(rot, base=500000.0, factor=8.0):
    """(cos, sin) pairs for every position, angles in 64 bits, frequencies scaled linearly for a long context."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1)) / factor
    a = torch.arange(TABLE_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack((a.cos(), a.sin()), dim=-1).to(torch.float32).contiguous()


def _cu(lens):
    return torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")


def _pages(lens, page, g):
    """A block table over a shuffled pool with a few pages to spare, and the pool's size."""
    need = [max(1, -(-n // page)) for n in lens]
    pool = sum(need) + 5
    ids = torch.randperm(pool, generator=g, device="cuda")[: sum(need)].to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    counts = torch.tensor(need, device="cuda")
    table[torch.arange(max(need), device="cuda")[None, :] < counts[:, None]] = ids
    return table, pool


def _power_of_two(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _cache(pool, kv_heads, page, dim, g):
    """Cached values of about unit size under scales of 2^-6 .. 2^-4."""
    scale = _power_of_two(torch.randint(-6, -3, (pool, kv_heads), generator=g, device="cuda"))
    x = _randn(g, pool, kv_heads, page, dim) / scale[:, :, None, None]
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "gemm4":
        m, n, k = case["tokens"], case["n"], case["k"]
        t = TYPES[case["dtype"]]
        s["x"] = _randn(g, m, k).to(t)
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = ((_randn(g, n, k // case["group"]).abs() + 0.5) * 0.005).to(torch.bfloat16)
        return s
    t, d = TYPES[case["dtype"]], case["dim"]
    if op == "rope":
        n, h, hk = case["tokens"], case["heads"], case["kv_heads"]
        s["qkv"] = _randn(g, n, (h + 2 * hk) * d).to(t)  # rows of a fused q|k|v projection
        s["q"] = s["qkv"][:, : h * d].unflatten(1, (h, d))
        s["k"] = s["qkv"][:, h * d : (h + hk) * d].unflatten(1, (hk, d))
        s["positions"] = torch.randint(0, TABLE_POSITIONS, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["table"] = _rope_table(case["rot"])
        return s
    first, second = _lens(case)
    hk, page = case["kv_heads"], case["page"]
    if op == "append":
        n = sum(second)
        qkv = _randn(g, n, (hk + 2 * hk) * d).to(t)
        s["k"] = qkv[:, hk * d : 2 * hk * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, 2 * hk * d :].unflatten(1, (hk, d))
        s["past"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        s["cu"] = _cu(second)
        s["table"] = _rope_table(case["rot"]) if case["rot"] else None
        s["block_table"], pool = _pages([a + b for a, b in zip(first, second)], page, g)
    else:
        n, h = sum(second), case["heads"]
        s["q"] = _randn(g, n, h, d).to(t)
        s["kv_lens"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        s["cu"] = _cu(second) if case["q_max"] > 1 else None
        s["block_table"], pool = _pages(first, page, g)
        s["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    s["ck"], s["sk"] = _cache(pool, hk, page, d, g)
    s["cv"], s["sv"] = _cache(pool, hk, page, d, g)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "gemm4": _plain_gemm4}[s["op"]](s)


def _run_own(s):
    import tile_sparse_gemm_b200 as tsg

    layout = "interleaved" if s.get("interleaved") else "half"
    if s["op"] == "rope":
        return tsg.patch_rope(s["q"], s["k"], s["positions"], s["table"], layout=layout, backward=s["backward"])
    if s["op"] == "gemm4":
        return tsg.patch_gemm4(s["x"], tsg.Weight4(s["codes"], s["scales"], s["group"]))
    cache = tsg.KvCache8(s["ck"], s["cv"], s["sk"], s["sv"])
    if s["op"] == "append":
        tsg.patch_kv8_append(s["k"], s["v"], cache, s["block_table"], s["past"], s["cu"], table=s["table"], layout=layout)
        return s["ck"], s["cv"], s["sk"], s["sv"]
    return tsg.patch_attn_kv8(s["q"], cache, s["block_table"], s["kv_lens"], s["cu"], causal=s["causal"],
                              workspace=s["workspace"], want_lse=True)


def _rotate(x, cs, interleaved, sign):
    """x [T][H][D] in 32 bits; cs [T][rot/2][2]: pair i turned by angle i (against it for sign -1), the rest kept."""
    rot = 2 * cs.shape[1]
    c, sn = cs[:, None, :, 0], sign * cs[:, None, :, 1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * sn, b * c + a * sn), dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y = torch.cat((a * c - b * sn, b * c + a * sn), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_rope(s):
    cs = s["table"][s["positions"].long()]
    sign = -1.0 if s["backward"] else 1.0
    return tuple(_rotate(x.float(), cs, s["interleaved"], sign).to(x.dtype) for x in (s["q"], s["k"]))


def _needed_scale(amax):
    """The least power of two (within the exponent range) that brings amax within e4m3."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    return _power_of_two(torch.where(amax > 0, e, SCALE_EXP_MIN))


def _plain_append(s):
    page, n, hk = s["page"], s["k"].shape[0], s["k"].shape[1]
    if n == 0:
        return s["ck"], s["cv"], s["sk"], s["sv"]
    t = torch.arange(n, device="cuda")
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    pos = s["past"].long()[b] + t - s["cu"].long()[b]
    where, off = s["block_table"].long()[b, pos // page], pos % page
    k = s["k"].float()
    if s["table"] is not None:
        k = _rotate(k, s["table"][pos], s["interleaved"], 1.0)
    # a page that held tokens before this call keeps a scale at least its own
    past, cap = s["past"].long(), s["block_table"].shape[1] - 1
    head = (past % page > 0) & (s["cu"][1:] > s["cu"][:-1])
    first = s["block_table"].long().gather(1, (past // page).clamp(max=cap)[:, None])[:, 0][head]
    held = (torch.arange(page, device="cuda") < (past % page)[head][:, None])[:, None, :, None]
    for x, cache, scale in ((k, s["ck"], s["sk"]), (s["v"].float(), s["cv"], s["sv"])):
        amax = torch.zeros(scale.shape, device="cuda").scatter_reduce_(
            0, where[:, None].expand(n, hk), x.abs().amax(-1), "amax")
        new = _needed_scale(amax)
        old = scale[first]
        new[first] = torch.maximum(new[first], old)
        raw = cache.view(torch.uint8)
        kept = raw[first]
        less = (kept.view(E4M3).float() * (old / new[first])[:, :, None, None]).to(E4M3).view(torch.uint8)
        raw[first] = torch.where(held, less, kept)
        scale[where] = new[where]
        y = (x / new[where][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        raw[where, :, off] = y.view(torch.uint8)
    return s["ck"], s["cv"], s["sk"], s["sv"]


def _plain_attn(s):
    q, kv_lens, h, hk, d = s["q"], s["kv_lens"].long(), s["heads"], s["kv_heads"], s["dim"]
    batch, span = kv_lens.numel(), s["block_table"].shape[1] * s["page"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(batch + 1, device="cuda")
    most, n = s["q_max"], q.shape[0]
    bt = s["block_table"].long()

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[bt].view(E4M3).float() * scale[bt][..., None, None]  # [B][P][Hk][page][D]
        return x.transpose(1, 2).reshape(batch, hk, span, d)

    t = torch.arange(n, device="cuda")
    b = torch.bucketize(t, cu[1:], right=True)
    i = t - cu[b]
    qs = torch.zeros(batch, most, h, d, device="cuda")
    qs[b, i] = q.float()
    qs = qs.view(batch, most, hk, h // hk, d).transpose(1, 2).reshape(batch, hk, most * (h // hk), d)
    score = (qs @ gathered(s["ck"], s["sk"]).transpose(2, 3)).view(batch, hk, most, h // hk, span) / math.sqrt(d)
    at = torch.arange(span, device="cuda")
    hidden = (at >= kv_lens[:, None])[:, None, :].expand(batch, most, span)
    if s["causal"]:
        q_lens = cu[1:] - cu[:-1]
        last = (kv_lens - q_lens)[:, None] + torch.arange(most, device="cuda")
        hidden = hidden | (at > last[:, :, None])
    score = score.masked_fill(hidden[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = p.view(batch, hk, -1, span) @ gathered(s["cv"], s["sv"])
    out = out.view(batch, hk, most, h // hk, d) / total.clamp(min=1e-30)
    lse = (total.log() + top)[..., 0]
    return out.transpose(1, 2).reshape(batch, most, h, d)[b, i].to(q.dtype), lse.transpose(1, 2).reshape(batch, most, h)[b, i]


def _plain_gemm4(s):
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).flatten(1)
    w = (c.float() - 8.0).unflatten(1, (-1, s["group"])) * s["scales"].float()[..., None]
    return (s["x"].float() @ w.flatten(1).T).to(s["x"].dtype)


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn, "gemm4": _exact_gemm4}[case["op"]](s)


def _turned(x, cs, interleaved, back):
    """Pairs as complex numbers times e^(i angle), or its conjugate."""
    rot = 2 * cs.shape[1]
    if rot == 0:
        return x
    turn = torch.complex(cs[..., 0], -cs[..., 1] if back else cs[..., 1])[:, None, :]
    lo = torch.arange(0, rot, 2, device="cuda") if interleaved else torch.arange(rot // 2, device="cuda")
    hi = lo + (1 if interleaved else rot // 2)
    z = torch.complex(x[..., lo], x[..., hi]) * turn
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rope(s):
    cs = s["table"].double()[s["positions"].long()]
    return tuple(_turned(x.double(), cs, s["interleaved"], s["backward"]) for x in (s["q"], s["k"]))


def _exact_append(s):
    past, cu, bt = s["past"].tolist(), s["cu"].tolist(), s["block_table"].tolist()
    page = s["page"]
    caches = [s["ck"].double(), s["cv"].double()]
    scales = [s["sk"].double(), s["sv"].double()]
    for b, p0 in enumerate(past):
        at = p0
        while at < p0 + cu[b + 1] - cu[b]:
            n = min(page - at % page, p0 + cu[b + 1] - cu[b] - at)
            rows = slice(cu[b] + at - p0, cu[b] + at - p0 + n)
            k = s["k"][rows].double()
            if s["table"] is not None:
                k = _turned(k, s["table"][at : at + n].double(), s["interleaved"], False)
            to, o = bt[b][at // page], at % page
            for x, cache, scale in zip((k, s["v"][rows].double()), caches, scales):
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 2)).clamp(min=1e-300) / E4M3_MAX)))
                need = need.clamp(2.0**SCALE_EXP_MIN, 2.0**SCALE_EXP_MAX)
                if o:
                    need = torch.maximum(need, scale[to])
                    cache[to, :, :o] *= (scale[to] / need)[:, None, None]
                scale[to] = need
                cache[to, :, o : o + n] = (x / need[None, :, None]).transpose(0, 1)
            at += n
    return (*caches, *scales)  # the caches before their rounding to 8 bits


def _exact_attn(s):
    kv_lens = s["kv_lens"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(len(kv_lens) + 1))
    h, hk, d = s["heads"], s["kv_heads"], s["dim"]
    if sum(kv_lens) * hk > 6_000_000:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(kv_lens):
        m = cu[b + 1] - cu[b]
        if n == 0 or m == 0:
            continue
        ids = s["block_table"][b, : -(-n // s["page"])].long()
        k, v = (torch.cat(list(c.view(torch.uint8)[ids].view(E4M3).double() * sc[ids].double()[..., None, None]), dim=1)[:, :n]
                for c, sc in ((s["ck"], s["sk"]), (s["cv"], s["sv"])))  # [Hk][n][D]
        for j in range(hk):
            q = s["q"][cu[b] : cu[b + 1], j * (h // hk) : (j + 1) * (h // hk)].double()
            z = torch.einsum("mgd,nd->gmn", q, k[j]) * d**-0.5
            if s["causal"]:
                z = torch.where(torch.ones(m, n, dtype=torch.bool, device="cuda").tril(n - m), z, -math.inf)
            total = torch.logsumexp(z, dim=-1)
            w = torch.exp(z - total.masked_fill(total == -math.inf, 0.0)[..., None])
            out[cu[b] : cu[b + 1], j * (h // hk) : (j + 1) * (h // hk)] = torch.einsum("gmn,nd->mgd", w, v[j])
            lse[cu[b] : cu[b + 1], j * (h // hk) : (j + 1) * (h // hk)] = total.T
    return out, lse


def _exact_gemm4(s):
    n, k, g = s["n"], s["k"], s["group"]
    y = torch.zeros(s["tokens"], n, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // k)
    for a in range(0, n, step):
        codes, scales = s["codes"][a : a + step], s["scales"][a : a + step].double()
        w = torch.empty(codes.shape[0], k, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        w -= 8.0
        w *= torch.repeat_interleave(scales, g, dim=1)
        y[:, a : a + step] = s["x"].double() @ w.T
    return y
