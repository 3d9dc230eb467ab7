"""Plain 64-bit forms of the decoder-layer operators (rotary positions, the paged
8-bit cache, attention over it, 4-bit linears), with the error bounds the GPU tests use."""
import math

import torch

E4M3_MAX = 448.0
HALF = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}  # half a step, relative
TINY = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25, torch.float32: 2.0**-150}  # half the smallest step
U32 = 2.0**-24


def turned(d, positions, table, layout="half", backward=False):
    """The rotation of d [T][H][D] (64 bits) by its positions' rows of the table."""
    rot = 2 * table.shape[1]
    cs = table.double()[positions.long()][:, None]
    c, s = cs[..., 0], cs[..., 1] * (-1.0 if backward else 1.0)
    ia, ib = pairs(rot, layout)
    y = d.clone()
    y[..., ia], y[..., ib] = d[..., ia] * c - d[..., ib] * s, d[..., ib] * c + d[..., ia] * s
    return y


def pairs(rot, layout):
    ia = torch.arange(0, rot, 2) if layout == "interleaved" else torch.arange(rot // 2)
    return ia, ia + (1 if layout == "interleaved" else rot // 2)


def rope(x, positions, table, layout="half", backward=False):
    """(y, bound): the rotation of x [T][H][D] in 64 bits, and how far a result in
    x's type may be from it: half a step of the type, and for fp32 arithmetic two
    products and one sum, each off by 2^-24 of a value below |a| + |b| times the amplitude."""
    d = x.double()
    ia, ib = pairs(2 * table.shape[1], layout)
    amp = table.double().abs().sum(-1)[positions.long()][:, None]
    size = torch.zeros_like(d)
    size[..., ia] = size[..., ib] = (d[..., ia].abs() + d[..., ib].abs()) * amp
    y = turned(d, positions, table, layout, backward)
    return y, HALF[x.dtype] * y.abs() + 4 * U32 * size + TINY[x.dtype]


def needed_scale(amax):
    """Least 2^e, e in -100 .. 119, with amax <= 448 * 2^e (amax a 64-bit tensor)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 119)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e)


def attention(q, cache_k, cache_v, ks, vs, block_table, kv_lens, cu_q, scale, causal=True, window=0):
    """(out, lse, bound): softmax(scale q K^T) V in 64 bits, sequence by sequence.

    Bound on the output: half a step of its type, and against sum p |v|: the
    probabilities enter the product as fp16 (2^-11) and carry the error of their
    fp32 scores, and the sum l is fp32: 2^-11 more for both.  A probability below
    fp16's normal range is off by up to 2^-25 of the largest one: n 2^-25 max|v| / l."""
    T, H, D = q.shape
    hk = cache_k.shape[1]
    page = cache_k.shape[2]
    g = H // hk
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, n in enumerate(kv_lens):
        r0, r1 = cu_q[b], cu_q[b + 1]
        m = r1 - r0
        if m <= 0 or n == 0:
            continue
        ids = block_table[b, : -(-n // page)].long()
        k = (cache_k.view(torch.uint8)[ids].view(cache_k.dtype).double() * ks[ids].double()[..., None, None])
        v = (cache_v.view(torch.uint8)[ids].view(cache_v.dtype).double() * vs[ids].double()[..., None, None])
        k, v = (x.permute(1, 0, 2, 3).reshape(hk, -1, D)[:, :n] for x in (k, v))
        x = q[r0:r1].double().view(m, hk, g, D)
        s = torch.einsum("mhgd,hnd->mhgn", x, k) * scale
        at = torch.arange(n, device=q.device)
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        hidden = torch.zeros(m, n, dtype=torch.bool, device=q.device)
        if causal:
            hidden |= at > pos
        if window:
            hidden |= at <= pos - window
        s = s.masked_fill(hidden[:, None, None, :], -math.inf)
        ls = torch.logsumexp(s, -1)
        p = torch.exp(s - ls.masked_fill(ls == -math.inf, 0.0)[..., None])
        # a token that a row does not see has no part in it, whatever it holds
        seen = (~hidden).double()
        vz = torch.nan_to_num(v, nan=0.0)
        o = torch.einsum("mhgn,hnd->mhgd", p, vz)
        o = o + torch.where(torch.einsum("mn,hnd->mhd", seen, v.isnan().double()) > 0, math.nan, 0.0)[:, :, None]
        mag = torch.einsum("mhgn,hnd->mhgd", p, vz.abs())
        top = p.amax(-1, keepdim=True).clamp(min=1e-300)
        bd = 2.0**-10 * mag + n * 2.0**-25 * vz.abs().amax(1)[None, :, None] * top
        out[r0:r1], lse[r0:r1] = o.reshape(m, H, D), ls.reshape(m, H)
        bound[r0:r1] = bd.reshape(m, H, D)
    bound = bound + HALF[q.dtype] * out.nan_to_num().abs() + TINY[q.dtype]
    return out, lse, bound


def gemm4(x, codes, scales, group):
    """(y, bound): X W^T in 64 bits; bound: half a step of the type and K fp32 additions
    (and products by the scale) of 2^-24 against sum |x| |w|."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double() - 8.0
    w = c * scales.double().repeat_interleave(group, 1)
    y = x.double() @ w.T
    mag = x.double().abs() @ w.abs().T
    return y, HALF[x.dtype] * y.abs() + (w.shape[1] + 2) * U32 * mag + TINY[x.dtype]
