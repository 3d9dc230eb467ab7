"""The decoder-layer operators at the ends of their ranges: page scales far apart, values near a type's limits."""
import math

import pytest
import torch

import _decoder_ref as ref
import tile_sparse_gemm_b200 as tsg
from test_gpu_decoder import F8, copy_of, gen, i32, pages_of, random_cache, within

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32

# (queries per sequence, query heads, key/value heads): tiles of 8, 16 and 128 rows
TILES = [(1, 4, 2), (3, 8, 2), (90, 2, 1)]


def attention_of_own(q, c, bt, kv, m, scale, causal, window):
    """(out, lse, bound) in 64 bits; m queries a sequence.  A token's part p |v| is off by what its own
    probability is: fp16 rounds it by 2^-11 or, small beside the sequence's largest, by 2^-25 of that, never by
    more than itself; fp32 scores and sums add 2^-11 at most.  Another page's values have no part in it."""
    T, H, D = q.shape
    hk, page = c.k.shape[1:3]
    g = H // hk
    out, bound = torch.zeros(T, H, D, dtype=torch.float64, device="cuda"), torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(kv):
        at, pos = torch.arange(n, device="cuda"), torch.arange(n - m, n, device="cuda")[:, None]
        hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        hidden |= (at > pos) if causal else False
        hidden |= (at <= pos - window) if window else False
        lo = 0 if not window else max(0, n - m - window + 1)  # pages before it may be anywhere
        ids = bt[b, : -(-n // page)].long()
        ids[: lo // page] = 0
        k, v = ((x.view(torch.uint8)[ids].view(F8).double() * s[ids].double()[..., None, None]).transpose(0, 1).reshape(hk, -1, D)[:, :n]
                for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        k[:, :lo] = v[:, :lo] = 0.0
        rows = slice(b * m, (b + 1) * m)
        s = torch.einsum("mhgd,hnd->mhgn", q[rows].double().view(m, hk, g, D), k) * scale
        s = s.masked_fill(hidden[:, None, None, :].expand_as(s), -math.inf)
        ls = torch.logsumexp(s, -1)
        p = torch.exp(s - ls[..., None].nan_to_num(neginf=0.0))
        off = 2.0**-10 * p + torch.minimum(p, 2.0**-25 * p.amax(-1, keepdim=True))
        out[rows] = torch.einsum("mhgn,hnd->mhgd", p, v).reshape(m, H, D)
        bound[rows] = torch.einsum("mhgn,hnd->mhgd", off, v.abs()).reshape(m, H, D)
        lse[rows] = ls.reshape(m, H)
    return out, lse, bound + ref.HALF[q.dtype] * out.abs() + ref.TINY[q.dtype]


def attend(tile, D, dtype, edit, page=16, kv=(700, 333), causal=True, window=0, scale=None, seed=0):
    m, H, hk = tile
    g = gen(seed)
    bt, n_pages = pages_of(list(kv), page, g)
    c = random_cache(n_pages, hk, page, D, g)
    q = torch.randn(m * len(kv), H, D, generator=g, device="cuda").to(dtype)
    q = edit(q, c, bt)
    st = tsg.new_status()
    scale = 1 / math.sqrt(D) if scale is None else scale
    cu = i32([m * i for i in range(len(kv) + 1)])
    out, lse = tsg.patch_attn_kv8(q, c, bt, i32(list(kv)), cu, scale, causal, window, want_lse=True, status=st)
    assert tsg.patch_read_status(st) == (0, 0)
    want, wl, bound = attention_of_own(q, c, bt, kv, m, scale, causal, window)
    within(out, want, bound, "out")
    near = (lse.double() - wl).abs() <= 2.0**-12 * (1 + wl.abs())
    assert bool((near | (lse.double() == wl)).all())
    return out, c, bt


@pytest.mark.parametrize("far", [12, 20, 24, 40, 90, 119])
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
@pytest.mark.parametrize("tile", TILES)
def test_attn_values_under_a_large_scale_without_weight(tile, D, dtype, far):
    """A page whose values have a scale up to 2^119 and no weight to speak of: the others keep their bits."""
    def edit(q, c, bt):
        q[..., 0] = 8.0
        for b, j in ((0, 3), (0, 30), (1, 0)):
            ids = int(bt[b, j])
            c.k[ids] = torch.zeros_like(c.k[ids].float()).to(F8)
            c.k[ids, :, :, 0] = torch.full_like(c.k[ids, :, :, 0].float(), -256.0).to(F8)
            c.k_scale[ids] = 16.0  # scores of -2896 and less: probabilities of 0 in any format
            c.v_scale[ids] = 2.0**far
        return q
    attend(tile, D, dtype, edit)


@pytest.mark.parametrize("spread", [6, 15, 30, 60])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("D,dtype", [(128, FP16), (64, BF16)])
@pytest.mark.parametrize("tile", TILES)
def test_attn_values_under_scales_far_apart(tile, D, dtype, page, spread):
    """Value scales over 2^-spread .. 2^spread, page by page, each page's scores falling with its scale so that small
    ones count; elements of the large pages are zero in half of the columns, where nothing hides the small ones."""
    def edit(q, c, bt):
        g = gen(spread)
        e = torch.randint(-spread, spread + 1, c.v_scale.shape, generator=g, device="cuda").float()
        e -= max(0, spread - 6) if dtype is FP16 else 0  # results within the type
        c.v_scale.copy_(2.0**e)
        v = c.v.float()
        v[..., ::2] *= (e <= 0)[..., None, None]
        c.v.copy_(v.to(F8))
        return q
    attend(tile, D, dtype, edit, page=page, seed=1)
    attend(tile, D, dtype, edit, page=page, causal=False, seed=2)


@pytest.mark.parametrize("tile", TILES)
def test_attn_values_under_the_least_and_largest_scales(tile):
    def edit(low, high):
        def f(q, c, bt):
            c.v_scale.fill_(2.0**-5)
            c.v_scale[bt[0, ::3].long()] = low
            c.v_scale[bt[1, 1::2].long()] = high
            return q
        return f
    attend(tile, 128, BF16, edit(2.0**-100, 2.0**100), seed=3)  # pages of zeros have the least scale
    attend(tile, 64, BF16, edit(2.0**100, 2.0**-100), seed=4)

    def first(value):
        def f(q, c, bt):
            c.v_scale.fill_(2.0**-5)
            c.v_scale[bt[:, 0].long()] = value
            return q
        return f
    for value in (0.0, 2.0**-100, 2.0**-30, 2.0**30, 2.0**110):
        attend(tile, 128, BF16, first(value), seed=5)

    def alone(value):
        def f(q, c, bt):
            c.v_scale.fill_(value)
            return q
        return f
    for value in (2.0**-100, 2.0**-60, 2.0**40, 2.0**100):
        attend(tile, 64, BF16, alone(value), seed=6)


@pytest.mark.parametrize("m,H", [(1, 1), (3, 4), (90, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_queries_at_the_ends_of_bf16(m, H, D):
    """One token in view, so lse is its score: rows whose largest element is bf16's largest, 2^127, 2^126, its least
    normal and its least number at all.  A row is divided by a power of two and then off by 2^-25 (fp16) or, in
    128-row tiles, 2^-17 of its largest element, or there by 2^-136 if that is more; D fp32 additions beside."""
    g = gen(41)
    tops = [torch.finfo(BF16).max, 2.0**127, 2.0**126, 2.0**-126, 2.0**-133, -torch.finfo(BF16).max]
    B = len(tops)
    cache = random_cache(B, 1, 16, D, g)
    q = torch.zeros(B * m, H, D, dtype=BF16, device="cuda")
    for b, top in enumerate(tops):
        x = torch.rand(m, H, D, generator=g, device="cuda").double() - 0.5
        x[..., 3] = 1.0
        q[b * m : (b + 1) * m] = (x * top).to(BF16)
        cache.k_scale[b] = 2.0**100 if abs(top) < 1 else 2.0**-4
    bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    cu = i32([m * b for b in range(B + 1)])
    scales = [2.0**-122 if abs(t) > 1 else 2.0**22 for t in tops]
    for scale in sorted(set(scales)):
        st = tsg.new_status()
        out, lse = tsg.patch_attn_kv8(q, cache, bt, i32([1] * B), cu, scale, False, want_lse=True, status=st)
        assert tsg.patch_read_status(st) == (0, 0)
        for b in [b for b in range(B) if scales[b] == scale]:
            rows = slice(b * m, (b + 1) * m)
            k = cache.k[b, 0, 0].double() * cache.k_scale[b, 0].double()
            x = q[rows].double()
            bound = scale * ((2.0**-16 if m > 64 else 2.0**-24) * x.abs().amax(-1) * k.abs().sum()
                             + 2.0**-136 * k.abs().sum() + 3 * (D + 2) * 2.0**-24 * (x.abs() @ k.abs())) + 1e-30
            within(lse[rows], (x @ k) * scale, bound, f"lse {tops[b]}")
            v = (cache.v[b, 0, 0].double() * cache.v_scale[b, 0].double()).expand(m, H, D)
            within(out[rows], v, 2.0**-8 * v.abs() + 1e-30, f"out {tops[b]}")


@pytest.mark.parametrize("N,K,group", [(5000, 4096, 32), (9000, 2080, 32), (700, 12800, 64), (96, 16384 + 32, 32), (3000, 24576, 128)])
def test_gemm4_ctas_that_share_an_sm_or_not(N, K, group):
    """X, its sums and the scales take shared memory by tokens, K and group: two CTAs an SM, one, or slices of K."""
    g = gen(N)
    w = tsg.Weight4(torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                    (0.5 + torch.rand(N, K // group, generator=g, device="cuda")).to(BF16), group)
    for M in (1, 3, 4, 5, 8, 9, 13, 16):
        x = torch.randn(M, K, generator=g, device="cuda").to(FP16)
        within(tsg.patch_gemm4(x, w), *ref.gemm4(x, w.codes, w.scales, group), f"M={M}")


FAR_BELOW = 2.0**-35  # of the largest of a token's 128 elements: what one of them may be off by


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("place", range(8))
def test_gemm4_elements_far_below_the_largest(dtype, place):
    """Elements 2^-32 to 2^-34 of the largest of their 128, which has a group of its own with weights of zero: each place of
    the operand order (8 elements) in turn holds them.  Beside FAR_BELOW of the largest, fp32 sums of up to 15 |x| s and
    8 |x| s, an addition a k, each off by 2^-24."""
    N, K, group, M = 64, 512, 32, 5
    g = gen(71)
    c = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    c.view(N, -1, 64)[:, :, :16] = 0x88  # the first group of each 128 k
    w = tsg.Weight4(c, (0.5 + torch.rand(N, K // group, generator=g, device="cuda")).to(BF16), group)
    k = torch.arange(K, device="cuda")
    e = torch.randint(22, 25, (M, K), generator=g, device="cuda").double()
    x = torch.where((k % 8 == place) & (k % 128 >= 32), (1 + torch.rand(M, K, generator=g, device="cuda").double()) * 2.0**-e, 0.0)
    x[:, 5::128] = 1024.0
    x = x.to(dtype)
    y, bound = ref.gemm4(x, c, w.scales, group)
    wd = (torch.stack((c & 15, c >> 4), -1).flatten(1).double() - 8.0).abs() * w.scales.double().repeat_interleave(group, 1)
    s = w.scales.double().repeat_interleave(group, 1) * (k % 128 >= 32)
    few = (k % 8 == place).double()
    bound = bound + 2.0**-24 * 23 * (group + 2) * x.double().abs() @ s.T + FAR_BELOW * 1024.0 * few @ wd.T
    within(tsg.patch_gemm4(x, w), y, bound)


def test_gemm4_a_token_with_an_infinity_is_nan():
    g = gen(72)
    w = tsg.patch_quantize4(torch.randn(40, 256, generator=g, device="cuda"), 64)
    for dtype in (BF16, FP16):
        x = torch.randn(12, 256, generator=g, device="cuda").to(dtype)
        clean = tsg.patch_gemm4(x, w)
        x[3, 70], x[9, 255] = math.inf, -math.inf
        y = tsg.patch_gemm4(x, w)
        rest = [m for m in range(12) if m not in (3, 9)]
        assert bool(y[[3, 9]].isnan().all()) and torch.equal(y[rest], clean[rest])


def state(c):
    return [t.view(torch.uint8).clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


@pytest.mark.parametrize("many", [False, True])  # small CTAs and page-wide ones
def test_append_beyond_the_table_writes_neither_keys_nor_values(many):
    """A page with a token whose position has no angles is left as it is, keys, values and both scales; others are not."""
    page, d, hk = 16, 64, 2
    g = gen(81)
    table = tsg.patch_rope_table(40, d)
    new = 20 if many else 1
    past = [39, 40, 47, 30] if not many else [24, 32, 30]
    B = len(past)
    bt = i32([[4 * b + j for j in range(4)] for b in range(B)])
    cache = random_cache(4 * B, hk, page, d, g)
    k, v = ((4 * torch.randn(B * new, hk, d, generator=g, device="cuda")).to(BF16) for _ in range(2))
    for b, p in enumerate(past):
        was = state(cache)
        st = tsg.new_status()
        rows = slice(b * new, (b + 1) * new)
        tsg.patch_kv8_append(k[rows], v[rows], cache, bt[b : b + 1], i32([p]), i32([0, new]), table, status=st)
        bad = p + new > 40
        assert tsg.patch_read_status(st)[1] == (tsg.DEV_BOUNDS if bad else 0)
        now = state(cache)
        for q in range(4 * B):
            first, last = max(p, (q - 4 * b) * page), min(p + new, (q - 4 * b + 1) * page)  # of this call's tokens in it
            written = q // 4 == b and first < last <= 40
            for i, (x, y) in enumerate(zip(was, now)):
                same = torch.equal(x[q], y[q])
                assert same or written, (p, q, i)
                assert not (same and written and i < 2), (p, q, i)  # a scale may stay


@pytest.mark.parametrize("page,B", [(16, 1), (64, 40)])
@pytest.mark.parametrize("past,new", [(-1, 1), (-5, 3), (-20, 20), (-3, 40), (-(2**31), 1)])
def test_append_to_a_negative_length_is_refused(page, B, past, new):
    """The only wrong sequence of a call, alone or last of many: reported, nothing of it stored, the others as ever."""
    d, hk = 64, 2
    g = gen(82)
    lens, news = [3] * (B - 1) + [past], [new] * B
    bt = torch.arange(4 * B, dtype=torch.int32, device="cuda").view(B, 4)
    cache = random_cache(4 * B, hk, page, d, g)
    was, other = state(cache), copy_of(cache)
    x = torch.randn(B * new, hk, d, generator=g, device="cuda").to(BF16)
    cu = i32([new * b for b in range(B + 1)])
    st = tsg.new_status()
    tsg.patch_kv8_append(x, x, cache, bt, i32(lens), cu, status=st)
    assert tsg.patch_read_status(st)[1] == tsg.DEV_BOUNDS
    for a, b in zip(was, state(cache)):
        assert torch.equal(a[4 * (B - 1) :], b[4 * (B - 1) :])
    if B > 1:
        tsg.patch_kv8_append(x[:-new], x[:-new], other, bt[:-1].contiguous(), i32(lens[:-1]), cu[:-1])
        for a, b in zip(state(other), state(cache)):
            assert torch.equal(a[: 4 * (B - 1)], b[: 4 * (B - 1)])
    if new == 1:
        st.zero_()
        tsg.patch_kv8_append(x, x, cache, bt, i32(lens), status=st)
        assert tsg.patch_read_status(st)[1] == tsg.DEV_BOUNDS
    st.zero_()  # no new tokens: nothing to refuse
    tsg.patch_kv8_append(x[:0], x[:0], cache, bt, i32(lens), i32([0] * (B + 1)), status=st)
    assert tsg.patch_read_status(st) == (0, 0)


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("window", [1, 37, 150])
def test_attn_pages_before_the_window(window, tile, D, page):
    """Pages that no query sees any more may have been given back: their ids are anything, without a report, or theirs
    are pages of others, full of NaN under any scale."""
    m, kv = tile[0], (700, 333)
    for spoilt in (-1, 2**31 - 1, None):
        def edit(q, c, bt):
            for b, n in enumerate(kv):
                gone = max(0, n - m - window + 1) // page
                if spoilt is not None:
                    bt[b, :gone] = spoilt
                else:
                    ids = bt[b, :gone].long()
                    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
                        x.view(torch.uint8)[ids] = 0x7F
                        s[ids] = math.inf
            return q
        attend(tile, D, BF16, edit, page=page, kv=kv, window=window)


def test_quantize4_weights_beyond_a_fp16_scale():
    """amax / 7 above 65504: the scale is fp16's largest number, the weights saturate, zeros stay zeros."""
    w = torch.zeros(3, 128, device="cuda")
    w[0, :4] = torch.tensor([1e6, -1e6, 3e5, -4e4])
    w[1, 5:7] = torch.tensor([3.4e38, -3.4e38])
    w[2, 0] = 458528.0  # 7 times the largest scale
    q = tsg.patch_quantize4(w, 64, FP16)
    c = torch.stack((q.codes & 15, q.codes >> 4), -1).flatten(1).int() - 8
    assert bool((q.scales[:, 0] == 65504.0).all()) and bool((q.scales[:, 1] == 0.0).all())
    want = torch.zeros_like(c)
    want[0, :4] = torch.tensor([7, -8, 5, -1], dtype=torch.int32)
    want[1, 5:7] = torch.tensor([7, -8], dtype=torch.int32)
    want[2, 0] = 7
    assert torch.equal(c, want)
    x = torch.zeros(1, 128, dtype=BF16, device="cuda")
    x[0, 10] = 1.0
    assert not tsg.patch_gemm4(x, q).any()
    assert torch.equal(tsg.patch_quantize4(w, 64, BF16).scales[:, 0].float(), (w[:, :64].abs().amax(1) / 7).to(BF16).float())


@pytest.mark.parametrize("kv,m,H,hk,D,dtype", [([1500], 1, 32, 32, 128, BF16), ([100 + 233 * i for i in range(30)], 1, 32, 8, 128, BF16),
                                               ([90000], 1, 32, 8, 128, FP16), ([3000, 50, 4321], 9, 14, 2, 64, BF16),
                                               ([1000, 5000], 300, 32, 8, 128, FP16)])
def test_attn_repeats_itself(kv, m, H, hk, D, dtype):
    """Tiles are cut between warps and CTAs, whose parts are joined in their order, whoever comes last: the same bits."""
    g = gen(91)
    bt, n_pages = pages_of(kv, 32, g)
    c = random_cache(n_pages, hk, 32, D, g)
    q = torch.randn(m * len(kv), H, D, generator=g, device="cuda").to(dtype)
    args = (q, c, bt, i32(kv), i32([m * i for i in range(len(kv) + 1)]))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    out, lse = tsg.patch_attn_kv8(*args, want_lse=True)
    for i in range(12):
        if i % 2:
            flush.fill_(i)
        again, l = tsg.patch_attn_kv8(*args, want_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, l)


def test_gemm4_k_whose_x_passes_32_bits():
    """16 tokens of 2^26 and a few k: X has 2^31 bytes and more, taken in slices; a token at a time in 64 bits."""
    N, K, group, M = 3, 2**26 + 128, 128, 16
    g = gen(101)
    w = tsg.Weight4(torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                    (0.5 + torch.rand(N, K // group, generator=g, device="cuda")).to(BF16), group)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float16)
    st = tsg.new_status()
    y = tsg.patch_gemm4(x, w, status=st)
    assert tsg.patch_read_status(st) == (0, 0)
    for m in (0, 7, 15):
        want, mag = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
        for k0 in range(0, K, 1 << 23):
            k1 = min(K, k0 + (1 << 23))
            c, s = w.codes[:, k0 // 2 : k1 // 2], w.scales[:, k0 // group : k1 // group]
            a, _ = ref.gemm4(x[m : m + 1, k0:k1], c, s, group)
            want += a[0]
            mag += (8 * s.double().repeat_interleave(group, 1) * x[m, k0:k1].double().abs()).sum(1)
        # 8 warps' sums of K / 8 each: a block of 256 k adds its part to a running sum, off by 2^-24 of what that holds
        within(y[m], want, ref.HALF[FP16] * want.abs() + 2.0**-24 * (K / 2048) ** 0.5 * mag, f"token {m}")
