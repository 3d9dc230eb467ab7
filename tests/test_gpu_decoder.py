"""GPU parity of the decoder-layer operators beside the linears with plain 64-bit forms:
rotary positions, appending to and attending over the paged 8-bit cache, 4-bit linears."""
import math

import pytest
import torch

import _decoder_ref as ref
import tile_sparse_gemm_b200 as tsg

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available() and torch.cuda.get_device_capability()[0] == 10
    tsg.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(got, want, bound, what=""):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN elsewhere"
    held = ~want.isnan()  # a NaN is right where it is, and has no distance
    err = ((got - want).abs() / bound)[held]
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


# ---------------------------------------------------------------- rotary positions


def test_rope_table_scalings():
    """Angles in 64 bits at far positions: fp32 results within half a step (and the last bit of a 64-bit sine)."""
    n, rot, base, c = 70000, 64, 10000.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    w = base ** (-2 * i / rot)
    bands = w.clone()
    for j, f in enumerate(w.tolist()):
        l = 2 * math.pi / f
        if l > c / 1.0:
            bands[j] = f / 8
        elif l >= c / 4.0:
            s = (c / l - 1.0) / (4.0 - 1.0)
            bands[j] = (1 - s) * f / 8 + s * f
    lo = max(math.floor(rot * math.log(c / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
    hi = min(math.ceil(rot * math.log(c / (1 * 2 * math.pi)) / (2 * math.log(base))), rot - 1)
    r = ((i - lo) / (hi - lo)).clamp(0, 1)
    yarn, amp = w * (1 - r) + w / 8 * r, 0.1 * math.log(8.0) + 1.0
    for kind, want, a in (("plain", w, 1.0), ("linear", w / 8, 1.0), ("bands", bands, 1.0), ("yarn", yarn, amp)):
        t = tsg.patch_rope_table(n, rot, base, scaling=kind, factor=8.0 if kind != "plain" else 1.0,
                                 original_positions=c).double().cpu()
        ang = torch.arange(n, dtype=torch.float64)[:, None] * want
        for z, f in ((t[..., 0], ang.cos()), (t[..., 1], ang.sin())):
            # frequencies differ by a few 2^-53, angles below 7e4: 1e-10 is far above it
            assert float(((z - f * a).abs() - 2.0**-24 * 1.25).max()) <= 1e-10, kind


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H,Hk,D,rot", [(1, 1, 0, 64, 64), (1, 32, 8, 128, 128), (37, 14, 2, 64, 32),
                                          (5, 3, 1, 80, 32), (9, 2, 2, 16, 16), (2, 1, 1, 1024, 512),
                                          (513, 7, 1, 128, 64)])
def test_rope(T, H, Hk, D, rot, dtype, layout):
    g = gen(T + D)
    qkv = torch.randn(T, (H + 2 * Hk) * D, generator=g, device="cuda").to(dtype)
    q = qkv[:, : H * D].unflatten(1, (H, D))
    k = qkv[:, H * D : (H + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    table = tsg.patch_rope_table(5000, rot, scaling="yarn", factor=4.0, original_positions=1024)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    st = tsg.new_status()
    for backward in (False, True):
        qo, ko = tsg.patch_rope(q, k, pos, table, layout, backward, status=st)
        within(qo, *ref.rope(q, pos, table, layout, backward), "q")
        if Hk:
            within(ko, *ref.rope(k, pos, table, layout, backward), "k")
        else:
            assert ko is None
    # in place through strided views gives the same bits and touches nothing else
    qkv2 = qkv.clone()
    q2 = qkv2[:, : H * D].unflatten(1, (H, D))
    k2 = qkv2[:, H * D : (H + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    tsg.patch_rope(q2, k2, pos, table, layout, True, q_out=q2, k_out=k2, status=st)
    assert torch.equal(q2, qo) and (k2 is None or torch.equal(k2, ko))
    assert torch.equal(qkv2[:, (H + Hk) * D :], qkv[:, (H + Hk) * D :])
    assert tsg.patch_read_status(st) == (0, 0)


def test_rope_padding_and_positions_out_of_range():
    g = gen(3)
    q = torch.randn(4, 2, 64, generator=g, device="cuda").to(BF16)
    table = tsg.patch_rope_table(10, 64)
    out = torch.full_like(q, 7.0)
    st = tsg.new_status()
    tsg.patch_rope(q, None, i32([3, -1, 9, 0]), table, q_out=out, status=st)
    assert tsg.patch_read_status(st) == (0, 0) and bool((out[1] == 7.0).all())
    within(out[[0, 2, 3]], *ref.rope(q[[0, 2, 3]], i32([3, 9, 0]), table))
    out.fill_(7.0)
    tsg.patch_rope(q, None, i32([10, -2, 2, 2**31 - 1]), table, q_out=out, status=st)
    assert tsg.patch_read_status(st)[1] == tsg.DEV_BOUNDS and bool((out[[0, 1, 3]] == 7.0).all())
    within(out[[2]], *ref.rope(q[[2]], i32([2]), table))


def test_rope_gradient_against_differences():
    """sum(w * rope(x)) in fp32: the gradient from backward=True against central differences of the 64-bit form
    (the rotation is linear, so differences are exact up to rounding)."""
    g = gen(5)
    x = torch.randn(3, 2, 32, generator=g, device="cuda")
    w = torch.randn(3, 2, 32, generator=g, device="cuda")
    table = tsg.patch_rope_table(100, 16, scaling="yarn", factor=4.0, original_positions=32)
    pos = i32([0, 99, 41])
    for layout in ("half", "interleaved"):
        grad, _ = tsg.patch_rope(w, None, pos, table, layout, backward=True)
        for t, h, d in ((0, 0, 0), (1, 1, 3), (1, 0, 15), (2, 1, 8), (2, 0, 31)):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[t, h, d] = 1.0
            f = [(w.double() * ref.turned(x.double() + s * e, pos, table, layout)).sum() for s in (1.0, -1.0)]
            assert abs(float(grad[t, h, d]) - float(f[0] - f[1]) / 2) <= 1e-5


# ---------------------------------------------------------------- the paged 8-bit cache


def pages_of(lens, page, g, spare=3):
    need = [max(1, -(-n // page)) for n in lens]
    ids = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(need)), -7, dtype=torch.int32, device="cuda")  # unused entries are invalid
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at : at + n]
        at += n
    return bt, sum(need) + spare


def random_cache(n_pages, hk, page, d, g):
    c = tsg.new_kv_cache8(n_pages, hk, page, d)
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        s.copy_(2.0 ** torch.randint(-7, -3, s.shape, generator=g, device="cuda").float())
        x.copy_((torch.randn(x.shape, generator=g, device="cuda") / s[..., None, None]).clamp(-448, 448).to(F8))
    return c


def copy_of(c):
    return tsg.KvCache8(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone())


def check_append(before, after, k, v, bt, past, cu, table, layout):
    """Every byte and scale of the cache after an append against the 64-bit form."""
    page, d = before.k.shape[2:]
    for name, x, c0, c1, s0, s1 in (("k", k, before.k, after.k, before.k_scale, after.k_scale),
                                    ("v", v, before.v, after.v, before.v_scale, after.v_scale)):
        raw0, raw1 = c0.view(torch.uint8), c1.view(torch.uint8)
        want_raw, want_s = raw0.clone(), s0.clone()
        for b, p0 in enumerate(past):
            at, stop = p0, p0 + cu[b + 1] - cu[b]
            while at < stop:
                n = min(page - at % page, stop - at)
                rows = x[cu[b] + at - p0 : cu[b] + at - p0 + n]
                y, err = rows.double(), torch.zeros_like(rows.double())
                if name == "k" and table is not None:
                    pos = torch.arange(at, at + n, device="cuda")
                    y, err = ref.rope(rows.float(), pos, table, layout)
                to, o = int(bt[b, at // page]), at % page
                mag = torch.where(y.isfinite(), y.abs(), 0.0).amax((0, 2))
                scale = ref.needed_scale(mag)
                if o:
                    scale = torch.maximum(scale, s0[to].double())
                    old, new = c0[to, :, :o].double(), c1[to, :, :o].double()
                    ratio = (s0[to].double() / scale)[:, None, None]
                    # a power of two: only e4m3's smallest step (2^-9) rounds
                    near = (new - old * ratio).abs() <= torch.where(ratio == 1.0, 0.0, 2.0**-10)
                    assert bool((near | (new.isnan() & old.isnan())).all()), name
                    want_raw[to, :, :o] = raw1[to, :, :o]
                assert torch.equal(s1[to].double(), scale), f"{name}: scale of page {to}"
                z = (y / scale[:, None]).transpose(0, 1)
                got = c1[to, :, o : o + n].double()
                assert torch.equal(got.isnan(), z.isnan()), name
                lim = z.clamp(-448.0, 448.0)
                # half a step of e4m3 and the fp32 rotation's error under the same scale
                tol = torch.maximum(2.0**-4 * lim.abs(), torch.full_like(lim, 2.0**-10)) * (1 + 2.0**-20)
                tol = tol + (err / scale[:, None]).transpose(0, 1).nan_to_num()
                assert bool((((got - lim).abs() <= tol) | got.isnan()).all()), f"{name}: values"
                want_raw[to, :, o : o + n] = raw1[to, :, o : o + n]
                want_s[to] = s1[to]
                at += n
        assert torch.equal(raw1, want_raw) and torch.equal(s1, want_s), f"{name}: something else was written"


@pytest.mark.parametrize("page,d,hk,dtype,layout,rot", [
    (16, 64, 2, BF16, "half", 64), (32, 128, 1, FP16, "interleaved", 128), (64, 128, 8, BF16, "half", 64),
    (128, 128, 3, FP16, "half", 16), (128, 64, 2, BF16, "interleaved", 32), (64, 64, 5, FP16, "half", 0)])
@pytest.mark.parametrize("past,new", [([0], [1]), ([15, 16, 0, 33], [1, 1, 1, 1]), ([7, 0, 130, 64, 3], [0, 300, 1, 64, 2]),
                                      ([5] * 70, [1] * 70)])
def test_append(page, d, hk, dtype, layout, rot, past, new):
    g = gen(page + d + len(past))
    total = [a + b for a, b in zip(past, new)]
    bt, n_pages = pages_of(total, page, g)
    cache = random_cache(n_pages, hk, page, d, g)
    T = sum(new)
    # magnitudes from tiny to large, so that scales shrink, stay and grow
    x = torch.randn(T + 2, 3 * hk * d, generator=g, device="cuda")
    x *= 2.0 ** torch.randint(-6, 7, (T + 2, 1), generator=g, device="cuda")
    x = x.to(dtype)
    k, v = (x[:, i * hk * d : (i + 1) * hk * d].unflatten(1, (hk, d)) for i in (1, 2))
    table = tsg.patch_rope_table(512, rot) if rot else None
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    before, st = copy_of(cache), tsg.new_status()
    single = all(n == 1 for n in new)
    # two rows behind the last sequence: not read
    tsg.patch_kv8_append(k, v, cache, bt, i32(past), i32(cu), table, layout, status=st)
    assert tsg.patch_read_status(st) == (0, 0)
    check_append(before, cache, k, v, bt, past, cu, table, layout)
    if single:  # the form for one token per sequence: the same bits
        other = copy_of(before)
        tsg.patch_kv8_append(k[:T], v[:T], other, bt, i32(past), None, table, layout, status=st)
        assert torch.equal(other.k.view(torch.uint8), cache.k.view(torch.uint8))
        assert torch.equal(other.v_scale, cache.v_scale)
    # again: a call that changes nothing any more
    once = copy_of(cache)
    tsg.patch_kv8_append(k, v, cache, bt, i32(past), i32(cu), table, layout, status=st)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in
               ((once.k, cache.k), (once.v, cache.v), (once.k_scale, cache.k_scale), (once.v_scale, cache.v_scale)))


def test_append_special_values():
    """Zeros, infinities, NaN, subnormals and the type's largest values; one token at a time into one page."""
    page, d, hk = 16, 64, 1
    cache = tsg.new_kv_cache8(1, hk, page, d)
    cache.k_scale.fill_(math.nan)  # a fresh page takes no notice of what it held
    bt, st = i32([[0]]), tsg.new_status()
    rows = torch.zeros(5, hk, d, dtype=BF16, device="cuda")
    rows[1, 0, :3] = torch.tensor([math.inf, -math.inf, 2.0])
    rows[2, 0, :2] = torch.tensor([math.nan, 1.0])
    rows[3, 0, :2] = torch.tensor([2.0**-130, 3e38])
    rows[4, 0, 0] = torch.finfo(BF16).max
    for i in range(5):
        was = copy_of(cache)
        tsg.patch_kv8_append(rows[i : i + 1], rows[i : i + 1], cache, bt, i32([i]), status=st)
        check_append(was, cache, rows[i : i + 1], rows[i : i + 1], bt, [i], [0, 1], None, "half")
    assert tsg.patch_read_status(st) == (0, 0)


def test_append_bad_pages_and_positions_are_refused_on_the_device():
    page, d, hk = 16, 64, 2
    g = gen(9)
    cache = random_cache(4, hk, page, d, g)
    k = torch.randn(3, hk, d, generator=g, device="cuda").to(BF16)
    was = copy_of(cache)
    for bt, past, table in (([[4], [-1], [2**31 - 1]], [0, 3, 5], None),       # pages outside the pool
                            ([[0], [1], [2]], [16, 1000000, -1], None),        # outside the block table
                            ([[0], [1], [2]], [8, 9, 15], tsg.patch_rope_table(8, 64))):  # outside the table
        st = tsg.new_status()
        tsg.patch_kv8_append(k, k, cache, i32(bt), i32(past), None, table, status=st)
        assert tsg.patch_read_status(st)[1] == tsg.DEV_BOUNDS
        if table is None:
            assert torch.equal(cache.k.view(torch.uint8), was.k.view(torch.uint8))
            assert torch.equal(cache.v.view(torch.uint8), was.v.view(torch.uint8))
        else:
            assert torch.equal(cache.k.view(torch.uint8), was.k.view(torch.uint8))


# ---------------------------------------------------------------- attention over it


def run_attn(B, H, Hk, D, page, kv, q_lens, dtype, causal=True, window=0, seed=0, pad_rows=0, scale=None, edit=None):
    g = gen(seed + B + H + D)
    bt, n_pages = pages_of(kv, page, g)
    cache = random_cache(n_pages, Hk, page, D, g)
    cu = [sum(q_lens[:i]) for i in range(B + 1)]
    T = cu[-1] + pad_rows
    q = torch.randn(T, H * D + 64, generator=g, device="cuda").to(dtype)[:, 64:].unflatten(1, (H, D))
    # what lies behind a sequence's tokens in its last page is NaN: nothing may come of it
    for b, n in enumerate(kv):
        if n % page:
            for c in (cache.k, cache.v):
                c.view(torch.uint8)[int(bt[b, n // page]), :, n % page :] = 0x7F
    if edit:
        q = edit(q, cache, bt)
    st = tsg.new_status()
    out = torch.full((T, H, D), 3.0, dtype=dtype, device="cuda")
    o, lse = tsg.patch_attn_kv8(q, cache, bt, i32(kv), None if all(m == 1 for m in q_lens) and not pad_rows else i32(cu),
                                scale, causal, window, out=out, want_lse=True, status=st)
    assert tsg.patch_read_status(st) == (0, 0)
    n = cu[-1]
    want, wl, bound = ref.attention(q[:n], cache.k, cache.v, cache.k_scale, cache.v_scale, bt, kv, cu,
                                    1.0 / math.sqrt(D) if scale is None else scale, causal, window)
    within(o[:n], want, bound, "out")
    assert bool((o[n:] == 3.0).all())
    fin = wl.isfinite()
    assert torch.equal(torch.isfinite(lse[:n]), fin) and torch.equal(lse[:n].double()[~fin].isnan(), wl[~fin].isnan())
    # fp32 scores and sum: 2^-12 of absolute error is far above both
    assert bool(((lse[:n].double() - wl).abs()[fin] <= 2.0**-12 * (1 + wl.abs()[fin])).all())
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hk,D", [(4, 4, 128), (8, 2, 128), (14, 2, 64), (3, 3, 64), (16, 1, 128), (8, 1, 64)])
def test_attn_decode_lengths(H, Hk, D, page):
    kv = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1023]
    run_attn(len(kv), H, Hk, D, page, kv, [1] * len(kv), BF16 if D == 128 else FP16)


@pytest.mark.parametrize("B,kv", [(1, [1]), (1, [40000]), (3, [20000, 5, 0]), (200, [37 * i % 1500 for i in range(200)])])
@pytest.mark.parametrize("H,Hk,D,dtype", [(8, 8, 128, FP16), (8, 2, 64, BF16)])
def test_attn_decode_batches(B, kv, H, Hk, D, dtype):
    run_attn(B, H, Hk, D, 64, kv, [1] * B, dtype, seed=1)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 70)])
@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 64), (14, 2, 64, 16), (2, 2, 128, 128), (16, 1, 64, 32)])
def test_attn_several_queries(H, Hk, D, page, causal, window):
    """Ragged query counts: none, one, more than the keys (rows that see nothing), many; rows behind the last sequence."""
    kv = [100, 7, 0, 300, 64, 1000, 33]
    q = [1, 20, 3, 0, 64, 131, 33]
    run_attn(7, H, Hk, D, page, kv, q, BF16, causal, window, seed=2, pad_rows=5)


def test_attn_large_and_small_values():
    """Queries near fp16's and bf16's ends, keys that make sharp and flat softmaxes, a scale of 0 and a negative one."""
    def big(q, cache, bt):
        q = q.clone()
        q[0] *= 2.0**60
        q[1] *= 2.0**-60
        q[2] = 0.0
        return q
    run_attn(4, 8, 2, 128, 64, [300, 200, 77, 500], [1, 1, 1, 1], BF16, scale=2.0**-62, seed=3, edit=big)
    run_attn(4, 8, 2, 128, 64, [300, 200, 77, 500], [1, 1, 1, 1], FP16, scale=0.0, seed=3)
    run_attn(4, 8, 2, 128, 64, [300, 200, 77, 500], [1, 1, 1, 1], FP16, scale=-0.3, seed=3)

    def scales(q, cache, bt):  # pages of one sequence under very different scales
        for s in (cache.k_scale, cache.v_scale):
            s.mul_(2.0 ** torch.randint(-14, 6, s.shape, device="cuda", generator=gen(4)).float())
        return q
    run_attn(3, 8, 2, 128, 16, [300, 200, 77], [1, 4, 1], BF16, seed=5, edit=scales)


def test_attn_nan_reaches_only_the_rows_that_see_it():
    def edit(q, cache, bt):
        page = int(bt[0, 2])  # tokens 32 .. 47 of sequence 0
        cache.v.view(torch.uint8)[page, 0, 8, 5] = 0x7F
        return q
    # 20 queries at positions 30 .. 49: token 40 is seen from position 40 on
    run_attn(2, 4, 2, 64, 16, [50, 60], [20, 2], BF16, seed=6, edit=edit)
    # the same with 128-row tiles: 170 queries at positions 0 .. 169, a second NaN behind the first tile's last position
    def more(q, cache, bt):
        q = edit(q, cache, bt)
        cache.v.view(torch.uint8)[int(bt[0, 9]), 1, 3, 63] = 0xFF
        cache.k.view(torch.uint8)[int(bt[1, 8]), 1, 1, 2] = 0x7F  # a key: whole rows from position 129 on
        return q
    run_attn(2, 4, 2, 64, 16, [170, 150], [170, 150], BF16, seed=6, edit=more)


@pytest.mark.parametrize("H,Hk,D,page,dtype", [(8, 2, 128, 64, BF16), (14, 2, 64, 16, FP16), (4, 4, 128, 32, FP16),
                                               (16, 1, 64, 128, BF16)])
@pytest.mark.parametrize("kv,q", [([64], [64]), ([5000], [130]), ([1, 700, 0, 2000], [300, 70, 90, 1999]),
                                  ([256] * 40, [65 + i for i in range(40)])])
def test_attn_prompts(H, Hk, D, page, dtype, kv, q):
    """Many queries per sequence: tiles of 128 rows, whole ones and cut ones, ragged, some without keys."""
    run_attn(len(kv), H, Hk, D, page, kv, q, dtype, seed=12, pad_rows=1)
    run_attn(len(kv), H, Hk, D, page, kv, q, dtype, causal=False, seed=13, scale=-0.05)


@pytest.mark.parametrize("B", [257, 449, 1000])
@pytest.mark.parametrize("many", [False, True])
def test_attn_more_sequences_than_threads(B, many):
    """Shares of the work are found by a CTA of 256 or 448 threads, a sequence each at a time."""
    q_lens = [(7 * i) % 23 + 10 * many for i in range(B)] if many else [i % 3 for i in range(B)]
    run_attn(B, 8, 1, 64, 16, [n + (5 * i) % 40 for i, n in enumerate(q_lens)], q_lens, FP16)


def test_append_more_sequences_than_threads():
    past, new = [(11 * i) % 37 for i in range(700)], [(5 * i) % 4 for i in range(700)]
    test_append(16, 64, 2, BF16, "half", 64, past, new)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_prompt_scores_of_wide_queries(D, dtype):
    """One token in view, so lse is its score: with 128-row tiles the queries are sums of e4m3 numbers,
    off by at most 2^-17 of a row's largest element; D fp32 additions of up to three terms beside."""
    g, m = gen(31), 300
    q = torch.randn(m, 1, D, generator=g, device="cuda").double()
    q *= torch.exp2(-20 * torch.rand(m, 1, D, generator=g, device="cuda").double())
    q[: m // 2] *= 2.0 ** (100 if dtype == BF16 else 12)
    q[3], q[4, :, 5], q[5, :, :1] = 0.0, math.inf, math.nan
    q = q.to(dtype)
    cache = random_cache(1, 1, 16, D, g)
    bt, lens, cu = i32([[0]]), i32([1]), i32([0, m])
    out, lse = tsg.patch_attn_kv8(q, cache, bt, lens, cu, causal=False, want_lse=True)
    k = cache.k[0, 0, 0].double() * cache.k_scale[0, 0].double()
    x, f = q[:, 0].double(), 1 / math.sqrt(D)
    bound = f * (2.0**-17 * x.abs().amax(1) * k.abs().sum() + 3 * (D + 2) * 2.0**-24 * (x.abs() @ k.abs())) + 1e-30
    want = (x @ k) * f
    want[4] = math.nan  # an infinite score has no softmax
    within(lse[:, 0], want, bound, "lse")
    v = cache.v[0, 0, 0].double() * cache.v_scale[0, 0].double()
    within(out[:, 0], torch.where(want.isnan()[:, None], math.nan, v.expand(m, D)), 2.0**-8 * v.abs() + 1e-30, "out")


def test_attn_bad_lengths_and_pages_read_as_zeros():
    g = gen(8)
    cache = random_cache(4, 2, 16, 64, g)
    q = torch.randn(3, 4, 64, generator=g, device="cuda").to(BF16)
    st = tsg.new_status()
    out, lse = tsg.patch_attn_kv8(q, cache, i32([[0, 1], [2, 9], [-1, 3]]), i32([33, 32, -4]), want_lse=True, status=st)
    assert tsg.patch_read_status(st)[1] == tsg.DEV_BOUNDS
    assert bool(torch.isfinite(out).all()) and bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())


def test_attn_workspace_is_reused_by_calls_of_other_sizes_and_by_graphs():
    g = gen(11)
    cache = random_cache(400, 2, 64, 128, g)
    jobs = []
    for B, n in ((1, 20000), (5, 3000), (64, 300)):
        bt = torch.randint(0, 400, (B, -(-n // 64)), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.randint(1, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        jobs.append((torch.randn(B, 8, 128, generator=g, device="cuda").to(BF16), bt, lens))
    alone = [tsg.patch_attn_kv8(q, cache, bt, lens) for q, bt, lens in jobs]
    ws = torch.zeros(max(max(tsg.patch_attn_kv8_workspace_size(q.shape[0], q.shape[0], 8, cache) for q, _, _ in jobs), 16),
                     dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(a) for a in alone]

    def all_of_them():
        for (q, bt, lens), o in zip(jobs, outs):
            tsg.patch_attn_kv8(q, cache, bt, lens, workspace=ws, out=o)

    for _ in range(2):
        all_of_them()
        assert all(torch.equal(a, o) for a, o in zip(alone, outs))
    graphs = []
    for _ in range(2):  # two graphs that share the workspace, replayed in turn
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            all_of_them()
        graphs.append(gr)
    for gr in graphs + graphs:
        for o in outs:
            o.zero_()
        gr.replay()
        assert all(torch.equal(a, o) for a, o in zip(alone, outs))


# ---------------------------------------------------------------- 4-bit linears


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("sdtype", [BF16, FP16])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (17, 64, 64), (33, 128, 32), (100, 128, 128), (129, 1056, 32),
                                       (64, 2112, 64), (1000, 896, 128), (128, 4864, 32), (3, 11008, 128)])
def test_gemm4(N, K, group, sdtype, dtype):
    g = gen(N + K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(N, K // group, generator=g, device="cuda") * 0.02).to(sdtype)
    w = tsg.Weight4(codes, scales, group)
    for M in (1, 2, 7, 8, 9, 16):
        x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
        out = torch.full((M + 1, N), 5.0, dtype=dtype, device="cuda")
        tsg.patch_gemm4(x, w, out[:M])
        within(out[:M], *ref.gemm4(x, codes, scales, group), f"M={M}")
        assert bool((out[M] == 5.0).all())
        assert torch.equal(out[:M], tsg.patch_gemm4(x, w))  # deterministic
    assert tsg.patch_gemm4(x[:0], w).shape == (0, N)


@pytest.mark.parametrize("M,N,K,group", [(14, 577, 11072, 64), (9, 2366, 4192, 32), (8, 4096, 14336, 128), (16, 1000, 14336, 64),
                                         (1, 256, 14336, 128), (4, 2000, 12320, 32), (16, 3000, 8192, 128), (1, 33, 2048, 64)])
def test_gemm4_parts_of_k(M, N, K, group):
    """Few rows or many tokens: clusters of CTAs with a part of K each."""
    g = gen(N + K)
    w = tsg.Weight4(torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                    (0.5 + torch.rand(N, K // group, generator=g, device="cuda")).to(FP16), group)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    y = tsg.patch_gemm4(x, w)
    within(y, *ref.gemm4(x, w.codes, w.scales, group))
    for _ in range(20):
        assert torch.equal(tsg.patch_gemm4(x, w), y)


@pytest.mark.parametrize("M", [1, 11])
@pytest.mark.parametrize("N,K,group", [(40000, 128, 32), (30011, 320, 64), (30000, 1824, 32)])
def test_gemm4_many_rows_of_few_blocks(N, K, group, M):
    """Fewer blocks of 256 k than warps that share them, and several row groups a CTA."""
    g = gen(N + K)
    w = tsg.Weight4(torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                    (0.5 + torch.rand(N, K // group, generator=g, device="cuda")).to(BF16), group)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    within(tsg.patch_gemm4(x, w), *ref.gemm4(x, w.codes, w.scales, group))


def test_gemm4_rows_with_infinities_and_nan():
    g = gen(2)
    w = tsg.patch_quantize4(torch.randn(40, 256, generator=g, device="cuda"), 64)
    x = torch.randn(5, 256, generator=g, device="cuda").to(BF16)
    clean = tsg.patch_gemm4(x, w)
    x[3, 70] = math.nan
    y = tsg.patch_gemm4(x, w)
    assert bool(y[3].isnan().all()) and torch.equal(y[[0, 1, 2, 4]], clean[[0, 1, 2, 4]])


@pytest.mark.parametrize("dtype,sdtype", [(BF16, BF16), (FP16, FP16), (FP32, FP16), (FP32, BF16)])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (37, 384, 64), (300, 1280, 128)])
def test_quantize4(N, K, group, dtype, sdtype):
    g = gen(K)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).to(dtype)
    w[0, :group] = 0.0
    q = tsg.patch_quantize4(w, group, sdtype)
    amax = w.double().abs().view(N, -1, group).amax(-1)
    # the scale: amax / 7 rounded to fp32 and then to its type
    assert bool(((q.scales.double() - amax / 7).abs() <= (ref.HALF[sdtype] + 2.0**-23) * amax / 7 + ref.TINY[sdtype]).all())
    c = torch.stack((q.codes & 15, q.codes >> 4), -1).flatten(1).double() - 8
    s = q.scales.double().repeat_interleave(group, 1)
    # every weight to its nearest code: half a step, and the fp32 division's rounding
    assert bool(((w.double() - c * s).abs() <= s * (0.5 + 8 * 2.0**-23)).all())
    assert bool((c[0, :group] == 0).all())
    # pruned weights stay exactly zero
    pruned = w.clone()
    pruned[:, 1::2] = 0.0
    cp = tsg.patch_quantize4(pruned, group, sdtype).codes
    assert bool((cp >> 4 == 8).all())


# ---------------------------------------------------------------- streams, devices, together


def test_on_another_stream_and_captured():
    g = gen(21)
    x = torch.randn(3, 512, generator=g, device="cuda").to(BF16)
    w = tsg.patch_quantize4(torch.randn(256, 512, generator=g, device="cuda"))
    want = tsg.patch_gemm4(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    tsg.patch_gemm4(x, w, y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    with torch.cuda.stream(s):
        z = tsg.patch_gemm4(x, w)
    s.synchronize()
    assert torch.equal(z, want)


@pytest.mark.parametrize("H,Hk,D", [(4, 2, 64), (8, 8, 128)])
def test_a_layers_attention_together(H, Hk, D):
    """q|k|v by the hybrid linear, rotary positions, append, attention, then o in 4 bits: a prompt and
    three decode steps, each stage against its 64-bit form on the tensors it was given, the decode
    step captured into a graph and replayed with the same bits."""
    import numpy as np

    import oracle
    import synth_inputs as si
    from _util import bits_of, check_gemm, to_dev, to_dev_bf16

    C = 256
    N = (H + 2 * Hk) * D
    wb = si.gen_w(N, C, 3, 1)
    bm, ids = si.tiles_exact(N, C, 0.5, 3, 1), si.patterns_top2(wb)
    st = tsg.new_status()
    pw = tsg.patch_pack(to_dev_bf16(wb), to_dev(bm), to_dev(ids), int(bm.sum()), status=st)
    wo = tsg.patch_quantize4(torch.randn(C, H * D, generator=gen(1), device="cuda") * 0.02, 64)
    table = tsg.patch_rope_table(512, D)
    page, B = 16, 3
    lens, steps = [5, 33, 16], 3
    bt, n_pages = pages_of([n + steps for n in lens], page, gen(2))
    cache = tsg.new_kv_cache8(n_pages, Hk, page, D)
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    gws = torch.zeros(max(tsg.patch_gemm_workspace_size(64, pw), tsg.patch_gemm_workspace_size(3, pw), 16),
                      dtype=torch.uint8, device="cuda")

    def step(x, past, pos, kv_lens, cu):
        qkv = tsg.patch_gemm(x, pw, workspace=gws, status=st)
        q = qkv[:, : H * D].unflatten(1, (H, D))
        k, v = (qkv[:, (H + i * Hk) * D : (H + (i + 1) * Hk) * D].unflatten(1, (Hk, D)) for i in (0, 1))
        tsg.patch_kv8_append(k, v, cache, bt, past, cu, table, status=st)
        q0 = q.clone()
        tsg.patch_rope(q, None, pos, table, q_out=q, status=st)
        a = tsg.patch_attn_kv8(q, cache, bt, kv_lens, cu, workspace=ws, status=st)
        return qkv, q0, k, v, q, a

    past = [0] * B
    new = lens
    x = to_dev_bf16(si.gen_x(sum(new), C, 3, 2))
    for s in range(steps + 1):
        cu = [sum(new[:i]) for i in range(B + 1)]
        pos = i32([p + i for p, n in zip(past, new) for i in range(n)])
        kv = [p + n for p, n in zip(past, new)]
        before = copy_of(cache)
        args = (x, i32(past), pos, i32(kv), i32(cu) if s == 0 else None)
        qkv, q0, k, v, q, a = step(*args)
        y = tsg.patch_gemm4(a.reshape(a.shape[0], -1), wo) if s else None
        assert tsg.patch_read_status(st) == (0, 0)
        want = oracle.hybrid_gemm(bits_of(x), wb, bm, ids)
        full = qkv.clone()
        full[:, : H * D] = q0.reshape(q0.shape[0], -1)
        check_gemm(bits_of(full), np.asarray(want), "qkv")
        within(q, *ref.rope(q0, pos, table), "rope")
        check_append(before, cache, k, v, bt, past, cu, table, "half")
        o, _, bound = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, bt, kv, cu, 1 / math.sqrt(D))
        within(a, o, bound, "attention")
        if y is not None:
            within(y, *ref.gemm4(a.reshape(a.shape[0], -1), wo.codes, wo.scales, 64), "o")
            after = copy_of(cache)
            for t, f in ((cache.k, before.k), (cache.v, before.v)):
                t.view(torch.uint8).copy_(f.view(torch.uint8))
            cache.k_scale.copy_(before.k_scale)
            cache.v_scale.copy_(before.v_scale)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                a2 = step(*args)[-1]
                y2 = tsg.patch_gemm4(a2.reshape(a2.shape[0], -1), wo)
            graph.replay()
            assert torch.equal(y2, y) and torch.equal(cache.k.view(torch.uint8), after.k.view(torch.uint8))
        past, new = kv, [1] * B
        x = to_dev_bf16(si.gen_x(B, C, 3, 10 + s))
