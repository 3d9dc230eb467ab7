"""Host checks of the decoder-layer operators' C ABI: refused before any device query or launch (no GPU needed)."""
import ctypes

import pytest
import torch

import tile_sparse_gemm_b200 as tsg
from tile_sparse_gemm_b200 import build as tsg_build
from tile_sparse_gemm_b200 import decoder as dec

P = ctypes.c_void_p
F = 0x10000  # never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module")
def lib():
    tsg_build.build()
    return tsg.lib()


def heads(n=4, data=F, ts=1024, hs=128):
    return ctypes.byref(dec._Heads(data, n, ts, hs))


def cache(k=F, v=F, ks=F, vs=F, n_pages=8, hk=4, page=64, d=128):
    return ctypes.byref(dec._Cache8(k, v, ks, vs, n_pages, hk, page, d))


def test_rope_table_refusals(lib):
    def call(n_pos=10, rot=64, kind=0, base=1e4, factor=2.0, orig=100.0, low=1.0, high=4.0, amp=1.0, table=F, cfg=True):
        c = dec._RopeConfig(kind, 0, base, factor, orig, low, high, amp)
        return lib.patch_rope_table(n_pos, rot, ctypes.byref(c) if cfg else None, table, None)

    inf, nan = float("inf"), float("nan")
    for kw in (dict(cfg=False), dict(table=None), dict(base=1.0), dict(base=nan), dict(base=inf), dict(kind=4),
               dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=1, factor=nan), dict(kind=2, orig=0.0),
               dict(kind=2, low=4.0), dict(kind=3, high=inf), dict(kind=3, orig=-1.0), dict(amp=nan)):
        assert call(**kw) == 1, kw
    for kw in (dict(n_pos=0), dict(n_pos=1 << 31), dict(rot=0), dict(rot=7), dict(rot=2048)):
        assert call(**kw) == 2, kw
    assert call(table=F + 4) == 3


def test_rope_refusals(lib):
    def call(q=heads(), k=heads(), qo=heads(), ko=heads(), T=3, D=128, dtype=0, pos=F, table=F, n_pos=10, rot=128,
             layout=0):
        return lib.patch_rope(q, k, qo, ko, T, D, dtype, pos, table, n_pos, rot, layout, 0, None, None)

    assert call(T=0) == 0 and call(T=0, q=heads(data=None), pos=None) == 0  # no tokens: no-op
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(T=-1), dict(dtype=3), dict(layout=2),
               dict(qo=heads(5)), dict(ko=heads(3)), dict(pos=None), dict(table=None), dict(q=heads(data=None)),
               dict(q=heads(0), qo=heads(0))):
        assert call(**kw) == 1, kw
    for kw in (dict(D=12), dict(D=132), dict(D=2048), dict(rot=0), dict(rot=24), dict(rot=144), dict(n_pos=0),
               dict(T=1 << 31), dict(q=heads(65533), qo=heads(65533)), dict(k=heads(1 << 62), ko=heads(1 << 62))):
        assert call(**kw) == 2, kw
    for kw in (dict(q=heads(data=F + 2)), dict(qo=heads(ts=1025)), dict(k=heads(hs=4)), dict(table=F + 8),
               dict(pos=F + 2)):
        assert call(**kw) == 3, kw


def test_append_refusals(lib):
    def call(k=heads(), v=heads(), T=3, dtype=0, c=cache(), bt=F, mp=4, past=F, cu=F, B=3, table=F, n_pos=10, rot=128,
             layout=0):
        return lib.patch_kv8_append(k, v, T, dtype, c, bt, mp, past, cu, B, table, n_pos, rot, layout, None, None)

    assert call(T=0) == 0 and call(B=0) == 0
    for kw in (dict(k=None), dict(v=None), dict(c=None), dict(c=cache(k=None)), dict(c=cache(vs=None)), dict(T=-1),
               dict(B=-1), dict(dtype=2), dict(layout=-1), dict(cu=None, T=2), dict(k=heads(3)), dict(bt=None),
               dict(past=None), dict(v=heads(data=None))):
        assert call(**kw) == 1, kw
    for kw in (dict(c=cache(page=8)), dict(c=cache(page=256)), dict(c=cache(d=96)), dict(c=cache(n_pages=0)),
               dict(rot=8), dict(rot=256), dict(rot=0), dict(table=None), dict(n_pos=0), dict(mp=-1)):
        assert call(**kw) == 2, kw
    for kw in (dict(k=heads(data=F + 8)), dict(v=heads(ts=12)), dict(c=cache(v=F + 1)), dict(table=F + 4),
               dict(past=F + 1), dict(bt=F + 2)):
        assert call(**kw) == 3, kw


def test_attn_refusals(lib):
    def call(q=heads(8), T=3, dtype=1, c=cache(), bt=F, mp=4, lens=F, cu=F, B=3, scale=0.1, causal=1, window=0,
             out=heads(8), lse=None):
        return lib.patch_attn_kv8(q, T, dtype, c, bt, mp, lens, cu, B, scale, causal, window, out, lse, F, 0, None,
                                  None, 0)

    assert call(T=0) == 0 and call(B=0) == 0
    for kw in (dict(q=None), dict(out=None), dict(c=None), dict(dtype=2), dict(T=-1), dict(B=-1), dict(window=-1),
               dict(window=3, causal=0), dict(scale=float("nan")), dict(out=heads(4)), dict(cu=None, T=4),
               dict(lens=None), dict(bt=None), dict(q=heads(8, data=None))):
        assert call(**kw) == 1, kw
    for kw in (dict(q=heads(6), out=heads(6)), dict(q=heads(128), out=heads(128)), dict(c=cache(d=256)),
               dict(c=cache(page=48)), dict(mp=-1)):
        assert call(**kw) == 2, kw
    for kw in (dict(q=heads(8, ts=1020)), dict(out=heads(8, data=F + 2)), dict(lens=F + 2), dict(lse=F + 1)):
        assert call(**kw) == 3, kw
    n = ctypes.c_size_t(9)
    assert lib.patch_attn_kv8_workspace_size(0, 3, 8, cache(), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.patch_attn_kv8_workspace_size(3, 3, 7, cache(), ctypes.byref(n)) == 2
    assert lib.patch_attn_kv8_workspace_size(3, 3, 8, cache(), None) == 1


def test_weight4_refusals(lib):
    def w(N=16, K=256, group=64, sd=0, codes=F, scales=F):
        return ctypes.byref(dec._Weight4(N, K, group, sd, codes, scales))

    def gemm(x=F, M=2, dtype=0, weight=w(), y=F):
        return lib.patch_gemm4(x, M, dtype, weight, y, None, None)

    assert gemm(M=0) == 0 and gemm(M=0, x=None, y=None) == 0
    for kw in (dict(M=-1), dict(M=17), dict(dtype=2), dict(weight=None), dict(x=None), dict(y=None),
               dict(weight=w(group=16)), dict(weight=w(sd=2)), dict(weight=w(codes=None)), dict(weight=w(scales=None))):
        assert gemm(**kw) == 1, kw
    for kw in (dict(weight=w(N=0)), dict(weight=w(K=96)), dict(weight=w(K=0)), dict(weight=w(N=1 << 31))):
        assert gemm(**kw) == 2, kw
    for kw in (dict(weight=w(codes=F + 8)), dict(weight=w(scales=F + 2)), dict(x=F + 4), dict(y=F + 1)):
        assert gemm(**kw) == 3, kw
    assert lib.patch_quantize4(None, 0, w(), None) == 1
    assert lib.patch_quantize4(F, 5, w(), None) == 1
    assert lib.patch_quantize4(F, 0, w(K=32), None) == 2
    assert lib.patch_quantize4(F + 2, 0, w(), None) == 3


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and devices: the binding's own checks (CPU tensors never reach the library)."""
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tsg.patch_rope(x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2))
    with pytest.raises(ValueError):
        tsg.patch_rope_table(10, 64, scaling="other")
    with pytest.raises(ValueError):
        tsg.new_kv_cache8(4, 2, 48, 64, device="cpu")
    with pytest.raises(ValueError):
        tsg.new_kv_cache8(4, 2, 16, 96, device="cpu")
    c = tsg.new_kv_cache8(4, 2, 16, 64, device="cpu")
    assert c.stored_bytes == 2 * 4 * 2 * 16 * 64 + 8 * 4 * 2
    with pytest.raises(ValueError):
        tsg.patch_attn_kv8(x, c, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        tsg.patch_quantize4(torch.zeros(4, 96), 64)
    w = tsg.Weight4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.float16), 64)
    assert (w.N, w.K, w.stored_bytes) == (4, 64, 4 * 32 + 8)
    with pytest.raises(ValueError):
        tsg.patch_gemm4(torch.zeros(1, 64, dtype=torch.bfloat16), w)
