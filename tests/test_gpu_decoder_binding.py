"""The decoder-layer calls through the compiled extension and through Python: the same results, the same refusals."""
import pytest
import torch

import tile_sparse_gemm_b200 as tsg
from tile_sparse_gemm_b200 import decoder as dec

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
B, H, HK, D, PAGE, N_PAGES = 3, 8, 2, 64, 16, 12


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def world():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    w = dict(q=randn(B, H, D), k=randn(B, HK, D), v=randn(B, HK, D), table=tsg.patch_rope_table(64, D),
             pos=i32([3, 0, 40]), bt=i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]]), past=i32([3, 0, 40]), lens=i32([4, 1, 41]),
             cu=i32([0, 1, 2, 3]), ws=torch.zeros(1 << 25, dtype=torch.uint8, device="cuda"), st=tsg.new_status(),
             x=randn(5, 256), w4=tsg.patch_quantize4(randn(96, 256), 64), qkv=randn(B, H + 2 * HK, D, dtype=FP16))
    w["cache"] = tsg.new_kv_cache8(N_PAGES, HK, PAGE, D)
    tsg.patch_kv8_append(w["k"], w["v"], w["cache"], w["bt"], w["past"])
    return w


def calls(w):
    """name -> (function, arguments, keywords), as documented."""
    c, q16 = w["cache"], w["qkv"]
    yield "rope", tsg.patch_rope, (w["q"], w["k"], w["pos"], w["table"]), {}
    yield "rope q", tsg.patch_rope, (w["q"], None, w["pos"], w["table"]), dict(layout="interleaved", backward=True)
    yield "rope slices", tsg.patch_rope, (q16[:, :H], q16[:, H : H + HK], w["pos"], w["table"]), dict(status=w["st"])
    yield "rope permuted", tsg.patch_rope, (w["q"].transpose(0, 1).contiguous().transpose(0, 1), None, w["pos"], w["table"]), {}
    yield "rope none", tsg.patch_rope, (w["q"][:0], w["k"][:0], w["pos"][:0], w["table"]), {}
    yield "append", tsg.patch_kv8_append, (w["k"], w["v"], c, w["bt"], w["past"]), {}
    yield "append rotated", tsg.patch_kv8_append, (w["k"], w["v"], c, w["bt"], w["past"], w["cu"], w["table"]), \
        dict(layout="interleaved", status=w["st"])
    yield "attn", tsg.patch_attn_kv8, (w["q"], c, w["bt"], w["lens"]), dict(workspace=w["ws"])
    yield "attn lse", tsg.patch_attn_kv8, (q16[:, :H], c, w["bt"], w["lens"], w["cu"]), \
        dict(workspace=w["ws"], want_lse=True, scale=0.2, causal=False, status=w["st"], wait_limit_us=1000000)
    yield "attn window", tsg.patch_attn_kv8, (w["q"], c, w["bt"], w["lens"]), dict(workspace=w["ws"], window=7)
    yield "gemm4", tsg.patch_gemm4, (w["x"], w["w4"]), {}
    yield "gemm4 fp16", tsg.patch_gemm4, (w["x"].half(), w["w4"]), dict(status=w["st"])


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def test_same_results(world, monkeypatch):
    c = world["cache"]
    state = lambda: [t.view(torch.uint8).clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]  # noqa: E731
    start = state()
    for name, f, args, kw in calls(world):
        def put_back():
            for t, s in zip((c.k, c.v, c.k_scale, c.v_scale), start):
                t.view(torch.uint8).copy_(s)

        slow = flat(f(*args, **kw, stream=torch.cuda.current_stream()))
        after = state()
        put_back()
        with monkeypatch.context() as m:  # Python's way is shut: the extension has taken the call
            m.setattr(dec, "_call", None)
            fast = flat(f(*args, **kw))
        assert all(torch.equal(x, y) for x, y in zip(state(), after)), name
        put_back()
        assert len(fast) == len(slow), name
        for x, y in zip(fast, slow):
            assert x.dtype == y.dtype and x.stride() == y.stride() and torch.equal(x, y), name
    assert tsg.patch_read_status(world["st"]) == (0, 0)


def test_same_outputs_given(world):
    q, k = world["q"].clone(), world["k"].clone()
    want = tsg.patch_rope(q, k, world["pos"], world["table"])
    got = tsg.patch_rope(q, k, world["pos"], world["table"], q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    out = torch.zeros(B, H + 1, D, dtype=BF16, device="cuda")
    args = (world["q"], world["cache"], world["bt"], world["lens"])
    got = tsg.patch_attn_kv8(*args, out=out[:, 1:], workspace=world["ws"])
    assert torch.equal(got, tsg.patch_attn_kv8(*args, workspace=world["ws"])) and not out[:, 0].any()
    y = torch.zeros(5, 96, dtype=BF16, device="cuda")
    assert tsg.patch_gemm4(world["x"], world["w4"], y) is y and torch.equal(y, tsg.patch_gemm4(world["x"], world["w4"]))


def bad_calls(w):
    """Every one is refused on the host, before any launch."""
    q, k, v, pos, table, c, bt, lens, ws = (w[n] for n in ("q", "k", "v", "pos", "table", "cache", "bt", "lens", "ws"))
    other = tsg.KvCache8(c.k, c.v[:-1], c.k_scale, c.v_scale)
    x, w4 = w["x"], w["w4"]
    for args, kw in (((q, k, pos.long(), table), {}), ((q, k, pos[:2], table), {}), ((q.cpu(), k, pos, table), {}),
                     ((q, k.cpu(), pos, table), {}), ((q, k.half(), pos, table), {}), ((q.double(), None, pos, table), {}),
                     ((q, k, pos, table[..., 0]), {}), ((q[:, :, ::2], None, pos, table), {}), ((q[0], None, pos, table), {}),
                     ((q, k, pos, table), dict(layout="pairs")), ((q, None, pos, table), dict(k_out=k)),
                     ((q, k, pos, table), dict(q_out=k)), ((q, k, pos, table), dict(status=pos.float())),
                     ((q, k, pos, tsg.patch_rope_table(64, 2 * D)), {})):
        yield tsg.patch_rope, args, kw
    for args, kw in (((k, v[:2], c, bt, lens), {}), ((k.float(), v.float(), c, bt, lens), {}), ((k, v, other, bt, lens), {}),
                     ((k, v, c, bt.long(), lens), {}), ((k, v, c, bt[0], lens), {}), ((k, v, c, bt, lens[:2]), {}),
                     ((k, v, c, bt, lens, w["cu"][:3]), {}), ((k[:2], v[:2], c, bt, lens), {}),
                     ((k, v, c, bt, lens), dict(layout=3)), ((q, q, c, bt, lens), {}), ((k, v, c, bt.t(), lens), {})):
        yield tsg.patch_kv8_append, args, kw
    for args, kw in (((q, other, bt, lens), {}), ((q[:, :7], c, bt, lens), {}), ((q.float(), c, bt, lens), {}),
                     ((q, c, bt.cpu(), lens), {}), ((q, c, bt, lens.float()), {}), ((q[:2], c, bt, lens), {}),
                     ((q, c, bt, lens), dict(scale=float("nan"))), ((q, c, bt, lens), dict(window=-1)),
                     ((q, c, bt, lens), dict(out=k)), ((q, c, bt, lens), dict(workspace=ws[:64])),
                     ((q, c, bt, lens), dict(workspace=ws[1:])), ((q, c, bt, lens), dict(workspace=ws.view(torch.int32)))):
        yield tsg.patch_attn_kv8, args, dict(workspace=ws) | kw
    for args, kw in (((x[:, :128], w4), {}), ((x.float(), w4), {}), ((x.t(), w4), {}), ((x, tsg.Weight4(w4.codes, w4.scales, 128)), {}),
                     ((x, tsg.Weight4(w4.codes, w4.scales, 16)), {}), ((x, tsg.Weight4(w4.codes, w4.scales.float(), 64)), {}),
                     ((x.repeat(4, 1), w4), {}), ((x, w4, torch.zeros(5, 95, dtype=BF16, device="cuda")), {}),
                     ((x.cpu(), w4), {})):
        yield tsg.patch_gemm4, args, kw


def test_same_refusals(world):
    for i, (f, args, kw) in enumerate(bad_calls(world)):
        with pytest.raises((ValueError, tsg.PatchError)) as fast:
            f(*args, **kw)
        with pytest.raises((ValueError, tsg.PatchError)) as slow:
            f(*args, **kw, stream=torch.cuda.current_stream())
        assert type(fast.value) is type(slow.value) and str(fast.value) == str(slow.value), (i, f.__name__)
