"""Calls on a stream of their own while the current one is busy: results, workspaces and zero-fills are that stream's."""
import pytest
import torch

import tile_sparse_gemm_b200 as tsg
from test_gpu_decoder import gen, i32, random_cache

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def busy_and_dirty(nbytes):
    """Work for the current stream, and memory on it, freed, that holds anything but zeros."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.full((nbytes,), 0xAB, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    del t


@pytest.mark.parametrize("m", [1, 100])
def test_attn_without_a_workspace(m):
    """A tile cut between CTAs counts arrivals in the workspace, whose zeros must come before them."""
    g = gen(51)
    n, H = 20000, 8
    cache = random_cache(n // 64 + 1, 2, 64, 128, g)
    bt = torch.randperm(n // 64 + 1, generator=g, device="cuda").to(torch.int32)[None]
    q = torch.randn(m, H, 128, generator=g, device="cuda").to(BF16)
    args = (q, cache, bt, i32([n]), i32([0, m]))
    want, lse = tsg.patch_attn_kv8(*args, want_lse=True)
    size = tsg.patch_attn_kv8_workspace_size(m, 1, H, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        busy_and_dirty(size)
        out, l = tsg.patch_attn_kv8(*args, want_lse=True, stream=s)
        s.synchronize()
        with torch.cuda.stream(s):
            same = torch.equal(out, want) and torch.equal(l, lse)
        assert same
        torch.cuda.synchronize()


def test_results_outlive_their_last_use_on_the_callers_stream():
    """A result dropped while the caller's stream still reads it is not handed out to the other stream's next call."""
    g = gen(52)
    w = tsg.patch_quantize4(torch.randn(4096, 512, generator=g, device="cuda"))
    x = torch.randn(8, 512, generator=g, device="cuda").to(BF16)
    want = tsg.patch_gemm4(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = tsg.patch_gemm4(x, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    got = y + 0  # read late on the caller's stream
    del y
    other = [tsg.patch_gemm4(-x, w, stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(o, -want) for o in other)


def test_hybrid_decode_gemm_without_a_workspace():
    """The decode kernel's counters and sums lie in a workspace that must be zero before it runs."""
    import oracle
    import synth_inputs as si
    from _util import bits_of, check_gemm, to_dev, to_dev_bf16

    N, K, M = 2048, 2048, 16
    w, bm = si.gen_w(N, K, 3, 1), si.tiles_exact(N, K, 0.5, 3, 1)
    ids = si.patterns_top2(w)
    pw = tsg.patch_pack(to_dev_bf16(w), to_dev(bm), to_dev(ids), int(bm.sum()))
    x = si.gen_x(M, K, 3, 2)
    xd = to_dev_bf16(x)
    want = oracle.hybrid_gemm(x, w, bm, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call in (lambda: tsg.patch_gemm(xd, pw, stream=s), lambda: tsg.patch_gemm_chain([(xd, pw, None, False)], stream=s)[0],
                 lambda: tsg.patch_gemm_group([(xd, pw, None)], stream=s)[0]):
        busy_and_dirty(tsg.patch_gemm_workspace_size(M, pw))
        y = call()
        s.synchronize()
        with torch.cuda.stream(s):
            got = bits_of(y)
        check_gemm(got, want, "another stream")
        torch.cuda.synchronize()
