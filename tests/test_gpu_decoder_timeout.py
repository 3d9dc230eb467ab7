"""Attention's bounded waits with a limit of 1 us.  Where one runs out, its copies still under way, the kernel reports
it, lets them land and returns; after zeroing the workspace the same call gives its results.  The 128-row tiles wait
for products and conversions and do run out; copies alone, which the few-row tiles wait for, may come before the
limit is looked at."""
import math

import pytest
import torch

import _decoder_ref as ref
import tile_sparse_gemm_b200 as tsg
from test_gpu_decoder import gen, i32, pages_of, random_cache, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("kv,q", [([8000 - 37 * i for i in range(48)], [1] * 48), ([4000 + 99 * i for i in range(24)], [3, 4, 2, 3] * 6),
                                  ([2500, 300, 5000], [400, 70, 130])])
def test_attn_wait_that_runs_out(kv, q):
    g = gen(61)
    H, Hk, D, page = 32, 8, 128, 32
    bt, n_pages = pages_of(kv, page, g)
    cache = random_cache(n_pages, Hk, page, D, g)
    cu = [sum(q[:i]) for i in range(len(q) + 1)]
    x = torch.randn(cu[-1], H, D, generator=g, device="cuda").to(BF16)
    args = (x, cache, bt, i32(kv), i32(cu))
    ws = torch.zeros(tsg.patch_attn_kv8_workspace_size(cu[-1], len(kv), H, cache), dtype=torch.uint8, device="cuda")
    want, lse, bound = ref.attention(x, cache.k, cache.v, cache.k_scale, cache.v_scale, bt, kv, cu, 1 / math.sqrt(D))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    ran_out = 0
    for _ in range(5):
        flush.fill_(1)  # the cache is not in L2: its copies take longer than the limit
        st = tsg.new_status()
        out = tsg.patch_attn_kv8(*args, workspace=ws, status=st, wait_limit_us=1)
        code, bits = tsg.patch_read_status(st)
        assert (code, bits) in ((0, 0), (7, tsg.DEV_TIMEOUT))
        if code:
            ran_out += 1
            ws.zero_()
        else:
            within(out, want, bound)
        st.zero_()
        out = tsg.patch_attn_kv8(*args, workspace=ws, status=st)
        assert tsg.patch_read_status(st) == (0, 0)
        within(out, want, bound, "after the timeout")
        assert not ws[: 4 * 148].any()
    assert ran_out > 0 or max(q) < 64
