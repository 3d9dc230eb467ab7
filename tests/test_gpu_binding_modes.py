"""Under a torch dispatch mode the decoder-layer calls allocate where the mode sees it."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import tile_sparse_gemm_b200 as tsg

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.ops = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.ops.append(str(func))
        return func(*args, **(kwargs or {}))


def test_outputs_are_allocated_through_the_dispatcher():
    x = torch.randn(2, 4, 64, device="cuda").bfloat16()
    pos, table = torch.zeros(2, dtype=torch.int32, device="cuda"), tsg.patch_rope_table(8, 64)
    cache = tsg.new_kv_cache8(2, 4, 16, 64)
    bt, one = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    w = tsg.patch_quantize4(torch.randn(32, 64, device="cuda"), 64)
    y = torch.randn(3, 64, device="cuda").bfloat16()
    for call, outputs in ((lambda: tsg.patch_rope(x, x, pos, table), 2),
                          (lambda: tsg.patch_attn_kv8(x[:1], cache, bt, one, want_lse=True, workspace=ws), 2),
                          (lambda: tsg.patch_gemm4(y, w), 1)):
        plain = call()
        with Seen() as mode:
            seen = call()
        assert sum("aten.empty" in op for op in mode.ops) == outputs, mode.ops
        for a, b in zip(plain if outputs > 1 else (plain,), seen if outputs > 1 else (seen,)):
            assert torch.equal(a, b)
