"""Calls on a stream of their own: what they allocate is allocated, and zero-filled, on that stream (no GPU needed:
allocations and launches are recorded, none is made)."""
import contextlib

import pytest
import torch

import tile_sparse_gemm_b200 as tsg
from tile_sparse_gemm_b200 import decoder as dec

BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32


class FakeStream:
    cuda_stream = 77
    device = torch.device("cpu")


@pytest.fixture
def log(monkeypatch):
    """[(what, stream)] of every allocation, launch and record_stream, in order."""
    events, current = [], ["current"]

    @contextlib.contextmanager
    def stream(s):
        was, current[0] = current[0], s
        yield
        current[0] = was

    for name in ("empty", "zeros"):
        def make(*a, _f=getattr(torch, name), _n=name, **k):
            events.append((_n, current[0]))
            return _f(*a, **k)
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: events.append(("record", s)))
    monkeypatch.setattr(dec, "_cuda", lambda t, name: t.device)
    monkeypatch.setattr(dec, "_call", lambda name, device, stream, *a, **k: events.append(("launch", stream)))
    monkeypatch.setattr(dec, "patch_attn_kv8_workspace_size", lambda *a: 4096)
    return events


def check(events, s, outputs, workspaces=0):
    made = [e for e in events if e[0] in ("empty", "zeros")]
    assert made == [("empty", s)] * outputs + [("zeros", s)] * workspaces, events
    # what is returned may be used on the caller's stream and dropped there
    assert events.count(("record", "current")) == outputs, events
    assert ("launch", s) in events and events.index(("launch", s)) > max(map(events.index, made))


def test_decoder_calls(log):
    s = FakeStream()
    q = torch.ones(3, 4, 64, dtype=BF16)
    pos, table = torch.ones(3, dtype=I32), torch.ones(8, 32, 2)
    tsg.patch_rope(q, q, pos, table, stream=s)
    check(log, s, 2)
    log.clear()
    tsg.patch_rope_table(8, 64, device="cpu", stream=s)
    check(log, s, 1)
    cache = tsg.KvCache8(*(torch.ones(5, 4, 16, 64).to(torch.float8_e4m3fn) for _ in range(2)), *(torch.ones(5, 4) for _ in range(2)))
    log.clear()
    tsg.patch_attn_kv8(q, cache, torch.ones(3, 2, dtype=I32), pos, want_lse=True, stream=s)
    check(log, s, 2, 1)
    w = tsg.Weight4(torch.ones(6, 32, dtype=torch.uint8), torch.ones(6, 1, dtype=BF16), 64)
    log.clear()
    tsg.patch_gemm4(torch.ones(2, 64, dtype=BF16), w, stream=s)
    check(log, s, 1)
    log.clear()
    tsg.patch_quantize4(torch.ones(6, 64), 64, stream=s)
    check(log, s, 2)


class FakeLib:
    """Every entry point returns PATCH_OK; those that take a stream are launches on it."""

    def __init__(self, events):
        self.events = events

    def __getattr__(self, name):
        def call(*a):
            if not name.endswith("_size") and not name.endswith("_sizes"):
                at = next(x for x in a if getattr(x, "value", None) == FakeStream.cuda_stream)
                self.events.append(("launch", at.value))
            return 0
        return call


def test_hybrid_calls(log, monkeypatch):
    s = FakeStream()
    monkeypatch.setattr(tsg, "lib", lambda: FakeLib(log))
    monkeypatch.setattr(tsg, "_dev", lambda t, name: None)
    N = K = 128
    u8 = torch.uint8
    W, x = torch.ones(N, K, dtype=BF16), torch.ones(4, K, dtype=BF16)
    pw = tsg.PackedWeight(N, K, 0, torch.ones(16, dtype=u8), torch.ones(16, dtype=u8), torch.ones(16, dtype=u8))
    for call in (lambda: tsg.patch_gemm(x, pw, stream=s), lambda: tsg.patch_gemm_chain([(x, pw, None, False)], stream=s),
                 lambda: tsg.patch_gemm_group([(x, pw, None)], stream=s), lambda: tsg.patch_gemm_mlp(x, pw, pw, stream=s),
                 lambda: tsg.patch_check_weight(pw, stream=s)):
        log.clear()
        call()
        made = [e[1] for e in log if e[0] in ("empty", "zeros")]
        assert made and all(m is s for m in made), log
        assert log[-1] == ("launch", FakeStream.cuda_stream), log
