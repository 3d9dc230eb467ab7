"""The decoder layer beside its linears: rotary positions, a paged 8-bit
key/value cache and attention over it, and linears with 4-bit weights.

Thin binding over the C ABI (include/patch.h), like the rest of the package: it
checks and marshals arguments, every step runs in the library's sm_100a
kernels.  The calls run on the tensors' own device and on `stream` (default:
that device's current stream), launch only libpatch kernels, allocate only the
outputs and workspace they are not given (on that stream), never synchronise and
can be captured in a CUDA graph.  Who passes a `stream` orders it after the inputs'
writers and before the results' readers, and keeps the inputs until it is done.  A
device status word is optional: `status=new_status()` collects what the kernels report
(patch_read_status).  Nothing is recorded for autograd; patch_rope(backward=True) is
the gradient of patch_rope.

The calls of a decode step take less time on the device than their checks take
in Python, so the ordinary ones (as documented, current device and stream) go
through a compiled extension, csrc/decoder_binding.cpp.  It leaves every other
call, the wrong ones among them, to the same checks here, which name the fault;
without it (another torch than it was built for) all calls come here.
"""
from __future__ import annotations

import ctypes
import math
import warnings
from dataclasses import dataclass

import torch

from . import PatchError, _check, _new, lib

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # PATCH_DTYPE_*
LAYOUTS = {"half": 0, "interleaved": 1}                           # PATCH_ROPE_HALF / PATCH_ROPE_INTERLEAVED
ROPE_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}  # PATCH_ROPE_*
KV8_PAGES = (16, 32, 64, 128)
KV8_HEAD_DIMS = (64, 128)
GROUPS4 = (32, 64, 128)


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _RopeConfig(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_positions", "low_freq", "high_freq", "amplitude")]


class _Cache8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int64) for n in ("n_pages", "kv_heads", "page", "head_dim")]


class _Weight4(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


def signatures() -> dict:
    """ctypes argument types of this module's entry points."""
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    H, C, W = (ctypes.POINTER(t) for t in (_Heads, _Cache8, _Weight4))
    return {
        "patch_rope_table": [I64, I64, ctypes.POINTER(_RopeConfig), P, P],
        "patch_rope": [H, H, H, H, I64, I64, I32, P, P, I64, I64, I32, I32, P, P],
        "patch_kv8_append": [H, H, I64, I32, C, P, I64, P, P, I64, P, I64, I64, I32, P, P],
        "patch_attn_kv8_workspace_size": [I64, I64, I64, C, ctypes.POINTER(SZ)],
        "patch_attn_kv8": [H, I64, I32, C, P, I64, P, P, I64, ctypes.c_float, I32, I64, H, P, P, SZ, P, P,
                           ctypes.c_uint64],
        "patch_quantize4": [P, I32, W, P],
        "patch_gemm4": [P, I64, I32, W, P, P, P],
    }


_byref = ctypes.byref
# the current device and stream without torch.cuda's wrappers (absent from CPU-only builds of torch)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_binding = None


class _ThroughPython:
    """In the place of the extension: leaves every call to the way through Python."""

    @staticmethod
    def rope(*_):
        return None

    append = attn = gemm4 = rope


def _fast():
    """The compiled extension, bound to the library's entry points; where it is missing, the same calls are made from here."""
    global _binding
    if _binding is None:
        library = lib()
        try:
            from . import _decoder_binding
        except ImportError as e:
            warnings.warn(f"the compiled binding is missing or was built for another torch ({e}): calls take their way through "
                          "Python, some 10 us more each; build it with `python -m tile_sparse_gemm_b200.build`", stacklevel=3)
            _binding = _ThroughPython
        else:
            _decoder_binding.bind(*(ctypes.cast(getattr(library, "patch_" + f), ctypes.c_void_p).value
                                    for f in ("rope", "kv8_append", "attn_kv8", "gemm4")))
            _binding = _decoder_binding
    return _binding


def _call(name: str, device: torch.device, stream, *args, tail=()):
    """Run a C entry point with `device` current: name(*args, stream, *tail)."""
    f = getattr(lib(), name)
    index = device.index
    if _raw_device() != index:
        with torch.cuda.device(device):
            code = f(*args, _raw_stream(index) if stream is None else stream.cuda_stream, *tail)
    else:
        code = f(*args, _raw_stream(index) if stream is None else stream.cuda_stream, *tail)
    if code:
        _check(code, name)


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    """The device of the tensor that decides a call's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _tensor(t: torch.Tensor, name: str, device, dtype, shape=None) -> int:
    """Address of a contiguous tensor of this device, type and shape."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous() or (shape is not None and t.shape != shape):
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype(t: torch.Tensor, name: str, allowed=(torch.bfloat16, torch.float16)) -> int:
    d = t.dtype
    if d not in allowed:
        raise ValueError(f"{name} is {d}, expected one of {[str(x) for x in allowed]}")
    return DTYPES[d]


def _heads(t: torch.Tensor, name: str, device, dtype, shape=None) -> _Heads:
    """[T][H][D] rows of heads: any token and head strides, elements in a row."""
    if t.dtype is not dtype or t.device != device or t.dim() != 3 or (shape is not None and t.shape != shape):
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
        if t.dim() != 3:
            raise ValueError(f"{name} must be [tokens][heads][head_dim]")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    tok, head, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return _Heads(t.data_ptr(), t.shape[1], tok, head)


def _new_heads(t: torch.Tensor, stream) -> tuple[torch.Tensor, _Heads]:
    """A contiguous output of t's shape, type and device."""
    T, H, D = t.shape
    out = _new((T, H, D), t.dtype, t.device, stream)
    return out, _Heads(out.data_ptr(), H, H * D, D)


def _status(status, device) -> int | None:
    return None if status is None else _tensor(status, "status", device, torch.int32)


# ---- rotary positions


def patch_rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_positions: float = 0.0, low_freq: float = 1.0, high_freq: float | None = None,
                     amplitude: float | None = None, device="cuda", stream=None) -> torch.Tensor:
    """(cos, sin) of every position's angles, fp32 [n_pos][rot_dim // 2][2], from 64-bit angles.

    scaling for long contexts: "plain", "linear" (positions divided by factor),
    "bands" (by wavelength against original_positions: LLaMA-3's rule, low_freq 1
    and high_freq 4 by default) or "yarn" (a ramp between the pairs that turn
    low_freq, 1, and high_freq, 32, times; amplitude 0.1 ln(factor) + 1 by default)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r}, expected one of {list(ROPE_SCALINGS)}")
    if high_freq is None:
        high_freq = 32.0 if scaling == "yarn" else 4.0
    if amplitude is None:
        amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
    cfg = _RopeConfig(ROPE_SCALINGS[scaling], 0, base, factor, original_positions, low_freq, high_freq, amplitude)
    if n_pos < 1 or rot_dim < 2:
        raise PatchError(2, "patch_rope_table")
    table = _new((n_pos, rot_dim // 2, 2), torch.float32, device, stream)
    _call("patch_rope_table", table.device, stream, n_pos, rot_dim, _byref(cfg), table.data_ptr())
    return table


def _table(table: torch.Tensor, device) -> tuple[int, int, int]:
    p = _tensor(table, "table", device, torch.float32)
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError("table must be [n_pos][rot_dim // 2][2] (patch_rope_table)")
    return p, shape[0], 2 * shape[1]


def _layout(layout: str) -> int:
    if layout not in LAYOUTS:
        raise ValueError(f"layout {layout!r}, expected one of {list(LAYOUTS)}")
    return LAYOUTS[layout]


def patch_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: torch.Tensor,
               layout: str = "half", backward: bool = False, q_out: torch.Tensor | None = None,
               k_out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Rotary positions of q [T][H][D] and k [T][Hk][D] (or None) in one launch: (q_out, k_out).

    bf16, fp16 or fp32; any token and head strides (slices of a fused q|k|v
    projection).  The first 2 * table.shape[1] elements of each head turn, the
    rest is copied.  positions int32 [T]; a token at -1 (padding) is skipped.
    backward=True turns the other way (times the table's amplitude): the
    gradient of the inputs from the gradient of the outputs.  Pass
    q_out=q, k_out=k to work in place."""
    if stream is None:
        r = _fast().rope(q, k, positions, table, layout, backward, q_out, k_out, status)
        if type(r) is int and r:
            _check(r, "patch_rope")
        if r is not None:
            return r
    dev, dtype = _cuda(q, "q"), q.dtype
    hq = _heads(q, "q", dev, dtype)
    dt = _dtype(q, "q", DTYPES)
    T, _, D = q.shape
    tab, n_pos, rot = _table(table, dev)
    pos = _tensor(positions, "positions", dev, torch.int32, (T,))
    if q_out is None:
        q_out, ho = _new_heads(q, stream)
    else:
        ho = _heads(q_out, "q_out", dev, dtype, q.shape)
    hk = hko = None
    if k is not None:
        hk = _byref(_heads(k, "k", dev, dtype, (T, k.shape[1], D)))
        if k_out is None:
            k_out, hko = _new_heads(k, stream)
        else:
            hko = _heads(k_out, "k_out", dev, dtype, k.shape)
        hko = _byref(hko)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call("patch_rope", dev, stream, _byref(hq), hk, _byref(ho), hko, T, D, dt, pos, tab, n_pos, rot, _layout(layout),
          1 if backward else 0, None if status is None else _status(status, dev))
    return q_out, k_out


# ---- the paged 8-bit cache


@dataclass
class KvCache8:
    """A paged key/value cache in 8 bits: e4m3 pages [n_pages][kv_heads][page][head_dim] and
    one power-of-two scale per page and head, fp32 [n_pages][kv_heads], for keys and for values."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def struct(self) -> _Cache8:
        k = self.k
        shape, f8, dev = k.shape, torch.float8_e4m3fn, k.device
        if len(shape) != 4:
            raise ValueError("cache.k must be [n_pages][kv_heads][page][head_dim]")
        n, h, page, d = shape
        return _Cache8(_tensor(k, "cache.k", dev, f8), _tensor(self.v, "cache.v", dev, f8, shape),
                       _tensor(self.k_scale, "cache.k_scale", dev, torch.float32, (n, h)),
                       _tensor(self.v_scale, "cache.v_scale", dev, torch.float32, (n, h)), n, h, page, d)

    @property
    def stored_bytes(self) -> int:
        return 2 * self.k.numel() + 8 * self.k_scale.numel()


def new_kv_cache8(n_pages: int, kv_heads: int, page: int, head_dim: int, device="cuda") -> KvCache8:
    """An empty cache of n_pages pages of `page` tokens."""
    if page not in KV8_PAGES or head_dim not in KV8_HEAD_DIMS:
        raise ValueError(f"page {page} (expected {KV8_PAGES}) or head_dim {head_dim} (expected {KV8_HEAD_DIMS})")
    k, v = (torch.zeros((n_pages, kv_heads, page, head_dim), dtype=torch.float8_e4m3fn, device=device)
            for _ in range(2))
    return KvCache8(k, v, *(torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)))


def _block_table(block_table: torch.Tensor, device) -> tuple[int, int, int]:
    p = _tensor(block_table, "block_table", device, torch.int32)
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [batch][max_pages]")
    return p, shape[0], shape[1]


def patch_kv8_append(k: torch.Tensor, v: torch.Tensor, cache: KvCache8, block_table: torch.Tensor,
                     past_lens: torch.Tensor, cu_new: torch.Tensor | None = None, table: torch.Tensor | None = None,
                     layout: str = "half", status: torch.Tensor | None = None, stream=None) -> None:
    """Store new tokens' keys and values (bf16 or fp16 [T][Hk][D], any token and head strides) in the cache.

    Sequence b holds past_lens[b] tokens (int32) and gets rows cu_new[b] ..
    cu_new[b + 1] - 1 (int32 [batch + 1]; None: one token each) at the positions
    that follow, in the pages of block_table (int32 [batch][max_pages]).  With a
    table (patch_rope_table) the keys are rotated to their positions on the way."""
    if stream is None:
        r = _fast().append(k, v, cache.k, cache.v, cache.k_scale, cache.v_scale, block_table, past_lens, cu_new, table,
                           layout, status)
        if type(r) is int and r:
            _check(r, "patch_kv8_append")
        if r is not None:
            return
    dev, dtype = _cuda(cache.k, "cache.k"), k.dtype
    c = cache.struct()
    dt = _dtype(k, "k")
    T = k.shape[0]
    shape = (T, c.kv_heads, c.head_dim)
    hk, hv = _heads(k, "k", dev, dtype, shape), _heads(v, "v", dev, dtype, shape)
    bt, batch, max_pages = _block_table(block_table, dev)
    past = _tensor(past_lens, "past_lens", dev, torch.int32, (batch,))
    cu = None if cu_new is None else _tensor(cu_new, "cu_new", dev, torch.int32, (batch + 1,))
    tab, n_pos, rot = (None, 0, 0) if table is None else _table(table, dev)
    _call("patch_kv8_append", dev, stream, _byref(hk), _byref(hv), T, dt, _byref(c), bt, max_pages, past, cu, batch,
          tab, n_pos, rot, _layout(layout), _status(status, dev))


def patch_attn_kv8_workspace_size(n_tokens: int, batch: int, q_heads: int, cache: KvCache8) -> int:
    b, c = ctypes.c_size_t(), cache.struct()
    with torch.cuda.device(cache.k.device):
        _check(lib().patch_attn_kv8_workspace_size(n_tokens, batch, q_heads, ctypes.byref(c), ctypes.byref(b)),
               "patch_attn_kv8_workspace_size")
    return b.value


def patch_attn_kv8(q: torch.Tensor, cache: KvCache8, block_table: torch.Tensor, kv_lens: torch.Tensor,
                   cu_q: torch.Tensor | None = None, scale: float | None = None, causal: bool = True, window: int = 0,
                   out: torch.Tensor | None = None, want_lse: bool = False, workspace: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, wait_limit_us: int = 0, stream=None):
    """Attention of q (bf16 or fp16 [T][H][D]) over the cache: out, or (out, lse fp32 [T][H]) with want_lse.

    Sequence b's queries are rows cu_q[b] .. cu_q[b + 1] - 1 (None: one each)
    and it holds kv_lens[b] tokens, its new ones included (int32 both).  causal:
    a query sees the tokens up to its own position; window > 0: only the last
    `window` of them.  A query that sees none gives zeros and lse -inf.  scale
    defaults to 1 / sqrt(D).  workspace: patch_attn_kv8_workspace_size bytes
    (uint8), zero-filled once, reusable by any later call on the same stream."""
    if stream is None:
        r = _fast().attn(q, cache.k, cache.v, cache.k_scale, cache.v_scale, block_table, kv_lens, cu_q, scale, causal, window,
                         out, want_lse, workspace, status, wait_limit_us)
        if type(r) is int and r:
            _check(r, "patch_attn_kv8")
        if r is not None:
            return r
    dev, dtype = _cuda(cache.k, "cache.k"), q.dtype
    c = cache.struct()
    hq = _heads(q, "q", dev, dtype)
    dt = _dtype(q, "q")
    T, H, D = shape = q.shape
    if D != c.head_dim or H % c.kv_heads:
        raise ValueError(f"q has {H} heads of {D}, the cache {c.kv_heads} of {c.head_dim}")
    bt, batch, max_pages = _block_table(block_table, dev)
    lens = _tensor(kv_lens, "kv_lens", dev, torch.int32, (batch,))
    cu = None if cu_q is None else _tensor(cu_q, "cu_q", dev, torch.int32, (batch + 1,))
    if out is None:
        out, ho = _new_heads(q, stream)
    else:
        ho = _heads(out, "out", dev, dtype, shape)
    lse = _new((T, H), torch.float32, dev, stream) if want_lse else None
    if workspace is None:
        workspace = _new((max(patch_attn_kv8_workspace_size(T, batch, H, cache), 16),), torch.uint8, dev, stream, zero=True)
    ws = _tensor(workspace, "workspace", dev, torch.uint8)
    _call("patch_attn_kv8", dev, stream, _byref(hq), T, dt, _byref(c), bt, max_pages, lens, cu, batch,
          1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, window, _byref(ho),
          None if lse is None else lse.data_ptr(), ws, workspace.numel(), _status(status, dev), tail=(wait_limit_us,))
    return (out, lse) if want_lse else out


# ---- linears with 4-bit weights


@dataclass
class Weight4:
    """A linear weight in 4 bits: W[n][k] = (code - 8) * scales[n][k // group], codes
    u8 [N][K // 2] with the even k in the low half of a byte."""
    codes: torch.Tensor
    scales: torch.Tensor  # bf16 or fp16 [N][K // group]
    group: int

    @property
    def N(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return 2 * self.codes.shape[1]

    def struct(self) -> _Weight4:
        codes, scales, group = self.codes, self.scales, self.group
        if group not in GROUPS4:
            raise ValueError(f"group {group}, expected one of {GROUPS4}")
        shape = codes.shape
        if len(shape) != 2 or 2 * shape[1] % group:
            raise ValueError(f"codes must be [N][K / 2] with K a multiple of the group ({group})")
        n, k, dev = shape[0], 2 * shape[1], codes.device
        return _Weight4(n, k, group, _dtype(scales, "scales"), _tensor(codes, "codes", dev, torch.uint8),
                        _tensor(scales, "scales", dev, scales.dtype, (n, k // group)))

    @property
    def stored_bytes(self) -> int:
        return self.codes.numel() + self.scales.numel() * self.scales.element_size()


def patch_quantize4(W: torch.Tensor, group: int = 128, scale_dtype: torch.dtype = torch.bfloat16,
                    stream=None) -> Weight4:
    """W (bf16, fp16 or fp32 [N][K]) to 4 bits by rounding under per-group scales amax / 7."""
    if W.dim() != 2:
        raise ValueError("W must be [N][K]")
    N, K = W.shape
    if group not in GROUPS4 or K % group:
        raise ValueError(f"group {group}: expected one of {GROUPS4} that divides K = {K}")
    if scale_dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"scale_dtype {scale_dtype}, expected torch.bfloat16 or torch.float16")
    dev = _cuda(W, "W")
    p = _tensor(W, "W", dev, W.dtype)
    w4 = Weight4(_new((N, K // 2), torch.uint8, dev, stream), _new((N, K // group), scale_dtype, dev, stream), group)
    st = w4.struct()
    _call("patch_quantize4", dev, stream, p, _dtype(W, "W", DTYPES), _byref(st))
    return w4


def patch_gemm4(X: torch.Tensor, weight: Weight4, Y: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X * W^T for up to 16 tokens (bf16 or fp16 [M][K]) and a 4-bit weight, fp32 sums."""
    if stream is None:
        r = _fast().gemm4(X, weight.codes, weight.scales, weight.group, Y, status)
        if type(r) is int and r:
            _check(r, "patch_gemm4")
        if r is not None:
            return r
    dev, dtype = _cuda(weight.codes, "codes"), X.dtype
    st = weight.struct()
    n, k = st.N, st.K
    if X.dim() != 2 or X.shape[1] != k:
        raise ValueError(f"X has shape {tuple(X.shape)}, weight has K={k}")
    M = X.shape[0]
    dt = _dtype(X, "X")
    x = _tensor(X, "X", dev, dtype)
    if Y is None:
        Y = _new((M, n), dtype, dev, stream)
    _call("patch_gemm4", dev, stream, x, M, dt, _byref(st), _tensor(Y, "Y", dev, dtype, (M, n)),
          _status(status, dev))
    return Y
