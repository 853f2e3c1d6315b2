"""Exact IO-aware attention for NVIDIA B200 (sm_100a): Python binding.

A thin ctypes layer over the C ABI in include/fa.h (libfa_b200.so, built
in-tree by `python exact_io_aware_44_b200/build.py`). It only marshals
arguments: it checks shapes and dtypes, allocates outputs with torch, and
passes raw device pointers and the current CUDA stream. Every step of the
attention path runs in the library's CUDA kernels. There is no CPU fallback:
importing this package fails if the library is missing.

    o, lse = fwd(q, k, v, causal=True)           # bf16 (tensor cores) or fp32
    dq, dk, dv = bwd(q, k, v, o, lse, do, causal=True)

Serving from a cache (d = 128): `decode` (bf16), `cache_store` and `decode_fp8` (8 bits,
a scale for each block of tokens and head), `block_bounds`, `select_blocks` and
`decode_blocks` (only the blocks that a bound of the scores selects), `cache_weights` and
`cache_evict` (keep the tokens that attention uses).

Layouts: q, o, do: [B, Hq, N, d]; k, v: [B, Hkv, N, d]; lse: [B, Hq, N] float32.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

__all__ = ["head_shard", "fwd", "fwd_fp8", "decode", "decode_raw", "decode_workspace_bytes", "bwd", "fwd_raw", "fwd_fp8_raw", "bwd_raw", "bwd_phases_raw", "workspace_bytes", "get_status", "set_wait_budget_ns",
           "selftest_wait_timeout", "get_progress", "FAError", "LIB_PATH", "lib", "STATUS",
           "cache_store", "decode_fp8", "block_bounds", "select_blocks", "decode_blocks", "cache_weights", "cache_evict",
           "decode_fp8_workspace_bytes", "select_blocks_workspace_bytes", "decode_blocks_workspace_bytes"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa_b200.so")

STATUS = {0: "FA_OK", -1: "FA_ERR_INVALID_ARG", -2: "FA_ERR_UNSUPPORTED", -3: "FA_ERR_ALIGNMENT",
          -4: "FA_ERR_LAUNCH", -5: "FA_ERR_DEVICE_TIMEOUT", -6: "FA_ERR_NO_DEVICE"}

# exported symbols and their C signatures (must match include/fa.h)
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
SIGNATURES = {
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_fwd_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_fwd_fp8": (_I, [_P, _P, _P, _F, _F, _F, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_fwd_e5m2": (_I, [_P, _P, _P, _F, _F, _F, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "fa_decode_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_bwd_preprocess": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_bwd_main": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_bwd_convert": (_I, [_P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "fa_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "fa_get_status": (_I, [_P]),
    "fa_get_progress": (_I, [_P, _I, _P]),
    "fa_set_wait_budget_ns": (None, [ctypes.c_uint64]),
    "fa_selftest_wait_timeout": (_I, [ctypes.c_uint64, _P]),
    "fa_cache_store": (_I, [_P] * 7 + [_I] * 6 + [_P]),
    "fa_block_bounds": (_I, [_P] * 3 + [_I] * 7 + [_P]),
    "fa_select_blocks_workspace_bytes": (ctypes.c_size_t, [_I] * 7),
    "fa_select_blocks": (_I, [_P] * 6 + [_I] * 12 + [_P]),
    "fa_decode_fp8_workspace_bytes": (ctypes.c_size_t, [_I] * 8),
    "fa_decode_fp8": (_I, [_P] * 9 + [_I] * 8 + [_F, _I, _P]),
    "fa_decode_blocks_workspace_bytes": (ctypes.c_size_t, [_I] * 10),
    "fa_decode_blocks": (_I, [_P] * 10 + [_I] * 10 + [_F, _I, _P]),
    "fa_cache_weights": (_I, [_P] * 6 + [_I] * 9 + [_F, _P]),
    "fa_cache_evict": (_I, [_P] * 13 + [_I] * 9 + [_P]),
    "fa_error_string": (ctypes.c_char_p, [_I]),
    "fa_version": (_I, []),
}


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = lib.fa_error_string(code).decode() if lib is not None else STATUS.get(code, "?")
        super().__init__(f"{where}: {STATUS.get(code, code)} ({msg})")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python exact_io_aware_44_b200/build.py` "
                          "(there is no CPU fallback)")
    so = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(so, name)
        fn.restype = res
        fn.argtypes = args
    return so


lib = _load()


def _check(code: int, where: str):
    if code != 0:
        raise FAError(code, where)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, Hq, N, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, Nk, dk) != (B, N, d):
        raise ValueError(f"k shape {tuple(k.shape)} does not match q shape {tuple(q.shape)}")
    return B, Hq, Hkv, N, d


def _require(t, name, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, Hq, Hkv, N, d, causal, scale, stream_ptr, f32=False):
    """The C call itself on raw device pointers (ints); returns the status code."""
    fn = lib.fa_fwd_f32 if f32 else lib.fa_fwd
    return fn(_P(q_ptr), _P(k_ptr), _P(v_ptr), _P(o_ptr), _P(lse_ptr), B, Hq, Hkv, N, d, int(bool(causal)),
              float(scale), _P(stream_ptr))


def fwd(q, k, v, causal: bool = True, scale: float | None = None, out=None, lse=None, stream=None):
    """Forward pass. bf16 inputs run on the tensor cores (d in {64, 128, 256});
    float32 inputs run the fp32 CUDA-core kernel. Returns (o, lse)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q, k, v must be bfloat16 or float32")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, dtype, q.device)
    if v.shape != k.shape:
        raise ValueError("v must have the shape of k")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    _require(out, "out", dtype, q.device)
    _require(lse, "lse", torch.float32, q.device)
    fn = lib.fa_fwd_f32 if dtype == torch.float32 else lib.fa_fwd
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, int(bool(causal)), scale,
              _stream_ptr(stream)), "fa_fwd")
    return out, lse


def fwd_fp8_raw(q_ptr, k_ptr, v_ptr, descale_q, descale_k, descale_v, o_ptr, lse_ptr, B, Hq, Hkv, N, d, causal,
                scale, stream_ptr, e5m2=False):
    """fa_fwd_fp8 (or fa_fwd_e5m2) on raw device pointers (ints); returns the status code."""
    fn = lib.fa_fwd_e5m2 if e5m2 else lib.fa_fwd_fp8
    return fn(_P(q_ptr), _P(k_ptr), _P(v_ptr), float(descale_q), float(descale_k), float(descale_v),
              _P(o_ptr), _P(lse_ptr), B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _P(stream_ptr))


def fwd_fp8(q, k, v, descale_q: float, descale_k: float, descale_v: float, causal: bool = True,
            scale: float | None = None, out=None, lse=None, stream=None):
    """Forward pass on FP8 inputs (torch.float8_e4m3fn or torch.float8_e5m2, all
    three the same, d = 128) with one descale per tensor: the real inputs are
    descale_q * q, descale_k * k, descale_v * v. Returns (o, lse) with o in bf16.
    `scale` defaults to 1/sqrt(d)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if q.dtype not in (torch.float8_e4m3fn, torch.float8_e5m2):
        raise TypeError("q, k, v must be torch.float8_e4m3fn or torch.float8_e5m2")
    e5m2 = q.dtype == torch.float8_e5m2
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, q.dtype, q.device)
    if v.shape != k.shape:
        raise ValueError("v must have the shape of k")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    _require(out, "out", torch.bfloat16, q.device)
    _require(lse, "lse", torch.float32, q.device)
    fn = lib.fa_fwd_e5m2 if e5m2 else lib.fa_fwd_fp8
    _check(fn(_ptr(q), _ptr(k), _ptr(v), float(descale_q), float(descale_k), float(descale_v), _ptr(out),
              _ptr(lse), B, Hq, Hkv, N, d, int(bool(causal)), scale, _stream_ptr(stream)), "fa_fwd_fp8")
    return out, lse


def head_shard(B: int, Hq: int, Hkv: int, rank: int, world: int):
    """The query and key/value heads one rank computes when a problem is split
    across `world` GPUs by heads (no exchange between ranks: every (batch, kv head)
    group is independent in the forward and the backward).

    Heads are counted on the flattened [B * H] axis of the [B, H, N, d] layout, so
    a rank's share is one contiguous slice: query heads [q0, q1) and kv heads
    [k0, k1), cut at GQA group boundaries, with group counts differing by at most
    one between ranks. The slice is a valid problem of its own with B = 1,
    Hq = q1 - q0, Hkv = k1 - k0 (query head i of the slice reads kv head
    i // (Hq / Hkv) of its slice). Returns (q0, q1, k0, k1); an empty slice when
    world exceeds the number of groups."""
    if world < 1 or not 0 <= rank < world or Hkv < 1 or Hq % Hkv:
        raise ValueError("invalid shard request")
    groups, g = B * Hkv, Hq // Hkv
    base, extra = divmod(groups, world)
    k0 = rank * base + min(rank, extra)
    k1 = k0 + base + (1 if rank < extra else 0)
    return k0 * g, k1 * g, k0, k1


def decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits=0) -> int:
    return int(lib.fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, int(num_splits)))


def decode_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, ws_ptr, B, Hq, Hkv, Nq, Nk, d, causal, scale, num_splits,
               stream_ptr):
    """fa_decode on raw device pointers (ints); returns the status code."""
    return lib.fa_decode(_P(q_ptr), _P(k_ptr), _P(v_ptr), _P(o_ptr), _P(lse_ptr), _P(ws_ptr), B, Hq, Hkv, Nq, Nk,
                         d, int(bool(causal)), float(scale), int(num_splits), _P(stream_ptr))


def decode(q, k, v, causal: bool = True, scale: float | None = None, num_splits: int = 0, out=None, lse=None,
           workspace=None, stream=None):
    """Attention of q [B, Hq, Nq, d] (the last Nq positions) against a key/value
    cache k, v [B, Hkv, Nk, d], all bf16, split along the keys; d = 64 or 128. At
    d = 128 a GQA group's (Hq / Hkv) * Nq query rows form one unit up to 32 rows,
    else blocks of 128 rows (always at d = 64). num_splits = 0: one CTA per SM, each an equal slice of all units'
    128-key chunks; > 0: units * num_splits CTAs. Returns (o, lse)."""
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, dk) != (B, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B, Hkv, Nk, d] with q's B and d")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    if workspace is None:
        nbytes = decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    _check(lib.fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(workspace), B, Hq, Hkv, Nq, Nk, d,
                         int(bool(causal)), scale, int(num_splits), _stream_ptr(stream)), "fa_decode")
    return out, lse


# ---------------------------------------------------------------------------
# cache operators: an 8-bit cache, sparse attention over selected blocks, eviction
# ---------------------------------------------------------------------------

# These calls take a few microseconds on the device for short caches, so the wrappers are kept
# lean: shapes and types are checked once per combination (functools.lru_cache on the
# functions named _..._plan), every tensor's device and contiguity on every call, and pointers
# and streams are passed as ints.

_torch = None
_C = None


def _t():
    """torch, imported once."""
    global _torch, _C
    if _torch is None:
        import torch
        _torch, _C = torch, torch._C
    return _torch


def _raw_stream(t, stream):
    """The raw current stream if `t` is on the current device and no other stream is asked
    for, else None: the call then repeats itself under `_placed`."""
    _t()
    dev = t.get_device()
    if stream is None and dev >= 0 and dev == _C._cuda_getDevice():
        return _C._cuda_getCurrentRawStream(dev)
    return None


@contextlib.contextmanager
def _placed(t, stream):
    """Makes the device of `t` and `stream` current: outputs and workspaces that the call
    allocates then belong to the stream that its kernels run on."""
    torch = _t()
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield


def _here(dev, *tensors):
    """Every tensor is on device `dev` and contiguous."""
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            if t.get_device() != dev:
                raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, expected device {dev}")
            raise ValueError(f"a tensor of shape {tuple(t.shape)} must be contiguous")


def _is(name, shape, dtype, want_shape, want_dtype):
    if dtype != want_dtype:
        raise TypeError(f"{name} must be {want_dtype}, got {dtype}")
    if tuple(shape) != tuple(want_shape):
        raise ValueError(f"{name} must have shape {tuple(want_shape)}, got {tuple(shape)}")


def _counts(*counts):
    """Counts on their way into C, where they are ints: ctypes would drop the upper bits."""
    for n in counts:
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"a size or count of {n} does not fit in 32 bits")


def _spec(t):
    return None if t is None else (t.shape, t.dtype)


def _cache_plan(k, block, lens, k_scale, v, v_scale):
    """Checks the specs of a cache and of what belongs to it; returns (fp8, B, Hkv, Nk, d)."""
    torch = _t()
    shape, dtype = k
    if len(shape) != 4:
        raise ValueError("a cache is [B, Hkv, Nk, d]")
    fp8 = dtype == torch.float8_e4m3fn
    if not fp8 and dtype != torch.bfloat16:
        raise TypeError(f"a cache is torch.float8_e4m3fn or torch.bfloat16, got {dtype}")
    if block not in (16, 32, 64, 128):
        raise ValueError(f"block must be 16, 32, 64 or 128, got {block}")
    B, Hkv, Nk, d = shape
    _counts(*shape)
    if v is not None:
        _is("v", *v, shape, dtype)
    for s, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s is not None:
            if not fp8:
                raise ValueError(f"{n} belongs to an 8-bit cache")
            _is(n, *s, (B, Hkv, -(-Nk // block)), torch.float32)
    if lens is not None:
        _is("lens", *lens, (B,), torch.int32)
    return fp8, B, Hkv, Nk, d


def _query_plan(q, B, d):
    """Checks the spec of queries; returns (Hq, Nq)."""
    shape, dtype = q
    if len(shape) != 4 or shape[0] != B or shape[3] != d:
        raise ValueError(f"q must be [{B}, Hq, Nq, {d}], got {tuple(shape)}")
    if dtype != _t().bfloat16:
        raise TypeError(f"q must be torch.bfloat16, got {dtype}")
    _counts(*shape)
    return shape[1], shape[2]


def _scales_given(fp8, *scales):
    if fp8 and any(s is None for s in scales):
        raise ValueError("an 8-bit cache needs its scales")


def _at(t):
    return None if t is None else t.data_ptr()


def _nbytes(shape, dtype):
    return math.prod(shape) * dtype.itemsize


def _overlap(ptr, sizes):
    """Whether an output shares a byte with another of the contiguous tensors at `ptr`: `sizes` has the bytes
    of each and whether it is an output."""
    end = out_end = 0  # of what came before, and of the outputs among it
    for at, (n, is_out) in sorted(zip(ptr, sizes)):
        if at < (end if is_out else out_end) and n:
            return True
        n += at
        if n > end:
            end = n
        if is_out and n > out_end:
            out_end = n
    return False


def _workspace(workspace, nbytes, q):
    """The caller's workspace if it is large enough, or a new one."""
    if workspace is None:
        return q.new_empty(max(nbytes, 256), dtype=_torch.uint8)
    _here(q.get_device(), workspace)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace needs {nbytes} contiguous bytes")
    return workspace


def _outputs(q, out, lse):
    if out is None:
        out = _torch.empty_like(q)
    else:
        _is("out", out.shape, out.dtype, q.shape, _torch.bfloat16)
    if lse is None:
        B, Hq, Nq, _ = q.shape
        lse = q.new_empty((B, Hq, Nq), dtype=_torch.float32)
    else:
        _is("lse", lse.shape, lse.dtype, q.shape[:3], _torch.float32)
    return out, lse


@functools.lru_cache(maxsize=4096)
def _store_plan(x, y, k, v, k_scale, v_scale, block, lens):
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, k_scale, v, v_scale)
    if not fp8:
        raise TypeError("cache_store writes a torch.float8_e4m3fn cache")
    _scales_given(True, k_scale, v_scale)
    shape, dtype = x
    if len(shape) != 4 or (shape[0], shape[1], shape[3]) != (B, Hkv, d):
        raise ValueError("k, v must be [B, Hkv, n_new, d] with the cache's B, Hkv and d")
    _is("k", shape, dtype, shape, _t().bfloat16)
    _is("v", *y, shape, _t().bfloat16)
    _counts(*shape)
    return B, Hkv, shape[2], Nk, d


def cache_store(k, v, cache_k, cache_v, k_scale, v_scale, block: int, lens=None, stream=None):
    """Appends the tokens k, v [B, Hkv, n_new, d] (bf16) to an 8-bit cache cache_k, cache_v
    [B, Hkv, Nk, d] (torch.float8_e4m3fn) with scales [B, Hkv, ceil(Nk / block)], in place, at
    the positions [lens - n_new, lens): lens [B] int32 counts them already (None: the
    cache's end). The four tensors written must not overlap. Returns (cache_k, cache_v, k_scale, v_scale)."""
    B, Hkv, n_new, Nk, d = _store_plan(_spec(k), _spec(v), _spec(cache_k), _spec(cache_v), _spec(k_scale), _spec(v_scale),
                                       block, _spec(lens))
    pk, pv, pks, pvs = cache_k.data_ptr(), cache_v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
    if pk == pv or pks == pvs:
        raise ValueError("cache_k and cache_v, and their scales, must not be the same memory")
    raw = _raw_stream(cache_k, stream)
    if raw is None:
        with _placed(cache_k, stream):
            return cache_store(k, v, cache_k, cache_v, k_scale, v_scale, block, lens)
    _here(cache_k.get_device(), k, v, cache_k, cache_v, k_scale, v_scale, lens)
    _check(lib.fa_cache_store(k.data_ptr(), v.data_ptr(), pk, pv, pks, pvs, _at(lens), B, Hkv, n_new, Nk, d, block, raw),
           "fa_cache_store")
    return cache_k, cache_v, k_scale, v_scale


def decode_fp8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block, num_splits=0) -> int:
    _counts(B, Hq, Hkv, Nq, Nk, d, block, num_splits)
    return int(lib.fa_decode_fp8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block, int(num_splits)))


@functools.lru_cache(maxsize=4096)
def _decode_fp8_plan(q, k, v, k_scale, v_scale, block, lens, num_splits):
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, k_scale, v, v_scale)
    if not fp8:
        raise TypeError("decode_fp8 reads a torch.float8_e4m3fn cache; `decode` reads bf16")
    _scales_given(True, k_scale, v_scale)
    Hq, Nq = _query_plan(q, B, d)
    return B, Hq, Hkv, Nq, Nk, d, decode_fp8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block, num_splits)


def decode_fp8(q, k, v, k_scale, v_scale, block: int, lens=None, causal: bool = True, scale: float | None = None,
               num_splits: int = 0, out=None, lse=None, workspace=None, stream=None):
    """`decode` against an 8-bit cache: q [B, Hq, Nq, d] bf16, k, v [B, Hkv, Nk, d]
    torch.float8_e4m3fn, k_scale, v_scale [B, Hkv, ceil(Nk / block)] float32, d = 128. lens
    [B] int32: the tokens that each sequence holds (None: Nk). Made for the few rows of a decode
    step: a group's (Hq / Hkv) * Nq rows read the keys once for every 16 of them. Returns (o, lse)."""
    B, Hq, Hkv, Nq, Nk, d, nbytes = _decode_fp8_plan(_spec(q), _spec(k), _spec(v), _spec(k_scale), _spec(v_scale), block,
                                                     _spec(lens), num_splits)
    raw = _raw_stream(q, stream)
    if raw is None:
        with _placed(q, stream):
            return decode_fp8(q, k, v, k_scale, v_scale, block, lens, causal, scale, num_splits, out, lse, workspace)
    out, lse = _outputs(q, out, lse)
    _here(q.get_device(), q, k, v, k_scale, v_scale, lens, out, lse)
    ws = _workspace(workspace, nbytes, q)
    _check(lib.fa_decode_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                             out.data_ptr(), lse.data_ptr(), ws.data_ptr(), _at(lens), B, Hq, Hkv, Nq, Nk, d, block,
                             1 if causal else 0, 1.0 / math.sqrt(d) if scale is None else float(scale), num_splits, raw),
           "fa_decode_fp8")
    return out, lse


@functools.lru_cache(maxsize=4096)
def _bounds_plan(k, block, lens, bounds, n_new):
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, None, None, None)
    _counts(n_new)
    if n_new < 0 or (n_new > 0 and bounds is None):
        raise ValueError("n_new > 0 refreshes the bounds that are passed in")
    shape = (B, Hkv, -(-Nk // block), 2, d)
    if bounds is not None:
        _is("bounds", *bounds, shape, k[1])
    return fp8, B, Hkv, Nk, d, shape


def block_bounds(k, block: int, lens=None, n_new: int = 0, bounds=None, stream=None):
    """Per-channel minimum and maximum of every block of a cache k [B, Hkv, Nk, d] (8-bit or
    bf16), as [B, Hkv, ceil(Nk / block), 2, d] in the cache's type. With n_new > 0 only the
    blocks that hold the newest n_new tokens are refreshed in `bounds`."""
    fp8, B, Hkv, Nk, d, shape = _bounds_plan(_spec(k), block, _spec(lens), _spec(bounds), n_new)
    raw = _raw_stream(k, stream)
    if raw is None:
        with _placed(k, stream):
            return block_bounds(k, block, lens, n_new, bounds)
    if bounds is None:  # blocks without a token keep what they hold: zeros
        bounds = _torch.zeros(shape, dtype=k.dtype, device=k.device)
    _here(k.get_device(), k, lens, bounds)
    _check(lib.fa_block_bounds(k.data_ptr(), bounds.data_ptr(), _at(lens), int(fp8), B, Hkv, Nk, d, block, n_new, raw),
           "fa_block_bounds")
    return bounds


def select_blocks_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block) -> int:
    _counts(B, Hq, Hkv, Nq, Nk, d, block)
    return int(lib.fa_select_blocks_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block))


@functools.lru_cache(maxsize=4096)
def _select_plan(q, bounds, n_select, block, Nk, k_scale, lens, out, n_first, n_last):
    torch = _t()
    shape, dtype = bounds
    if len(shape) != 5 or shape[3] != 2:
        raise ValueError("bounds must be [B, Hkv, ceil(Nk / block), 2, d]")
    B, Hkv, n_blocks, _, d = shape
    if block not in (16, 32, 64, 128):
        raise ValueError(f"block must be 16, 32, 64 or 128, got {block}")
    if Nk < 1 or n_blocks != -(-Nk // block):
        raise ValueError(f"bounds hold {n_blocks} blocks, a cache of {Nk} tokens has {-(-Nk // block)}")
    fp8 = dtype == torch.float8_e4m3fn
    if not fp8 and dtype != torch.bfloat16:
        raise TypeError(f"bounds must be torch.float8_e4m3fn or torch.bfloat16, got {dtype}")
    _scales_given(fp8, k_scale)
    if k_scale is not None:
        if not fp8:
            raise ValueError("k_scale belongs to an 8-bit cache")
        _is("k_scale", *k_scale, (B, Hkv, n_blocks), torch.float32)
    if lens is not None:
        _is("lens", *lens, (B,), torch.int32)
    Hq, Nq = _query_plan(q, B, d)
    _counts(n_select, n_first, n_last)
    if n_select < 1:
        raise ValueError("n_select must be at least 1")
    if n_first < 0 or n_last < 0:
        raise ValueError(f"n_first and n_last must not be negative, got {n_first} and {n_last}")
    if n_first + n_last > n_select:
        raise ValueError(f"n_first + n_last must not exceed n_select, got {n_first} + {n_last} of {n_select}")
    if out is not None:
        _is("out", *out, (B, Hkv, Nq, n_select), torch.int32)
    return fp8, B, Hq, Hkv, Nq, d, select_blocks_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, block)


def select_blocks(q, bounds, n_select: int, block: int, Nk: int, k_scale=None, lens=None, n_first: int = 1,
                  n_last: int = 1, causal: bool = True, out=None, workspace=None, stream=None):
    """The n_select blocks that each query of q [B, Hq, Nq, d] attends to, by an upper bound of
    its scores in them: bounds [B, Hkv, ceil(Nk / block), 2, d] from `block_bounds`, k_scale for
    an 8-bit cache. The first n_first and the last n_last blocks that the query sees
    are always taken (n_first + n_last <= n_select). Returns int32 [B, Hkv, Nq, n_select], ascending, padded with -1."""
    fp8, B, Hq, Hkv, Nq, d, nbytes = _select_plan(_spec(q), _spec(bounds), n_select, block, Nk, _spec(k_scale),
                                                  _spec(lens), _spec(out), n_first, n_last)
    raw = _raw_stream(q, stream)
    if raw is None:
        with _placed(q, stream):
            return select_blocks(q, bounds, n_select, block, Nk, k_scale, lens, n_first, n_last, causal, out, workspace)
    if out is None:
        out = q.new_empty((B, Hkv, Nq, n_select), dtype=_torch.int32)
    _here(q.get_device(), q, bounds, k_scale, lens, out)
    ws = _workspace(workspace, nbytes, q)
    _check(lib.fa_select_blocks(q.data_ptr(), bounds.data_ptr(), _at(k_scale), out.data_ptr(), ws.data_ptr(), _at(lens),
                                int(fp8), B, Hq, Hkv, Nq, Nk, d, block, n_select, n_first, n_last, 1 if causal else 0,
                                raw), "fa_select_blocks")
    return out


def decode_blocks_workspace_bytes(fp8, B, Hq, Hkv, Nq, Nk, d, block, n_select, num_splits=0) -> int:
    _counts(B, Hq, Hkv, Nq, Nk, d, block, n_select, num_splits)
    return int(lib.fa_decode_blocks_workspace_bytes(int(bool(fp8)), B, Hq, Hkv, Nq, Nk, d, block, n_select,
                                                    int(num_splits)))


@functools.lru_cache(maxsize=4096)
def _decode_blocks_plan(q, k, v, idx, block, k_scale, v_scale, lens, num_splits):
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, k_scale, v, v_scale)
    _scales_given(fp8, k_scale, v_scale)
    Hq, Nq = _query_plan(q, B, d)
    if len(idx[0]) != 4:
        raise ValueError("idx must be [B, Hkv, Nq, n_select]")
    n_select = idx[0][3]
    _is("idx", *idx, (B, Hkv, Nq, n_select), _t().int32)
    return (fp8, B, Hq, Hkv, Nq, Nk, d, n_select,
            decode_blocks_workspace_bytes(fp8, B, Hq, Hkv, Nq, Nk, d, block, n_select, num_splits))


def decode_blocks(q, k, v, idx, block: int, k_scale=None, v_scale=None, lens=None, causal: bool = True,
                  scale: float | None = None, num_splits: int = 0, out=None, lse=None, workspace=None, stream=None):
    """`decode` over the blocks idx [B, Hkv, Nq, n_select] (int32, -1 for none) of each query
    alone, against a bf16 or an 8-bit cache (with its scales); d = 128. With every block listed
    it is `decode` against a bf16 cache of sequences of different lengths. Returns (o, lse)."""
    fp8, B, Hq, Hkv, Nq, Nk, d, n_select, nbytes = _decode_blocks_plan(_spec(q), _spec(k), _spec(v), _spec(idx), block,
                                                                       _spec(k_scale), _spec(v_scale), _spec(lens),
                                                                       num_splits)
    raw = _raw_stream(q, stream)
    if raw is None:
        with _placed(q, stream):
            return decode_blocks(q, k, v, idx, block, k_scale, v_scale, lens, causal, scale, num_splits, out, lse,
                                 workspace)
    out, lse = _outputs(q, out, lse)
    _here(q.get_device(), q, k, v, idx, k_scale, v_scale, lens, out, lse)
    ws = _workspace(workspace, nbytes, q)
    _check(lib.fa_decode_blocks(q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(k_scale), _at(v_scale), idx.data_ptr(),
                                out.data_ptr(), lse.data_ptr(), ws.data_ptr(), _at(lens), int(fp8), B, Hq, Hkv, Nq, Nk,
                                d, block, n_select, 1 if causal else 0,
                                1.0 / math.sqrt(d) if scale is None else float(scale), num_splits, raw),
           "fa_decode_blocks")
    return out, lse


@functools.lru_cache(maxsize=4096)
def _weights_plan(q, k, lse, acc, k_scale, block, lens):
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, k_scale, None, None)
    _scales_given(fp8, k_scale)
    Hq, Nq = _query_plan(q, B, d)
    _is("lse", *lse, (B, Hq, Nq), _t().float32)
    _is("acc", *acc, (B, Hkv, Nk), _t().float32)
    return fp8, B, Hq, Hkv, Nq, Nk, d


def cache_weights(q, k, lse, acc, k_scale=None, block: int = 64, lens=None, causal: bool = True,
                  scale: float | None = None, stream=None):
    """Adds to acc [B, Hkv, Nk] (float32, in place) the attention weight that the queries q
    [B, Hq, Nq, d] gave each key of a cache k (bf16, or 8-bit with k_scale): the sum of
    exp(S - lse) over the group's rows. lse [B, Hq, Nq] comes from an attention call over all of the
    sequence's keys (`fwd`, `decode`, `decode_fp8`); that of `decode_blocks` covers the listed blocks alone
    and makes every weight too large. Returns acc."""
    fp8, B, Hq, Hkv, Nq, Nk, d = _weights_plan(_spec(q), _spec(k), _spec(lse), _spec(acc), _spec(k_scale), block,
                                               _spec(lens))
    raw = _raw_stream(q, stream)
    if raw is None:
        with _placed(q, stream):
            return cache_weights(q, k, lse, acc, k_scale, block, lens, causal, scale)
    _here(q.get_device(), q, k, lse, acc, k_scale, lens)
    _check(lib.fa_cache_weights(q.data_ptr(), k.data_ptr(), _at(k_scale), lse.data_ptr(), acc.data_ptr(), _at(lens),
                                int(fp8), B, Hq, Hkv, Nq, Nk, d, block, 1 if causal else 0,
                                1.0 / math.sqrt(d) if scale is None else float(scale), raw), "fa_cache_weights")
    return acc


@functools.lru_cache(maxsize=4096)
def _evict_plan(k, v, acc, keep, recent, k_scale, v_scale, block, lens, out):
    torch = _t()
    fp8, B, Hkv, Nk, d = _cache_plan(k, block, lens, k_scale, v, v_scale)
    _scales_given(fp8, k_scale, v_scale)
    _is("acc", *acc, (B, Hkv, Nk), torch.float32)
    _counts(keep, recent)
    if keep < 1 or not 0 <= recent <= keep:
        raise ValueError("keep must be at least 1, recent from 0 to keep")
    cap = Nk
    if out is not None:
        if len(out) != (7 if fp8 else 5):
            raise ValueError(f"out must hold {7 if fp8 else 5} tensors")
        if len(out[0][0]) != 4:
            raise ValueError("out's cache is [B, Hkv, capacity, d]")
        cap = out[0][0][2]
        _counts(cap)
        if cap < min(keep, Nk):
            raise ValueError(f"out's cache holds {cap} tokens, {min(keep, Nk)} may be kept")
        want = (("k", (B, Hkv, cap, d), k[1]), ("v", (B, Hkv, cap, d), k[1]), ("acc", (B, Hkv, cap), torch.float32),
                ("idx", (B, Hkv, keep), torch.int32), ("lens", (B,), torch.int32),
                ("k_scale", (B, Hkv, -(-cap // block)), torch.float32),
                ("v_scale", (B, Hkv, -(-cap // block)), torch.float32))
        for o, (name, shape, dtype) in zip(out, want):
            _is(f"out {name}", *o, shape, dtype)
    sizes = [(0 if t is None else _nbytes(*t), False) for t in (k, v, acc, k_scale, v_scale, lens)]
    return fp8, B, Hkv, Nk, d, cap, sizes + [(_nbytes(*t), True) for t in out or ()]


def cache_evict(k, v, acc, keep: int, recent: int = 0, k_scale=None, v_scale=None, block: int = 64, lens=None, out=None,
                stream=None):
    """Cuts every head of a cache back to at most `keep` tokens: the newest `recent` and the
    others with the largest acc [B, Hkv, Nk], in their order, copied into a second
    cache. Returns (k, v, acc, idx, lens), for an 8-bit cache (k, v, acc, idx, lens,
    k_scale, v_scale): idx [B, Hkv, keep] int32 the old positions (-1 behind them), lens [B]
    int32 the new lengths. `out` is such a tuple to write into (its cache may have any
    capacity >= min(keep, Nk)) and overlaps neither the inputs nor itself; what lies behind the kept tokens stays
    as it is there. The new cache's blocks hold other tokens: `block_bounds` makes their bounds anew."""
    fp8, B, Hkv, Nk, d, cap, sizes = _evict_plan(_spec(k), _spec(v), _spec(acc), keep, recent, _spec(k_scale), _spec(v_scale),
                                                 block, _spec(lens), None if out is None else tuple(map(_spec, out)))
    ptr = [0 if t is None else t.data_ptr() for t in (k, v, acc, k_scale, v_scale, lens)]
    if out is not None:
        ptr += [o.data_ptr() for o in out]
        if _overlap(ptr, sizes):
            raise ValueError("out must not overlap the cache that is cut, nor itself")
    raw = _raw_stream(k, stream)
    if raw is None:
        with _placed(k, stream):
            return cache_evict(k, v, acc, keep, recent, k_scale, v_scale, block, lens, out)
    if out is None:
        torch = _torch
        out = [torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(acc),
               k.new_empty((B, Hkv, keep), dtype=torch.int32), k.new_empty((B,), dtype=torch.int32)]
        out += [torch.ones_like(k_scale), torch.ones_like(v_scale)] if fp8 else []
        ptr += [o.data_ptr() for o in out]
    _here(k.get_device(), k, v, acc, k_scale, v_scale, lens, *out)
    pk, pv, pacc, pks, pvs, plens, ok, ov, oacc, oidx, olens = ptr[:11]
    oks, ovs = ptr[11:] if fp8 else (0, 0)
    _check(lib.fa_cache_evict(pk, pv, pks, pvs, pacc, plens, ok, ov, oks, ovs, oacc, oidx, olens, int(fp8), B, Hkv, Nk, d,
                              block, keep, recent, cap, raw), "fa_cache_evict")
    return tuple(out)


def workspace_bytes(B, Hq, Hkv, N, d) -> int:
    return int(lib.fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def bwd_raw(q, k, v, o, lse, do, dq, dk, dv, ws, B, Hq, Hkv, N, d, causal, scale, stream_ptr):
    """The C call itself on raw device pointers (ints); returns the status code."""
    return lib.fa_bwd(_P(q), _P(k), _P(v), _P(o), _P(lse), _P(do), _P(dq), _P(dk), _P(dv), _P(ws), B, Hq, Hkv, N,
                      d, int(bool(causal)), float(scale), _P(stream_ptr))


def bwd_phases_raw(q, k, v, o, lse, do, dq, dk, dv, ws, B, Hq, Hkv, N, d, causal, scale, stream_ptr,
                   between=None):
    """fa_bwd as its three C calls (preprocess, main, convert) on raw pointers.
    `between(i)` (optional) is called before phase i = 0, 1, 2 and after the
    last (i = 3), e.g. to record CUDA events on the same stream. Returns the
    first nonzero status code, else 0."""
    c = int(bool(causal))
    st = _P(stream_ptr)
    calls = (lambda: lib.fa_bwd_preprocess(_P(o), _P(do), _P(ws), B, Hq, Hkv, N, d, st),
             lambda: lib.fa_bwd_main(_P(q), _P(k), _P(v), _P(lse), _P(do), _P(dk), _P(dv), _P(ws), B, Hq, Hkv, N, d,
                                     c, float(scale), st),
             lambda: lib.fa_bwd_convert(_P(dq), _P(ws), B, Hq, Hkv, N, d, float(scale), st))
    for i, call in enumerate(calls):
        if between is not None:
            between(i)
        rc = call()
        if rc != 0:
            return rc
    if between is not None:
        between(3)
    return 0


def bwd(q, k, v, o, lse, do, causal: bool = True, scale: float | None = None, workspace=None, out=None,
        stream=None):
    """Backward pass (bf16). Returns (dq, dk, dv)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _require(t, n, torch.bfloat16, q.device)
    _require(lse, "lse", torch.float32, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = workspace_bytes(B, Hq, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes")
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = out
    _check(lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                      _ptr(workspace), B, Hq, Hkv, N, d, int(bool(causal)), scale, _stream_ptr(stream)), "fa_bwd")
    return dq, dk, dv


def get_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib.fa_get_status(_stream_ptr(stream)))


def get_progress(n: int, stream=None):
    """Per-CTA progress words of the last forward / backward main-kernel launch
    (see fa_get_progress in include/fa.h), as a list of n ints."""
    buf = (ctypes.c_uint * max(int(n), 0))()
    rc = lib.fa_get_progress(ctypes.cast(buf, ctypes.c_void_p), int(n), _stream_ptr(stream))
    if rc < 0:
        raise FAError(rc, "fa_get_progress")
    return list(buf)[:rc]


def set_wait_budget_ns(ns: int):
    lib.fa_set_wait_budget_ns(int(ns))


def selftest_wait_timeout(budget_ns: int = 10_000_000, stream=None) -> int:
    return int(lib.fa_selftest_wait_timeout(int(budget_ns), _stream_ptr(stream)))
