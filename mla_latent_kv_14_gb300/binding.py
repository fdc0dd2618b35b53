"""ctypes binding of libmla (include/mla.h). Marshalling only: every step of the
decode runs in the library's CUDA kernels; PyTorch supplies device memory and
streams. Nothing here computes attention, and there is no fallback path: if
the shared library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

MLA_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "stale metadata",
                4: "out-of-range page or index skipped", 5: "device wait timed out", 6: "CUDA error",
                7: "FP8 path: a value beyond fp16 range was saturated"}
DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}

_lib = None
_lib_lock = threading.Lock()


class MLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} (status {status})")


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmla.so (built by ``mla_latent_kv_14_gb300.build``)."""
    global _lib
    with _lib_lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"libmla.so not built at {p}: run `python -m mla_latent_kv_14_gb300.build`")
        lib = ctypes.CDLL(p)
        c = ctypes
        vp, i32p = c.c_void_p, c.c_void_p
        lib.mla_status_string.restype = c.c_char_p
        lib.mla_status_string.argtypes = [c.c_int]
        lib.mla_num_sm_parts.restype = c.c_int
        lib.mla_num_sm_parts.argtypes = [c.c_int]
        lib.mla_num_sm_parts_for.restype = c.c_int
        lib.mla_num_sm_parts_for.argtypes = [c.c_int, c.c_int]
        lib.mla_metadata_size.restype = c.c_size_t
        lib.mla_metadata_size.argtypes = [c.c_int, c.c_int, c.c_int]
        lib.mla_workspace_size.restype = c.c_size_t
        lib.mla_workspace_size.argtypes = [c.c_int, c.c_int, c.c_int, c.c_int]
        lib.mla_get_metadata.restype = c.c_int
        lib.mla_get_metadata.argtypes = [i32p, c.c_int, c.c_int, c.c_int, c.c_int, c.c_int, c.c_int, c.c_int,
                                         c.c_int, c.c_int, vp, i32p, vp]
        lib.mla_decode_with_kvcache.restype = c.c_int
        lib.mla_decode_with_kvcache.argtypes = [vp, c.c_int, vp, c.c_int64, c.c_int, i32p, c.c_int, i32p, c.c_int,
                                                c.c_int, c.c_int, c.c_int, vp, i32p, c.c_int, c.c_float, c.c_int,
                                                c.c_int, i32p, c.c_int, vp, vp, vp, c.c_size_t, vp]
        for name in ("mla_decode_splitkv", "mla_combine_splits"):
            f = getattr(lib, name)
            f.restype = c.c_int
            f.argtypes = lib.mla_decode_with_kvcache.argtypes
        lib.mla_decode_with_kvcache_noalloc.restype = c.c_int
        lib.mla_decode_with_kvcache_noalloc.argtypes = lib.mla_decode_with_kvcache.argtypes[:-3] + [vp, vp]
        for name in ("mla_quantize_kv_fp8", "mla_quantize_kv_fp8_528", "mla_quantize_kv_fp4_288"):
            f = getattr(lib, name)
            f.restype = c.c_int
            f.argtypes = [vp, vp, c.c_int64, vp]
        lib.mla_read_status.restype = c.c_int
        lib.mla_read_status.argtypes = [vp, vp, c.POINTER(c.c_uint32)]
        for name in ("mla_absorb_q", "mla_up_project"):
            f = getattr(lib, name)
            f.restype = c.c_int
            f.argtypes = [vp, vp, vp, c.c_int, c.c_int, c.c_int, vp, vp]
        i32, i64 = c.c_int, c.c_int64
        rope = [vp, vp, i64, i32]  # positions, table, its rows, style
        lib.mla_append_kv.argtypes = [vp, i64, vp, i64, i32, vp] + rope + [i64, vp, i64, i32, i32, vp, vp]
        lib.mla_rotate_q.argtypes = [vp, i64, i64, vp, i64, i64, i32] + rope + [i64, i32, vp, vp]
        lib.mla_append_index_k.argtypes = [vp, i64, i32, vp] + rope + [i64, vp, i64, i32, i32, vp, vp]
        lib.mla_quantize_index_q.argtypes = [vp, i64, i64, i32, vp] + rope + [i64, i32, vp, vp, vp, vp]
        lib.mla_index_score.argtypes = [vp, i32, vp, vp, i32, i64, i32, vp, i32, vp, i32, i32, i32, i32, i32, vp,
                                        i64, i32, vp, vp]
        lib.mla_select_topk.argtypes = [vp, i64, i32, vp, i32, i32, i32, i32, i32, vp, i32, i64, i32, vp, vp, vp, vp]
        f32, size = c.c_float, c.c_size_t
        lib.mla_norm_rotate.argtypes = [vp, i64, i64, vp, f32, i32, i32, vp, i64, i64, vp, i64, i64, i32] + rope + [
            i64, i32, vp, vp]
        lib.mla_norm_append_kv.argtypes = [vp, i64, vp, i64, vp, f32, i32, vp] + rope + [
            i64, vp, i64, i32, i32, vp, i64, vp, vp]
        lib.mla_read_kv.argtypes = [vp, i64, i32, i32, vp, i32, vp, vp, i32, i64, vp, i64, i32, vp, vp]
        lib.mla_prefill.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, i32, vp, vp, vp, i32, i64, i64, i32,
                                    f32, i32, vp, i64, i64, vp, vp, size, vp, vp]
        lib.mla_prefill_workspace_size.restype = size
        lib.mla_prefill_workspace_size.argtypes = [i64, i64, i32, i32]
        for name in ("mla_append_kv", "mla_rotate_q", "mla_append_index_k", "mla_quantize_index_q",
                     "mla_index_score", "mla_select_topk", "mla_norm_rotate", "mla_norm_append_kv", "mla_read_kv",
                     "mla_prefill"):
            getattr(lib, name).restype = c.c_int
        lib.mla_set_test_stall.restype = None
        lib.mla_set_test_stall.argtypes = [c.c_uint32]
        if path is None:
            _lib = lib
        return lib


def _dev(device=None) -> torch.device:
    """A cuda device with an explicit index (the current one if unspecified)."""
    d = torch.device("cuda") if device is None else torch.device(device)
    if d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, where: str):
    if status != MLA_OK:
        raise MLAError(status, where)


def mla_num_sm_parts(device=None, h_q: int = 128) -> int:
    """Default number of SM parts of the decode kernel for `h_q` query heads."""
    n = load_library().mla_num_sm_parts_for(_dev(device).index, h_q)
    if n <= 0:
        raise MLAError(2 if n < 0 else 6, "mla_num_sm_parts")
    return n


class Metadata:
    """Split-KV schedule from :func:`mla_get_metadata` (device tensors)."""

    def __init__(self, meta: torch.Tensor, num_splits: torch.Tensor, parts: int, key: tuple):
        self.meta = meta
        self.num_splits = num_splits
        self.parts = parts
        self.key = key


# cache row formats (the kv_format argument; is_fp8=True is KV_FP8_656)
KV_16BIT, KV_FP8_656, KV_FP8_528, KV_FP4_288 = 0, 1, 2, 3
ROW_WIDTH = {KV_16BIT: 576, KV_FP8_656: 576, KV_FP8_528: 512, KV_FP4_288: 512}   # query / key width


def _kv_format(is_fp8: bool, kv_format: Optional[int]) -> int:
    if kv_format is None:
        return KV_FP8_656 if is_fp8 else KV_16BIT
    if kv_format not in ROW_WIDTH:
        raise MLAError(1, f"unknown kv_format {kv_format}")
    return int(kv_format)


def mla_get_metadata(cache_seqlens: Optional[torch.Tensor], s_q: int, h_q: int = 128, *, batch: Optional[int] = None,
                     topk: int = 0, is_fp8: bool = False, causal: bool = False, page_block: int = 64,
                     num_sm_parts: Optional[int] = None, device=None,
                     kv_format: Optional[int] = None) -> Tuple[Metadata, torch.Tensor]:
    """Compute the split-KV schedule on the device (no host sync)."""
    lib = load_library()
    fmt = _kv_format(is_fp8, kv_format)
    if cache_seqlens is not None:
        batch = int(cache_seqlens.shape[0])
        device = cache_seqlens.device
        assert cache_seqlens.dtype == torch.int32 and cache_seqlens.is_contiguous()
    assert batch is not None and device is not None
    device = _dev(device)
    parts = num_sm_parts or mla_num_sm_parts(device, h_q)
    nbytes = lib.mla_metadata_size(batch, s_q, parts)
    meta = torch.empty((nbytes + 3) // 4, dtype=torch.int32, device=device)
    num_splits = torch.empty(batch * s_q + 1, dtype=torch.int32, device=device)
    st = lib.mla_get_metadata(_ptr(cache_seqlens), batch, s_q, h_q, 1, topk, fmt, int(causal), page_block,
                              parts, _ptr(meta), _ptr(num_splits), _stream(device))
    _check(st, "mla_get_metadata")
    return Metadata(meta, num_splits, parts, (batch, s_q, h_q, topk, fmt, bool(causal))), num_splits


_ws_cache = {}
_ws_lock = threading.Lock()


def workspace_for(device: torch.device, nbytes: int) -> torch.Tensor:
    """A zero-initialised workspace cached per (device, stream); grown on demand."""
    device = _dev(device)
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws_cache[key] = ws
        return ws


def mla_decode_with_kvcache(q: torch.Tensor, kvcache: torch.Tensor, block_table: Optional[torch.Tensor],
                            cache_seqlens: Optional[torch.Tensor], head_dim_v: int, metadata: Metadata,
                            num_splits: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                            causal: bool = False, is_fp8: bool = False, indices: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, kv_format: Optional[int] = None,
                            _entry: str = "mla_decode_with_kvcache") -> Tuple[torch.Tensor, torch.Tensor]:
    """out [B, s_q, h_q, 512] (q dtype), lse [B, s_q, h_q] fp32 (natural log).
    ``kv_format`` picks the cache row format (KV_*); q is [B, s_q, h_q, 576],
    or 512 wide with the V4.1 rows (KV_FP8_528, KV_FP4_288)."""
    lib = load_library()
    fmt = _kv_format(is_fp8, kv_format)
    B, s_q, h_q, d_k = q.shape
    assert d_k == ROW_WIDTH[fmt] and q.is_contiguous() and kvcache.is_contiguous()
    dev = _dev(q.device)
    num_blocks, page_block = int(kvcache.shape[0]), int(kvcache.shape[1])
    if softmax_scale is None:
        softmax_scale = d_k ** -0.5
    if num_splits is None:
        num_splits = metadata.num_splits
    topk = int(indices.shape[-1]) if indices is not None else 0
    if out is None:
        out = torch.empty(B, s_q, h_q, head_dim_v, dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty(B, s_q, h_q, dtype=torch.float32, device=dev)
    wsb = lib.mla_workspace_size(B, s_q, h_q, metadata.parts)
    if workspace is None:
        workspace = workspace_for(dev, wsb)
    max_blocks = int(block_table.shape[1]) if block_table is not None else 0
    st = getattr(lib, _entry)(
        _ptr(q), DTYPE_CODES[q.dtype], _ptr(kvcache), num_blocks, page_block, _ptr(block_table), max_blocks,
        _ptr(cache_seqlens), B, s_q, h_q, head_dim_v, _ptr(metadata.meta), _ptr(num_splits), metadata.parts,
        float(softmax_scale), int(causal), fmt, _ptr(indices), topk, _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(dev))
    _check(st, _entry)
    return out, lse


def mla_decode_splitkv(*args, **kw):
    """Only the split-KV kernel of :func:`mla_decode_with_kvcache`."""
    return mla_decode_with_kvcache(*args, _entry="mla_decode_splitkv", **kw)


def mla_combine_splits(*args, **kw):
    """Only the combine of :func:`mla_decode_with_kvcache` (after mla_decode_splitkv)."""
    return mla_decode_with_kvcache(*args, _entry="mla_combine_splits", **kw)


def mla_decode_with_kvcache_noalloc(q: torch.Tensor, kvcache: torch.Tensor, block_table: Optional[torch.Tensor],
                                    cache_seqlens: Optional[torch.Tensor], head_dim_v: int, metadata: Metadata,
                                    num_splits: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                                    causal: bool = False, is_fp8: bool = False,
                                    indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                    lse: Optional[torch.Tensor] = None,
                                    status: Optional[torch.Tensor] = None,
                                    kv_format: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode using the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory on demand). ``out``/``lse``
    /``status`` are allocated here only when not given."""
    lib = load_library()
    fmt = _kv_format(is_fp8, kv_format)
    B, s_q, h_q, d_k = q.shape
    assert d_k == ROW_WIDTH[fmt] and q.is_contiguous() and kvcache.is_contiguous()
    dev = _dev(q.device)
    num_blocks, page_block = int(kvcache.shape[0]), int(kvcache.shape[1])
    if softmax_scale is None:
        softmax_scale = d_k ** -0.5
    if num_splits is None:
        num_splits = metadata.num_splits
    topk = int(indices.shape[-1]) if indices is not None else 0
    if out is None:
        out = torch.empty(B, s_q, h_q, head_dim_v, dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty(B, s_q, h_q, dtype=torch.float32, device=dev)
    max_blocks = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.mla_decode_with_kvcache_noalloc(
        _ptr(q), DTYPE_CODES[q.dtype], _ptr(kvcache), num_blocks, page_block, _ptr(block_table), max_blocks,
        _ptr(cache_seqlens), B, s_q, h_q, head_dim_v, _ptr(metadata.meta), _ptr(num_splits), metadata.parts,
        float(softmax_scale), int(causal), fmt, _ptr(indices), topk, _ptr(out), _ptr(lse), _ptr(status),
        _stream(dev))
    _check(st, "mla_decode_with_kvcache_noalloc")
    return out, lse


def mla_quantize_kv_fp8(kv: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 rows [..., 576] -> uint8 rows [..., 656] (the FP8 cache layout)."""
    lib = load_library()
    assert kv.dtype == torch.bfloat16 and kv.shape[-1] == 576 and kv.is_contiguous()
    n = kv.numel() // 576
    if out is None:
        out = torch.empty(*kv.shape[:-1], 656, dtype=torch.uint8, device=kv.device)
    st = lib.mla_quantize_kv_fp8(_ptr(kv), _ptr(out), n, _stream(kv.device))
    _check(st, "mla_quantize_kv_fp8")
    return out


def _quantize_v41(name: str, row_bytes: int, kv: torch.Tensor, out: Optional[torch.Tensor]) -> torch.Tensor:
    lib = load_library()
    assert kv.dtype == torch.bfloat16 and kv.shape[-1] == 512 and kv.is_contiguous()
    n = kv.numel() // 512
    if out is None:
        out = torch.empty(*kv.shape[:-1], row_bytes, dtype=torch.uint8, device=kv.device)
    st = getattr(lib, name)(_ptr(kv), _ptr(out), n, _stream(kv.device))
    _check(st, name)
    return out


def mla_quantize_kv_fp8_528(kv: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 rows [..., 512] -> uint8 rows [..., 528] (V4.1: e4m3 + UE8M0 per 32)."""
    return _quantize_v41("mla_quantize_kv_fp8_528", 528, kv, out)


def mla_quantize_kv_fp4_288(kv: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 rows [..., 512] -> uint8 rows [..., 288] (e2m1 + e4m3 per 16)."""
    return _quantize_v41("mla_quantize_kv_fp4_288", 288, kv, out)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise MLAError(1, f"unsupported dtype {t.dtype}")


def mla_absorb_q(q_nope: torch.Tensor, w_uk: torch.Tensor, q_out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q~ = W^UK_i^T q^C per head: q_nope [..., h, 128], w_uk [h, 128, 512] ->
    dims [0, 512) of q_out [..., h, 576] (allocated if not given; its RoPE dims
    are the caller's). ``status``: optional device status word (read it with
    :func:`mla_read_status`)."""
    lib = load_library()
    h = q_nope.shape[-2]
    assert q_nope.shape[-1] == 128 and tuple(w_uk.shape) == (h, 128, 512)
    assert q_nope.is_contiguous() and w_uk.is_contiguous() and w_uk.dtype == q_nope.dtype
    tokens = q_nope.numel() // (h * 128)
    if q_out is None:
        q_out = torch.zeros(*q_nope.shape[:-1], 576, dtype=q_nope.dtype, device=q_nope.device)
    assert q_out.is_contiguous() and q_out.dtype == q_nope.dtype and q_out.numel() == tokens * h * 576
    st = lib.mla_absorb_q(_ptr(q_nope), _ptr(w_uk), _ptr(q_out), tokens, h, _dtype_code(q_nope), _ptr(status),
                          _stream(q_nope.device))
    _check(st, "mla_absorb_q")
    return q_out


def mla_up_project(o_lat: torch.Tensor, w_uv: torch.Tensor, o_out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o = W^UV_i o~ per head: o_lat [..., h, 512], w_uv [h, 128, 512] -> [..., h, 128].
    ``status``: optional device status word (read it with :func:`mla_read_status`)."""
    lib = load_library()
    h = o_lat.shape[-2]
    assert o_lat.shape[-1] == 512 and tuple(w_uv.shape) == (h, 128, 512)
    assert o_lat.is_contiguous() and w_uv.is_contiguous() and w_uv.dtype == o_lat.dtype
    tokens = o_lat.numel() // (h * 512)
    if o_out is None:
        o_out = torch.empty(*o_lat.shape[:-1], 128, dtype=o_lat.dtype, device=o_lat.device)
    assert o_out.is_contiguous() and o_out.dtype == o_lat.dtype and o_out.numel() == tokens * h * 128
    st = lib.mla_up_project(_ptr(o_lat), _ptr(w_uv), _ptr(o_out), tokens, h, _dtype_code(o_lat), _ptr(status),
                            _stream(o_lat.device))
    _check(st, "mla_up_project")
    return o_out


def mla_read_status(workspace: Optional[torch.Tensor] = None, device=None) -> Tuple[int, int]:
    """Synchronise and return (status, bits) of a workspace, clearing it."""
    lib = load_library()
    dev = _dev(device)
    if workspace is None:
        workspace = workspace_for(dev, 256)
    bits = ctypes.c_uint32(0)
    st = lib.mla_read_status(_ptr(workspace), _stream(dev), ctypes.byref(bits))
    return st, int(bits.value)


def mla_set_test_stall(cycles: int) -> None:
    """Test hook of the time-out path: while non-zero, every decode, absorption,
    index-score and prompt-attention launch first waits ``cycles`` SM cycles on a barrier nothing
    arrives at, records a wait time-out and skips its work. 0 turns it off."""
    load_library().mla_set_test_stall(int(cycles))


# ---------------------------------------------------------------------------
# New tokens, index scores, selection
# ---------------------------------------------------------------------------
ROPE_PAIRS, ROPE_HALVES = 0, 1        # rope_style: pairs (2i, 2i+1), or (i, i+32)
INDEX_16BIT, INDEX_FP8 = 0, 1         # index_format
INDEX_DIM, INDEX_FP8_PAGE_BYTES = 128, 8448
_host = None


def load_host():
    """The extension module that checks and launches these calls (built with
    libmla.so; their time on the GPU is a few microseconds)."""
    global _host
    load_library()
    with _lib_lock:
        if _host is None:
            path = os.path.join(_HERE, "_host.so")
            if not os.path.exists(path):
                raise ImportError(f"_host.so not built at {path}: run `python -m mla_latent_kv_14_gb300.build`")
            spec = importlib.util.spec_from_file_location("mla_latent_kv_14_gb300._host", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.set_error(MLAError)
            _host = module
    return _host


def mla_rope_table(max_positions: int, base: float = 10000.0, inv_freq: Optional[torch.Tensor] = None,
                   scale: float = 1.0, device=None) -> torch.Tensor:
    """The rotation table [max_positions, 64] fp32: 32 cosines, then 32 sines, of
    position * inv_freq (base ** (-i / 32) unless given), times ``scale``. The
    angles are formed in 64 bits: far positions lose nothing."""
    dev = _dev(device)
    if inv_freq is None:
        inv_freq = base ** (-torch.arange(32, dtype=torch.float64) / 32)
    if tuple(inv_freq.shape) != (32,):
        raise MLAError(1, "mla_rope_table: inv_freq [32]")
    angle = torch.arange(max_positions, dtype=torch.float64, device=dev)[:, None] * inv_freq.to(dev, torch.float64)
    return torch.cat((angle.cos() * scale, angle.sin() * scale), 1).float()


def mla_append_kv(c_kv: torch.Tensor, k_rope: torch.Tensor, kvcache: torch.Tensor, slots: torch.Tensor,
                  positions: torch.Tensor, rope_table: torch.Tensor, kv_format: int = KV_16BIT,
                  rope_style: int = ROPE_PAIRS, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Append tokens to the paged cache in place: c_kv [n, 512] (V4.1 rows: 448)
    and k_rope [n, 64], which is rotated on the way; ``slots`` int32 [n] are cache
    rows (page * 64 + offset, negative: skip). Returns kvcache."""
    return (_host or load_host()).mla_append_kv(c_kv, k_rope, kvcache, slots, positions, rope_table, kv_format,
                                                 rope_style, status)


def mla_rotate_q(x: torch.Tensor, positions: torch.Tensor, rope_table: torch.Tensor,
                 out: Optional[torch.Tensor] = None, rope_style: int = ROPE_PAIRS,
                 status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate query rows: x [tokens, heads, 64] (any token and head strides, for
    example ``q[..., 128:]`` of the projection) -> out, of the same shape
    (``q_abs[..., 512:]``, ``x`` itself, or allocated). Rows of tokens whose
    position is negative are not written."""
    return (_host or load_host()).mla_rotate_q(x, positions, rope_table, out, rope_style, status)


def mla_append_index_k(k: torch.Tensor, index_cache: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor,
                       rope_table: torch.Tensor, index_format: int = INDEX_16BIT, rope_style: int = ROPE_PAIRS,
                       status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Append index keys k [n, 128] (dims [0, 64) are rotated) to the paged index
    cache in place: [num_blocks, 64, 1, 128] of k's type, or uint8 [num_blocks,
    8448] with INDEX_FP8. ``slots`` as in :func:`mla_append_kv`."""
    return (_host or load_host()).mla_append_index_k(k, index_cache, slots, positions, rope_table, index_format,
                                                      rope_style, status)


def mla_quantize_index_q(q: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor, rope_table: torch.Tensor,
                         rope_style: int = ROPE_PAIRS, q_out: Optional[torch.Tensor] = None,
                         weights_out: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Index queries q [tokens, heads, 128] (dims [0, 64) are rotated) as e4m3 rows,
    with each row's scale folded into ``weights`` fp32 [tokens, heads]. Returns
    (float8_e4m3fn [tokens, heads, 128], fp32 [tokens, heads]); rows of tokens
    whose position is negative are not written."""
    return (_host or load_host()).mla_quantize_index_q(q, weights, positions, rope_table, rope_style, q_out,
                                                        weights_out, status)


def mla_index_score(q: torch.Tensor, weights: torch.Tensor, index_cache: torch.Tensor, block_table: torch.Tensor,
                    cache_seqlens: torch.Tensor, width: Optional[int] = None, causal: bool = False, block: int = 1,
                    index_format: int = INDEX_16BIT, scores: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scores fp32 [B, s_q, width] of the cached tokens (block=1) or pages
    (block=64): sum_h weights[b, i, h] * relu(q[b, i, h] . k_t), -inf where
    nothing is visible. q [B, s_q, heads, 128] of the index cache's type (e4m3
    with INDEX_FP8); ``width`` defaults to what the block table reaches."""
    return (_host or load_host()).mla_index_score(q, weights, index_cache, block_table, cache_seqlens, width, causal,
                                                   block, index_format, scores, status)


def mla_select_topk(scores: torch.Tensor, cache_seqlens: torch.Tensor, topk: int, block_table: torch.Tensor,
                    num_blocks: int, causal: bool = False, block: int = 1, indices: Optional[torch.Tensor] = None,
                    lens: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The ``topk`` best visible columns of scores [B, s_q, width], in ascending
    position. block=1: (indices int32 [B, s_q, topk] of cache rows, -1 padded, and
    their number [B, s_q]); block=64: (pages [B, s_q, topk] and the tokens they
    hold [B, s_q]), the block table and lengths of a decode with B * s_q requests
    of one query. ``num_blocks``: pages of the cache that the rows index."""
    return (_host or load_host()).mla_select_topk(scores, cache_seqlens, topk, block_table, num_blocks, causal, block,
                                                   indices, lens, status)


# ---------------------------------------------------------------------------
# Prompts over the latent cache
# ---------------------------------------------------------------------------
def mla_norm_rotate(x: torch.Tensor, positions: torch.Tensor, rope_table: torch.Tensor,
                    weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rope_at: Optional[int] = None,
                    out: Optional[torch.Tensor] = None, rope_out: Optional[torch.Tensor] = None,
                    rope_style: int = ROPE_PAIRS, status: Optional[torch.Tensor] = None):
    """RMS norm of queries or keys for each head, with the rotation of dims
    [rope_at, rope_at + 64) in the same pass (the last 64 unless given): x [tokens,
    heads, dim] of any token and head strides -> out of the same shape (``x``
    itself, or allocated). With ``rope_out`` [tokens, heads, 64] (for example
    ``q_abs[..., 512:]``) the turned dims go there and out [tokens, heads, dim - 64]
    takes the others; returns (out, rope_out) then. ``weight`` [dim] of x's type.
    Rows of tokens whose position is negative are not written."""
    return (_host or load_host()).mla_norm_rotate(x, positions, rope_table, weight, eps, rope_at, out, rope_out,
                                                   rope_style, status)


def mla_norm_append_kv(c_kv: torch.Tensor, k_rope: torch.Tensor, weight: Optional[torch.Tensor], kvcache: torch.Tensor,
                       slots: torch.Tensor, positions: torch.Tensor, rope_table: torch.Tensor, eps: float = 1e-6,
                       kv_format: int = KV_16BIT, rope_style: int = ROPE_PAIRS, rows: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """:func:`mla_append_kv` with the latent dims RMS-normalised on the way
    (``weight`` [512], V4.1 rows [448], of c_kv's type, or None). ``rows`` [n, 576]
    (V4.1 rows: 512) optionally takes the same rows in 16 bits, for the prompt's
    own attention. Returns kvcache."""
    return (_host or load_host()).mla_norm_append_kv(c_kv, k_rope, weight, kvcache, slots, positions, rope_table, eps,
                                                      kv_format, rope_style, rows, status)


def mla_read_kv(kvcache: torch.Tensor, block_table: torch.Tensor, offsets: torch.Tensor, total: Optional[int] = None,
                starts: Optional[torch.Tensor] = None, kv_format: int = KV_16BIT, dtype: Optional[torch.dtype] = None,
                out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of the paged cache read back in 16 bits and packed: rows offsets[b] ..
    offsets[b + 1] of the result [total, 576] (V4.1 rows: 512) are the tokens of
    request b from ``starts[b]`` (0) on; the last 64 dims are the rotated ones.
    ``total`` or ``out`` gives the number of rows (offsets stay on the device).
    ``dtype`` of quantised rows: bf16 (default) or fp16."""
    code = -1 if dtype is None else DTYPE_CODES.get(dtype)
    if code is None:
        raise MLAError(1, f"mla_read_kv: dtype {dtype}")
    return (_host or load_host()).mla_read_kv(kvcache, block_table, offsets, total, starts, kv_format, code, out, status)


def mla_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, softmax_scale: float, causal: bool = True,
                prefix_lens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of many new tokens in the expanded form, over packed documents:
    q [tokens_q, heads, 192] (128 plain dims, 64 rotated), k_nope and v [tokens_k,
    heads, 128], k_rope [tokens_k, 64] shared by the heads; rows cu_seqlens_q[b] ..
    cu_seqlens_q[b + 1] attend to keys cu_seqlens_k[b] .. cu_seqlens_k[b + 1]. Causal:
    the last query sees all keys, each before it one fewer, and every query at least
    the first ``prefix_lens[b]``. Values must be finite: one that is not may reach
    queries shortly before its key too. Returns (out [tokens_q, heads, 128], lse fp32
    [tokens_q, heads]); a query that sees nothing gets 0 and -inf."""
    return (_host or load_host()).mla_prefill(q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, softmax_scale, causal,
                                               prefix_lens, out, lse, status)
