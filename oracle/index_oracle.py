"""Oracle for the writers of new tokens, the index score and the selection.

* Rotation of 64 dims: pair (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos),
  every product and sum rounded to fp32 (the operator's own definition, so
  that quantised rows compare bit for bit); pair i is dims (2i, 2i + 1), or
  (i, i + 32) with ``halves``.
* Index score: sum over heads of weight x max(0, q . k), in float64.
* Selection: the topk largest, equal ones in the order of their positions, NaN
  as -inf, the result in ascending position.
"""
from __future__ import annotations

import numpy as np
import torch

from .mla_oracle import E4M3_MAX, e4m3_encode_rne, encode_kv_fp4_288, encode_kv_fp8_528, quantize_kv_fp8, to_f64

_F32 = np.float32


def rope_table(positions: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [positions, 64]: 32 cosines, then 32 sines."""
    angle = np.arange(positions, dtype=np.float64)[:, None] * base ** (-np.arange(32) / 32.0)
    return np.concatenate((np.cos(angle), np.sin(angle)), axis=1).astype(_F32)


def rotate(x, row: np.ndarray, halves: bool, exact: bool = False) -> np.ndarray:
    """x [..., 64] (any 16-bit type) by table rows [..., 64]: fp32 values, or
    float64 without a rounding in between when ``exact``."""
    t = np.float64 if exact else _F32
    x = to_f64(x).astype(t)
    c, s = row[..., :32].astype(t), row[..., 32:].astype(t)
    a, b = (x[..., :32], x[..., 32:]) if halves else (x[..., 0::2], x[..., 1::2])
    lo, hi = a * c - b * s, a * s + b * c     # numpy rounds each step to t
    out = np.empty(np.broadcast(x, row).shape, dtype=t)
    if halves:
        out[..., :32], out[..., 32:] = lo, hi
    else:
        out[..., 0::2], out[..., 1::2] = lo, hi
    return out


def round_to(x: np.ndarray, dtype: torch.dtype) -> torch.Tensor:
    """fp32 values rounded once (to nearest even) to a 16-bit type."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=_F32)).to(dtype)


def append_rows(c_kv: torch.Tensor, k_rope: torch.Tensor, row: np.ndarray, halves: bool, kv_format: int) -> torch.Tensor:
    """The cache rows of new tokens as bytes, uint8 [n, row bytes]; kv_format as
    in the C ABI (0: 16-bit, 1: 656 B, 2: 528 B, 3: 288 B)."""
    rope = rotate(k_rope, row, halves)
    if kv_format <= 1:
        rows = torch.cat((c_kv, round_to(rope, c_kv.dtype)), dim=1).contiguous()
        return torch.from_numpy(quantize_kv_fp8(rows)) if kv_format else rows.view(torch.uint8)
    values = np.concatenate((to_f64(c_kv), rope.astype(np.float64)), axis=1)
    return torch.from_numpy(encode_kv_fp8_528(values) if kv_format == 2 else encode_kv_fp4_288(values))


def index_row_codes(x, row: np.ndarray, halves: bool):
    """Rows [..., 128] with dims [0, 64) rotated -> (fp32 values, e4m3 codes,
    fp32 scales amax / 448, 1 for a zero row)."""
    v = np.concatenate((rotate(x[..., :64], row, halves), to_f64(x[..., 64:]).astype(_F32)), axis=-1)
    amax = np.abs(v).max(axis=-1)
    scale = np.where(amax == 0, _F32(1.0), amax / _F32(E4M3_MAX)).astype(_F32)
    return v, e4m3_encode_rne((v / scale[..., None]).astype(_F32)), scale


def index_score(q: np.ndarray, weights: np.ndarray, keys: np.ndarray) -> np.ndarray:
    """q [n, h, 128], weights [n, h], keys [t, 128] -> float64 [n, t]."""
    return np.einsum("nh,nht->nt", weights, np.maximum(np.einsum("nhd,td->nht", q, keys), 0.0))


def index_score_error(q: np.ndarray, weights: np.ndarray, keys: np.ndarray) -> np.ndarray:
    """Bound of an fp32 evaluation's error, [n, t]. With u = 2^-24, a dot of 128
    exact products accumulated in fp32 (each step at worst cut off, one unit
    2u of what is summed) is off by at most 128 * 2u * sum |q_d k_d|; the
    positive part does not enlarge it; each of the h steps of the weighted sum
    rounds by u of at most the sum of its terms; a key's scale rounds once, as
    does its product."""
    u = 2.0 ** -24
    size = np.einsum("nh,nhd,td->nt", np.abs(weights), np.abs(q), np.abs(keys))
    return (2 * 128 + q.shape[1] + 2) * u * size


def page_max(scores: np.ndarray, page: int = 64) -> np.ndarray:
    pad = -scores.shape[-1] % page
    s = np.concatenate((scores, np.full(scores.shape[:-1] + (pad,), -np.inf)), axis=-1)
    return s.reshape(s.shape[:-1] + (-1, page)).max(axis=-1)


def select_topk(scores, n: int, topk: int, last: bool = False) -> np.ndarray:
    """Positions selected among scores[:n], ascending; ``last`` forces n - 1."""
    s = [float(v) for v in scores[:n]]
    key = [(-np.inf, 1) if np.isnan(v) else (v, 1) for v in s]
    if last and n:
        key[n - 1] = (np.inf, 2)
    order = sorted(range(n), key=lambda i: (-key[i][0], -key[i][1], i))
    return np.array(sorted(order[:topk]), dtype=np.int64)
