"""Oracle for prompts over the latent cache: norms, rows read back, and the
attention of many new tokens, in float64 from the definitions.

* RMS norm: x / sqrt(mean(x^2) + eps) * w.
* Attention of one document, per head: query i of n_q sees the keys below
  vis(i) = n_k, or causal n_k - n_q + i + 1, at least ``prefix``; scores are
  scale (q[:128] . k_nope + q[128:] . k_rope), softmax over the visible keys, the
  weighted sum of v. Nothing visible: 0 and -inf.
"""
from __future__ import annotations

import numpy as np

from .index_oracle import rotate
from .mla_oracle import dequantize_kv_fp4_288, dequantize_kv_fp8, dequantize_kv_fp8_528, to_f64


def rms_norm(x, weight=None, eps: float = 1e-6) -> np.ndarray:
    x = to_f64(x)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return y if weight is None else y * to_f64(weight)


def norm_rotate(x, weight, eps, row: np.ndarray, at: int, halves: bool) -> np.ndarray:
    """x [tokens, heads, d], table rows [tokens, 64] -> float64 of x's shape."""
    y = rms_norm(x, weight, eps)
    y[..., at:at + 64] = rotate(y[..., at:at + 64], row[:, None], halves, exact=True)
    return y


def norm_rotate_error(y: np.ndarray, at: int, halves: bool) -> np.ndarray:
    """Bound of an fp32 evaluation's error before the result's rounding, per
    element. With u = 2^-24: the d squares and their sum in any order are off by at
    most (d + 1) u of the sum, its root by half of that; the division, root, mean,
    eps and the products with it and the weight round 6 times: (d / 2 + 7) u of y.
    A turned value is a sum of two products, each rounded, and rounded itself: 2 u
    more of the sum of their sizes, which is below |y0| + |y1| of its pair as the
    rotation left it, times sqrt 2."""
    u, d = 2.0 ** -24, y.shape[-1]
    size = np.abs(y)
    turned = size[..., at:at + 64]
    a, b = (turned[..., :32], turned[..., 32:]) if halves else (turned[..., 0::2], turned[..., 1::2])
    both = np.sqrt(2.0) * (a + b)
    pair = np.concatenate((both, both), -1) if halves else np.repeat(both, 2, axis=-1)
    size = size.copy()
    size[..., at:at + 64] = pair
    return (d / 2 + 9) * u * size


def cached_rows(raw: np.ndarray, kv_format: int) -> np.ndarray:
    """Quantised rows (uint8) as the float64 values they hold."""
    return {1: dequantize_kv_fp8, 2: dequantize_kv_fp8_528, 3: dequantize_kv_fp4_288}[kv_format](raw)


def visible(n_q: int, n_k: int, causal: bool, prefix: int = 0) -> np.ndarray:
    """Keys that each query sees, [n_q]."""
    if not causal:
        return np.full(n_q, n_k)
    prefix = min(max(prefix, 0), n_k)
    return np.array([min(max(n_k - n_q + i + 1, prefix), n_k) for i in range(n_q)], dtype=np.int64)


def prefill(q, k_nope, k_rope, v, scale: float, seen: np.ndarray):
    """One document: q [n_q, h, 192], k_nope, v [n_k, h, 128], k_rope [n_k, 64],
    seen [n_q] -> (out [n_q, h, 128], lse [n_q, h], sum of weight x |v|, largest sum
    of |q k| over the visible keys [n_q, h])."""
    q, k_nope, k_rope, v = (to_f64(t) for t in (q, k_nope, k_rope, v))
    n_q, h = q.shape[:2]
    out, size = np.zeros((n_q, h, v.shape[-1])), np.zeros((n_q, h, v.shape[-1]))
    lse, dots = np.full((n_q, h), -np.inf), np.zeros((n_q, h))
    for i in range(n_q):
        n = int(seen[i])
        if n == 0:
            continue
        s = np.einsum("hd,jhd->hj", q[i, :, :128], k_nope[:n]) + np.einsum("hd,jd->hj", q[i, :, 128:], k_rope[:n])
        s *= scale
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(axis=1, keepdims=True)
        out[i] = np.einsum("hj,jhd->hd", p / total, v[:n])
        size[i] = np.einsum("hj,jhd->hd", p / total, np.abs(v[:n]))
        lse[i] = (m + np.log(total))[:, 0]
        dots[i] = (np.einsum("hd,jhd->hj", np.abs(q[i, :, :128]), np.abs(k_nope[:n]))
                   + np.einsum("hd,jd->hj", np.abs(q[i, :, 128:]), np.abs(k_rope[:n]))).max(axis=1)
    return out, lse, size, dots


def prefill_error(out, lse, size, dots, scale: float, seen, v_total, unit: float, fp16: bool):
    """Bounds of the result's error (per element of out, of lse). With u = 2^-24 and
    U = `unit`, half a step of the 16-bit type:
    a dot of 192 exact products accumulated in fp32 (each step at worst cut off, 2u
    of what is summed) is off by 192 * 2u * sum |q k|, as is its exponential relatively,
    times the scale; scaling, reference and the 2^x of the hardware (2^-22) add 8u of 1
    and 4u of |x| <= 2 * (|s| + |lse|), s being below scale * dots. Weights round to 16
    bits for the products with v (U each; fp16's smallest ones by 2^-25 of the largest
    weight at least, which is no larger than their sum), the products accumulate over n
    keys (2u each step), the result rounds once (U)."""
    u = 2.0 ** -24
    n = np.asarray(seen, np.float64)[:, None]
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    weight = 384 * u * scale * dots + 8 * u + 8 * u * (scale * dots + finite)      # relative error of one weight
    rel = 2 * weight + (2 * n + 64) * u
    bound = (U_OUT * unit) * np.abs(out) + (unit + rel)[..., None] * size
    if fp16:
        bound = bound + 2.0 ** -25 * (1 + np.asarray(v_total))
    return bound, weight + (n + 64) * u + 4 * u * finite


U_OUT = 1.01     # the result's own rounding is of the value computed, not of the exact one
