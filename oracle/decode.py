"""The decode-step operators on 4-bit tensors (oracle, test infrastructure
only): products of a few tokens with a 4-bit weight matrix, attention of one
new token per sequence over the paged INT4 cache, and page copies.

Sources on the pages:
  * QuaRot reviews, review 3 Questions: with Y = X H^T applied to activations
    and weights alike, X W^T is unchanged -- for a key cache the same statement
    says q . k is unchanged when both carry the rotation.
  * QuaRot reviews, final comments: the KV cache at 4 bits with the randomized
    Hadamard transform; the pages define no attention kernel, no paging and no
    window, so the definitions below are the textbook ones.

Everything is float64 on dequantized values; nothing here follows the CUDA
path's arrangement (no splitting, no running maximum, no rotated scores: keys
and values are rotated back first).
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_decode, e4m3_decode
from .hadamard import sylvester

HEAD = 128


def weights(fmt: str, codes, scales, zeros=None, tensor_scale=None) -> np.ndarray:
    """Unpacked codes [n, k] and their scales -> float64 weights, exactly."""
    c = np.asarray(codes, dtype=np.int64)
    n, k = c.shape
    if fmt == "int4_sym":
        q = np.where(c >= 8, c - 16, c).astype(np.float64)
        return q * np.asarray(scales, dtype=np.float32).astype(np.float64)[:, None]
    if fmt == "int4_asym":
        s = np.asarray(scales, dtype=np.float16).astype(np.float64)[..., None]
        z = np.asarray(zeros, dtype=np.float16).astype(np.float64)[..., None]
        return ((c.reshape(n, k // HEAD, HEAD) - z) * s).reshape(n, k)
    v = e2m1_decode(c)
    if fmt == "nvfp4":
        d = e4m3_decode(scales)[..., None] * np.float64(np.float32(tensor_scale))
        return (v.reshape(n, k // 16, 16) * d).reshape(n, k)
    if fmt == "mxfp4":
        d = np.ldexp(1.0, np.asarray(scales, dtype=np.int64) - 127)[..., None]
        return (v.reshape(n, k // 32, 32) * d).reshape(n, k)
    raise ValueError(fmt)


def gemv(x, w) -> np.ndarray:
    """y[j][i] = sum_k x[j][k] w[i][k]."""
    return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T


def visible(length: int, window: int, sinks: int) -> np.ndarray:
    """Positions a new token at the end of `length` cached tokens attends to."""
    t = np.arange(max(0, int(length)))
    return t if window == 0 else t[(t < sinks) | (t >= length - window)]


def cache_rows(table, page_size: int, num_slots: int, positions) -> np.ndarray:
    """Cache rows of the positions of one sequence; -1 where there is none."""
    page = np.asarray(table, dtype=np.int64)[positions // page_size]
    row = page * page_size + positions % page_size
    return np.where((page >= 0) & (row < num_slots), row, -1)


def dequant_heads(cache, rows, head: int) -> np.ndarray:
    """Stored (rotated) values of one head at the rows: codes are unpacked
    [slots, heads * 128], scales and zeros [slots, heads]."""
    codes, scales, zeros = cache
    u = np.asarray(codes)[rows, head * HEAD:(head + 1) * HEAD].astype(np.float64)
    z = np.asarray(zeros, dtype=np.float16)[rows, head].astype(np.float64)[:, None]
    s = np.asarray(scales, dtype=np.float16)[rows, head].astype(np.float64)[:, None]
    return (u - z) * s


def attn_decode(q, k_cache, v_cache, k_signs, v_signs, table, page_size, lens, scale,
                window=0, sinks=0) -> np.ndarray:
    """[batch, q_heads, 128] -> the same shape; see include/kq.h."""
    q = np.asarray(q, dtype=np.float64)
    batch, q_heads, _ = q.shape
    slots, heads = np.asarray(k_cache[1]).shape
    group = q_heads // heads
    h = sylvester(128).astype(np.float64) / np.sqrt(HEAD)
    one = np.ones(heads * HEAD)
    ks = (one if k_signs is None else np.asarray(k_signs, dtype=np.float64)).reshape(heads, HEAD)
    vs = (one if v_signs is None else np.asarray(v_signs, dtype=np.float64)).reshape(heads, HEAD)
    most = np.asarray(table).shape[1] * page_size
    out = np.zeros_like(q)
    for b in range(batch):
        rows = cache_rows(table[b], page_size, slots,
                          visible(min(int(lens[b]), most), window, sinks))
        rows = rows[rows >= 0]
        if rows.size == 0:
            continue
        for i in range(heads):
            keys = dequant_heads(k_cache, rows, i) @ h * ks[i]
            values = dequant_heads(v_cache, rows, i) @ h * vs[i]
            a = q[b, i * group:(i + 1) * group] @ keys.T * scale
            p = np.exp(a - a.max(axis=1, keepdims=True))
            out[b, i * group:(i + 1) * group] = p @ values / p.sum(axis=1, keepdims=True)
    return out


def copy_pages(array, pairs, page_size: int) -> np.ndarray:
    """array [layers, slots, width] after the copies (destinations distinct and
    no pair's source)."""
    out = np.array(array)
    pages = out.shape[1] // page_size
    for s, d in np.asarray(pairs, dtype=np.int64):
        if 0 <= s < pages and 0 <= d < pages:
            out[:, d * page_size:(d + 1) * page_size] = \
                array[:, s * page_size:(s + 1) * page_size]
    return out
