"""Plain numpy definition of the operators that extend a cached prompt.

Rotary positions (binary32 by definition), the rotated append, reading token
ranges back, and fp64 attention of a chunk of new tokens over the paged cache.
"Agent Memory Below the Prompt" (gist.science summary of arXiv 2603.04428), sec.
2.1 item 4: a prompt that extends a cached prefix grows the cache in place.
Shares nothing with the CUDA path.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from . import q4kv_oracle as O


def from_f32(x: np.ndarray, dtype: str) -> np.ndarray:
    """Round binary32 to the 16-bit type, to nearest even (bf16 as uint16 bits)."""
    x = np.asarray(x, np.float32)
    if dtype == "fp16":
        return x.astype(np.float16)
    u = x.view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rotary(x: np.ndarray, dtype: str, table: np.ndarray, positions: np.ndarray, axis: Sequence[int],
           interleaved: bool) -> np.ndarray:
    """x [B][T][H][D]; table [P][pairs][2] float32; positions [axes][B][T]."""
    xf = O.to_f32(x, dtype)
    out = xf.copy()
    half = table.shape[1]
    for f in range(half):
        cs = table[positions[axis[f]], f]                  # [B][T][2]
        c, s = (cs[..., i][..., None].astype(np.float32) for i in (0, 1))
        ia, ib = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        a, b = xf[..., ia], xf[..., ib]
        out[..., ia] = (a * c) - (b * s)
        out[..., ib] = (b * c) + (a * s)
    return from_f32(out, dtype)


def _tokens(pool: O.OraclePool, table: np.ndarray, n: int, unrotate_k: bool = False):
    ks, vs, ms = [], [], []
    for c in range(-(-n // O.BLOCK_TOKENS)):
        blk = int(table[c])
        k, v = pool.dequantize_block(blk, unrotate_k)
        ks.append(k)
        vs.append(v)
        ms.append(pool.masked(blk))
    return np.concatenate(ks, 1)[:, :n], np.concatenate(vs, 1)[:, :n], np.concatenate(ms)[:n]


def gather(pool: O.OraclePool, tables: np.ndarray, starts: Sequence[int], counts: Sequence[int],
           unrotate_k: bool = False):
    """Binary32 K_hat, V_hat [rows][Hkv][D], sequence after sequence."""
    out = ([], [])
    for b, (s, n) in enumerate(zip(starts, counts)):
        if n == 0:
            continue
        k, v, _ = _tokens(pool, tables[b], s + n, unrotate_k)
        out[0].append(k[:, s:].transpose(1, 0, 2))
        out[1].append(v[:, s:].transpose(1, 0, 2))
    empty = np.zeros((0, pool.hkv, pool.d), np.float32)
    return tuple(np.concatenate(x) if x else empty for x in out)


def extend_attention(pool: O.OraclePool, q: np.ndarray, q_dtype: str, tables: np.ndarray, seq_lens: Sequence[int],
                     n_new: Optional[Sequence[int]] = None, scale: Optional[float] = None, window: int = 0):
    """fp64 attention of q [B][T][Hq][D]; returns (out, bound).

    bound is a first-order bound on what rounding q_rot, K_hat, V_hat and the
    weights to fp16 once each can change: every logit by at most
    d_t = scale sum_c |q_c K_tc| 2 u with u = 2^-11, so the output by at most
    sum_t p_t |V_t - o| d_t + 2 u sum_t p_t |V_t|.
    """
    qf = O.to_f32(q, q_dtype).astype(np.float64)
    B, T, Hq, D = qf.shape
    g = Hq // pool.hkv
    scale = 1.0 / math.sqrt(D) if not scale or scale <= 0 else scale
    out, bound = np.zeros(qf.shape), np.zeros(qf.shape)
    u = 2.0 ** -11
    for b in range(B):
        t = T if n_new is None else int(n_new[b])
        if t == 0:
            continue
        n = int(seq_lens[b]) + t
        K, V, gone = _tokens(pool, tables[b], n)
        K, V = K.astype(np.float64), V.astype(np.float64)
        p_at = int(seq_lens[b]) + np.arange(t)[:, None]
        at = np.arange(n)[None]
        seen = at <= p_at
        if window:
            seen &= at > p_at - window
        for h in range(Hq):
            qv = qf[b, :t, h]
            if pool.k_rotated:
                qv = np.stack([O.rotate_f64(x) for x in qv])
            k, v = K[h // g], V[h // g]
            live = np.where(gone[:, None], 0.0, k)
            s = scale * (qv @ live.T)
            s = np.where(gone, O.SENTINEL_LOGIT, s)
            s = np.where(seen, s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ v
            d = scale * (np.abs(qv) @ np.abs(live).T) * 2 * u
            pd = p * d
            out[b, :t, h] = o
            bound[b, :t, h] = pd @ np.abs(v) + pd.sum(1, keepdims=True) * np.abs(o) + 2 * u * (p @ np.abs(v))
    return out, bound
