"""CPU oracle of the prompt side (fp64, numpy): rotary positions, the paged
cache, attention of a chunk of new tokens over it, and sampling from filtered
logits.

TEST INFRASTRUCTURE, as medusa_oracle.py: the plain statement of what the
calls compute, sharing no code with the product path.  Arrays come in already
widened to float64.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import numpy as np


def rope_freqs(rot: int, theta: float, scaling: str = "none", factor: float = 1.0,
               low: float = 1.0, high: float = 4.0, original: float = 8192.0
               ) -> Tuple[np.ndarray, float]:
    """Frequencies f_i (radians per position) and the factor on rotated
    elements.  low / high: full turns over the original length."""
    out, scale = [], 1.0
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "llama3":
            wavelength = 2.0 * math.pi / f
            if wavelength > original / low:
                f = f / factor
            elif wavelength > original / high:
                s = (original / wavelength - low) / (high - low)
                f = (1.0 - s) * f / factor + s * f
        elif scaling == "yarn":
            def index(turns):
                return rot * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
            a = max(math.floor(index(high)), 0)
            b = min(math.ceil(index(low)), rot - 1)
            ramp = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1.0 - ramp)
            scale = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out), scale


def rope(x: np.ndarray, positions: np.ndarray, freqs: np.ndarray, scale: float = 1.0,
         interleaved: bool = False, inverse: bool = False) -> np.ndarray:
    """x [T, H, dh] with its first 2 * len(freqs) elements rotated."""
    n = len(freqs)
    y = np.array(x, np.float64)
    for t, p in enumerate(positions):
        for i in range(n):
            a = float(p) * float(freqs[i]) * (-1.0 if inverse else 1.0)
            e0, e1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            x0, x1 = x[t, :, e0], x[t, :, e1]
            y[t, :, e0] = scale * (x0 * math.cos(a) - x1 * math.sin(a))
            y[t, :, e1] = scale * (x0 * math.sin(a) + x1 * math.cos(a))
    return y


def slots(cu_q: Sequence[int], kv_len: Sequence[int], T: int) -> np.ndarray:
    """[T, 2]: sequence and cache slot of each row, (-1, -1) behind the last."""
    out = np.full((T, 2), -1, dtype=np.int64)
    for b in range(len(kv_len)):
        n = cu_q[b + 1] - cu_q[b]
        for i in range(n):
            out[cu_q[b] + i] = (b, kv_len[b] - n + i)
    return out


def append(pool: np.ndarray, x: np.ndarray, table: np.ndarray, cu_q, kv_len) -> np.ndarray:
    """pool [n_pages, Hkv, page, dh] with the rows x [T, Hkv, dh] written at
    their slots (negative slots skipped)."""
    pool = np.array(pool)
    page = pool.shape[2]
    for t, (b, s) in enumerate(slots(cu_q, kv_len, x.shape[0])):
        if b >= 0 and s >= 0:
            pool[table[b, s // page], :, s % page] = x[t]
    return pool


def chunk_attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, table: np.ndarray, cu_q, kv_len,
                    scale: float) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """out [T, Hq, dh] (0 where a row sees nothing or lies behind the last
    sequence), and what error bounds need: sum_j p_j |v_j| (same shape),
    max_j sum_e |q_e k_je| * scale and the number of visible keys, per row and
    head."""
    T, Hq, dh = q.shape
    Hkv, page = K.shape[1], K.shape[2]
    out, absv = np.zeros((T, Hq, dh)), np.zeros((T, Hq, dh))
    mag, count = np.zeros((T, Hq)), np.zeros((T, Hq))
    where = slots(cu_q, kv_len, T)
    for b in range(len(kv_len)):
        ids = [int(x) for x in table[b, :-(-int(kv_len[b]) // page)]]
        if not ids:
            continue
        k = np.concatenate([K[i] for i in ids], axis=1)[:, :kv_len[b]]
        v = np.concatenate([V[i] for i in ids], axis=1)[:, :kv_len[b]]
        for t in range(cu_q[b], cu_q[b + 1]):
            n = int(where[t, 1]) + 1
            if n <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[h // (Hq // Hkv), :n], v[h // (Hq // Hkv), :n]
                s = kk @ q[t, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h], absv[t, h] = p @ vv, p @ np.abs(vv)
                mag[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
                count[t, h] = n
    return out, absv, mag, count


def sample_row(z: np.ndarray, u: float, temperature: float = 1.0, top_k: int = 0,
               top_p: float = 1.0, min_p: float = 0.0) -> Tuple[int, int, float]:
    """(token, kept, margin): margin is how far, relative to the masses
    compared, the nearest decision lies from flipping (inf when none)."""
    V = z.shape[0]
    order = sorted((v for v in range(V) if z[v] > -np.inf), key=lambda v: (-z[v], v))
    if temperature == 0.0 or top_k == 1:
        return order[0], 1, math.inf
    w = [math.exp(min((z[v] - z[order[0]]) / temperature, 0.0)) for v in order]
    n = len(order)
    if top_k > 0:
        n = min(n, top_k)
    margin = math.inf
    n_p = n
    if top_p < 1.0:
        total, before, n_p = math.fsum(w[:n]), 0.0, 0
        for i in range(n):
            if i > 0:
                margin = min(margin, abs(before - top_p * total) / total)
            if i > 0 and not before < top_p * total:
                break
            n_p, before = i + 1, before + w[i]
    if min_p > 0.0:
        for i in range(n):
            margin = min(margin, abs(w[i] - min_p) / min_p) if 0 < i else margin
        n = sum(1 for i in range(n) if w[i] >= min_p)
    n = max(1, min(n, n_p))
    kept = sorted(zip(order[:n], w[:n]))
    total, cum, token = math.fsum(x for _, x in kept), 0.0, None
    for v, x in kept:
        cum += x
        if n > 1 and v != kept[-1][0]:
            margin = min(margin, abs(cum - u * total) / total)
        if token is None and (cum > u * total or (u == 0.0 and x >= 0.0)):
            token = v
    return (kept[-1][0] if token is None else token), n, margin
