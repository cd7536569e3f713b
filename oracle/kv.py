"""Plain CPU oracle of the paged NVFP4 key/value cache: rotation, the cache's bytes,
and attention over cached values.

TEST INFRASTRUCTURE ONLY.  Only ``tests/``, ``__graft_entry__.smoke()`` and the
``cpu_baseline`` leg of ``bench.py`` may import, call or execute anything in this
package.  The HIP library never uses it; the two share no code.  numpy; the rotation
in fp32 in the order that include/nvfp4.h states (the codes of the rotated keys depend
on it), everything else in float64.

Cache layout: page = [head][page_size / 16 granules]; granule of 16 tokens, head
dimension D: K codes [16][D/2] at 0, K scales [16][D/16] at 8 D, V codes
[4 quads][16 parts][4 tokens][D/32] at 9 D, V scales [4 quads][D/16][4 tokens] at 17 D.
"""

from __future__ import annotations

import numpy as np

from . import nvfp4 as O


def rotate_f32(x, cos, sin, interleaved):
    """x fp32 [T, H, D]; cos, sin fp32 [T, R/2]: the rotation with every product and
    sum rounded to fp32."""
    x = np.asarray(x, dtype=np.float32)
    y = x.copy()
    R = 2 * cos.shape[1]
    c, s = cos[:, None].astype(np.float32), sin[:, None].astype(np.float32)
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., lo], x[..., hi]
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


def quantize_heads(x, g):
    """x [T, H, D] -> codes [T, H, D/2], scales [T, H, D/16] under g fp32 [H]."""
    T, H, D = x.shape
    codes, scales = O.quantize_rows(np.asarray(x, dtype=np.float64).reshape(T * H, D), np.tile(g, T))
    return codes.reshape(T, H, D // 2), scales.reshape(T, H, D // 16)


def byte_places(slot, head, Hkv, page, D):
    """(K codes [D/2], K scales [D/16], V codes, V scales): the byte addresses of one
    token of one head in the flat cache."""
    base = (slot // page) * (Hkv * page * D * 9 // 8) + (head * (page // 16) + (slot % page) // 16) * 18 * D
    r = slot % 16
    quad, e = r // 4, r % 4
    byte, blk = np.arange(D // 2), np.arange(D // 16)
    per = D // 32
    return (base + r * (D // 2) + byte, base + 8 * D + r * (D // 16) + blk,
            base + 9 * D + quad * 64 * per + (byte // per) * 4 * per + e * per + byte % per,
            base + 17 * D + quad * (D // 4) + blk * 4 + e)


def append(cache, k, v, slots, kg, vg, page):
    """The flat cache (uint8, changed in place) after k, v [T, H, D] went to their slots."""
    T, H, D = k.shape
    kc, ks = quantize_heads(k, kg)
    vc, vs = quantize_heads(v, vg)
    total = cache.size // (H * page * D * 9 // 8) * page
    for t in range(T):
        if not 0 <= slots[t] < total:
            continue
        for h in range(H):
            for at, new in zip(byte_places(int(slots[t]), h, H, page, D), (kc[t, h], ks[t, h], vc[t, h], vs[t, h])):
                cache[at] = new


def gather(cache, slots, Hkv, D, kg, vg, page):
    """(k, v) float64 [T, Hkv, D] of the slots' rows (outside the cache: zeros)."""
    total = cache.size // (Hkv * page * D * 9 // 8) * page
    k, v = np.zeros((len(slots), Hkv, D)), np.zeros((len(slots), Hkv, D))
    for t, slot in enumerate(slots):
        if not 0 <= slot < total:
            continue
        for h in range(Hkv):
            a, b, c, d = byte_places(int(slot), h, Hkv, page, D)
            k[t, h] = O.dequantize_rows(cache[a][None], cache[b][None], kg[h:h + 1])[0]
            v[t, h] = O.dequantize_rows(cache[c][None], cache[d][None], vg[h:h + 1])[0]
    return k, v


def attention(q, k, v, scale, window=0):
    """One sequence: q [m, Hq, D], the last m of the n tokens of k, v [n, Hkv, D].
    Returns (o [m, Hq, D], lse [m, Hq], weights [m, Hq, n]) in float64."""
    m, Hq, D = q.shape
    n, Hkv, _ = k.shape
    q = np.asarray(q, dtype=np.float64)
    o, lse, weights = np.zeros((m, Hq, D)), np.full((m, Hq), -np.inf), np.zeros((m, Hq, n))
    for i in range(m):
        p = n - m + i
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            s = scale * (k[lo:p + 1, kh] @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            lse[i, h] = top + np.log(w.sum())
            weights[i, h, lo:p + 1] = w / w.sum()
            o[i, h] = weights[i, h, lo:p + 1] @ v[lo:p + 1, kh]
    return o, lse, weights


def attention_bounds(q, k, v, weights, scale, out_dtype):
    """Bounds on |o - o64| (before the output's own rounding) and |lse - lse64| for a
    kernel that sums scores of exact f16 operands in fp32 and rounds its weights to f16
    (bf16 output) or to two f16 terms (fp32).

    A score's error: the fp32 sum of D products (gamma_D of the sum of magnitudes), the
    fp32 score factor and the subtraction of the maximum (4 u of the score and of the
    maximum), fp32 queries as two f16 terms (2^-21).  The weights inherit it relatively,
    numerator and denominator, plus exp2 (4 u), the f16 rounding, weights below the normal
    f16 range (2^-25 each, where the largest weight is at least 2^7), and the fp32 sums over
    n weights (gamma_n)."""
    u = 2.0 ** -24
    m, Hq, D = q.shape
    n, Hkv, _ = k.shape
    kr, vr = np.repeat(k, Hq // Hkv, 1), np.repeat(v, Hq // Hkv, 1)
    mag = abs(scale) * np.einsum("mhd,nhd->mhn", np.abs(np.asarray(q, dtype=np.float64)), np.abs(kr))
    mag = np.where(weights > 0, mag, 0).max(-1) if n else np.zeros((m, Hq))
    ds = ((D + 16) * u + (2.0 ** -21 if out_dtype == "f32" else 0)) * mag + 16 * u
    f16 = 2.0 ** -11 if out_dtype == "bf16" else 2.0 ** -21
    mean = np.einsum("mhn,nhd->mhd", weights, np.abs(vr)) if n else np.zeros(q.shape)
    most = np.abs(vr).max(0)[None] if n else 0.0
    o = (2 * ds[..., None] + f16 + 2 * (n + 16) * u) * mean * 1.01 + n * 2.0 ** -32 * most
    return o, ds + (n + 16) * u
