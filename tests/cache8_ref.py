"""The 8-bit cache's operators in 64 bits (numpy), from their definition, and the error bounds the tests use.

e4m3: sign, 4 exponent bits of bias 7, 3 fraction bits, 0x7F / 0xFF NaN.  A chunk's rows on one side share one scale."""
import math

import numpy as np


def _table():
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[b] = (math.nan if e == 15 and f == 7 else x) * (-1.0 if b & 128 else 1.0)
    return v


TABLE = _table()


def encode(x):
    """Bytes of the e4m3 values nearest to x (float64; halves to even, saturating, NaN -> 0x7F).  A zero keeps its sign."""
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    _, e = np.frexp(a)
    e = np.maximum(e - 1, -6)
    n = np.rint(np.ldexp(a, 3 - e)).astype(np.int64)              # units of 2^(e-3): 0..16, halves to even
    code = (e + 6) * 8 + n                                        # fraction overflow carries into the exponent
    code = np.where(n < 8, n, code)                               # subnormal (e == -6): the fraction itself
    return np.where(nan, 0x7F, np.minimum(code, 0x7E) | (np.signbit(x) * 128)).astype(np.uint8)


def scale_for(m):
    e = -100
    while e < 119 and m > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, data, scale, t0, C):
    """x [n,d] float64 into data [T,d] bytes and scale [nL] (one side of one kv-head), in place."""
    n = len(x)
    for c in range(t0 // C, (t0 + n - 1) // C + 1):
        a, b = max(t0, c * C), min(t0 + n, (c + 1) * C)
        new = x[a - t0:b - t0]
        s = scale_for(np.max(np.where(np.isfinite(new), np.abs(new), 0.0), initial=0.0))
        if a > c * C:
            old = float(scale[c])
            s = max(s, old)
            if s > old:
                data[c * C:a] = encode(TABLE[data[c * C:a]] * (old / s))
        scale[c] = s
        data[a:b] = encode(new / s)


def landmarks(k, u, scale):
    """k [rows,d], u [d] -> (L, beta)."""
    x = k @ u * scale
    x = x - x.max()
    e = np.exp(x)
    p = e / e.sum()
    return p @ k, math.log(e.sum()) - float(p @ x)


def attend_row(q, kd, vd, ks, vs, chunks, score, pos, C, scale):
    """One query group: q [G,d]; kd, vd [T,d] float64 values of the bytes; ks, vs [nL]; chunks [ns] (-1: empty slot);
    score [G,ns].  Returns (O [G,d], reach [G] = sum of w * largest |v| of the slot, logit magnitude [G])."""
    G, d = q.shape
    O, reach, mag = np.zeros((G, d)), np.zeros(G), np.zeros(G)
    for h in range(G):
        s = np.where(chunks < 0, -np.inf, score[h])
        if np.all(s == -np.inf):
            continue
        w = np.exp(s - s.max())
        w = w / w.sum()
        for j, c in enumerate(chunks):
            if w[j] == 0.0:
                continue
            a, b = c * C, min((c + 1) * C, pos + 1)
            k, v = kd[a:b] * ks[c], vd[a:b] * vs[c]
            x = k @ q[h] * scale
            mag[h] = max(mag[h], float(np.max(np.abs(k) @ np.abs(q[h]))) * scale)
            p = np.exp(x - x.max())
            O[h] += w[j] * (p / p.sum()) @ v
            reach[h] += w[j] * np.max(np.abs(v))
    return O, reach, mag


def half_step(dtype):
    """Half a rounding step relative to the value."""
    return {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]


def bound(reach, mag, ref, out, d, C, score_mag=0.0):
    """How far an output may be off.  Logits: a float32 dot product of d terms is within (d + 8) 2^-24 of the sum of its
    magnitudes `mag` (8: the query's and the scales' own roundings); a softmax weight moves by twice the largest logit error.
    The sums over C keys and the slots add (C + 40) 2^-24, the fusion weights 2 * 4 * 2^-24 of their scores.  With bf16
    results the weights of the value product may be rounded to 11 bits (2^-11 of `reach`), queries to 2^-17 of their
    row's largest (2 * 2^-17 * mag), and the result is rounded."""
    e = 2 * (d + 8) * 2.0 ** -24 * mag + (C + 40 + 8 * score_mag) * 2.0 ** -24
    if out == "bf16":
        e = e + 2.0 ** -11 + 2 * 2.0 ** -17 * mag
    return (e * reach)[..., None] + half_step(out) * np.abs(ref) + 1e-37
