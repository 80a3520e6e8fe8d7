"""Plain 64-bit NumPy definitions of the 8-bit operators.

Codes and scales: a group of values x has the scale s = max(max|x| * r, 2^-60)
(one float32 product, r the float32 nearest 1 / qmax; qmax 127 for int8, 448
for e4m3) and each value the code nearest to the exact quotient x / s, ties to even.  A group with a
non-finite value has the scale NaN and codes 0.  Test infrastructure only; it
shares no code with the library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

QMAX = {"int8": 127, "e4m3": 448}
FLOOR = np.float32(2.0 ** -60)


def e4m3_values() -> np.ndarray:
    """The value of every byte: sign, 4 exponent bits (bias 7), 3 fraction
    bits; exponent 0 is subnormal, 0x7F and 0xFF are NaN."""
    v = np.empty(256, np.float64)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        m = (f / 8.0) * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        v[b] = -m if b & 128 else m
        if (b & 127) == 127:
            v[b] = np.nan
    return v


E4M3 = e4m3_values()


def values(codes: np.ndarray, kind: str) -> np.ndarray:
    """Codes (int8, or e4m3 bytes as uint8) as float64."""
    return codes.astype(np.float64) if kind == "int8" else E4M3[codes.view(np.uint8)]


def scale_of(amax, kind: str) -> np.ndarray:
    """float32 scales of groups with largest magnitudes `amax`."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(all="ignore"):
        s = np.maximum(amax.astype(np.float32) * (np.float32(1) / np.float32(QMAX[kind])), FLOOR)
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def encode(x: np.ndarray, s: np.ndarray, kind: str) -> np.ndarray:
    """Codes of x under scales s (broadcast), as int8 or e4m3 bytes in uint8.
    A quotient of a bf16 (or integer times float32) value and a float32 scale
    is further than 2^-34 relative from any middle of two codes unless it is
    one, so the 64-bit quotient decides."""
    x, s = np.broadcast_arrays(np.asarray(x, np.float64), np.asarray(s, np.float64))
    with np.errstate(all="ignore"):
        v = np.where(np.isfinite(s) & np.isfinite(x), x / s, 0.0)
    if kind == "int8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8)
    mag = np.minimum(np.abs(v), 448.0)
    e = np.maximum(np.frexp(mag)[1] - 1, -6)       # mag in [2^e, 2^(e+1)) or subnormal
    step = np.ldexp(1.0, e - 3)
    q = np.rint(mag / step) * step
    e = np.maximum(np.frexp(q)[1] - 1, -6)
    frac = np.rint(q / np.ldexp(1.0, e - 3)).astype(np.int64)  # 8..15, or 0..7 subnormal
    b = np.where(frac >= 8, ((e + 7) << 3) + (frac - 8), frac)
    return (b | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def encode_one(x: float, s: float, kind: str) -> float:
    """The value of the code of one x / s in exact rational arithmetic."""
    v = Fraction(x) / Fraction(s)
    if kind == "int8":
        cand = [Fraction(i) for i in range(-127, 128)]
        odd = lambda i: i - 127                       # noqa: E731
    else:
        bytes_ = [b for b in range(256) if (b & 127) != 127 and b != 128]
        cand = [Fraction(float(E4M3[b])) for b in bytes_]
        odd = lambda i: bytes_[i]                     # noqa: E731
    d = [abs(c - v) for c in cand]
    best = min(d)
    at = [i for i, y in enumerate(d) if y == best]
    at.sort(key=lambda i: odd(i) & 1)                 # ties to the even code
    return float(cand[at[0]])


def quantise_rows(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """int8 codes and float32 scales of the rows of x."""
    with np.errstate(all="ignore"):
        amax = np.where(np.isfinite(x).all(1), np.abs(x).max(1), np.nan)
    s = scale_of(amax, "int8")
    return encode(x, s[:, None], "int8"), s


def dequantise_cache(codes, scale, kind: str, block: int) -> np.ndarray:
    """[B, Hkv, L, dh] values of a cache with a scale per `block` positions."""
    L = codes.shape[2]
    s = np.repeat(scale.astype(np.float64), block, axis=2)[:, :, :L, None]
    return values(codes, kind) * s


def append(codes, scale, new, ctx_len, new_len, kind: str, block: int):
    """One cache (K or V) after rows new[b, :new_len[b]] joined at ctx_len[b];
    returns new codes and scales.  new: float64 [B, n, Hkv, dh]."""
    codes, scale = codes.copy(), scale.copy()
    B, n, Hkv, dh = new.shape
    cap = codes.shape[2]
    for b in range(B):
        L, m = int(ctx_len[b]), int(new_len[b])
        if m < 0 or m > n or L < 0 or L + m > cap or m == 0:
            continue
        for g in range(Hkv):
            for k in range(L // block, (L + m - 1) // block + 1):
                lo, hi = max(k * block, L), min((k + 1) * block, L + m)
                x = new[b, lo - L:hi - L, g]
                amax = np.abs(x).max() if np.isfinite(x).all() else np.nan
                s = scale_of(amax, kind)[()]
                if k * block < L:
                    s_old = scale[b, g, k]
                    old = slice(k * block, L)
                    if s_old >= s or np.isnan(s_old):
                        s = s_old
                    elif np.isnan(s):
                        codes[b, g, old] = 0
                    else:
                        v = values(codes[b, g, old], kind) * np.float64(s_old)
                        codes[b, g, old] = encode(v, s, kind)
                codes[b, g, lo:hi] = encode(x, s, kind) if not np.isnan(s) else 0
                scale[b, g, k] = s
    return codes, scale


def linear(x, w_q, w_scale) -> np.ndarray:
    """x [M, K] (float64 of bf16), int8 weights [N, K]: unrounded float64."""
    q, s = quantise_rows(x)
    acc = q.astype(np.float64) @ w_q.astype(np.float64).T
    return acc * s.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None]


def attention(q, k_blk, v_blk, k, v, ctx_len):
    """softmax(q . [k_blk ; k[:L]] / sqrt(dh)) [v_blk ; v[:L]] for float64
    arrays; returns the output [B, S, Hq, dh], the mean of |value| under the
    softmax (the weight of a relative error of the probabilities) and the
    largest sum of |q||k| / sqrt(dh) of a row (that of a score's rounding)."""
    B, S, Hq, dh = q.shape
    Hkv = k_blk.shape[2]
    G = Hq // Hkv
    out = np.empty(q.shape)
    mass = np.empty(q.shape)
    reach = np.empty((B, S, Hq, 1))
    for b in range(B):
        L = int(ctx_len[b])
        for g in range(Hkv):
            keys = np.concatenate((k_blk[b, :, g], k[b, g, :L]))
            vals = np.concatenate((v_blk[b, :, g], v[b, g, :L]))
            hs = slice(g * G, (g + 1) * G)
            qq = q[b, :, hs].reshape(S * G, dh)
            s = qq @ keys.T / np.sqrt(dh)
            reach[b, :, hs] = (np.abs(qq) @ np.abs(keys).T).max(1).reshape(S, G, 1) / np.sqrt(dh)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[b, :, hs] = (p @ vals).reshape(S, G, dh)
            mass[b, :, hs] = (p @ np.abs(vals)).reshape(S, G, dh)
    return out, mass, reach


def vocab_logits(y, w_q, w_scale):
    """(argmax key w_scale * sum, logits without logit_scale), float64."""
    q, s = quantise_rows(y)
    key = (q.astype(np.float64) @ w_q.astype(np.float64).T) * w_scale.astype(np.float64)[None]
    return key, key * s.astype(np.float64)[:, None]
