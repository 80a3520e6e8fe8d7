"""Pins of the 8-bit oracle: codes against exact rational arithmetic and
torch's e4m3 type, scales, the append rule on worked examples."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from oracle import twotower_oracle as O
import tt_inputs


def _bf16(x):
    return O.from_bf16(tt_inputs.bf16_bits(np.asarray(x, np.float32)))


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(Q.E4M3, t.astype(np.float64))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_codes_are_the_nearest_in_exact_arithmetic(kind):
    rng = np.random.default_rng(1)
    x = _bf16(rng.standard_normal(300) * np.exp2(rng.integers(-12, 3, 300)))
    amax = np.abs(x).max()
    # values half way to a code when the scale is a short number, and the
    # half of the largest, whose quotient lies next to a middle
    x = np.concatenate([x, [amax, -amax, amax / 2, amax / 4, 0.0, -0.0]])
    for s in (Q.scale_of(amax, kind)[()], np.float32(0.25), np.float32(amax / 64)):
        x_in = x[np.abs(x) <= Q.QMAX[kind] * float(s)]
        got = Q.values(Q.encode(x_in, s, kind), kind)
        want = [Q.encode_one(float(v), float(s), kind) for v in x_in]
        np.testing.assert_array_equal(got, want)


def test_scale_floor_and_non_finite():
    np.testing.assert_array_equal(Q.scale_of([0.0, 127.0], "int8"),
                                  np.array([2.0 ** -60, 1.0], np.float32))
    assert np.isnan(Q.scale_of([np.inf, np.nan], "e4m3")).all()
    codes, s = Q.quantise_rows(np.array([[1.0, np.nan], [1.0, -2.0]]))
    assert np.isnan(s[0]) and (codes[0] == 0).all()
    assert s[1] == np.float32(2.0) * (np.float32(1) / np.float32(127))
    # 1 / s = 63.5 (1 - d), d the rounding of the scale: the exact quotient decides
    assert codes[1, 0] == Q.encode_one(1.0, float(s[1]), "int8") and codes[1, 1] == -127


def test_append_by_hand():
    """Blocks of 16, one head of two dims: three rows join five."""
    codes = np.zeros((1, 1, 32, 2), np.int8)
    scale = np.full((1, 1, 2), 7.0, np.float32)         # never written: must not matter
    first = np.full((1, 5, 1, 2), 127.0)
    codes, scale = Q.append(codes, scale, first, [0], [5], "int8", 16)
    assert scale[0, 0, 0] == 1.0 and scale[0, 0, 1] == 7.0
    assert (codes[0, 0, :5] == 127).all() and (codes[0, 0, 5:] == 0).all()
    # larger rows: the old codes shrink by half
    c2, s2 = Q.append(codes, scale, np.full((1, 3, 1, 2), 254.0), [5], [3], "int8", 16)
    assert s2[0, 0, 0] == 2.0 and (c2[0, 0, :5] == 64).all()   # 63.5 to even
    assert (c2[0, 0, 5:8] == 127).all()
    # smaller rows: the old scale stays
    c3, s3 = Q.append(codes, scale, np.full((1, 3, 1, 2), 3.0), [5], [3], "int8", 16)
    assert s3[0, 0, 0] == 1.0 and (c3[0, 0, 5:8] == 3).all() and (c3[0, 0, :5] == 127).all()
    # a run over a block's end, room checked, a short new_len
    c4, s4 = Q.append(codes, scale, np.full((1, 20, 1, 2), 1.0), [14], [20], "int8", 16)
    assert (c4 == codes).all()                                # 34 > 32: unchanged
    c5, s5 = Q.append(codes, scale, np.full((1, 20, 1, 2), 254.0), [14], [4], "int8", 16)
    assert s5[0, 0, 1] == 2.0 and (c5[0, 0, 14:18] == 127).all() and (c5[0, 0, 18:] == 0).all()


def test_attention_is_the_bf16_oracle_on_dequantised_keys():
    rng = np.random.default_rng(3)
    B, S, Hkv, G, dh, L = 2, 16, 2, 2, 64, 40
    q, kb, vb = (rng.standard_normal((B, S, h, dh)) for h in (Hkv * G, Hkv, Hkv))
    codes = rng.integers(-127, 128, (2, B, Hkv, L, dh)).astype(np.int8)
    scale = rng.random((2, B, Hkv, 3)).astype(np.float32) / 64
    k, v = (Q.dequantise_cache(codes[i], scale[i], "int8", 16) for i in (0, 1))
    cl = np.array([40, 17])
    out, mass, reach = Q.attention(q, kb, vb, k, v, cl)
    np.testing.assert_allclose(out, O.block_attention(q, kb, vb, k, v, cl), atol=1e-12)
    assert (np.abs(out) <= mass + 1e-12).all() and (reach > 0).all()


def test_linear_is_the_product_of_dequantised_factors():
    rng = np.random.default_rng(4)
    x = _bf16(rng.standard_normal((5, 64)))
    w = rng.integers(-127, 128, (7, 64)).astype(np.int8)
    ws = rng.random(7).astype(np.float32)
    codes, s = Q.quantise_rows(x)
    want = (codes * s[:, None].astype(np.float64)) @ (w * ws[:, None].astype(np.float64)).T
    np.testing.assert_allclose(Q.linear(x, w, ws), want, rtol=1e-12)
    assert np.abs(codes * s[:, None].astype(np.float64) - x).max() <= s.max() * 0.5001


@pytest.mark.parametrize("kind,qmax", [("int8", 127), ("e4m3", 448)])
def test_one_factor_rounds_a_group(kind, qmax):
    """A group under the scale s of its own largest value A: x times 1 / s moved by
    2^-22 against the sign of s - A / qmax rounds to the exact code, for every
    pair of significands, unless s is exact."""
    f32, exact = np.float32, 0
    x_all = (np.arange(128, 256)[:, None] / 128.0 * np.exp2(np.arange(-20.0, 1.0))).ravel()
    for m in range(128, 256):
        A = m / 128.0
        s = Q.scale_of(A, kind)[()]
        e = np.float64(s) * qmax - A
        if e == 0:
            exact += 1
            continue
        f = f32(f32(1) / s * f32(1 - np.copysign(2.0 ** -22, e)))
        x = x_all[x_all <= A].astype(f32)
        want = Q.values(Q.encode(x, s, kind), kind)
        if kind == "int8":                 # one rounding, of x * f + 1.5 * 2^23
            got = np.rint(x.astype(np.float64) * np.float64(f))
        else:                              # x * f to fp32, that to a code
            got = Q.values(Q.encode(x * f, f32(1), kind), kind)
        np.testing.assert_array_equal(got, want)
    assert exact in ((1, 2, 3) if kind == "int8" else range(1, 20))
