"""tt_block_denoise_attn_q8 over the range of magnitudes that its inputs may have:
scores, keys, values and scales near the ends of fp32.

Bounds are relative to what a row adds up (no fixed term): half a bf16 step of the
output, the fp16 rounding of every probability, twice the error of a score, and a few
fp32 roundings (tests/_q8.py has the same terms); beside them what fp16 drops of a
probability and of an own value, relative to the largest value that a row may read:
a probability below fp16's normal numbers is off by at most 2^-25 times the key's
code, which is at most 2^7 (2^15 for an own key), where the row's largest probability
is at least 2^10, and its code 2^7 where its block holds the largest value: 2^-35 of that
value (2^-27).  An own value has steps of at least 2^-124 (fp16's smallest times
2^-100, the smallest power of two that its tile may carry)."""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
import tt_inputs
from oracle import q8_oracle as Q
from tests import _q8 as H

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def bound(out, mass, reach, d, ctx_len, v_blk, vd):
    top = np.empty((d.B, 1, d.Hq, 1))
    for b in range(d.B):
        for h in range(d.Hq):
            g = h * d.Hkv // d.Hq
            top[b, 0, h, 0] = max(np.abs(v_blk[b, :, g]).max(),
                                  np.abs(vd[b, g, :ctx_len[b]]).max(initial=0.0))
    n = np.asarray(ctx_len, np.float64).reshape(-1, 1, 1, 1)
    return (np.abs(out) * H.U16
            + mass * (H.U_P + 2 * (d.dh + 8) * 2.0 ** -22 * reach + 2.0 ** -16)
            + top * (d.S * 2.0 ** -27 + n * 2.0 ** -35) + 2.0 ** -125)


def check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, ctx_len, splits=(0,)):
    """q, k, v: float64 arrays of bf16 numbers; the caches with their scales."""
    B, Hkv, cap = kc.shape[:3]
    d = tt_inputs.Dims(B=B, S=S, Hq=Hkv * G, Hkv=Hkv, dh=dh, V=512, L_cap=cap, ctx=("fixed", cap))
    q, k, v = (H.bf16(x) for x in (q, k, v))
    kd, vd = Q.dequantise_cache(kc, ks, kind, block), Q.dequantise_cache(vc, vs, kind, block)
    out, mass, reach = Q.attention(q[0], k[0], v[0], kd, vd, ctx_len)
    limit = bound(out, mass, reach, d, ctx_len, v[0], vd)
    for n in splits:
        tt.tt_set_attn_splits(n)
        try:
            got, ws = H.run_attention(d, tt.q8(kind, block), kind, (q[1], k[1], v[1]), kc, ks, vc, vs,
                                      ctx_len)
            assert tt.tt_device_status(ws) == 0
        finally:
            tt.tt_set_attn_splits(0)
        got = got.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all(), n
        err = np.abs(got - out)
        assert (err <= limit).all(), (n, np.nanmax(err / limit))
    return got


def inputs(seed, B, S, G, Hkv, dh, fq=1.0, fk=1.0, fv=1.0):
    rng = np.random.default_rng(seed)
    return rng, [rng.standard_normal((B, S, h, dh)) * f
                 for h, f in ((Hkv * G, fq), (Hkv, fk), (Hkv, fv))]


# more than 16 query rows per KV head, and at most 16: two kernels
SHAPES = [(16, 4, 64), (32, 16, 128), (1, 16, 128), (1, 1, 64)]
KINDS = [("int8", 64), ("e4m3", 16)]


# ------------------------------------------------- scores that all but vanish
@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", SHAPES)
@pytest.mark.parametrize("fq", [2.0 ** -64, 2.0 ** -75, 2.0 ** -100, 2.0 ** -124])
def test_tiny_queries_and_a_zero_key_block(kind, block, S, G, dh, fq):
    """The keys' last block is zeros under the smallest scale, in a tile that the
    context's end cuts."""
    rng, (q, k, v) = inputs(1, 2, S, G, 2, dh, fq)
    kc, ks = H.cache(rng, 2, 2, 300, dh, kind, block)
    vc, vs = H.cache(rng, 2, 2, 300, dh, kind, block)
    for b, n in enumerate((200, 131)):
        at = (n - 1) // block
        kc[b, :, at * block:] = 0
        ks[b, :, at:] = Q.FLOOR
    check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, [200, 131], (0, 3))


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -135, 2.0 ** -149])
def test_tiny_key_scales(kind, block, S, G, dh, scale):
    rng, (q, k, v) = inputs(2, 2, S, G, 1, dh)
    kc, ks = H.cache(rng, 2, 1, 200, dh, kind, block)
    vc, vs = H.cache(rng, 2, 1, 200, dh, kind, block)
    ks[:, :, 1:] = np.float32(scale)
    check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, [200, 77])


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", SHAPES)
@pytest.mark.parametrize("fq,fk", [(2.0 ** -62, 2.0 ** -62), (2.0 ** -80, 2.0 ** -80),
                                   (2.0 ** -120, 2.0 ** -120), (1.0, 2.0 ** -126),
                                   (2.0 ** -129, 2.0 ** 124), (2.0 ** 124, 2.0 ** -129)])
def test_tiny_own_keys(kind, block, S, G, dh, fq, fk):
    """Without a context, and with one whose keys are zeros.  (The last two
    pairs multiply to ordinary scores.)"""
    rng, (q, k, v) = inputs(3, 2, S, G, 1, dh, fq, fk)
    for cap, cl in ((0, [0, 0]), (140, [140, 0])):
        kc, ks = H.cache(rng, 2, 1, cap, dh, kind, block, 0.0)
        vc, vs = H.cache(rng, 2, 1, cap, dh, kind, block)
        check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, cl, (0, 2))


# ------------------------------------------ values far apart, far down, far up
@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", SHAPES)
@pytest.mark.parametrize("fv", [2.0 ** -80, 2.0 ** -110, 2.0 ** -113, 2.0 ** -120, 0.0])
def test_tiny_own_values(kind, block, S, G, dh, fv):
    """Without a context, with one, and with CTAs that hold one tile each, so that
    the own keys are a record of their own."""
    rng, (q, k, v) = inputs(4, 2, S, G, 1, dh, fv=fv)
    for cap, cl in ((0, [0, 0]), (256, [256, 256]), (256, [1, 130])):
        kc, ks = H.cache(rng, 2, 1, cap, dh, kind, block)
        vc, vs = H.cache(rng, 2, 1, cap, dh, kind, block)
        check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, cl, (0, 1, 6, 40))


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", SHAPES)
@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("own", [2.0 ** -104, 1.0, 2.0 ** 100])
@pytest.mark.parametrize("big_first", [True, False])
def test_value_scales_far_apart(kind, block, S, G, dh, big, own, big_first):
    """Blocks of zero values under the smallest scale beside very large values, own
    values of either kind: what a key weighs does not depend on its value."""
    rng, (q, k, v) = inputs(5, 2, S, G, 1, dh, fv=own)
    kc, ks = H.cache(rng, 2, 1, 320, dh, kind, block)
    vc, vs = H.cache(rng, 2, 1, 320, dh, kind, block, big)
    zero = np.arange(320) >= 192 if big_first else np.arange(320) < 192
    vc[:, :, zero] = 0
    vs[:, :, zero[::block]] = Q.FLOOR
    check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, [320, 250], (0, 1, 8, 40))


# --------------------------------------------------------- a peaked row
@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("S,G,dh", [(16, 4, 64), (1, 16, 128)])
@pytest.mark.parametrize("down", [17.0, 26.0, 31.0])
@pytest.mark.parametrize("at", [0, 40000])
def test_one_peak_over_a_long_context(kind, block, S, G, dh, down, at):
    """One key of value 0 takes nearly all the weight; 65536 others, each 2^-down of
    it, make the output."""
    L, cap = 65536, 65600
    kc = np.zeros((1, 1, cap, dh), np.int8 if kind == "int8" else np.uint8)
    vc = np.empty_like(kc)
    ks = np.full((1, 1, -(-cap // block)), 1 / 64, np.float32)
    vs = np.ones_like(ks)
    one = np.float32(1.0)
    vc[:] = Q.encode(np.ones(1), one, kind)[0]
    kc[0, 0, at] = Q.encode(np.ones(1), one, kind)[0]
    vc[0, 0, at] = 0
    # q . k / sqrt(dh) = sqrt(dh) * scale: `down` in log2 units
    ks[0, 0, at // block] = down / LOG2E / np.sqrt(dh)
    q, k, v = (np.full((1, S, h, dh), x) for h, x in ((G, 1.0), (1, 0.0), (1, 1.0)))
    check(S, G, dh, kind, block, q, k, v, kc, ks, vc, vs, [L], (0, 7))
