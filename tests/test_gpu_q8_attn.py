"""tt_block_denoise_attn_q8 against the 64-bit oracle on the dequantised cache.

Every element is held to the bound of its own roundings (tests/_q8.py): half a
bf16 step of the output, the fp16 rounding of the probabilities and the fp32
accumulation of the scores.
"""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
import tt_inputs
from oracle import q8_oracle as Q
from tests import _q8 as H

pytestmark = pytest.mark.gpu


def dims(B, S, Hq, Hkv, dh, L_cap):
    return tt_inputs.Dims(B=B, S=S, Hq=Hq, Hkv=Hkv, dh=dh, V=512, L_cap=L_cap,
                          ctx=("fixed", L_cap))


def check(d, kind, block, ctx_len, seed, spread=(1.0, 1.0), skew=0.0, splits=0, poison=True):
    rng = np.random.default_rng(seed)
    q, qb = H.bf16(rng.standard_normal((d.B, d.S, d.Hq, d.dh)))
    k, kb = H.bf16(rng.standard_normal((d.B, d.S, d.Hkv, d.dh)) * spread[0])
    v, vb = H.bf16(rng.standard_normal((d.B, d.S, d.Hkv, d.dh)) * spread[1])
    kc, ks = H.cache(rng, d.B, d.Hkv, d.L_cap, d.dh, kind, block, spread[0], skew)
    vc, vs = H.cache(rng, d.B, d.Hkv, d.L_cap, d.dh, kind, block, spread[1], skew)
    ctx_len = np.asarray(ctx_len)
    if poison:
        # what lies behind a sequence is never used: NaN codes (e4m3), NaN scales
        for b in range(d.B):
            if kind == "e4m3":
                kc[b, :, ctx_len[b]:] = 0x7F
                vc[b, :, ctx_len[b]:] = 0xFF
            first = -(-int(ctx_len[b]) // block)
            ks[b, :, first:] = np.nan
            vs[b, :, first:] = np.nan
    tt.tt_set_attn_splits(splits)
    try:
        got, ws = H.run_attention(d, tt.q8(kind, block), kind, (qb, kb, vb), kc, ks, vc, vs, ctx_len)
        assert tt.tt_device_status(ws) == 0
    finally:
        tt.tt_set_attn_splits(0)
    got = got.float().cpu().numpy().astype(np.float64)
    kd, vd = Q.dequantise_cache(kc, ks, kind, block), Q.dequantise_cache(vc, vs, kind, block)
    out, mass, reach = Q.attention(q, k, v, kd, vd, ctx_len)
    err = np.abs(got - out)
    bound = H.attention_bound(out, mass, reach, d.dh)
    rel = np.linalg.norm(got - out) / np.linalg.norm(out)
    print(f"worst {np.max(err / bound):.3f} of the bound, rel-L2 {rel:.2e}")
    assert np.isfinite(got).all()
    assert (err <= bound).all(), np.max(err / bound)
    return got


CASES = [
    # name, dims, type, block, context lengths, spreads of k and v, skew
    ("tiny", dims(1, 16, 4, 1, 64, 256), "int8", 16, [256], (1, 1), 0),
    ("ragged-i8", dims(4, 16, 32, 2, 128, 1000), "int8", 128, [1000, 777, 0, 1], (1, 1), 0),
    ("ragged-e4", dims(4, 16, 32, 2, 128, 1000), "e4m3", 64, [129, 128, 127, 640], (1, 1), 0),
    ("ar", dims(3, 1, 32, 2, 128, 700), "e4m3", 32, [700, 129, 0], (1, 1), 0),
    ("ar-one-key", dims(2, 1, 4, 4, 64, 40), "int8", 32, [1, 0], (1, 1), 0),
    ("no-cache", dims(2, 16, 4, 2, 64, 0), "int8", 128, [0, 0], (1, 1), 0),
    ("s32", dims(2, 32, 32, 2, 128, 300), "int8", 16, [300, 65], (1, 1), 0),
    ("s64-g4", dims(2, 64, 8, 2, 64, 300), "e4m3", 128, [300, 0], (1, 1), 0),
    ("s128", dims(1, 128, 32, 2, 128, 333), "int8", 64, [333], (1, 1), 0),
    ("g1", dims(2, 16, 4, 4, 64, 300), "e4m3", 16, [300, 17], (1, 1), 0),
    ("g2-odd-cap", dims(3, 16, 4, 2, 128, 203), "int8", 32, [203, 202, 16], (1, 1), 0),
    ("g64", dims(1, 16, 64, 1, 128, 150), "int8", 128, [150], (1, 1), 0),
    ("g128", dims(2, 32, 128, 1, 64, 200), "e4m3", 64, [200, 3], (1, 1), 0),
    ("batch200", dims(200, 16, 4, 1, 64, 130), "int8", 64, list(range(131)) + [130] * 69, (1, 1), 0),
    ("long", dims(1, 16, 16, 1, 128, 20000), "int8", 128, [19999], (1, 1), 0),
    ("sharp", dims(2, 16, 16, 1, 128, 600), "int8", 128, [600, 333], (4, 1), 0),
    # blocks whose magnitudes differ by up to 2^16, in keys and values
    ("skewed", dims(2, 16, 16, 1, 64, 600), "int8", 32, [600, 333], (0.02, 1), 8),
    ("skewed-e4", dims(2, 1, 16, 1, 64, 600), "e4m3", 16, [600, 333], (0.02, 1), 8),
    # very small and very large values
    ("small", dims(1, 16, 8, 1, 64, 200), "int8", 64, [200], (2.0 ** -20, 2.0 ** -30), 0),
    ("large", dims(1, 16, 8, 1, 64, 200), "e4m3", 64, [200], (1, 2.0 ** 60), 0),
]


@pytest.mark.parametrize("name,d,kind,block,cl,spread,skew", CASES, ids=[c[0] for c in CASES])
def test_matches_oracle(name, d, kind, block, cl, spread, skew):
    check(d, kind, block, cl, seed=len(name) * 7 + d.S, spread=spread, skew=skew)


@pytest.mark.parametrize("splits", [1, 3, 40, 300])
@pytest.mark.parametrize("S", [1, 16])
def test_any_number_of_ctas(splits, S):
    check(dims(2, S, 32, 2, 128, 1500), "int8", 64, [1500, 1111], seed=5, splits=splits)


def test_zero_blocks_and_extreme_codes():
    """Blocks of zeros (the smallest scale) beside ordinary ones, and the code
    -128 that only a caller can store."""
    d = dims(1, 16, 4, 1, 64, 256)
    rng = np.random.default_rng(2)
    (q, qb), (k, kb), (v, vb) = (H.bf16(rng.standard_normal((1, 16, h, 64))) for h in (4, 1, 1))
    kc, ks = H.cache(rng, 1, 1, 256, 64, "int8", 64)
    vc, vs = H.cache(rng, 1, 1, 256, 64, "int8", 64)
    vc[:, :, 64:128] = 0
    vs[:, :, 1] = Q.FLOOR
    kc[:, :, 192:] = 0
    ks[:, :, 3] = Q.FLOOR
    vc[0, 0, 5] = -128
    kc[0, 0, 6] = -128
    got, _ = H.run_attention(d, tt.q8("int8", 64), "int8", (qb, kb, vb), kc, ks, vc, vs, [256])
    out, mass, reach = Q.attention(q, k, v, Q.dequantise_cache(kc, ks, "int8", 64),
                                   Q.dequantise_cache(vc, vs, "int8", 64), [256])
    err = np.abs(got.float().cpu().numpy() - out)
    assert (err <= H.attention_bound(out, mass, reach, 64)).all()


def test_non_finite_scale_reaches_only_its_own_sequence_and_head():
    d = dims(2, 16, 8, 2, 64, 200)
    rng = np.random.default_rng(4)
    bits = [H.bf16(rng.standard_normal((2, 16, h, 64)))[1] for h in (8, 2, 2)]
    kc, ks = H.cache(rng, 2, 2, 200, 64, "int8", 32)
    vc, vs = H.cache(rng, 2, 2, 200, 64, "int8", 32)
    ks[0, 1, 2] = np.nan
    vs[1, 0, 3] = np.nan
    got, _ = H.run_attention(d, tt.q8("int8", 32), "int8", bits, kc, ks, vc, vs, [200, 200])
    bad = torch.isnan(got.view(2, 16, 2, 4, 64)).all(4).all(3).all(1).cpu().numpy()
    np.testing.assert_array_equal(bad, [[False, True], [True, False]])
    assert torch.isfinite(got.view(2, 16, 2, 4, 64)[0, :, 0]).all()
    assert torch.isfinite(got.view(2, 16, 2, 4, 64)[1, :, 1]).all()


def test_bad_length_is_clamped_and_recorded():
    d = dims(2, 16, 4, 1, 64, 100)
    rng = np.random.default_rng(6)
    bits = [H.bf16(rng.standard_normal((2, 16, h, 64)))[1] for h in (4, 1, 1)]
    kc, ks = H.cache(rng, 2, 1, 100, 64, "int8", 16)
    vc, vs = H.cache(rng, 2, 1, 100, 64, "int8", 16)
    args = (d, tt.q8("int8", 16), "int8", bits, kc, ks, vc, vs)
    got, ws = H.run_attention(*args, [105, -4])
    assert tt.tt_device_status(ws) == 1 and tt.tt_device_status(ws) == 0
    want, ws2 = H.run_attention(*args, [100, 0], ws=ws)
    assert tt.tt_device_status(ws2) == 0
    assert torch.equal(got, want)


def test_streams_graph_and_repeats():
    """The same bits on another stream, captured and replayed (also after the
    inputs changed in place), and a second call on the same workspace."""
    d = dims(3, 16, 32, 2, 128, 900)
    rng = np.random.default_rng(8)
    D, fmt = tt.dims(d), tt.q8("int8", 64)
    q, k, v = (H.up_bf16(H.bf16(rng.standard_normal((3, 16, h, 128)))[1]) for h in (32, 2, 2))
    kc, ks = (H.up_codes(x) if x.dtype != np.float32 else H.up(x)
              for x in H.cache(rng, 3, 2, 900, 128, "int8", 64))
    vc, vs = (H.up_codes(x) if x.dtype != np.float32 else H.up(x)
              for x in H.cache(rng, 3, 2, 900, 128, "int8", 64))
    cl = H.up(np.array([900, 0, 431], np.int32))
    ws = tt.workspace(D, tt.TT_WS_ATTN_Q8)
    ws.fill_(0xA5)
    outs = [torch.empty((3, 16, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    call = lambda o, s=None: tt.tt_block_denoise_attn_q8(D, fmt, q, k, v, kc, vc, ks, vs, cl, o, ws, s)  # noqa: E731
    call(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[1], side)
    torch.cuda.current_stream().wait_stream(side)
    call(outs[2])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[3])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[3])
    cl.copy_(H.up(np.array([17, 900, 128], np.int32)))
    q.neg_()
    g.replay()
    call(outs[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[3]) and torch.isfinite(outs[0]).all()


def test_writes_only_its_output():
    from tests.test_gpu_guards import Guarded, _check, _ws
    d = dims(3, 16, 32, 2, 128, 500)
    rng = np.random.default_rng(9)
    D = tt.dims(d)
    ins = {n: Guarded((3, 16, h, 128), torch.bfloat16,
                      H.up_bf16(H.bf16(rng.standard_normal((3, 16, h, 128)))[1]))
           for n, h in (("q", 32), ("k", 2), ("v", 2))}
    for n in ("kc", "vc"):
        c, s = H.cache(rng, 3, 2, 500, 128, "int8", 64)
        ins[n] = Guarded(c.shape, torch.int8, H.up(c))
        ins[n + "s"] = Guarded(s.shape, torch.float32, H.up(s))
    ins["cl"] = Guarded((3,), torch.int32, H.up(np.array([500, 377, 0], np.int32)))
    outs = {"out": Guarded((3, 16, 32, 128), torch.bfloat16), "ws": _ws(D, tt.TT_WS_ATTN_Q8)}
    tt.tt_block_denoise_attn_q8(D, tt.q8("int8", 64), *(ins[n].t for n in ("q", "k", "v", "kc", "vc",
                                                                           "kcs", "vcs", "cl")),
                                outs["out"].t, outs["ws"].t)
    _check(ins, outs)
    assert torch.isfinite(outs["out"].t).all()
