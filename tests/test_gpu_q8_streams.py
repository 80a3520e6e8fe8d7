"""8-bit calls at once, each on a stream and a workspace of its own: both forms of the
linear update (pairs of CTAs, a cluster that splits K), both attention kernels, the
append and the vocabulary step give the bits that each gives alone."""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
from tests import _q8 as H

pytestmark = pytest.mark.gpu


def linear(rng, rows, N, K):
    x = H.up_bf16(H.bf16(rng.standard_normal((rows, K)))[1])
    w = H.up(rng.integers(-127, 128, (N, K)).astype(np.int8))
    s = H.up(rng.random(N).astype(np.float32))
    out = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    ws = tt.linear_i8_workspace(rows, N, K)
    return [out], lambda st: tt.tt_linear_i8(rows, N, K, x, w, s, out, ws, st), lambda: out.zero_()


def attention(rng, S, lens):
    B, HQ, HKV, dh, cap = len(lens), 32, 2, 128, 2048
    D, fmt = tt.Dims(B, S, HQ, HKV, dh, HQ * dh, 512, cap), tt.q8("e4m3", 64)
    q, k, v = (H.up_bf16(H.bf16(rng.standard_normal((B, S, h, dh)))[1]) for h in (HQ, HKV, HKV))
    (kc, ks), (vc, vs) = (H.cache(rng, B, HKV, cap, dh, "e4m3", 64) for _ in range(2))
    kc, vc, ks, vs = H.up_codes(kc), H.up_codes(vc), H.up(ks), H.up(vs)
    cl = H.up(np.array(lens, np.int32))
    out = torch.zeros((B, S, HQ, dh), dtype=torch.bfloat16, device="cuda")
    ws = tt.workspace(D, tt.TT_WS_ATTN_Q8)
    return [out], lambda st: tt.tt_block_denoise_attn_q8(D, fmt, q, k, v, kc, vc, ks, vs, cl, out, ws,
                                                         st), lambda: out.zero_()


def append(rng):
    B, HKV, dh, cap, n = 8, 2, 128, 1000, 400
    d, fmt = tt.Dims(B, 1, HKV, HKV, dh, HKV * dh, 16, cap), tt.q8("int8", 128)
    new = [H.up_bf16(H.bf16(rng.standard_normal((B, n, HKV, dh)))[1]) for _ in range(2)]
    bufs = [torch.zeros((B, HKV, cap, dh), dtype=torch.int8, device="cuda") for _ in range(2)] + \
        [torch.zeros((B, HKV, 8), device="cuda") for _ in range(2)] + \
        [torch.zeros(B, dtype=torch.int32, device="cuda")]
    ws = tt.workspace(d, tt.TT_WS_APPEND_Q8)

    def reset():
        for x in bufs:
            x.zero_()
        bufs[4].fill_(37)
    return bufs, lambda st: tt.tt_append_ctx_q8(d, fmt, n, None, *new, *bufs, ws, st), reset


def vocab(rng):
    B, S, Hh, V = 4, 16, 1024, 20000
    D = tt.Dims(B, S, 16, 16, 64, Hh, V, 0)
    y = H.up_bf16(H.bf16(rng.standard_normal((B * S, Hh)))[1])
    w = H.up(np.clip(np.rint(rng.standard_normal((V, Hh)) * 31), -127, 127).astype(np.int8))
    sc = H.up((rng.uniform(0.5, 1.5, V) / 31 / 32).astype(np.float32))
    tok = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    m = torch.zeros((B, S), dtype=torch.uint8, device="cuda")
    conf, arg = torch.zeros((B, S), device="cuda"), tok.clone()
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = tt.workspace(D, tt.TT_WS_VOCAB_I8)

    def reset():
        tok.fill_(-1)
        m.fill_(1)
    return [tok, m, conf, arg, n], lambda st: tt.tt_vocab_confidence_commit_i8(
        D, y, w, sc, 0.3, 6.0, tok, m, conf, arg, n, ws, st), reset


def test_calls_at_once():
    rng = np.random.default_rng(21)
    jobs = [linear(rng, 700, 4608, 1024), linear(rng, 128, 4608, 1024), linear(rng, 16, 384, 256),
            attention(rng, 16, [2048, 0, 700, 1300]), attention(rng, 1, [2048, 5, 1999]),
            append(rng), vocab(rng)]
    alone = []
    for bufs, call, reset in jobs:
        reset()
        torch.cuda.synchronize()
        call(None)
        torch.cuda.synchronize()
        alone.append([x.clone() for x in bufs])
    streams = [torch.cuda.Stream() for _ in jobs]
    for turn in range(10):
        for _, _, reset in jobs:
            reset()
        torch.cuda.synchronize()
        order = rng.permutation(len(jobs))
        for i in order:
            jobs[i][1](streams[i])
        torch.cuda.synchronize()
        for (bufs, _, _), want in zip(jobs, alone):
            for x, y in zip(bufs, want):
                assert torch.equal(x, y), turn
