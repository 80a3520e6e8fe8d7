"""tt_quantize_rows_i8, tt_linear_i8 and tt_vocab_confidence_commit_i8 against
the 64-bit oracle.  Codes are compared bit for bit; the integer sums are
exact, so a linear output is off by its bf16 rounding (half a step, 2^-8
relative) and three fp32 roundings (of the sum, the two scales' product and
theirs), and a confidence by fp32 exponentials and sums."""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
from oracle import q8_oracle as Q
from oracle import twotower_oracle as O
from tests import _gpu as G
from tests import _q8 as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 64), (130, 256), (7, 4096), (5, 8208), (2, 131072)])
def test_quantised_rows(rows, K):
    rng = np.random.default_rng(K)
    x, bits = H.bf16(rng.standard_normal((rows, K)) * np.exp2(rng.integers(-9, 9, (rows, 1))))
    x[0, :] = 0.0
    if rows > 2:
        x[1, K // 2] = np.nan
        x[2, 3] = np.inf
    x, bits = H.bf16(x)
    q = torch.full((rows, K), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, dtype=torch.float32, device="cuda")
    tt.tt_quantize_rows_i8(rows, K, H.up_bf16(bits), q, s)
    want_q, want_s = Q.quantise_rows(x)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


def linear(rows, N, K, seed, extreme=False):
    rng = np.random.default_rng(seed)
    x, bits = H.bf16(rng.standard_normal((rows, K)))
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    ws = (rng.standard_normal(N) / 64).astype(np.float32)
    if extreme:                         # the largest sums the operands can make
        x, bits = H.bf16(np.sign(x))
        w = np.where(np.arange(N)[:, None] % 2, -128, 127).astype(np.int8) * np.ones((1, K), np.int8)
        x[0], bits[0] = H.bf16(np.ones(K))
    got = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    wsp = tt.linear_i8_workspace(rows, N, K)
    tt.tt_linear_i8(rows, N, K, H.up_bf16(bits), H.up(w), H.up(ws), got, wsp)
    assert tt.tt_device_status(wsp) == 0
    want = Q.linear(x, w, ws)
    got = got.float().cpu().numpy().astype(np.float64)
    err = np.abs(got - want)
    bound = np.abs(want) * (2.0 ** -8 + 4 * 2.0 ** -24) + 1e-38
    assert (err <= bound).all(), (np.max(err / bound), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("rows,N,K", [
    (1, 1, 16), (1, 8, 64), (16, 384, 256), (17, 389, 112), (128, 4608, 1024), (129, 257, 4096),
    (300, 1000, 2000), (5, 4608, 4096), (1, 9000, 4096), (64, 513, 8192), (2000, 72, 320), (3, 24, 131072),
    (257, 1024, 144), (128, 128, 16384),
    (300, 13001, 144), (257, 26000, 2064), (2100, 2600, 256), (1025, 6400, 128),
    (40000, 24, 64), (20000, 1, 16), (5, 20001, 64), (130, 20002, 48), (65, 65, 1040)])
def test_linear_matches_oracle(rows, N, K):
    linear(rows, N, K, rows + N + K)


@pytest.mark.parametrize("K", [4096, 131072])
def test_linear_largest_sums(K):
    linear(4, 40, K, 3, extreme=True)


def test_linear_zero_and_non_finite_rows():
    x = np.ones((4, 64), np.float32)
    x[1] = 0
    x[2, 7] = np.nan
    x[3, 9] = -np.inf
    w = np.ones((24, 64), np.int8)
    out = torch.empty((4, 24), dtype=torch.bfloat16, device="cuda")
    tt.tt_linear_i8(4, 24, 64, H.up_bf16(H.bf16(x)[1]), H.up(w), H.up(np.ones(24, np.float32)), out,
                    tt.linear_i8_workspace(4, 24, 64))
    assert (out[0] == 64).all() and (out[1] == 0).all() and torch.isnan(out[2:]).all()


def test_linear_writes_only_its_output():
    from tests.test_gpu_guards import Guarded, _check
    rng = np.random.default_rng(1)
    for rows, N, K in ((17, 389, 112), (128, 520, 512), (40, 24, 4096), (300, 13001, 64), (5, 20002, 64)):
        ins = dict(x=Guarded((rows, K), torch.bfloat16, H.up_bf16(H.bf16(rng.standard_normal((rows, K)))[1])),
                   w=Guarded((N, K), torch.int8, H.up(rng.integers(-127, 128, (N, K)).astype(np.int8))),
                   s=Guarded((N,), torch.float32, H.up(rng.random(N).astype(np.float32))))
        outs = dict(out=Guarded((rows, N), torch.bfloat16),
                    ws=Guarded((tt.tt_linear_i8_workspace_bytes(rows, N, K),), torch.uint8))
        tt.tt_linear_i8(rows, N, K, ins["x"].t, ins["w"].t, ins["s"].t, outs["out"].t, outs["ws"].t)
        _check(ins, outs)


def test_linear_graph_streams_repeats():
    rng = np.random.default_rng(2)
    rows, N, K = 96, 1032, 2048
    x = H.up_bf16(H.bf16(rng.standard_normal((rows, K)))[1])
    w, s = H.up(rng.integers(-127, 128, (N, K)).astype(np.int8)), H.up(rng.random(N).astype(np.float32))
    ws = tt.linear_i8_workspace(rows, N, K)
    ws.fill_(0xA5)
    a, b, c = (torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    tt.tt_linear_i8(rows, N, K, x, w, s, a, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tt.tt_linear_i8(rows, N, K, x, w, s, b, ws, side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tt.tt_linear_i8(rows, N, K, x, w, s, c, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    x.mul_(3)
    g.replay()
    tt.tt_linear_i8(rows, N, K, x, w, s, a, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, c)


# ------------------------------------------------------------ vocabulary
def vocab(B, S, Hh, V, gamma, scale, seed, masked=None, w=None, ws=None, y=None):
    rng = np.random.default_rng(seed)
    y, bits = H.bf16(rng.standard_normal((B * S, Hh)) if y is None else y)
    if w is None:
        w = np.clip(np.rint(rng.standard_normal((V, Hh)) * 31), -127, 127).astype(np.int8)
    if ws is None:
        ws = (rng.uniform(0.5, 1.5, V) / 31 / np.sqrt(Hh)).astype(np.float32)
    masked = np.ones((B, S), np.uint8) if masked is None else masked
    tokens = np.where(masked == 1, -1, rng.integers(0, V, (B, S))).astype(np.int32)
    D = tt.Dims(B, S, Hh // 64, Hh // 64, 64, Hh, V, 0)
    t_tok, t_m = H.up(tokens), H.up(masked)
    conf = torch.empty((B, S), dtype=torch.float32, device="cuda")
    amax = torch.empty((B, S), dtype=torch.int32, device="cuda")
    ncom = torch.empty((B,), dtype=torch.int32, device="cuda")
    wsp = tt.workspace(D, tt.TT_WS_VOCAB_I8)
    tt.tt_vocab_confidence_commit_i8(D, H.up_bf16(bits), H.up(w), H.up(ws), gamma, scale, t_tok, t_m,
                                     conf, amax, ncom, wsp)
    status = tt.tt_device_status(wsp)
    got = dict(tokens=t_tok.cpu().numpy(), masked=t_m.cpu().numpy(), conf=conf.cpu().numpy(),
               tok=amax.cpu().numpy(), n=ncom.cpu().numpy(), status=status)
    key, logits = Q.vocab_logits(y, w, ws)
    key = np.sort(key, 1)
    tok = np.argmax(logits, 1).reshape(B, S)
    # two keys nearer than the fp32 rounding of each may come out either way
    sure = ((key[:, -1] - key[:, -2] > 2.0 ** -22 * np.abs(key[:, -1]))
            | (key[:, -1] == key[:, -2])).reshape(B, S)
    p = np.exp((logits - logits.max(1, keepdims=True)) * scale)
    ref = dict(tok=tok, conf=(1 / p.sum(1)).reshape(B, S), sure=sure,
               reach=np.abs(logits).max() * scale)
    return got, ref, tokens, masked.astype(bool)


def check_vocab(got, ref, tokens, m, gamma, scale):
    assert got["status"] == 0
    # 2^-18 for the exponentials (2^-21 relative each) and the sums of 131072 of
    # them.  A logit x is held as fp32 (its integer sum, the product with the
    # column's scale: 2^-24 |x| each), so a term exp(x - max) is off by 2 * 2 *
    # 2^-24 max|x| relative, and the sum of terms by no more.
    tol = 2.0 ** -18 + 4 * 2.0 ** -24 * ref["reach"]
    np.testing.assert_allclose(got["conf"][m], ref["conf"][m], rtol=tol)
    assert (got["conf"][~m] == -1).all() and (got["tok"][~m] == -1).all()
    ok = m & ref["sure"]
    np.testing.assert_array_equal(got["tok"][ok], ref["tok"][ok])
    np.testing.assert_array_equal(got["tokens"][~m], tokens[~m])
    skipped = 0
    t2, m2, com, fb = O.commit(np.where(m, ref["conf"], np.nan), ref["tok"], tokens, m, gamma)
    for b in range(m.shape[0]):
        c = ref["conf"][b][m[b]]
        top = np.sort(c)[::-1]
        near = (np.abs(c - gamma) < tol * gamma).any() or (
            fb[b] and len(top) > 1 and 0 < top[0] - top[1] < 2 * tol * top[0])
        if near or not ref["sure"][b][m[b]].all():
            skipped += 1
            continue
        np.testing.assert_array_equal(got["masked"][b], m2[b].astype(np.uint8))
        np.testing.assert_array_equal(got["tokens"][b], t2[b])
        assert got["n"][b] == com[b].sum()
    return skipped


@pytest.mark.parametrize("B,S,Hh,V,gamma,scale", [
    (1, 1, 64, 2, 0.8, 1.0), (4, 16, 256, 1024, 0.8, 1.0), (4, 16, 256, 1000, 0.5, 12.0),
    (3, 32, 320, 5003, 0.3, 8.0), (9, 16, 1024, 9000, 0.8, 40.0), (2, 128, 128, 449, 0.9, 4.0),
    (20, 16, 512, 2250, 0.2, 8.0)])
def test_vocab_matches_oracle(B, S, Hh, V, gamma, scale):
    rng = np.random.default_rng(V)
    masked = (rng.random((B, S)) < 0.7).astype(np.uint8)
    masked[0, 0] = 1
    if B > 3:
        masked[2] = 0
    got = vocab(B, S, Hh, V, gamma, scale, V + S, masked=masked)
    skipped = check_vocab(*got, gamma, scale)
    assert skipped <= max(1, B // 8), skipped


def test_vocab_many_rows():
    """More rows than the fused planning takes (8192): the same commit rule."""
    rng = np.random.default_rng(9)
    masked = (rng.random((520, 16)) < 0.5).astype(np.uint8)
    got = vocab(520, 16, 64, 300, 0.4, 6.0, 10, masked=masked)
    assert check_vocab(*got, 0.4, 6.0) <= 4


def test_vocab_nothing_masked():
    got, ref, tokens, m = vocab(2, 16, 128, 300, 0.9, 1.0, 3, masked=np.zeros((2, 16), np.uint8))
    assert got["status"] == 0 and (got["n"] == 0).all() and (got["conf"] == -1).all()
    np.testing.assert_array_equal(got["tokens"], tokens)


def test_vocab_full_size():
    """The mid-size vocabulary step, 16 rows against the oracle."""
    masked = np.zeros((4, 16), np.uint8)
    masked[:, ::4] = 1
    got = vocab(4, 16, 4096, 131072, 0.5, 8.0, 1, masked=masked)
    assert check_vocab(*got, 0.5, 8.0) <= 1


def test_vocab_ties_take_the_lowest_id():
    rng = np.random.default_rng(5)
    w = np.clip(np.rint(rng.standard_normal((1500, 128)) * 20), -127, 127).astype(np.int8)
    ws = np.full(1500, 0.01, np.float32)
    for far in (700, 900, 1499):
        w[far] = w[3]
    w[4], w[1100] = w[230], w[230]
    got, ref, tokens, m = vocab(4, 16, 128, 1500, 0.9, 3.0, 6, w=w, ws=ws)
    np.testing.assert_array_equal(got["tok"], ref["tok"])
    # a vocabulary of equal rows: token 0, confidence 1 / V
    got, ref, tokens, m = vocab(2, 16, 64, 500, 0.9, 3.0, 7, w=np.ones((500, 64), np.int8),
                                ws=np.full(500, 0.5, np.float32))
    assert (got["tok"] == 0).all()
    np.testing.assert_allclose(got["conf"], 1 / 500, rtol=2.0 ** -18)


def test_vocab_zero_and_non_finite_rows():
    rng = np.random.default_rng(8)
    y = rng.standard_normal((32, 128))
    y[3] = 0.0
    got, ref, tokens, m = vocab(2, 16, 128, 300, 0.9, 1.0, 8, y=y)
    assert got["status"] == 0 and got["tok"][0, 3] == 0
    np.testing.assert_allclose(got["conf"][0, 3], 1 / 300, rtol=2.0 ** -18)
    y[20, 5] = np.nan
    bad, ref, tokens, m = vocab(2, 16, 128, 300, 0.9, 1.0, 8, y=y)
    assert bad["status"] == 6 and bad["n"][1] >= 1      # reported, and the step still goes on
    for k in ("tokens", "masked", "conf", "tok", "n"):  # the other sequence is as before
        np.testing.assert_array_equal(bad[k][0], got[k][0])


def test_vocab_extreme_logit_scales():
    """A row's factor that underflows makes every logit equal, one that overflows
    leaves the largest alone; neither is a NaN."""
    y = np.random.default_rng(12).standard_normal((16, 128))
    y[3] = 0.0                                       # scale 2^-60
    got, ref, tokens, m = vocab(1, 16, 128, 300, 0.9, 1e-35, 12, y=y)
    assert got["status"] == 0
    np.testing.assert_allclose(got["conf"], 1 / 300, rtol=2.0 ** -18)
    got, ref, tokens, m = vocab(1, 16, 128, 300, 0.9, 3e38, 12, y=y * 2.0 ** 9)
    assert got["status"] == 0
    sure = ref["sure"].copy()
    sure[0, 3] = False
    assert sure.sum() > 12 and (got["conf"][sure] == 1).all()
    np.testing.assert_array_equal(got["tok"][sure], ref["tok"][sure])


def test_vocab_captured_twice_on_their_own_workspaces():
    rng = np.random.default_rng(11)
    B, S, Hh, V = 3, 16, 256, 3000
    D = tt.Dims(B, S, 4, 4, 64, Hh, V, 0)
    w = H.up(np.clip(np.rint(rng.standard_normal((V, Hh)) * 31), -127, 127).astype(np.int8))
    ws = H.up((rng.uniform(0.5, 1.5, V) / 500).astype(np.float32))
    sets, alive = [], []
    for i in range(2):
        y = H.up_bf16(H.bf16(rng.standard_normal((B * S, Hh)))[1])
        st = dict(tok=torch.full((B, S), -1, dtype=torch.int32, device="cuda"),
                  m=torch.ones((B, S), dtype=torch.uint8, device="cuda"),
                  conf=torch.empty((B, S), device="cuda"),
                  arg=torch.empty((B, S), dtype=torch.int32, device="cuda"),
                  n=torch.empty((B,), dtype=torch.int32, device="cuda"))
        wsp = tt.workspace(D, tt.TT_WS_VOCAB_I8)
        call = lambda st=st, y=y, wsp=wsp: tt.tt_vocab_confidence_commit_i8(  # noqa: E731
            D, y, w, ws, 0.6, 10.0, st["tok"], st["m"], st["conf"], st["arg"], st["n"], wsp)
        call()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in st.items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        sets.append((g, st, want))
        alive.append((y, wsp))                      # the captured calls read them
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for (g, st, want), s in zip(sets, (a, b)):
            st["tok"].fill_(-1)
            st["m"].fill_(1)
        torch.cuda.synchronize()
        for (g, st, want), s in zip(sets, (a, b)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, st, want in sets:
            for k in st:
                assert torch.equal(st[k], want[k]), k
    G.workspace(D, tt.TT_WS_VOCAB)                  # the bf16 step's workspace is its own kind
