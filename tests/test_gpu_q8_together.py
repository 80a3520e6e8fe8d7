"""The 8-bit operators in a row, as a server runs them: weights quantised once,
prompts through the linear update into the cache, blocks denoised step by step
against that cache (linear update, attention, modulation, vocabulary step) and
appended to it when they are committed.  Every stage is held to the oracle on
the inputs it had; the whole run is repeated from captured graphs."""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
from oracle import q8_oracle as Q
from oracle import twotower_oracle as O
from tests import _gpu as G
from tests import _q8 as H

pytestmark = pytest.mark.gpu

B, S, HQ, HKV, DH, V, CAP, N = 3, 16, 4, 2, 64, 1000, 150, 70
HID, NQKV = HQ * DH, (HQ + 2 * HKV) * DH
PROMPT = [70, 0, 33]
GAMMA, SCALE = 0.25, 4.0


def empty(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


class Server:
    """Buffers of the run; `prompt`, `step` and `append` only enqueue work."""

    def __init__(self, kind, block, seed):
        rng = np.random.default_rng(seed)
        self.kind, self.block = kind, block
        self.D, self.f = tt.Dims(B, S, HQ, HKV, DH, HID, V, CAP), tt.q8(kind, block)
        bits = lambda *s, f=1.0: H.up_bf16(H.bf16(rng.standard_normal(s) * f)[1])  # noqa: E731
        self.u, self.w = bits(NQKV, HID, f=1 / 16), bits(V, HID, f=1 / 16)
        self.emb, self.mod = bits(V + 1, HID), bits(2, HID, f=0.1)
        self.px, self.pos = bits(B * N, HID), bits(B * S, HID)
        self.uq, self.us = empty(NQKV, HID, dtype=torch.int8), empty(NQKV, dtype=torch.float32)
        self.wq, self.wscale = empty(V, HID, dtype=torch.int8), empty(V, dtype=torch.float32)
        tt.tt_quantize_rows_i8(NQKV, HID, self.u, self.uq, self.us)
        tt.tt_quantize_rows_i8(V, HID, self.w, self.wq, self.wscale)
        self.plen = H.up(np.array(PROMPT, np.int32))
        self.pqkv, self.qkv = empty(B, N, NQKV), empty(B, S, NQKV)
        t = torch.int8 if kind == "int8" else torch.float8_e4m3fn
        self.codes = [empty(B, HKV, CAP, DH, dtype=t) for _ in range(2)]
        self.scales = [empty(B, HKV, -(-CAP // block), dtype=torch.float32) for _ in range(2)]
        self.ctx = empty(B, dtype=torch.int32)
        self.x, self.att, self.y = empty(B * S, HID), empty(B, S, HQ, DH), empty(B * S, HID)
        self.q, self.k, self.v = empty(B, S, HQ, DH), empty(B, S, HKV, DH), empty(B, S, HKV, DH)
        self.t = empty(B, dtype=torch.float32)
        self.tokens, self.masked = empty(B, S, dtype=torch.int32), empty(B, S, dtype=torch.uint8)
        self.conf, self.arg = empty(B, S, dtype=torch.float32), empty(B, S, dtype=torch.int32)
        self.n = empty(B, dtype=torch.int32)
        self.ws = {w: tt.workspace(self.D, w) for w in (tt.TT_WS_ATTN_Q8, tt.TT_WS_APPEND_Q8,
                                                        tt.TT_WS_VOCAB_I8, tt.TT_WS_ADALN)}
        self.lws = tt.linear_i8_workspace(B * N, NQKV, HID)

    def start(self):
        self.ctx.zero_()
        for x in self.codes + self.scales:
            x.view(torch.uint8).zero_()

    def block_start(self):
        self.tokens.fill_(-1)
        self.masked.fill_(1)

    def _append(self, n, new_len, qkv):
        k, v = (qkv[..., a:a + HKV * DH].unflatten(2, (HKV, DH))
                for a in (HID, HID + HKV * DH))
        tt.tt_append_ctx_q8(self.D, self.f, n, new_len, k, v, *self.codes, *self.scales, self.ctx,
                            self.ws[tt.TT_WS_APPEND_Q8])

    def prompt(self):
        tt.tt_linear_i8(B * N, NQKV, HID, self.px, self.uq, self.us, self.pqkv, self.lws)
        self._append(N, self.plen, self.pqkv)

    def rows(self):
        idx = torch.where(self.masked != 0, V, self.tokens).long().view(-1)
        torch.index_select(self.emb, 0, idx, out=self.x)
        self.x.add_(self.pos)
        tt.tt_linear_i8(B * S, NQKV, HID, self.x, self.uq, self.us, self.qkv, self.lws)

    def step(self):
        self.rows()
        self.q.copy_(self.qkv[..., :HID].unflatten(2, (HQ, DH)))
        self.k.copy_(self.qkv[..., HID:HID + HKV * DH].unflatten(2, (HKV, DH)))
        self.v.copy_(self.qkv[..., HID + HKV * DH:].unflatten(2, (HKV, DH)))
        tt.tt_block_denoise_attn_q8(self.D, self.f, self.q, self.k, self.v, *self.codes,
                                    *self.scales, self.ctx, self.att, self.ws[tt.TT_WS_ATTN_Q8])
        self.t.copy_(self.masked.float().mean(1))
        tt.tt_adaln_modulate(self.D, self.att, self.mod, self.t, self.y, self.ws[tt.TT_WS_ADALN])
        tt.tt_vocab_confidence_commit_i8(self.D, self.y, self.wq, self.wscale, GAMMA, SCALE,
                                         self.tokens, self.masked, self.conf, self.arg, self.n,
                                         self.ws[tt.TT_WS_VOCAB_I8])

    def append(self):
        self.rows()
        self._append(S, None, self.qkv)

    def status(self):
        return [tt.tt_device_status(w) for w in (*self.ws.values(), self.lws)]


def check_linear(x, out, uq, us):
    want = Q.linear(x, uq, us)
    bound = np.abs(want) * (2.0 ** -8 + 4 * 2.0 ** -24) + 1e-38   # one bf16 rounding, three fp32
    assert (np.abs(G.host_f64(out).reshape(want.shape) - want) <= bound).all()


def kv_of(qkv, n):
    x = G.host_f64(qkv).reshape(B, n, NQKV)
    return [x[..., a:a + HKV * DH].reshape(B, n, HKV, DH) for a in (HID, HID + HKV * DH)]


@pytest.mark.parametrize("kind,block", [("int8", 64), ("e4m3", 16)])
def test_prompt_then_blocks(kind, block):
    s = Server(kind, block, 5)
    host = {n: G.host_f64(getattr(s, n)) for n in ("u", "w", "px")}
    for w, q, sc in (("u", s.uq, s.us), ("w", s.wq, s.wscale)):
        want = Q.quantise_rows(host[w])
        np.testing.assert_array_equal(q.cpu().numpy(), want[0])
        np.testing.assert_array_equal(sc.cpu().numpy(), want[1])
    uq, us, wq, wsc = (x.cpu().numpy() for x in (s.uq, s.us, s.wq, s.wscale))

    # ---- one stage at a time against the oracle
    s.start()
    cdt = np.int8 if kind == "int8" else np.uint8
    cache = [(np.zeros((B, HKV, CAP, DH), cdt), np.zeros((B, HKV, -(-CAP // block)), np.float32))
             for _ in range(2)]
    ctx = np.zeros(B, np.int64)

    def appended(new, m):
        nonlocal cache, ctx
        cache = [Q.append(c, sc, x, ctx, m, kind, block) for (c, sc), x in zip(cache, new)]
        ctx = ctx + np.asarray(m)
        for (c, sc), gc, gs in zip(cache, s.codes, s.scales):
            np.testing.assert_array_equal(gc.view(torch.int8).cpu().numpy().view(cdt), c)
            np.testing.assert_array_equal(gs.cpu().numpy(), sc)
        np.testing.assert_array_equal(s.ctx.cpu().numpy(), ctx)

    s.prompt()
    check_linear(host["px"], s.pqkv, uq, us)
    appended(kv_of(s.pqkv, N), PROMPT)
    steps, unsure, committed = [], 0, []
    for _ in range(2):
        s.block_start()
        for n_steps in range(1, S + 1):
            before = s.tokens.cpu().numpy().copy(), s.masked.cpu().numpy().copy()
            s.step()
            check_linear(G.host_f64(s.x), s.qkv, uq, us)
            q, k, v = (G.host_f64(x) for x in (s.q, s.k, s.v))
            kd, vd = (Q.dequantise_cache(c, sc, kind, block) for c, sc in cache)
            out, mass, reach = Q.attention(q, k, v, kd, vd, ctx)
            err = np.abs(G.host_f64(s.att) - out)
            assert (err <= H.attention_bound(out, mass, reach, DH)).all()
            key, lg = Q.vocab_logits(G.host_f64(s.y), wq, wsc)
            top = np.sort(key, 1)
            m = before[1].astype(bool)
            ok = m & (top[:, -1] - top[:, -2] > 2.0 ** -22 * np.abs(top[:, -1])).reshape(B, S)
            unsure += int((m & ~ok).sum())
            np.testing.assert_array_equal(s.arg.cpu().numpy()[ok], lg.argmax(1).reshape(B, S)[ok])
            conf = 1 / np.exp((lg - lg.max(1, keepdims=True)) * SCALE).sum(1).reshape(B, S)
            # as in the vocabulary step's own test
            np.testing.assert_allclose(s.conf.cpu().numpy()[m], conf[m],
                                       rtol=2.0 ** -18 + 4 * 2.0 ** -24 * np.abs(lg).max() * SCALE)
            # the commit rule, on the confidences and tokens that the call reports
            t2, m2, com, _ = O.commit(np.where(m, s.conf.cpu().numpy().astype(np.float64), np.nan),
                                      s.arg.cpu().numpy(), *before[:1], m, GAMMA)
            np.testing.assert_array_equal(s.tokens.cpu().numpy(), t2)
            np.testing.assert_array_equal(s.masked.cpu().numpy(), m2.astype(np.uint8))
            np.testing.assert_array_equal(s.n.cpu().numpy(), com.sum(1))
            if not m2.any():
                break
        assert not s.masked.any()
        committed.append(s.tokens.clone())
        s.append()
        appended(kv_of(s.qkv, S), [S] * B)
        steps.append(n_steps)
    assert unsure <= 2 and max(steps) > 1 and s.status() == [0] * 5
    final = [x.clone() for x in s.codes + s.scales]

    # ---- the same run from graphs, all of it on one stream and one set of workspaces
    graphs = {}
    for name in ("prompt", "block_start", "step", "append"):
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            getattr(s, name)()
    s.start()
    graphs["prompt"].replay()
    for n_steps, want in zip(steps, committed):
        graphs["block_start"].replay()
        for _ in range(n_steps):
            graphs["step"].replay()
        graphs["append"].replay()
        assert torch.equal(s.tokens, want)
    assert s.status() == [0] * 5
    for x, want in zip(s.codes + s.scales, final):
        assert torch.equal(x.view(torch.uint8), want.view(torch.uint8))
