"""tt_append_ctx_q8 against the 64-bit oracle, bit for bit."""
import numpy as np
import pytest
import torch

import block_wise_diffusion_b200 as tt
from oracle import q8_oracle as Q
from tests import _q8 as H

pytestmark = pytest.mark.gpu


def dims(B, Hkv, dh, L_cap):
    return tt.Dims(B, 1, Hkv, Hkv, dh, Hkv * dh, 16, L_cap)


class Cache:
    def __init__(self, rng, B, Hkv, dh, L_cap, kind, block):
        self.kind, self.block = kind, block
        self.host = [H.cache(rng, B, Hkv, L_cap, dh, kind, block, 0.5) for _ in range(2)]
        self.codes = [H.up_codes(c) for c, _ in self.host]
        self.scale = [H.up(s) for _, s in self.host]
        self.ws = tt.workspace(dims(B, Hkv, dh, L_cap), tt.TT_WS_APPEND_Q8)

    def append(self, d, new, ctx_len, new_len, strided):
        """Both sides: the library in place, the oracle on the host copy.  new: two
        (float64, bits) pairs [B, n, Hkv, dh]."""
        B, n, Hkv, dh = new[0][0].shape
        if strided:                    # column ranges of one projection's rows
            both = torch.full((B, n, 2 * Hkv * dh + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
            t = [both[:, :, i * Hkv * dh:(i + 1) * Hkv * dh].view(B, n, Hkv, dh) for i in (0, 1)]
        else:                          # the layout of a bf16 context cache
            both = torch.full((2, B, Hkv, n + 3, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
            t = [both[i, :, :, :n].transpose(1, 2) for i in (0, 1)]
        for x, (_, bits) in zip(t, new):
            x.copy_(H.up_bf16(bits))
        cl = H.up(np.asarray(ctx_len, np.int32))
        nl = None if new_len is None else H.up(np.asarray(new_len, np.int32))
        tt.tt_append_ctx_q8(d, tt.q8(self.kind, self.block), n, nl, t[0], t[1], *self.codes,
                            *self.scale, cl, self.ws)
        m = [n] * B if new_len is None else new_len
        self.host = [Q.append(c, s, x, ctx_len, m, self.kind, self.block)
                     for (c, s), (x, _) in zip(self.host, new)]
        return cl.cpu().numpy()

    def check(self):
        for (c, s), gc, gs in zip(self.host, self.codes, self.scale):
            np.testing.assert_array_equal(gs.cpu().numpy(), s)
            g = gc.view(torch.int8).cpu().numpy().view(c.dtype)
            if not np.array_equal(g, c):
                at = np.argwhere(g != c)
                raise AssertionError(f"{len(at)} codes differ, first at {at[0]}: "
                                     f"{g[tuple(at[0])]} for {c[tuple(at[0])]}")


def rows(rng, B, n, Hkv, dh, spread=1.0):
    return [H.bf16(rng.standard_normal((B, n, Hkv, dh)) * spread) for _ in range(2)]


CASES = [
    # B, Hkv, dh, L_cap, block, n, ctx_len, new_len
    (1, 1, 64, 16, 16, 1, [0], None),
    (1, 1, 64, 17, 16, 1, [16], None),
    (3, 2, 128, 500, 128, 16, [0, 127, 484], None),
    (3, 2, 128, 500, 32, 37, [5, 463, 31], None),
    (4, 1, 64, 300, 64, 300, [0, 10, 299, 300], [300, 290, 1, 0]),
    (2, 4, 64, 1000, 16, 700, [0, 123], [700, 1]),
    (2, 2, 128, 400, 128, 257, [1, 100], [257, 129]),
]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("strided", [True, False])
def test_append_matches_oracle(kind, i, strided):
    B, Hkv, dh, cap, block, n, cl, nl = CASES[i]
    rng = np.random.default_rng(i + 10)
    c = Cache(rng, B, Hkv, dh, cap, kind, block)
    got = c.append(dims(B, Hkv, dh, cap), rows(rng, B, n, Hkv, dh), cl, nl, strided)
    assert tt.tt_device_status(c.ws) == 0
    c.check()
    np.testing.assert_array_equal(got, np.asarray(cl) + (nl if nl is not None else n))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_scales_grow_block_by_block(kind):
    """Sixteen appends of a few rows whose magnitude rises and falls: the older
    codes are rounded again each time the scale of their block grows."""
    rng = np.random.default_rng(3)
    d = dims(2, 2, 64, 200)
    c = Cache(rng, 2, 2, 64, 200, kind, 128)
    cl = np.array([0, 9])
    for step in range(16):
        n = int(rng.integers(1, 12))
        cl = c.append(d, rows(rng, 2, n, 2, 64, 2.0 ** rng.integers(-6, 7)), cl, None, True)
    c.check()


# (127 and multiples of 7: the scales of int8 and e4m3 that are exact, so that
# middles are met)
@pytest.mark.parametrize("amaxes", [(1.0, 1.9921875, 3.0, 2.0 ** -40 * 1.3125),
                                    (1.984375, 1.75, 2.0 ** 20 * 2.625, 2.0 ** -30 * 1.984375)])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_every_quotient_rounds_exactly(kind, amaxes):
    """Values that lie at, next to and between the middles of two codes: bf16
    neighbours of (c + 1/2) s for every code, and the half of the largest."""
    rng = np.random.default_rng(7)
    block, dh = 128, 128
    x = np.empty((4, 4, block, dh))
    for i, amax in enumerate(amaxes):
        amax = H.bf16(np.array([amax]))[0][0]
        s = float(Q.scale_of(amax, kind)[()])
        v = np.unique(np.abs(Q.values(np.arange(-127, 128).astype(np.int8), kind) if kind == "int8"
                             else Q.E4M3[np.isfinite(Q.E4M3)]))
        mid = (v[1:] + v[:-1]) / 2 * s
        near = np.concatenate([mid, mid * (1 + 2.0 ** -8), mid * (1 - 2.0 ** -8), v * s,
                               [amax, amax / 2, amax / 4, 0]])
        near = H.bf16(near)[0]
        near = near[near <= amax]
        x[i] = rng.choice(near, (4, block, dh)) * rng.choice([-1, 1], (4, block, dh))
        x[i, :, 0, 0] = amax
    new = [H.bf16(x.transpose(0, 2, 1, 3)), H.bf16(-x.transpose(0, 2, 1, 3))]
    c = Cache(rng, 4, 4, dh, block, kind, block)
    c.append(dims(4, 4, dh, block), new, [0] * 4, None, True)
    c.check()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_zeros_extremes_and_non_finite_rows(kind):
    rng = np.random.default_rng(8)
    d = dims(4, 1, 64, 64)
    c = Cache(rng, 4, 1, 64, 64, kind, 32)
    new = rows(rng, 4, 40, 1, 64)
    x = new[0][0].copy()
    x[0] = 0.0
    x[1] *= 2.0 ** 100
    x[2, 3] = np.nan
    x[2, 35, 0, 5] = -np.inf
    x[3] *= 2.0 ** -100
    cl = c.append(d, [H.bf16(x), new[1]], [0, 5, 10, 20], None, True)
    c.check()
    # a block whose scale is NaN stays so
    c.append(d, rows(rng, 4, 2, 1, 64), cl, None, True)
    c.check()


def test_refused_sequences_stay_as_they_were():
    rng = np.random.default_rng(9)
    d = dims(5, 1, 64, 50)
    c = Cache(rng, 5, 1, 64, 50, "int8", 16)
    cl = [45, -1, 51, 10, 20]
    got = c.append(d, rows(rng, 5, 10, 1, 64), cl, [10, 3, 0, 11, 10], True)
    assert tt.tt_device_status(c.ws) == 1
    np.testing.assert_array_equal(got, [45, -1, 51, 10, 30])
    c.check()


def test_captured_append_replays():
    """A captured append run three times equals three appends."""
    rng = np.random.default_rng(12)
    d, fmt = dims(3, 2, 128, 400), tt.q8("int8", 64)
    c = Cache(rng, 3, 2, 128, 400, "int8", 64)
    new = rows(rng, 3, 16, 2, 128)
    k, v = (H.up_bf16(b) for _, b in new)
    cl = H.up(np.array([0, 50, 301], np.int32))
    keep = [x.clone() for x in (*c.codes, *c.scale, cl)]
    call = lambda: tt.tt_append_ctx_q8(d, fmt, 16, None, k, v, *c.codes, *c.scale, cl, c.ws)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x, y in zip((*c.codes, *c.scale, cl), keep):
        x.copy_(y)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    lens = np.array([0, 50, 301])
    for _ in range(3):
        c.host = [Q.append(a, s, x, lens, [16] * 3, "int8", 64) for (a, s), (x, _) in zip(c.host, new)]
        lens = lens + 16
    np.testing.assert_array_equal(cl.cpu().numpy(), lens)
    c.check()


def test_binding_refuses_other_shapes():
    d, fmt = dims(2, 2, 64, 64), tt.q8("int8", 16)
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    k = z(2, 4, 2, 64, dtype=torch.bfloat16)
    rest = (z(2, 2, 64, 64, dtype=torch.int8), z(2, 2, 64, 64, dtype=torch.int8), z(2, 2, 4), z(2, 2, 4),
            z(2, dtype=torch.int32), tt.workspace(d, tt.TT_WS_APPEND_Q8))
    with pytest.raises(ValueError, match="shape"):
        tt.tt_append_ctx_q8(d, fmt, 5, None, k, k, *rest)
    with pytest.raises(ValueError, match="shape"):
        tt.tt_append_ctx_q8(d, fmt, 4, None, k, k.float(), *rest)
    with pytest.raises(ValueError, match="same strides"):
        tt.tt_append_ctx_q8(d, fmt, 4, None, k, k.transpose(1, 2).contiguous().transpose(1, 2), *rest)
    with pytest.raises(ValueError, match="holds"):
        tt.tt_append_ctx_q8(d, fmt, 4, None, k, k, rest[0], rest[1], z(2, 2, 3), *rest[3:])
