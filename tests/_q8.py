"""Helpers of the 8-bit GPU tests: seeded caches, uploads, elementwise bounds."""
from __future__ import annotations

import numpy as np
import torch

import block_wise_diffusion_b200 as tt
import tt_inputs
from oracle import q8_oracle as Q
from oracle import twotower_oracle as O

U16 = 2.0 ** -8      # half a bf16 step, relative
U_P = 2.0 ** -11     # half an fp16 step: the rounding of a probability


def bf16(x):
    """float64 values of x rounded to bf16, and their bits."""
    bits = tt_inputs.bf16_bits(np.asarray(x, np.float32))
    return O.from_bf16(bits), bits


def up_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def up_codes(codes):
    t = torch.from_numpy(np.ascontiguousarray(codes)).cuda()
    return t if codes.dtype == np.int8 else t.view(torch.float8_e4m3fn)


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def cache(rng, B, Hkv, L_cap, dh, kind, block, spread=1.0, skew=0.0):
    """A cache as appending fills it: every block's codes reach the largest
    code and its scale is that of its rows.  `skew`: spread of the blocks'
    magnitudes in powers of two."""
    nb = -(-L_cap // block)
    x, _ = bf16(rng.standard_normal((B, Hkv, nb, block, dh)) * spread
                * np.exp2(rng.uniform(-skew, skew, (B, Hkv, nb, 1, 1)).round()))
    s = Q.scale_of(np.abs(x).max((3, 4)), kind) if nb else np.zeros((B, Hkv, 0), np.float32)
    c = Q.encode(x, s[..., None, None], kind).reshape(B, Hkv, nb * block, dh)[:, :, :L_cap]
    return np.ascontiguousarray(c), s


def attention_bound(out, mass, reach, dh):
    """|error| of an output element: its bf16 rounding; the fp16 rounding of
    every probability; twice the error of a score (dh products and the sums
    of their fp32 accumulation, at most 2^-22 relative each where the tensor
    core truncates) and a few fp32 roundings of the exponential and the
    normaliser (2^-16 in all)."""
    return np.abs(out) * U16 + mass * (U_P + 2 * (dh + 8) * 2.0 ** -22 * reach + 2.0 ** -16) \
        + 2.0 ** -40


def run_attention(d, fmt, kind, bits, kc, ks, vc, vs, ctx_len, out=None, ws=None, stream=None):
    D = tt.dims(d)
    out = out if out is not None else torch.full((d.B, d.S, d.Hq, d.dh), float("nan"),
                                                 dtype=torch.bfloat16, device="cuda")
    ws = ws if ws is not None else tt.workspace(D, tt.TT_WS_ATTN_Q8)
    tt.tt_block_denoise_attn_q8(D, fmt, *(up_bf16(b) for b in bits), up_codes(kc), up_codes(vc),
                                up(ks), up(vs), up(np.asarray(ctx_len, np.int32)), out, ws, stream)
    return out, ws
