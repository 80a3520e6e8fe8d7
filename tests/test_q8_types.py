"""An 8-bit cache whose tensor type is not its format's is refused by the binding (on
the host: refusals come before any launch)."""
import pytest
import torch

import block_wise_diffusion_b200 as tt
from block_wise_diffusion_b200 import build

FAKE = 1 << 20
B, S, HQ, HKV, DH, CAP = 2, 16, 4, 2, 64, 50


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def attention(f, k, v):
    d = tt.Dims(B, S, HQ, HKV, DH, HQ * DH, 1000, CAP)
    tt.tt_block_denoise_attn_q8(d, f, FAKE, FAKE, FAKE, k, v, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0)


@pytest.mark.parametrize("kind,other", [("int8", torch.float8_e4m3fn), ("e4m3", torch.int8),
                                        ("e4m3", torch.float8_e5m2), ("int8", torch.bfloat16)])
def test_attention_refuses_the_other_type(kind, other):
    x = torch.zeros((B, HKV, CAP, DH), dtype=other)
    for k, v, name in ((x, FAKE, "k_ctx"), (FAKE, x, "v_ctx")):
        with pytest.raises(ValueError, match=f"{name} is torch"):
            attention(tt.q8(kind, 16), k, v)


@pytest.mark.parametrize("kind,dtype", [("int8", torch.int8), ("e4m3", torch.float8_e4m3fn),
                                        ("int8", torch.uint8), ("e4m3", torch.uint8)])
def test_its_own_type_and_bytes_pass_on(kind, dtype):
    x = torch.zeros((B, HKV, CAP, DH), dtype=dtype)
    with pytest.raises(ValueError, match="CUDA tensors only"):   # the next check
        attention(tt.q8(kind, 16), x, FAKE)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,other", [("int8", torch.float8_e4m3fn), ("e4m3", torch.int8)])
def test_append_refuses_the_other_type(kind, other):
    d = tt.Dims(B, 1, HKV, HKV, DH, HKV * DH, 16, CAP)
    z = lambda *s, dtype: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    new = z(B, 3, HKV, DH, dtype=torch.bfloat16)
    own = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    good, bad = (z(B, HKV, CAP, DH, dtype=t) for t in (own, other))
    scale, cl = z(B, HKV, 4, dtype=torch.float32), z(B, dtype=torch.int32)
    ws = tt.workspace(d, tt.TT_WS_APPEND_Q8)
    call = lambda k, v: tt.tt_append_ctx_q8(d, tt.q8(kind, 16), 3, None, new, new, k, v, scale,  # noqa: E731
                                            scale.clone(), cl, ws)
    for k, v, name in ((bad, good, "k_ctx"), (good, bad, "v_ctx")):
        with pytest.raises(ValueError, match=f"{name} is torch"):
            call(k, v)
    assert (cl == 0).all()
    call(good, good.clone())
    assert (cl == 3).all()
