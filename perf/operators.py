"""Cases of the 8-bit operators: attention over a context cache held in 8 bits,
appending rows to that cache, the 8-bit linear update and the 8-bit vocabulary
projection with the confidence commit.

``run`` computes them in plain torch operations, or, with ``own``, through the
framework's entry points.  Sizes are those of the framework's own workloads
(tiny, mid, loop64, long, ragged) and generic ones around them.
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
FLOOR = 2.0 ** -60  # smallest scale


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one short sequence of a small model: launch latency
        dict(name="attn-tiny", op="attn", kv="int8", block=16, B=1, S=16, Hkv=1, G=4, dh=64, L=256,
             ragged=False),
        # a small serving batch
        dict(name="attn-mid", op="attn", kv="int8", block=128, B=8, S=16, Hkv=2, G=16, dh=128,
             L=4096, ragged=False),
        # one position per sequence (the autoregressive step), ragged lengths
        dict(name="attn-ar", op="attn", kv="e4m3", block=64, B=64, S=1, Hkv=2, G=16, dh=128,
             L=8192, ragged=True),
        # few long sequences
        dict(name="attn-long", op="attn", kv="int8", block=128, B=4, S=16, Hkv=2, G=16, dh=128,
             L=65536, ragged=False),
        # a large batch of mixed lengths
        dict(name="attn-ragged", op="attn", kv="e4m3", block=32, B=48, S=16, Hkv=2, G=16, dh=128,
             L=32768, ragged=True),
        # a committed block of 16 positions joins every sequence's cache
        dict(name="append-block", op="append", kv="int8", block=128, B=64, n=16, Hkv=2, dh=128,
             L=8192, ragged=False),
        # prompts of mixed lengths enter empty caches
        dict(name="append-prompt", op="append", kv="e4m3", block=64, B=16, n=8192, Hkv=2, dh=128,
             L=0, ragged=True),
        # the linear update of a small model's block
        dict(name="linear-tiny", op="linear", M=16, N=384, K=256),
        # the linear update [q|k|v] of 8 and of 128 sequences' blocks
        dict(name="linear-mid", op="linear", M=128, N=4608, K=4096),
        dict(name="linear-wide", op="linear", M=2048, N=4608, K=4096),
        # the vocabulary step: a small batch, partly committed; 64 fresh blocks
        dict(name="vocab-mid", op="vocab", B=8, S=16, H=4096, V=131072, masked=0.6, scale=1.0),
        dict(name="vocab-64", op="vocab", B=64, S=16, H=4096, V=131072, masked=1.0, scale=8.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "linear", "vocab"])
    if op == "attn":
        while True:
            c = dict(op=op, kv=rng.choice(["int8", "e4m3"]), block=rng.choice([16, 32, 64, 128]),
                     B=_log(rng, 1, 64), S=rng.choice([1, 16, 16, 32, 64, 128]),
                     Hkv=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 8, 16, 32]),
                     dh=rng.choice([64, 128]), L=_log(rng, 1, 65536), ragged=rng.random() < 0.5)
            if c["Hkv"] * c["G"] * c["dh"] <= 8192 and c["S"] * c["G"] <= 2048 and \
                    c["B"] * c["S"] * c["Hkv"] * c["G"] * c["L"] * c["dh"] <= 5e10 and \
                    c["B"] * c["Hkv"] * c["L"] * c["dh"] <= 1.5e8:
                return c
    if op == "append":
        while True:
            c = dict(op=op, kv=rng.choice(["int8", "e4m3"]), block=rng.choice([16, 32, 64, 128]),
                     B=_log(rng, 1, 64), n=_log(rng, 1, 8192), Hkv=rng.choice([1, 2, 4, 8]),
                     dh=rng.choice([64, 128]), L=rng.choice([0, _log(rng, 1, 8192)]),
                     ragged=rng.random() < 0.5)
            if c["B"] * c["Hkv"] * c["n"] * c["dh"] <= 3.4e7 and \
                    c["B"] * c["Hkv"] * (c["n"] + c["L"]) * c["dh"] <= 1.5e8:
                return c
    if op == "linear":
        while True:
            c = dict(op=op, M=_log(rng, 1, 2048), N=_log(rng, 8, 9000), K=64 * _log(rng, 2, 128))
            if c["M"] * c["N"] * c["K"] <= 3.8e10:
                return c
    while True:
        c = dict(op=op, B=_log(rng, 1, 64), S=rng.choice([1, 16, 16, 32, 64, 128]),
                 H=128 * _log(rng, 2, 48), V=_log(rng, 1000, 131072), masked=rng.uniform(0.3, 1.0),
                 scale=rng.choice([1.0, 8.0, 12.0]))
        if c["B"] * c["S"] <= 1024 and c["B"] * c["S"] * c["V"] * c["H"] <= 5e11:
            return c


# ---------------------------------------------------------------- inputs
def _scales(blk_amax, kv):
    """Scale of a block (or row) from its largest magnitude, in 32 bits."""
    return torch.clamp(blk_amax.float() / QMAX[kv], min=FLOOR)


def _code(x, s, kv):
    """x / s rounded to the nearest code, ties to even; quotients in 64 bits,
    since a value half way between two codes has to go the right way."""
    v = x.double() / s.double()
    if kv == "int8":
        return torch.round(v).clamp_(-127, 127).to(torch.int8)
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20)))
    step = torch.exp2(e.clamp_(min=-6) - 3)
    return (torch.round(v / step) * step).clamp_(-448, 448).float().to(torch.float8_e4m3fn)


def _pieces(n, most=1 << 24):
    return max(1, -(-n // most))


def _lengths(c, g, dev):
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], dtype=torch.int32, device=dev)
    lo = max(1, c["L"] // 64)
    return torch.randint(lo, c["L"] + 1, (c["B"],), generator=g, device=dev).to(torch.int32)


def _cache(c, g, dev, cap, spread):
    """One 8-bit cache and its scales, as appending in whole blocks fills it."""
    B, Hkv, dh, blk, kv = c["B"], c["Hkv"], c["dh"], c["block"], c["kv"]
    nb = -(-cap // blk)
    q = torch.empty((B, Hkv, cap, dh), dtype=DTYPE[kv], device=dev)
    s = torch.ones((B, Hkv, nb), dtype=torch.float32, device=dev)
    step = max(1, (1 << 25) // max(1, cap * dh))
    flat, fs = q.view(B * Hkv, cap, dh), s.view(B * Hkv, nb)
    for i in range(0, B * Hkv, step):
        x = torch.randn((min(step, B * Hkv - i), nb * blk, dh), generator=g, device=dev) * spread
        x = x.to(torch.bfloat16).view(-1, nb, blk, dh)
        sc = _scales(x.abs().amax((2, 3)), kv)
        v = x.float() / sc[:, :, None, None]
        v = torch.round(v).to(torch.int8) if kv == "int8" else v.to(torch.float8_e4m3fn)
        flat[i:i + step] = v.view(-1, nb * blk, dh)[:, :cap]
        fs[i:i + step] = sc
    return q, s


def _rows(shape, g, dev, scale=1.0):
    return (torch.randn(shape, generator=g, device=dev) * scale).to(torch.bfloat16)


def _weight(n, k, g, dev):
    """int8 weights with a scale for each output channel."""
    q = torch.empty((n, k), dtype=torch.int8, device=dev)
    s = torch.empty((n,), dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // k)
    for i in range(0, n, step):
        w = torch.randn((min(step, n - i), k), generator=g, device=dev) / math.sqrt(k)
        s[i:i + step] = _scales(w.abs().amax(1), "int8")
        q[i:i + step] = torch.round(w / s[i:i + step, None]).to(torch.int8)
    return q, s


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = dict(case=c)
    if c["op"] == "attn":
        B, S, Hkv, Hq, dh = c["B"], c["S"], c["Hkv"], c["Hkv"] * c["G"], c["dh"]
        st["k_ctx"], st["k_scale"] = _cache(c, g, dev, c["L"], 1.0)
        st["v_ctx"], st["v_scale"] = _cache(c, g, dev, c["L"], 1.0)
        st["ctx_len"] = _lengths(c, g, dev)
        st["q_blk"] = _rows((B, S, Hq, dh), g, dev)
        st["k_blk"] = _rows((B, S, Hkv, dh), g, dev)
        st["v_blk"] = _rows((B, S, Hkv, dh), g, dev)
        st["out"] = torch.empty((B, S, Hq, dh), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "append":
        B, Hkv, dh, n = c["B"], c["Hkv"], c["dh"], c["n"]
        cap = c["L"] + n
        st["k_ctx"], st["k_scale"] = _cache(c, g, dev, cap, 0.8)
        st["v_ctx"], st["v_scale"] = _cache(c, g, dev, cap, 0.8)
        # sequences end anywhere inside a block; the prompts' ragged lengths
        # leave padding rows behind the shorter ones
        back = torch.randint(0, min(c["block"], c["L"]) + 1, (B,), generator=g, device=dev)
        st["ctx_len0"] = (c["L"] - back).to(torch.int32)
        st["ctx_len"] = st["ctx_len0"].clone()
        st["new_len"] = torch.randint(n // 2, n + 1, (B,), generator=g, device=dev).to(torch.int32) \
            if c["ragged"] else None
        # k and v are column ranges of one projection's rows
        kv = _rows((B, n, 2 * Hkv * dh), g, dev)
        st["k_new"] = kv[:, :, :Hkv * dh].view(B, n, Hkv, dh)
        st["v_new"] = kv[:, :, Hkv * dh:].view(B, n, Hkv, dh)
    elif c["op"] == "linear":
        st["x"] = _rows((c["M"], c["K"]), g, dev)
        st["w"], st["ws"] = _weight(c["N"], c["K"], g, dev)
        st["out"] = torch.empty((c["M"], c["N"]), dtype=torch.bfloat16, device=dev)
    else:
        B, S = c["B"], c["S"]
        st["y"] = _rows((B * S, c["H"]), g, dev)
        st["w"], st["ws"] = _weight(c["V"], c["H"], g, dev)
        m = torch.rand((B, S), generator=g, device=dev) < c["masked"]
        m[:, 0] |= ~m.any(1)
        tok = torch.randint(0, c["V"], (B, S), generator=g, device=dev)
        st["masked0"] = m.to(torch.uint8)
        st["tokens0"] = torch.where(m, torch.full_like(tok, -1), tok).to(torch.int32)
        st["masked"], st["tokens"] = st["masked0"].clone(), st["tokens0"].clone()
        st["gamma"] = 0.5
        st["conf"] = torch.empty((B, S), dtype=torch.float32, device=dev)
        st["argmax"] = torch.empty((B, S), dtype=torch.int32, device=dev)
        st["n"] = torch.empty((B,), dtype=torch.int32, device=dev)
    return st


# ------------------------------------------------------------ plain forms
def _attn(st):
    c = st["case"]
    B, S, Hkv, G, dh, L, blk = c["B"], c["S"], c["Hkv"], c["G"], c["dh"], c["L"], c["block"]
    f = torch.float32
    ks = st["k_scale"].repeat_interleave(blk, 2)[:, :, :L, None]
    vs = st["v_scale"].repeat_interleave(blk, 2)[:, :, :L, None]
    k = torch.cat((st["k_blk"].to(f).transpose(1, 2), st["k_ctx"].to(f) * ks), 2)
    v = torch.cat((st["v_blk"].to(f).transpose(1, 2), st["v_ctx"].to(f) * vs), 2)
    q = st["q_blk"].to(f).view(B, S, Hkv, G, dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, dh)
    sc = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(dh)
    pos = torch.arange(S + L, device=q.device) - S
    sc = torch.where((pos[None] < st["ctx_len"][:, None])[:, None, None], sc, -math.inf)
    sc -= sc.amax(3, keepdim=True)
    p = torch.exp_(sc)
    o = torch.matmul(p, v) / p.sum(3, keepdim=True)
    o = o.view(B, Hkv, S, G, dh).permute(0, 2, 1, 3, 4).reshape(B, S, Hkv * G, dh)
    return o.to(torch.bfloat16)


def _append_one(c, new, cache, scale, len0, new_len):
    """The blocks that the new rows touch, as [B, Hkv, blocks, block, dh]: the
    first starts at the block that holds the sequence's end."""
    B, Hkv, dh, n, blk, kv = c["B"], c["Hkv"], c["dh"], c["n"], c["block"], c["kv"]
    dev, cap = cache.device, cache.shape[2]
    nb = -(-n // blk) + 1
    first = (len0 // blk).long()
    b = torch.arange(B, device=dev)[:, None]
    pos = first[:, None] * blk + torch.arange(nb * blk, device=dev)  # cache positions
    src = pos - len0[:, None]
    is_new = (src >= 0) & (src < new_len[:, None])
    is_old = src < 0
    rows = new[b, src.clamp(0, n - 1)].permute(0, 2, 1, 3)  # [B, Hkv, nb*blk, dh]
    at = pos.clamp(max=cap - 1)
    old = cache.view(torch.int8)[b, :, at].permute(0, 2, 1, 3).contiguous().view(cache.dtype)
    blocks = first[:, None] + torch.arange(nb, device=dev)
    in_scale = blocks.clamp(max=scale.shape[2] - 1)
    s_old = scale[b, :, in_scale].permute(0, 2, 1)
    shape = (B, Hkv, nb, blk, dh)
    x = torch.where(is_new[:, None, :, None], rows.float(), 0.0).view(shape)
    s = _scales(x.abs().amax((3, 4)), kv)
    s[:, :, 0] = torch.where(is_old[:, None, 0], torch.maximum(s[:, :, 0], s_old[:, :, 0]), s[:, :, 0])
    q_new = _code(x, s[..., None, None], kv)
    q_old = _code(old.view(shape)[:, :, :1].double() * s_old[:, :, :1, None, None].double(),
                  s[:, :, :1, None, None], kv)
    bytes_new = q_new.view(torch.int8)
    o = is_old.view(B, 1, nb, blk, 1)[:, :, :1]
    bytes_new[:, :, :1] = torch.where(o, q_old.view(torch.int8), bytes_new[:, :, :1])
    write = is_new | (is_old & is_new[:, :blk].any(1, keepdim=True))
    bi, pi = torch.nonzero(write, as_tuple=True)
    flat = bytes_new.view(B, Hkv, nb * blk, dh)
    cache.view(torch.int8)[bi, :, pos[bi, pi]] = flat[bi, :, pi]
    touched = is_new.view(B, nb, blk).any(2)
    bi, ki = torch.nonzero(touched, as_tuple=True)
    scale[bi, :, blocks[bi, ki]] = s[bi, :, ki]


def _append(st):
    c = st["case"]
    len0 = st["ctx_len"]
    new_len = st["new_len"] if st["new_len"] is not None else torch.full_like(len0, c["n"])
    _append_one(c, st["k_new"], st["k_ctx"], st["k_scale"], len0, new_len)
    _append_one(c, st["v_new"], st["v_ctx"], st["v_scale"], len0, new_len)
    st["ctx_len"] += new_len


def _quantised_rows(x):
    s = _scales(x.abs().amax(1), "int8")
    return _code(x, s[:, None], "int8"), s


def _linear(st):
    xq, xs = _quantised_rows(st["x"])
    acc = torch.matmul(xq.float(), st["w"].float().t())  # whole numbers below 2^24
    return (acc * (xs[:, None] * st["ws"][None])).to(torch.bfloat16)


def _vocab(st):
    c = st["case"]
    B, S, V = c["B"], c["S"], c["V"]
    yq, ys = _quantised_rows(st["y"])
    logits = torch.empty((B * S, V), dtype=torch.float32, device=yq.device)
    yf = yq.float()
    for i in range(0, V, 32768):  # 32-bit weights a piece at a time
        logits[:, i:i + 32768] = torch.matmul(yf, st["w"][i:i + 32768].float().t())
    logits *= st["ws"][None]
    top = logits.amax(1, keepdim=True)
    ids = torch.arange(V, dtype=torch.int32, device=yq.device)
    tok = torch.where(logits == top, ids[None], V).amin(1).view(B, S).to(torch.int32)
    conf = 1.0 / torch.exp((logits - top) * (ys * c["scale"])[:, None]).sum(1).view(B, S)
    return _commit(st, tok, conf)


def _commit(st, tok, conf):
    m = st["masked"] != 0
    S = m.shape[1]
    cand = m & (conf >= st["gamma"])
    seen = torch.where(m, conf, -1.0)
    ids = torch.arange(S, device=m.device)[None]
    best = torch.where(seen == seen.amax(1, keepdim=True), ids, S).amin(1, keepdim=True)
    alone = m & (ids == best) & ~cand.any(1, keepdim=True)
    take = cand | alone
    tokens = torch.where(take, tok, st["tokens"])
    return dict(tokens=tokens, masked=(m & ~take).to(torch.uint8),
                conf=seen.to(torch.float32), argmax=torch.where(m, tok, -1).to(torch.int32),
                n=take.sum(1).to(torch.int32))


# -------------------------------------------------------------------- run
def run(state):
    st, op = state, state["case"]["op"]
    if op == "append":
        st["ctx_len"].copy_(st["ctx_len0"])  # the same append again
    if op == "vocab":
        st["tokens"].copy_(st["tokens0"])
        st["masked"].copy_(st["masked0"])
    if own:
        return _run_own(st, op)
    if op == "attn":
        return _attn(st)
    if op == "linear":
        return _linear(st)
    if op == "vocab":
        return _vocab(st)
    _append(st)
    return _append_result(st)


def _append_result(st):
    # codes in units of their block's scale, and the scales
    return dict(k=st["k_ctx"], v=st["v_ctx"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                ctx_len=st["ctx_len"])


def _run_own(st, op):
    import block_wise_diffusion_b200 as tt
    c = st["case"]
    if "ws_own" not in st:  # dims and workspace, kept by the program
        if op == "linear":
            st["ws_own"] = tt.linear_i8_workspace(c["M"], c["N"], c["K"])
        elif op == "vocab":
            heads = c["H"] // 64
            st["dims"] = tt.Dims(c["B"], c["S"], heads, heads, 64, c["H"], c["V"], 0)
            st["ws_own"] = tt.workspace(st["dims"], tt.TT_WS_VOCAB_I8)
        else:
            st["fmt"] = tt.q8(c["kv"], c["block"])
            G, cap = (c["G"], c["L"]) if op == "attn" else (1, c["L"] + c["n"])
            st["dims"] = tt.Dims(c["B"], c.get("S", 1), c["Hkv"] * G, c["Hkv"], c["dh"],
                                 c["Hkv"] * G * c["dh"], 1024, cap)
            st["ws_own"] = tt.workspace(st["dims"], tt.TT_WS_ATTN_Q8 if op == "attn" else
                                        tt.TT_WS_APPEND_Q8)
    if op == "attn":
        tt.tt_block_denoise_attn_q8(st["dims"], st["fmt"], st["q_blk"], st["k_blk"], st["v_blk"],
                                    st["k_ctx"], st["v_ctx"], st["k_scale"], st["v_scale"],
                                    st["ctx_len"], st["out"], st["ws_own"])
        return st["out"]
    if op == "append":
        tt.tt_append_ctx_q8(st["dims"], st["fmt"], c["n"], st["new_len"], st["k_new"], st["v_new"],
                            st["k_ctx"], st["v_ctx"], st["k_scale"], st["v_scale"], st["ctx_len"],
                            st["ws_own"])
        return _append_result(st)
    if op == "linear":
        tt.tt_linear_i8(c["M"], c["N"], c["K"], st["x"], st["w"], st["ws"], st["out"], st["ws_own"])
        return st["out"]
    tt.tt_vocab_confidence_commit_i8(st["dims"], st["y"], st["w"], st["ws"], st["gamma"],
                                     c["scale"], st["tokens"], st["masked"], st["conf"],
                                     st["argmax"], st["n"], st["ws_own"])
    return dict(tokens=st["tokens"], masked=st["masked"], conf=st["conf"], argmax=st["argmax"],
                n=st["n"])


# ------------------------------------------------------------------- work
def _mean_len(c):
    return (max(1, c["L"] // 64) + c["L"]) / 2 if c["ragged"] else c["L"]


def work(case):
    c = case
    if c["op"] == "attn":
        L, rows = _mean_len(c), c["B"] * c["S"] * c["Hkv"]
        kv = 2 * c["B"] * c["Hkv"] * L * (c["dh"] + 4 / c["block"])
        return dict(bytes=kv + 2 * rows * c["dh"] * (2 * c["G"] + 2),
                    flops=4 * rows * c["G"] * (L + c["S"]) * c["dh"])
    if c["op"] == "append":
        n = c["n"] * (0.75 if c["ragged"] else 1.0)
        vals = 2 * c["B"] * c["Hkv"] * n * c["dh"]
        return dict(bytes=3 * vals + 4 * vals / (c["dh"] * c["block"]), flops=3 * vals)
    if c["op"] == "linear":
        return dict(bytes=c["N"] * c["K"] + 4 * c["N"] + 2 * c["M"] * (c["K"] + c["N"]),
                    flops=2 * c["M"] * c["N"] * c["K"])
    rows = c["B"] * c["S"] * c["masked"]
    return dict(bytes=c["V"] * c["H"] + 4 * c["V"] + 2 * rows * c["H"] + 13 * c["B"] * c["S"],
                flops=2 * rows * c["V"] * c["H"])


# ------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    c, st = case, prepare(case, seed)
    d = torch.float64
    if c["op"] == "attn":
        out = torch.zeros(st["out"].shape, dtype=d, device="cuda")
        for b in range(c["B"]):
            n = int(st["ctx_len"][b])
            nb = -(-n // c["block"])
            for h in range(c["Hkv"]):
                def rows(codes, scale, blk_rows):
                    full = torch.zeros((nb * c["block"], c["dh"]), dtype=d, device="cuda")
                    full[:n] = codes[b, h, :n].to(torch.float32).to(d)
                    full = full.view(nb, c["block"], c["dh"]) * scale[b, h, :nb].to(d)[:, None, None]
                    return torch.cat((full.reshape(-1, c["dh"])[:n], blk_rows[b, :, h].to(d)))
                k = rows(st["k_ctx"], st["k_scale"], st["k_blk"])
                v = rows(st["v_ctx"], st["v_scale"], st["v_blk"])
                q = st["q_blk"][b, :, h * c["G"]:(h + 1) * c["G"]].to(d)
                w = torch.softmax(torch.einsum("sgd,kd->sgk", q, k) * c["dh"] ** -0.5, -1)
                out[b, :, h * c["G"]:(h + 1) * c["G"]] = torch.einsum("sgk,kd->sgd", w, v)
        return out
    if c["op"] == "append":
        # only the scales are computed numbers; the codes are whole multiples of them
        lens = st["ctx_len0"].tolist()
        new = st["new_len"].tolist() if st["new_len"] is not None else [c["n"]] * c["B"]
        blk = c["block"]
        res = {}
        for name in ("k", "v"):
            s = st[name + "_scale"].to(d)
            mag = st[name + "_new"].to(d).abs().amax(3)  # [B, n, Hkv]
            for b in range(c["B"]):
                if new[b] == 0:
                    continue
                lo, hi = lens[b] // blk, (lens[b] + new[b] - 1) // blk
                pad = torch.zeros(((hi - lo + 1) * blk, c["Hkv"]), dtype=d, device="cuda")
                pad[lens[b] - lo * blk:lens[b] - lo * blk + new[b]] = mag[b, :new[b]]
                got = (pad.view(-1, blk, c["Hkv"]).amax(1) / QMAX[c["kv"]]).clamp(min=FLOOR).t()
                if lens[b] % blk:
                    got[:, 0] = torch.maximum(got[:, 0], s[b, :, lo])
                s[b, :, lo:hi + 1] = got
            res[name + "_scale"] = s
        return dict(k=None, v=None, k_scale=res["k_scale"], v_scale=res["v_scale"], ctx_len=None)

    def codes(x):
        a = x.to(d).abs().amax(1, keepdim=True)
        s = (a.float() / 127).clamp(min=FLOOR).to(d)  # a scale is a 32-bit number
        return torch.round(x.to(d) / s), s
    if c["op"] == "linear":
        q, s = codes(st["x"])
        out = torch.empty((c["M"], c["N"]), dtype=d, device="cuda")
        for i in range(0, c["N"], 4096):
            out[:, i:i + 4096] = (q @ st["w"][i:i + 4096].to(d).t()) * s * st["ws"][i:i + 4096].to(d)
        return out
    B, S = c["B"], c["S"]
    q, s = codes(st["y"])
    lg = torch.empty((B * S, c["V"]), dtype=d, device="cuda")
    for i in range(0, c["V"], 16384):
        lg[:, i:i + 16384] = (q @ st["w"][i:i + 16384].to(d).t()) * s * st["ws"][i:i + 16384].to(d)
    tok = lg.argmax(1).view(B, S)
    conf = torch.softmax(lg.mul_(c["scale"]), 1).amax(1).view(B, S).cpu()
    m0 = st["masked0"].cpu().bool()
    tokens, left = st["tokens0"].cpu().clone(), m0.clone()
    tok = tok.cpu()
    n = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        at = [p for p in range(S) if m0[b, p] and conf[b, p] >= st["gamma"]]
        if not at and bool(m0[b].any()):
            at = [max((p for p in range(S) if m0[b, p]), key=lambda p: (float(conf[b, p]), -p))]
        for p in at:
            tokens[b, p], left[b, p] = int(tok[b, p]), False
        n[b] = len(at)
    return dict(tokens=tokens, masked=left.to(torch.uint8),
                conf=torch.where(m0, conf, torch.full_like(conf, -1.0)),
                argmax=torch.where(m0, tok, torch.full_like(tok, -1)).to(torch.int32), n=n)
