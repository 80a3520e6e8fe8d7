"""Python binding of libtwotower (argument marshalling only).

Every function with a ``tt_`` name calls the C entry point of the same name
in ``libtwotower.so`` (built in-tree by ``block_wise_diffusion_b200.build``)
with raw device pointers taken from torch tensors.  Nothing here computes:
torch provides device memory and streams; all arithmetic runs in the
library's sm_100a kernels.  There is no CPU path: if the library or a CUDA
device is missing, the calls raise.  Before a call, every tensor argument is
checked to hold at least the bytes of the shape include/twotower.h documents
for it, since the kernels address each buffer from the dims alone.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "TTError", "Dims", "lib", "lib_path", "dims", "workspace", "tt_workspace_bytes",
    "tt_block_denoise_attn", "tt_adaln_modulate", "tt_vocab_confidence_commit",
    "tt_denoise_block_loop", "tt_denoise_block_loop_layers", "tt_decode_blocks",
    "tt_vocab_confidence_commit_noalloc", "tt_loop_last_step",
    "tt_device_status", "tt_launch_count", "tt_set_attn_splits", "tt_set_loop_graphs",
    "tt_status_string", "tt_last_error", "EXPORTS", "tt_profile_enable", "tt_profile_read",
    "tt_selftest_timeout",
    "profile_table", "KERNEL_KINDS",
    "TT_WS_ATTN", "TT_WS_ADALN", "TT_WS_VOCAB", "TT_WS_LOOP",
    "Q8", "q8", "tt_block_denoise_attn_q8", "tt_append_ctx_q8", "tt_quantize_rows_i8",
    "tt_linear_i8", "tt_linear_i8_workspace_bytes", "linear_i8_workspace",
    "tt_vocab_confidence_commit_i8",
    "TT_WS_ATTN_Q8", "TT_WS_APPEND_Q8", "TT_WS_VOCAB_I8", "TT_Q8_INT8", "TT_Q8_E4M3",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libtwotower.so")

TT_WS_ATTN, TT_WS_ADALN, TT_WS_VOCAB, TT_WS_LOOP = 0, 1, 2, 3
TT_WS_ATTN_Q8, TT_WS_APPEND_Q8, TT_WS_VOCAB_I8 = 4, 5, 6
TT_Q8_INT8, TT_Q8_E4M3 = 0, 1
STATUS = {0: "TT_OK", 1: "TT_ERR_INVALID_ARG", 2: "TT_ERR_UNSUPPORTED", 3: "TT_ERR_WORKSPACE",
          4: "TT_ERR_CUDA", 5: "TT_ERR_TIMEOUT", 6: "TT_ERR_INTERNAL"}

# Every symbol the header declares.
EXPORTS = (
    "tt_status_string", "tt_last_error", "tt_workspace_bytes", "tt_device_status",
    "tt_launch_count", "tt_set_attn_splits", "tt_set_loop_graphs", "tt_block_denoise_attn",
    "tt_adaln_modulate",
    "tt_vocab_confidence_commit", "tt_denoise_block_loop", "tt_profile_enable", "tt_profile_read",
    "tt_vocab_confidence_commit_noalloc", "tt_selftest_timeout", "tt_denoise_block_loop_layers",
    "tt_decode_blocks", "tt_loop_last_step", "tt_block_denoise_attn_q8", "tt_append_ctx_q8",
    "tt_quantize_rows_i8", "tt_linear_i8_workspace_bytes", "tt_linear_i8",
    "tt_vocab_confidence_commit_i8",
)
KERNEL_KINDS = ("plan", "embed", "gemm_qkv", "attn", "merge", "adaln", "gemm_vocab", "commit",
                "gather", "init", "splitk_reduce", "append", "attn_plan", "attn_q8", "merge_q8",
                "append_q8", "quant_i8", "gemm_i8", "gemm_vocab_i8")


class TTError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}: {detail}")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "S", "Hq", "Hkv", "dh", "H", "V", "L_cap")]


class Q8(ctypes.Structure):
    """Format of an 8-bit context cache (tt_q8): element type and positions per scale."""
    _fields_ = [("type", ctypes.c_int32), ("block", ctypes.c_int32)]


class _RowStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "token", "head")]


_P = ctypes.c_void_p
_lib = None


def lib() -> ctypes.CDLL:
    """Load libtwotower.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(
                f"{lib_path} is missing: build it with `python -m block_wise_diffusion_b200.build`")
        L = ctypes.CDLL(lib_path)
        L.tt_status_string.restype = ctypes.c_char_p
        L.tt_status_string.argtypes = [ctypes.c_int]
        L.tt_last_error.restype = ctypes.c_char_p
        L.tt_last_error.argtypes = []
        L.tt_workspace_bytes.restype = ctypes.c_size_t
        L.tt_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
        L.tt_device_status.restype = ctypes.c_int
        L.tt_device_status.argtypes = [_P, _P]
        L.tt_selftest_timeout.restype = ctypes.c_int
        L.tt_selftest_timeout.argtypes = [_P, ctypes.c_int32, _P]
        L.tt_launch_count.restype = ctypes.c_uint64
        L.tt_launch_count.argtypes = []
        L.tt_set_attn_splits.restype = ctypes.c_int
        L.tt_set_attn_splits.argtypes = [ctypes.c_int32]
        L.tt_set_loop_graphs.restype = ctypes.c_int
        L.tt_set_loop_graphs.argtypes = [ctypes.c_int32]
        L.tt_profile_enable.restype = ctypes.c_int
        L.tt_profile_enable.argtypes = [ctypes.c_int32]
        L.tt_profile_read.restype = ctypes.c_int
        L.tt_profile_read.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_int64)]
        L.tt_block_denoise_attn.restype = ctypes.c_int
        L.tt_block_denoise_attn.argtypes = [ctypes.POINTER(Dims)] + [_P] * 7 + [_P, ctypes.c_size_t, _P]
        L.tt_adaln_modulate.restype = ctypes.c_int
        L.tt_adaln_modulate.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.tt_vocab_confidence_commit.restype = ctypes.c_int
        L.tt_vocab_confidence_commit.argtypes = (
            [ctypes.POINTER(Dims), _P, _P, ctypes.c_float, ctypes.c_float] + [_P] * 5
            + [_P, ctypes.c_size_t, _P])
        L.tt_vocab_confidence_commit_noalloc.restype = ctypes.c_int
        L.tt_vocab_confidence_commit_noalloc.argtypes = (
            [ctypes.POINTER(Dims), _P, _P, ctypes.c_float, ctypes.c_float] + [_P] * 5 + [_P])
        L.tt_denoise_block_loop.restype = ctypes.c_int
        L.tt_denoise_block_loop.argtypes = (
            [ctypes.POINTER(Dims)] + [_P] * 8 + [ctypes.c_float, ctypes.c_float, ctypes.c_int32]
            + [_P] * 5 + [_P, ctypes.c_size_t, _P])
        L.tt_decode_blocks.restype = ctypes.c_int
        L.tt_decode_blocks.argtypes = (
            [ctypes.POINTER(Dims), ctypes.c_int32] + [_P] * 9
            + [ctypes.c_float, ctypes.c_float] + [_P] * 4 + [_P, ctypes.c_size_t, _P])
        L.tt_loop_last_step.restype = ctypes.c_int
        L.tt_loop_last_step.argtypes = [ctypes.POINTER(Dims), _P, ctypes.c_size_t] + [_P] * 5 + [_P]
        L.tt_denoise_block_loop_layers.restype = ctypes.c_int
        L.tt_denoise_block_loop_layers.argtypes = (
            [ctypes.POINTER(Dims), ctypes.c_int32] + [_P] * 8
            + [ctypes.c_float, ctypes.c_float, ctypes.c_int32] + [_P] * 5
            + [_P, ctypes.c_size_t, _P])
        dims_p, q8_p = ctypes.POINTER(Dims), ctypes.POINTER(Q8)
        L.tt_block_denoise_attn_q8.restype = ctypes.c_int
        L.tt_block_denoise_attn_q8.argtypes = [dims_p, q8_p] + [_P] * 9 + [_P, ctypes.c_size_t, _P]
        L.tt_append_ctx_q8.restype = ctypes.c_int
        L.tt_append_ctx_q8.argtypes = (
            [dims_p, q8_p, ctypes.c_int32, _P, _P, _P, ctypes.POINTER(_RowStrides)] + [_P] * 5
            + [_P, ctypes.c_size_t, _P])
        L.tt_quantize_rows_i8.restype = ctypes.c_int
        L.tt_quantize_rows_i8.argtypes = [ctypes.c_int32, ctypes.c_int32] + [_P] * 4
        L.tt_linear_i8_workspace_bytes.restype = ctypes.c_size_t
        L.tt_linear_i8_workspace_bytes.argtypes = [ctypes.c_int32] * 3
        L.tt_linear_i8.restype = ctypes.c_int
        L.tt_linear_i8.argtypes = [ctypes.c_int32] * 3 + [_P] * 5 + [ctypes.c_size_t, _P]
        L.tt_vocab_confidence_commit_i8.restype = ctypes.c_int
        L.tt_vocab_confidence_commit_i8.argtypes = (
            [dims_p, _P, _P, _P, ctypes.c_float, ctypes.c_float] + [_P] * 5
            + [_P, ctypes.c_size_t, _P])
        _lib = L
    return _lib


def dims(d) -> Dims:
    """tt_dims from any object with B, S, Hq, Hkv, dh, V, L_cap (and H) fields."""
    H = getattr(d, "H", d.Hq * d.dh)
    return Dims(d.B, d.S, d.Hq, d.Hkv, d.dh, H, d.V, d.L_cap)


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("libtwotower takes CUDA tensors only (no CPU path)")
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return x.data_ptr()


def _nbytes(x) -> int:
    return x.numel() * x.element_size() if hasattr(x, "numel") else 0


def _sized(x, name: str, nbytes: int) -> int | None:
    """_ptr(x) after checking that a tensor holds at least ``nbytes``: the
    shape include/twotower.h documents for the argument times its element
    size.  The kernels address these buffers from the dims alone, so a short
    tensor would be read or written past its end.  Raw integer addresses
    carry no size and pass unchecked."""
    if x is not None and not isinstance(x, int) and _nbytes(x) < nbytes:
        raise ValueError(f"{name} holds {_nbytes(x)} bytes; these dims need {nbytes}")
    return _ptr(x)


def _ctx_bytes(d: Dims) -> int:
    """bf16 [B, Hkv, L_cap, dh]: one context cache (K or V) of one layer."""
    return d.B * d.Hkv * d.L_cap * d.dh * 2


def _u_t_bytes(d: Dims) -> int:
    """bf16 [H + 2*Hkv*dh, H]: one layer's linear update."""
    return (d.H + 2 * d.Hkv * d.dh) * d.H * 2


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != 0:
        raise TTError(code, where, lib().tt_last_error().decode())


def tt_status_string(code: int) -> str:
    return lib().tt_status_string(code).decode()


def tt_last_error() -> str:
    return lib().tt_last_error().decode()


def tt_launch_count() -> int:
    return int(lib().tt_launch_count())


def tt_set_attn_splits(n: int) -> None:
    _check(lib().tt_set_attn_splits(n), "tt_set_attn_splits")


def tt_set_loop_graphs(on: int) -> None:
    _check(lib().tt_set_loop_graphs(on), "tt_set_loop_graphs")


def tt_profile_enable(on: bool) -> None:
    _check(lib().tt_profile_enable(1 if on else 0), "tt_profile_enable")


def tt_profile_read(kind: int) -> tuple[float, int]:
    """(total ms, launches) of one kernel kind since profiling was enabled."""
    ms, n = ctypes.c_double(0), ctypes.c_int64(0)
    _check(lib().tt_profile_read(kind, ctypes.byref(ms), ctypes.byref(n)), "tt_profile_read")
    return ms.value, n.value


def profile_table() -> dict:
    """{kernel kind name: (total ms, launches)} for every kind that ran."""
    out = {}
    for k, name in enumerate(KERNEL_KINDS):
        ms, n = tt_profile_read(k)
        if n:
            out[name] = (ms, n)
    return out


def tt_workspace_bytes(d: Dims, which: int) -> int:
    n = lib().tt_workspace_bytes(ctypes.byref(d), which)
    if n == 0:
        raise TTError(1, "tt_workspace_bytes", tt_last_error())
    return int(n)


def workspace(d: Dims, which: int, device="cuda"):
    """A torch uint8 device buffer of tt_workspace_bytes(d, which) bytes."""
    import torch
    return torch.empty(tt_workspace_bytes(d, which), dtype=torch.uint8, device=device)


def tt_selftest_timeout(ws, limit_us: int, stream=None) -> None:
    """Make one bounded device wait run out on purpose (see the header)."""
    _check(lib().tt_selftest_timeout(_ptr(ws), int(limit_us), _stream(stream)),
           "tt_selftest_timeout")


def tt_device_status(ws, stream=None) -> int:
    """Synchronise and return (and clear) the device error code in `ws`."""
    return int(lib().tt_device_status(_ptr(ws), _stream(stream)))


def tt_block_denoise_attn(d: Dims, q_blk, k_blk, v_blk, k_ctx, v_ctx, ctx_len, out, ws,
                          stream=None) -> None:
    rows = d.B * d.S
    _check(lib().tt_block_denoise_attn(
        ctypes.byref(d), _sized(q_blk, "q_blk", rows * d.Hq * d.dh * 2),
        _sized(k_blk, "k_blk", rows * d.Hkv * d.dh * 2),
        _sized(v_blk, "v_blk", rows * d.Hkv * d.dh * 2), _sized(k_ctx, "k_ctx", _ctx_bytes(d)),
        _sized(v_ctx, "v_ctx", _ctx_bytes(d)), _sized(ctx_len, "ctx_len", d.B * 4),
        _sized(out, "out", rows * d.Hq * d.dh * 2), _ptr(ws), _nbytes(ws),
        _stream(stream)), "tt_block_denoise_attn")


def tt_adaln_modulate(d: Dims, x, shift_scale, t, y, ws, stream=None) -> None:
    rows = d.B * d.S
    _check(lib().tt_adaln_modulate(
        ctypes.byref(d), _sized(x, "x", rows * d.H * 2),
        _sized(shift_scale, "shift_scale", 2 * d.H * 2), _sized(t, "t", d.B * 4),
        _sized(y, "y", rows * d.H * 2), _ptr(ws), _nbytes(ws), _stream(stream)),
        "tt_adaln_modulate")


def tt_vocab_confidence_commit(d: Dims, y, w, gamma: float, logit_scale: float, tokens, masked,
                               conf_out, argmax_out, n_committed, ws, stream=None) -> None:
    _check(lib().tt_vocab_confidence_commit(
        ctypes.byref(d), *_vocab_args(d, y, w, gamma, logit_scale, tokens, masked, conf_out,
                                      argmax_out, n_committed),
        _ptr(ws), _nbytes(ws), _stream(stream)), "tt_vocab_confidence_commit")


def _vocab_args(d: Dims, y, w, gamma, logit_scale, tokens, masked, conf_out, argmax_out,
                n_committed) -> tuple:
    rows = d.B * d.S
    return (_sized(y, "y", rows * d.H * 2), _sized(w, "w", d.V * d.H * 2), float(gamma),
            float(logit_scale), _sized(tokens, "tokens", rows * 4),
            _sized(masked, "masked", rows), _sized(conf_out, "conf_out", rows * 4),
            _sized(argmax_out, "argmax_out", rows * 4),
            _sized(n_committed, "n_committed", d.B * 4))


def tt_vocab_confidence_commit_noalloc(d: Dims, y, w, gamma: float, logit_scale: float,
                                       tokens, masked, conf_out, argmax_out, n_committed,
                                       stream=None) -> None:
    """tt_vocab_confidence_commit without a workspace, for callers that cannot
    allocate device memory; its scratch is a 16 MiB array built into the
    library (calls that overlap on the GPU must be serialised)."""
    _check(lib().tt_vocab_confidence_commit_noalloc(
        ctypes.byref(d), *_vocab_args(d, y, w, gamma, logit_scale, tokens, masked, conf_out,
                                      argmax_out, n_committed), _stream(stream)),
        "tt_vocab_confidence_commit_noalloc")


def tt_denoise_block_loop(d: Dims, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t, shift_scale, w,
                          gamma: float, logit_scale: float, max_steps: int, tokens, masked,
                          steps_taken, commit_step, ws, stream=None) -> int:
    """Runs the loop; returns the number of steps that did work."""
    steps_run = ctypes.c_int32(0)
    _check(lib().tt_denoise_block_loop(
        ctypes.byref(d), *_loop_args(d, 1, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t, shift_scale,
                                     w),
        float(gamma), float(logit_scale), int(max_steps),
        *_state_args(d, tokens, masked, steps_taken, commit_step),
        ctypes.addressof(steps_run), _ptr(ws), _nbytes(ws), _stream(stream)),
        "tt_denoise_block_loop")
    return int(steps_run.value)


def _loop_args(d: Dims, n_layers: int, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t, shift_scale,
               w) -> tuple:
    """Checked pointers of the loop's inputs; per-layer tensors hold n_layers
    stacked copies (layer outermost)."""
    nl = max(int(n_layers), 0)
    return (_sized(k_ctx, "k_ctx", nl * _ctx_bytes(d)), _sized(v_ctx, "v_ctx", nl * _ctx_bytes(d)),
            _sized(ctx_len, "ctx_len", d.B * 4), _sized(emb, "emb", d.V * d.H * 2),
            _sized(e_mask, "e_mask", d.H * 2), _sized(u_t, "u_t", nl * _u_t_bytes(d)),
            _sized(shift_scale, "shift_scale", nl * 2 * d.H * 2),
            _sized(w, "w", d.V * d.H * 2))


def _state_args(d: Dims, tokens, masked, steps_taken, commit_step) -> tuple:
    rows = d.B * d.S
    return (_sized(tokens, "tokens", rows * 4), _sized(masked, "masked", rows),
            _sized(steps_taken, "steps_taken", d.B * 4),
            _sized(commit_step, "commit_step", rows * 4))


def tt_decode_blocks(d: Dims, n_blocks: int, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t,
                     shift_scale, w, u_ctx, gamma: float, logit_scale: float, tokens,
                     steps_taken, commit_step, ws, stream=None) -> int:
    """n_blocks blocks one after the other, each joining the context once
    committed (k_ctx, v_ctx and ctx_len are updated in place); returns the
    total number of steps that did work."""
    steps_run = ctypes.c_int32(0)
    nb = max(int(n_blocks), 0)
    rows = d.B * d.S
    _check(lib().tt_decode_blocks(
        ctypes.byref(d), int(n_blocks),
        *_loop_args(d, 1, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t, shift_scale, w),
        _sized(u_ctx, "u_ctx", 2 * d.Hkv * d.dh * d.H * 2), float(gamma), float(logit_scale),
        _sized(tokens, "tokens", nb * rows * 4), _sized(steps_taken, "steps_taken", nb * d.B * 4),
        _sized(commit_step, "commit_step", nb * rows * 4),
        ctypes.addressof(steps_run), _ptr(ws), _nbytes(ws), _stream(stream)),
        "tt_decode_blocks")
    return int(steps_run.value)


def tt_denoise_block_loop_layers(d: Dims, n_layers: int, k_ctx, v_ctx, ctx_len, emb, e_mask,
                                 u_t, shift_scale, w, gamma: float, logit_scale: float,
                                 max_steps: int, tokens, masked, steps_taken, commit_step, ws,
                                 stream=None) -> int:
    """The loop over n_layers denoiser layers (per-layer tensors stacked with
    the layer outermost); returns the number of steps that did work."""
    steps_run = ctypes.c_int32(0)
    _check(lib().tt_denoise_block_loop_layers(
        ctypes.byref(d), int(n_layers),
        *_loop_args(d, n_layers, k_ctx, v_ctx, ctx_len, emb, e_mask, u_t, shift_scale, w),
        float(gamma), float(logit_scale), int(max_steps),
        *_state_args(d, tokens, masked, steps_taken, commit_step),
        ctypes.addressof(steps_run), _ptr(ws), _nbytes(ws), _stream(stream)),
        "tt_denoise_block_loop_layers")
    return int(steps_run.value)


def tt_loop_last_step(d: Dims, ws, y_rows, row_ids, conf, argmax, stream=None) -> int:
    """Copy out what the loop's last working step fed the vocabulary and the
    commit rule (data copies only): the compacted adaLN rows into y_rows
    [B*S, H] bf16, their row indices b*S+s into row_ids [B*S] int32, and the
    confidence / argmax of each position masked at the start of the step into
    conf [B*S] float32 and argmax [B*S] int32 (-1 elsewhere).  Returns the
    number of compacted rows."""
    rows = d.B * d.S
    n = ctypes.c_int32(0)
    _check(lib().tt_loop_last_step(
        ctypes.byref(d), _ptr(ws), _nbytes(ws), _sized(y_rows, "y_rows", rows * d.H * 2),
        _sized(row_ids, "row_ids", rows * 4), _sized(conf, "conf", rows * 4),
        _sized(argmax, "argmax", rows * 4), ctypes.addressof(n), _stream(stream)),
        "tt_loop_last_step")
    return int(n.value)


# --------------------------------------------------------------- 8-bit serving
def q8(kind: str, block: int) -> Q8:
    """Format of an 8-bit context cache: kind "int8" or "e4m3", `block` context
    positions (16, 32, 64 or 128) per scale."""
    return Q8({"int8": TT_Q8_INT8, "e4m3": TT_Q8_E4M3}[kind], int(block))


_torch = None


def _device() -> int:
    """The current device: these calls launch there, on its current stream
    unless another is given, so every tensor has to live there."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch.cuda.current_device() if _torch.cuda.is_initialized() else -1


def _arg(x, name: str, nbytes: int, dev: int) -> int | None:
    """Address of a tensor argument after the checks of _sized and of its
    device, with as few tensor calls as they take: a small call's time is the
    host's.  Raw integer addresses carry no size and pass unchecked."""
    if x is None or type(x) is int:
        return x
    if x.nbytes < nbytes:
        raise ValueError(f"{name} holds {x.nbytes} bytes; these dims need {nbytes}")
    at = x.get_device()
    if at < 0:
        raise ValueError("libtwotower takes CUDA tensors only (no CPU path)")
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if at != dev:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{dev}")
    return x.data_ptr()


def _codes_arg(x, name: str, nbytes: int, dev: int, f: Q8) -> int | None:
    """_arg for 8-bit codes: a tensor has the format's type, or is plain bytes (uint8)."""
    if x is not None and type(x) is not int and x.dtype != _torch.uint8:
        want = {TT_Q8_INT8: _torch.int8, TT_Q8_E4M3: _torch.float8_e4m3fn}.get(f.type, x.dtype)
        if x.dtype != want:
            raise ValueError(f"{name} is {x.dtype}, the format's codes are {want}")
    return _arg(x, name, nbytes, dev)


def _raw_stream(stream, dev: int) -> int | None:
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else _stream(None)
    return stream if type(stream) is int else stream.cuda_stream


def tt_block_denoise_attn_q8(d: Dims, f: Q8, q_blk, k_blk, v_blk, k_ctx, v_ctx, k_scale, v_scale,
                             ctx_len, out, ws, stream=None) -> None:
    """tt_block_denoise_attn over a context cache held in 8 bits: codes
    [B, Hkv, L_cap, dh] (int8 or float8_e4m3fn as f has it, or their bytes) and one float32 scale per
    `f.block` positions and KV head."""
    B, S, Hq, Hkv, dh, L_cap, block = d.B, d.S, d.Hq, d.Hkv, d.dh, d.L_cap, f.block
    q, kv, ctx = 2 * B * S * Hq * dh, 2 * B * S * Hkv * dh, B * Hkv * L_cap * dh
    ns = 4 * B * Hkv * -(-L_cap // block) if block > 0 else 0
    dev = _device()
    code = lib().tt_block_denoise_attn_q8(
        d, f, _arg(q_blk, "q_blk", q, dev), _arg(k_blk, "k_blk", kv, dev),
        _arg(v_blk, "v_blk", kv, dev), _codes_arg(k_ctx, "k_ctx", ctx, dev, f),
        _codes_arg(v_ctx, "v_ctx", ctx, dev, f), _arg(k_scale, "k_scale", ns, dev),
        _arg(v_scale, "v_scale", ns, dev), _arg(ctx_len, "ctx_len", 4 * B, dev),
        _arg(out, "out", q, dev), _arg(ws, "ws", 0, dev), _nbytes(ws), _raw_stream(stream, dev))
    if code:
        _check(code, "tt_block_denoise_attn_q8")


def _rows_arg(x, name: str, shape: tuple, dev: int) -> tuple[int, tuple]:
    """Address and strides of a [B, n, Hkv, dh] bf16 tensor with a dense last
    dimension; a dimension of one element has no stride of its own (0)."""
    at, st = x.get_device(), x.stride()
    if at < 0:
        raise ValueError("libtwotower takes CUDA tensors only (no CPU path)")
    if x.shape != shape or x.element_size() != 2 or st[3] != 1:
        raise ValueError(f"{name} must be a 16-bit tensor of shape {shape} with a dense last "
                         f"dimension; got {tuple(x.shape)}, strides {st}")
    if at != dev:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{dev}")
    return x.data_ptr(), tuple(0 if k == 1 else a for k, a in zip(shape[:3], st))


def tt_append_ctx_q8(d: Dims, f: Q8, n: int, new_len, k_new, v_new, k_ctx, v_ctx, k_scale, v_scale,
                     ctx_len, ws, stream=None) -> None:
    """Quantise the first new_len[b] (or all n, with new_len None) rows of
    k_new / v_new [B, n, Hkv, dh] onto the end of each sequence's 8-bit cache;
    ctx_len grows in place.  k_new and v_new may be strided views (the last
    dimension dense, both with the same strides)."""
    B, Hkv, dh, L_cap, block = d.B, d.Hkv, d.dh, d.L_cap, f.block
    ctx, ns = B * Hkv * L_cap * dh, 4 * B * Hkv * -(-L_cap // block) if block > 0 else 0
    dev, shape = _device(), (B, n, Hkv, dh)
    k_ptr, st = _rows_arg(k_new, "k_new", shape, dev)
    v_ptr, sv = _rows_arg(v_new, "v_new", shape, dev)
    if st != sv:
        raise ValueError(f"k_new and v_new need the same strides; got {st} and {sv}")
    code = lib().tt_append_ctx_q8(
        d, f, n, _arg(new_len, "new_len", 4 * B, dev), k_ptr, v_ptr, _RowStrides(*st),
        _codes_arg(k_ctx, "k_ctx", ctx, dev, f), _codes_arg(v_ctx, "v_ctx", ctx, dev, f),
        _arg(k_scale, "k_scale", ns, dev), _arg(v_scale, "v_scale", ns, dev),
        _arg(ctx_len, "ctx_len", 4 * B, dev), _arg(ws, "ws", 0, dev), _nbytes(ws),
        _raw_stream(stream, dev))
    if code:
        _check(code, "tt_append_ctx_q8")


def tt_quantize_rows_i8(rows: int, K: int, x, q, scale, stream=None) -> None:
    """int8 codes q [rows, K] and float32 scales [rows] of bf16 x [rows, K]
    (weights: a row per output channel)."""
    dev = _device()
    code = lib().tt_quantize_rows_i8(
        rows, K, _arg(x, "x", 2 * rows * K, dev), _arg(q, "q", rows * K, dev),
        _arg(scale, "scale", 4 * rows, dev), _raw_stream(stream, dev))
    if code:
        _check(code, "tt_quantize_rows_i8")


def tt_linear_i8_workspace_bytes(rows: int, N: int, K: int) -> int:
    n = lib().tt_linear_i8_workspace_bytes(int(rows), int(N), int(K))
    if n == 0:
        raise TTError(1, "tt_linear_i8_workspace_bytes", tt_last_error())
    return int(n)


def linear_i8_workspace(rows: int, N: int, K: int, device="cuda"):
    """A torch uint8 device buffer of tt_linear_i8_workspace_bytes(rows, N, K) bytes."""
    import torch
    return torch.empty(tt_linear_i8_workspace_bytes(rows, N, K), dtype=torch.uint8, device=device)


def tt_linear_i8(rows: int, N: int, K: int, x, w_q, w_scale, out, ws, stream=None) -> None:
    """out [rows, N] = bf16(x [rows, K] . (w_q * w_scale)^T), x quantised per
    row to int8, the sums exact in 32-bit integers."""
    dev = _device()
    code = lib().tt_linear_i8(
        rows, N, K, _arg(x, "x", 2 * rows * K, dev), _arg(w_q, "w_q", N * K, dev),
        _arg(w_scale, "w_scale", 4 * N, dev), _arg(out, "out", 2 * rows * N, dev),
        _arg(ws, "ws", 0, dev), _nbytes(ws), _raw_stream(stream, dev))
    if code:
        _check(code, "tt_linear_i8")


def tt_vocab_confidence_commit_i8(d: Dims, y, w_q, w_scale, gamma: float, logit_scale: float,
                                  tokens, masked, conf_out, argmax_out, n_committed, ws,
                                  stream=None) -> None:
    """tt_vocab_confidence_commit with int8 weights w_q [V, H], one float32
    scale per token, and y quantised per row."""
    B, H, V = d.B, d.H, d.V
    rows, dev = B * d.S, _device()
    code = lib().tt_vocab_confidence_commit_i8(
        d, _arg(y, "y", 2 * rows * H, dev), _arg(w_q, "w_q", V * H, dev),
        _arg(w_scale, "w_scale", 4 * V, dev), gamma, logit_scale,
        _arg(tokens, "tokens", 4 * rows, dev), _arg(masked, "masked", rows, dev),
        _arg(conf_out, "conf_out", 4 * rows, dev), _arg(argmax_out, "argmax_out", 4 * rows, dev),
        _arg(n_committed, "n_committed", 4 * B, dev), _arg(ws, "ws", 0, dev), _nbytes(ws),
        _raw_stream(stream, dev))
    if code:
        _check(code, "tt_vocab_confidence_commit_i8")
