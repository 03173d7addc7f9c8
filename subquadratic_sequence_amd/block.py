"""ctypes binding of the operators around the long convolution in a block: the
gated linear recurrence, the gated feed-forward block and the group norm (argument marshalling and checks only; the computation
is in libhyena.so).

Tensors are on one GPU, which need not be the current one; work goes to that
GPU's current stream, where workspaces are allocated too.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from .hyena import ACT_NONE, ACT_SILU, GlrInputs, HyenaError, _check, _dtype_code, lib

# A decoding step is a few microseconds of GPU time, so what a call costs on the
# host counts: addresses are passed as plain integers, workspace sizes are
# remembered, and the current GPU is only switched where it has to be.
_NO_SWITCH = contextlib.nullcontext()


def _p(t):
    return None if t is None else t.data_ptr()


def _on(first, *tensors):
    """(a context that makes the tensors' GPU current, that GPU's current stream); all
    tensors have to be on one GPU."""
    dev = first.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not {dev}")
    guard = _NO_SWITCH if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    return guard, torch._C._cuda_getCurrentRawStream(dev.index)


@functools.lru_cache(maxsize=1024)
def _need(query, *sizes):
    """Bytes of a workspace; sizes outside the supported range raise."""
    n = getattr(lib(), query)(*sizes)
    if n == 0:
        raise HyenaError(2, query)
    return n


def _scratch(ws, like, query, *sizes):
    """The workspace of a call: the caller's, or a new one."""
    need = _need(query, *sizes)
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    if ws.device != like.device:
        raise ValueError(f"workspace on {ws.device}, tensors on {like.device}")
    if not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return ws


def _nbytes(t):
    return t.numel() * t.element_size()


def _tensor(t, name, shape, dtype):
    """A contiguous tensor of this shape and dtype, or None."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, dtype):
    """Strides of a tensor with contiguous rows, in elements, without its last
    dimension (0 for dimensions of size 1)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if 1 in shape:
        return [s if n > 1 else 0 for s, n in zip(strides[:-1], shape)]
    return strides[:-1]


# ------------------------------------------------- gated linear recurrence


def hyena_glr_workspace_bytes(B, L, D, dtype) -> int:
    return lib().hyena_glr_workspace_bytes(B, L, D, dtype)


def hyena_glr_bwd_workspace_bytes(B, L, D, dtype) -> int:
    return lib().hyena_glr_bwd_workspace_bytes(B, L, D, dtype)


def _glr_inputs(v, f, g, bias, h0, reset, lens, pad_zero):
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v: expected a tensor [B, L, D]")
    shape, dtype = v.shape, v.dtype
    B, L, D = shape
    dt = _dtype_code(v)
    sv, sf = _rows(v, "v", shape, dtype), _rows(f, "f", shape, dtype)
    sg = (0, 0) if g is None else _rows(g, "g", shape, dtype)
    _tensor(bias, "bias", (D,), torch.float32)
    _tensor(h0, "h0", (B, D), torch.float32)
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _tensor(reset, "reset", (B, L), torch.uint8)
    _tensor(lens, "lens", (B,), torch.int32)
    return GlrInputs(B, L, D, dt, _p(v), _p(f), _p(g), *sv, *sf, *sg, _p(bias), _p(h0), _p(reset), _p(lens),
                     pad_zero)


def hyena_glr_fwd(v, f, g=None, bias=None, h0=None, reset=None, lens=None, y=None, h_last=None, ws=None):
    """y_t = h_t silu(g_t) with h_t = a_t h_{t-1} + (1 - a_t) v_t, a = sigmoid(f + bias).

    v, f, g, y [B, L, D] (float32 or bfloat16, contiguous rows: column blocks of one
    tensor are fine); bias [D], h0 and h_last [B, D] float32; reset [B, L] uint8 or
    bool; lens [B] int32. The state after the last position goes to h_last, if
    given (not h0 itself). Positions behind lens are left as they are in a given y, zero otherwise."""
    c = _glr_inputs(v, f, g, bias, h0, reset, lens, y is None)
    if y is not None:
        sy = _rows(y, "y", v.shape, v.dtype)
    _tensor(h_last, "h_last", (c.B, c.D), torch.float32)
    # other workgroups still read the old state and rows when the first ones write
    if h_last is not None and h_last.data_ptr() == c.h0:
        raise ValueError("h_last may not be h0")
    if y is not None and y.data_ptr() in (c.v, c.f, c.g):
        raise ValueError("y may not be v, f or g")
    guard, stream = _on(v, f, g, bias, h0, reset, lens, y, h_last)
    with guard:
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            sy = y.stride()[:-1]
        ws = _scratch(ws, v, "hyena_glr_workspace_bytes", c.B, c.L, c.D, c.dtype)
        _check(lib().hyena_glr_fwd(ctypes.byref(c), _p(y), *sy, _p(h_last), _p(ws), _nbytes(ws), stream),
               "hyena_glr_fwd")
    return y


def hyena_glr_bwd(v, f, dy, g=None, bias=None, h0=None, reset=None, lens=None, dh_last=None, dp=None, ws=None):
    """Gradients of sum(dy * y) + sum(dh_last * h_last) of hyena_glr_fwd: a dict with
    dv, df (and dg, if g is given; dtype of v), dbias [D] and dh0 [B, D] (float32).
    dv, df, dg are the column blocks of one tensor dp [B, L, 3D] (2D without g), in
    the dict too: the gradient of the projection that v, f, g come from."""
    c = _glr_inputs(v, f, g, bias, h0, reset, lens, False)
    B, L, D = v.shape
    n = 2 if g is None else 3
    sdy = _rows(dy, "dy", v.shape, v.dtype)
    _tensor(dh_last, "dh_last", (B, D), torch.float32)
    _tensor(dp, "dp", (B, L, n * D), v.dtype)
    guard, stream = _on(v, f, g, bias, h0, reset, lens, dy, dh_last, dp)
    with guard:
        if dp is None:
            dp = torch.empty(B, L, n * D, dtype=v.dtype, device=v.device)
        out = dict(dp=dp, dv=dp[..., :D], df=dp[..., D:2 * D], dbias=torch.empty(D, device=v.device),
                   dh0=torch.empty(B, D, device=v.device))
        if g is not None:
            out["dg"] = dp[..., 2 * D:]
        ws = _scratch(ws, v, "hyena_glr_bwd_workspace_bytes", B, L, D, c.dtype)
        _check(lib().hyena_glr_bwd(ctypes.byref(c), _p(dy), *sdy, _p(dh_last), _p(out["dv"]), _p(out["df"]),
                                   _p(out.get("dg")), L * n * D, n * D, _p(out["dbias"]), _p(out["dh0"]), _p(ws),
                                   _nbytes(ws), stream), "hyena_glr_bwd")
    return out


def hyena_glr_step(state, v, f, g=None, bias=None, slots=None, state_out=None, y=None):
    """One position of B sequences: v, f, g, y [B, D]; state [S, D] float32, advanced
    in place or into state_out (only the rows of state it advances). slots [B] int32: the
    row of state of each sequence (default: row r); rows with a slot outside [0, S) are skipped (zero in a new y),
    rows that share a slot are consecutive positions of one sequence."""
    if not isinstance(v, torch.Tensor) or v.dim() != 2:
        raise ValueError("v: expected a tensor [B, D]")
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state: expected a tensor [S, D]")
    shape, dtype = v.shape, v.dtype
    B, D = shape
    S = state.shape[0]
    dt = _dtype_code(v)
    _tensor(state, "state", (S, D), torch.float32)
    _tensor(state_out, "state_out", (S, D), torch.float32)
    _tensor(bias, "bias", (D,), torch.float32)
    _tensor(slots, "slots", (B,), torch.int32)
    sv, sf = _rows(v, "v", shape, dtype), _rows(f, "f", shape, dtype)
    sg = (0,) if g is None else _rows(g, "g", shape, dtype)
    pad_zero = y is None
    if y is not None:
        sy = _rows(y, "y", shape, dtype)
    if state_out is None:
        state_out = state
    guard, stream = _on(v, f, g, bias, slots, state, state_out, y)
    with guard:
        if y is None:
            y = torch.empty(B, D, dtype=dtype, device=v.device)
            sy = (D,)
        _check(lib().hyena_glr_step(B, D, S, dt, _p(v), *sv, _p(f), *sf, _p(g), *sg, _p(bias), _p(slots), _p(state),
                                    _p(state_out), _p(y), *sy, pad_zero, stream), "hyena_glr_step")
    return y


# ---------------------------------------------- gated feed-forward block


def hyena_ffn_workspace_bytes(M, D, F, dtype) -> int:
    return lib().hyena_ffn_workspace_bytes(M, D, F, dtype)


def hyena_ffn_bwd_workspace_bytes(M, D, F, dtype) -> int:
    return lib().hyena_ffn_bwd_workspace_bytes(M, D, F, dtype)


def _ffn_shape(x, w_in, w_out):
    """(M, D, F) of x [..., D]: its leading dimensions are M rows."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a tensor [..., D]")
    if not isinstance(w_out, torch.Tensor) or w_out.dim() != 2:
        raise ValueError("w_out: expected a tensor [F, D]")
    D, F = x.shape[-1], w_out.shape[0]
    M = 1
    for n in x.shape[:-1]:
        M *= n
    _tensor(x, "x", x.shape, x.dtype)
    _tensor(w_out, "w_out", (F, D), x.dtype)
    if w_in is None:
        raise TypeError("w_in: expected a torch tensor")
    _tensor(w_in, "w_in", (D, 2 * F), x.dtype)
    return M, D, F


def hyena_ffn_fwd(x, w_in, w_out, act=ACT_SILU, y=None, ws=None):
    """y = (p * act(q)) w_out with (p, q) = x w_in: x, y [..., D], w_in [D, 2F] (the
    columns of p, then those of q), w_out [F, D], all float32 or bfloat16."""
    M, D, F = _ffn_shape(x, w_in, w_out)
    dt = _dtype_code(x)
    _tensor(y, "y", x.shape, x.dtype)
    guard, stream = _on(x, w_in, w_out, y)
    with guard:
        if y is None:
            y = torch.empty_like(x)
        ws = _scratch(ws, x, "hyena_ffn_workspace_bytes", M, D, F, dt)
        _check(lib().hyena_ffn_fwd(M, D, F, dt, act, _p(x), _p(w_in), _p(w_out), _p(y), _p(ws), _nbytes(ws),
                                   stream), "hyena_ffn_fwd")
    return y


def hyena_ffn_bwd(x, w_in, w_out, dy, act=ACT_SILU, ws=None):
    """Gradients of sum(dy * y), y = hyena_ffn_fwd(x, w_in, w_out, act): a dict with dx,
    dw_in, dw_out (shapes and dtype of x, w_in, w_out)."""
    M, D, F = _ffn_shape(x, w_in, w_out)
    dt = _dtype_code(x)
    if dy is None:
        raise TypeError("dy: expected a torch tensor")
    _tensor(dy, "dy", x.shape, x.dtype)
    guard, stream = _on(x, w_in, w_out, dy)
    with guard:
        g = dict(dx=torch.empty_like(x), dw_in=torch.empty_like(w_in), dw_out=torch.empty_like(w_out))
        ws = _scratch(ws, x, "hyena_ffn_bwd_workspace_bytes", M, D, F, dt)
        _check(lib().hyena_ffn_bwd(M, D, F, dt, act, _p(x), _p(w_in), _p(w_out), _p(dy), _p(g["dx"]), _p(g["dw_in"]),
                                   _p(g["dw_out"]), _p(ws), _nbytes(ws), stream), "hyena_ffn_bwd")
    return g


# ------------------------------------------------ group norm, channels last


def hyena_group_norm_workspace_bytes(B, S, C, G, dtype) -> int:
    return lib().hyena_group_norm_workspace_bytes(B, S, C, G, dtype)


def hyena_group_norm_bwd_workspace_bytes(B, S, C, G, dtype) -> int:
    return lib().hyena_group_norm_bwd_workspace_bytes(B, S, C, G, dtype)


def _norm_shape(x):
    """(B, S, C) of x [B, ..., C]; two dimensions are rows by themselves (S = 1)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x: expected a tensor [B, ..., C]")
    S = 1
    for n in x.shape[1:-1]:
        S *= n
    return x.shape[0], S, x.shape[-1]


def hyena_group_norm_fwd(x, groups, gamma=None, beta=None, eps=1e-5, act=ACT_NONE, lens=None, y=None, mean=None,
                         rstd=None, ws=None):
    """y = act(gamma (x - mean) rstd + beta) for x [B, ..., C] (channels last; float32 or
    bfloat16), mean and rstd over the positions of a sample and the C / groups
    channels of a group. gamma, beta [C] float32; lens [B] int32: positions in use;
    mean, rstd [B, groups] float32 receive the statistics (the backward takes them).
    y may be x. Positions behind lens are left as they are in a given y, zero otherwise."""
    B, S, C = _norm_shape(x)
    dt = _dtype_code(x)
    _tensor(x, "x", x.shape, x.dtype)
    _tensor(gamma, "gamma", (C,), torch.float32)
    _tensor(beta, "beta", (C,), torch.float32)
    _tensor(lens, "lens", (B,), torch.int32)
    _tensor(y, "y", x.shape, x.dtype)
    _tensor(mean, "mean", (B, groups), torch.float32)
    _tensor(rstd, "rstd", (B, groups), torch.float32)
    guard, stream = _on(x, gamma, beta, lens, y, mean, rstd)
    pad_zero = False
    with guard:
        if y is None:
            y, pad_zero = torch.empty_like(x), True
        ws = _scratch(ws, x, "hyena_group_norm_workspace_bytes", B, S, C, groups, dt)
        _check(lib().hyena_group_norm_fwd(B, S, C, groups, dt, act, eps, _p(x), _p(gamma), _p(beta), _p(lens), pad_zero,
                                          _p(y), _p(mean), _p(rstd), _p(ws), _nbytes(ws), stream),
               "hyena_group_norm_fwd")
    return y


def hyena_group_norm_bwd(x, dy, groups, mean, rstd, gamma=None, beta=None, act=ACT_NONE, lens=None, dx=None, ws=None):
    """Gradients of sum(dy * y), y = hyena_group_norm_fwd(x, ...), mean and rstd as it
    wrote them: a dict with dx (dtype of x, zero behind lens; dx may be dy) and
    dgamma, dbeta [C] float32 (also where gamma or beta were left out)."""
    B, S, C = _norm_shape(x)
    dt = _dtype_code(x)
    _tensor(x, "x", x.shape, x.dtype)
    _tensor(dy, "dy", x.shape, x.dtype)
    _tensor(gamma, "gamma", (C,), torch.float32)
    _tensor(beta, "beta", (C,), torch.float32)
    _tensor(lens, "lens", (B,), torch.int32)
    _tensor(dx, "dx", x.shape, x.dtype)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            raise ValueError(f"{name}: the forward's statistics are needed")
        _tensor(t, name, (B, groups), torch.float32)
    guard, stream = _on(x, dy, gamma, beta, lens, mean, rstd, dx)
    with guard:
        d = torch.empty(2, C, device=x.device)  # neighbours: their sums take one launch
        out = dict(dx=torch.empty_like(x) if dx is None else dx, dgamma=d[0], dbeta=d[1])
        ws = _scratch(ws, x, "hyena_group_norm_bwd_workspace_bytes", B, S, C, groups, dt)
        _check(lib().hyena_group_norm_bwd(B, S, C, groups, dt, act, _p(x), _p(dy), _p(gamma), _p(beta), _p(lens),
                                          _p(mean), _p(rstd), _p(out["dx"]), _p(out["dgamma"]), _p(out["dbeta"]),
                                          _p(ws), _nbytes(ws), stream), "hyena_group_norm_bwd")
    return out
