"""Binding of a recurrent block's other operators: the gated linear recurrence,
the gated feed-forward block and dropout, with their gradients (C ABI in
include/nrnn.h).

Argument marshalling only, as in the rest of the binding."""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._binding import _cu_device, _device_tensor, _space, load
from ._language import _at, _like, _result, _run, _storage, _with

RECURRENCE_ORDER = ("rate", "b_a", "b_i")


def _rows(t, rows: int, d: int, like: torch.Tensor, what: str):
    """A float32 (rows, d) tensor of states on the call's device, or None."""
    if t is None:
        return None
    t = _device_tensor(t, what)
    if tuple(t.shape) != (rows, d) or t.dtype != torch.float32 or t.device != like.device:
        raise ValueError(f"{what} must be float32 of shape {(rows, d)} on {like.device}")
    return t


def _recurrence_params(params, d: int, device) -> torch.Tensor:
    """(3, d) fp32 device tensor from a dict (rate, b_a, b_i) or a tensor."""
    if isinstance(params, torch.Tensor):   # as a decode step has them: nothing to do
        if params.dtype == torch.float32 and params.device == device and params.shape == (3, d) \
                and params.is_contiguous():
            return params
    elif isinstance(params, dict):
        params = torch.stack([torch.as_tensor(params[k]).to(device, torch.float32).reshape(-1)
                              for k in RECURRENCE_ORDER])
    params = torch.as_tensor(params)
    if tuple(params.shape) != (3, d):
        raise ValueError(f"params must have shape (3, {d}), got {tuple(params.shape)}")
    return params.to(device, torch.float32).contiguous()


def _recurrence_args(preact, params, cu_seqlens):
    preact = _device_tensor(preact, "preact")
    if preact.dim() != 3 or preact.shape[2] % 3:
        raise ValueError("preact must have shape (B, T, 3 d_h)")
    B, T, d = preact.shape[0], preact.shape[1], preact.shape[2] // 3
    code = _storage(preact)
    prm = _recurrence_params(params, d, preact.device)
    cu, S = _cu_device(cu_seqlens, B, T, preact.device)
    return preact, code, prm, B, T, d, cu, S


def _recurrence_space(workspace, B, T, d, code, S, backward, device):
    nbytes = load().nrnn_linear_recurrence_workspace_bytes(B, T, d, code, S, backward)
    if nbytes == 0:
        raise ValueError("invalid shape")
    return _space(workspace, nbytes, device), nbytes


def linear_recurrence(preact: torch.Tensor, params, cu_seqlens=None, state: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Gated linear recurrence over preact (B, T, 3 d_h), blocks [a | i | v] (what
    input_projection gives), float32/bfloat16:

        r = sig(P_a + b_a);  a = exp(-rate r);  i = sig(P_i + b_i)
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t v_t

    params: float32 (3, d_h), rows rate (>= 0), b_a, b_i, or a dict of them.
    cu_seqlens: a pack (B = 1), as newton_forward takes it.  state: float32 (B,
    d_h), for a pack one row per segment: the states before the first step
    (None: zeros).  Returns (H (B, T, d_h) in preact's dtype, the last states as
    float32, which a later call or linear_recurrence_step continues from)."""
    preact, code, prm, B, T, d, cu, S = _recurrence_args(preact, params, cu_seqlens)
    rows = S if cu is not None else B
    state = _rows(state, rows, d, preact, "state")
    H = _result(out, (B, T, d), preact, "out")
    last = torch.empty((rows, d), dtype=torch.float32, device=preact.device)
    ws, nbytes = _recurrence_space(workspace, B, T, d, code, S, 0, preact.device)
    _run("linear_recurrence", load().nrnn_linear_recurrence_forward, preact, preact.data_ptr(), code,
         prm.data_ptr(), B, T, d, _at(cu), S, _at(state), H.data_ptr(), last.data_ptr(), ws.data_ptr(), nbytes)
    return H, last


class LinearRecurrenceGrads(NamedTuple):
    gP: torch.Tensor
    gparams: torch.Tensor
    g_state: torch.Tensor | None


def linear_recurrence_backward(preact: torch.Tensor, params, H: torch.Tensor, gH: torch.Tensor,
                               cu_seqlens=None, state: torch.Tensor | None = None,
                               g_state: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None) -> LinearRecurrenceGrads:
    """Gradients of linear_recurrence() at its stored H, from gH = dL/dH and
    g_state = dL/d(last states), float32 (None: they took no part).  Returns (gP
    in preact's dtype, gparams (3, d_h) float32, dL/dstate float32 or None where
    no state was given)."""
    preact, code, prm, B, T, d, cu, S = _recurrence_args(preact, params, cu_seqlens)
    rows = S if cu is not None else B
    state, g_last = _rows(state, rows, d, preact, "state"), _rows(g_state, rows, d, preact, "g_state")
    both = []
    for t, what in ((H, "H"), (gH, "gH")):
        t = _device_tensor(t, what)
        if tuple(t.shape) != (B, T, d) or t.dtype != preact.dtype or t.device != preact.device:
            raise ValueError(f"{what} must be (B, T, d_h) in preact's dtype and on its device")
        both.append(t)
    gP = torch.empty_like(preact)
    gparams = torch.empty((3, d), dtype=torch.float32, device=preact.device)
    g0 = None if state is None else torch.empty_like(state)
    ws, nbytes = _recurrence_space(workspace, B, T, d, code, S, 1, preact.device)
    _run("linear_recurrence_backward", load().nrnn_linear_recurrence_backward, preact, preact.data_ptr(), code,
         prm.data_ptr(), B, T, d, _at(cu), S, _at(state), both[0].data_ptr(), both[1].data_ptr(), _at(g_last),
         gP.data_ptr(), gparams.data_ptr(), _at(g0), ws.data_ptr(), nbytes)
    return LinearRecurrenceGrads(gP, gparams, g0)


def linear_recurrence_step(params, state: torch.Tensor | None, preact: torch.Tensor,
                           out: torch.Tensor | None = None, state_out: torch.Tensor | None = None):
    """One step per slot: preact (slots, 3 d_h), state float32 (slots, d_h) (None:
    zeros).  Returns (h (slots, d_h) in preact's dtype, the new state as float32);
    state_out may be state."""
    preact = _device_tensor(preact, "preact")
    if preact.dim() != 2 or preact.shape[1] % 3:
        raise ValueError("preact must have shape (slots, 3 d_h)")
    slots, d = preact.shape
    d //= 3
    code = _storage(preact)
    prm = _recurrence_params(params, d, preact.device)
    state = _rows(state, slots, d, preact, "state")
    h = _result(out, (slots, d), preact, "out")
    if state_out is None:
        state_out = torch.empty((slots, d), dtype=torch.float32, device=preact.device) if state is None \
            else torch.empty_like(state)
    elif state_out.dtype != torch.float32 or state_out.shape != h.shape \
            or state_out.device != preact.device or not state_out.is_contiguous():
        raise ValueError(f"state_out must be a contiguous float32 {(slots, d)} tensor on {preact.device}")
    _run("linear_recurrence_step", load().nrnn_linear_recurrence_step, preact, preact.data_ptr(), code,
         prm.data_ptr(), slots, d, _at(state), h.data_ptr(), state_out.data_ptr())
    return h, state_out


def _mlp_args(x, W_in, W_out):
    x, W_in, W_out = _device_tensor(x, "x"), _device_tensor(W_in, "W_in"), _device_tensor(W_out, "W_out")
    if x.dim() < 1 or W_out.dim() != 2:
        raise ValueError("x must have shape (..., d), W_in (2 f, d) and W_out (d, f)")
    d, f = W_out.shape
    if x.shape[-1] != d or W_in.shape != (2 * f, d):
        raise ValueError("x must have shape (..., d), W_in (2 f, d) and W_out (d, f)")
    if x.dtype != W_in.dtype or x.dtype != W_out.dtype:
        raise TypeError("x, W_in and W_out must share a dtype")
    _with(x, W_in, "W_in")
    _with(x, W_out, "W_out")
    if d == 0 or f == 0:
        raise ValueError("d and f must be positive")
    return x, W_in, W_out, _storage(x), x.numel() // d, d, f


def gated_mlp(x: torch.Tensor, W_in: torch.Tensor, W_out: torch.Tensor, keep: bool = False,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Gated feed-forward block y = (silu(x Wg^T) * (x Wu^T)) W_out^T: x (..., d),
    W_in (2 f, d) = the rows of Wg, then those of Wu, W_out (d, f), float32 or
    bfloat16.  keep=True returns (y, kept): an opaque tensor that
    gated_mlp_backward takes.

    bfloat16 rounds silu(a) b once between the products, and y: 1.41 times as far off
    as rounding the exact y.  Calls of at most 16 rows leave the first rounding out, so
    y of a decode step's row may differ by it from the same row of a longer call."""
    x, W_in, W_out, code, rows, d, f = _mlp_args(x, W_in, W_out)
    lib = load()
    y = torch.empty_like(x) if out is None else _result(out, x.shape, x, "out")
    nbytes = lib.nrnn_gated_mlp_workspace_bytes(rows, d, f, code, 2 if keep else 0)
    kept = None
    if keep:
        kept = torch.empty(lib.nrnn_gated_mlp_kept_bytes(rows, f, code), dtype=torch.uint8, device=x.device)
    ws = _space(workspace, nbytes, x.device)
    _run("gated_mlp", lib.nrnn_gated_mlp_forward, x, x.data_ptr(), W_in.data_ptr(), W_out.data_ptr(), code,
         rows, d, f, y.data_ptr(), _at(kept), ws.data_ptr(), nbytes)
    return (y, kept) if keep else y


def gated_mlp_backward(x: torch.Tensor, W_in: torch.Tensor, W_out: torch.Tensor, kept: torch.Tensor,
                       g: torch.Tensor, workspace: torch.Tensor | None = None):
    """(dL/dx, dL/dW_in, dL/dW_out) of gated_mlp() in x's dtype, from what it kept
    for the same x and weights and g = dL/dy.  bfloat16 rounds dL/da, dL/db and silu(a) b
    once before their products (not of at most 16 rows), and the results: 1.41 times as
    far off as rounding the exact gradients."""
    x, W_in, W_out, code, rows, d, f = _mlp_args(x, W_in, W_out)
    g = _like(g, x, "g")
    lib = load()
    if not isinstance(kept, torch.Tensor) or kept.dtype != torch.uint8 or kept.device != x.device \
            or kept.dim() != 1 or not kept.is_contiguous() \
            or kept.numel() != lib.nrnn_gated_mlp_kept_bytes(rows, f, code):
        raise ValueError("kept must be what gated_mlp(keep=True) returned for this x and these weights")
    nbytes = lib.nrnn_gated_mlp_workspace_bytes(rows, d, f, code, 1)
    gx, gW_in, gW_out = torch.empty_like(x), torch.empty_like(W_in), torch.empty_like(W_out)
    ws = _space(workspace, nbytes, x.device)
    _run("gated_mlp_backward", lib.nrnn_gated_mlp_backward, x, x.data_ptr(), W_in.data_ptr(), W_out.data_ptr(),
         kept.data_ptr(), g.data_ptr(), code, rows, d, f, gx.data_ptr(), gW_in.data_ptr(), gW_out.data_ptr(),
         ws.data_ptr(), nbytes)
    return gx, gW_in, gW_out


def dropout(x: torch.Tensor, p: float, seed, offset: int = 0, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """residual + x * keep / (1 - p) with a mask that is made from (seed, offset)
    and an element's place, never stored: the gradient with respect to x is the
    same call on the gradient, without residual.  seed: an int of 64 bits, or an
    int64 CUDA tensor of one element, read when the kernel runs (a captured graph
    draws another mask once it changes).  offset: an int of 64 bits, to tell apart
    the layers and steps of one seed.  out may be x or residual."""
    x = _device_tensor(x, "x")
    residual = _like(residual, x, "residual")
    code = _storage(x)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be between 0 and 1")
    at = None
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != x.device:
            raise ValueError(f"a seed tensor must be int64, of one element and on {x.device}")
        at, seed = seed.data_ptr(), 0
    y = torch.empty_like(x) if out is None else _result(out, x.shape, x, "out")
    _run("dropout", load().nrnn_dropout, x, x.data_ptr(), code, x.numel(), float(p), int(seed) & (1 << 64) - 1,
         at, int(offset) & (1 << 64) - 1, _at(residual), y.data_ptr())
    return y
