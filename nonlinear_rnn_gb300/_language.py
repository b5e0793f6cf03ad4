"""Binding of the operators of a language model around the recurrent layer:
the embedding lookup, the norms around a block and the cross entropy over the
vocabulary, with their gradients (C ABI in include/nrnn.h).

Argument marshalling only, as in the rest of the binding."""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._binding import BF16, F32, OK, _device_tensor, _raise, _space, load

I32, I64 = 0, 1


# A decode step's calls take a few microseconds on the GPU, so this path is kept
# short: the device is switched only if it has to be, and the stream is read
# without making a Stream object (together 3 us a call).
_INDEX_TYPES = {torch.int32: I32, torch.int64: I64}
_STORAGE_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _run(what: str, fn, t: torch.Tensor, *args) -> None:
    """fn(*args, stream) on t's device and that device's current stream."""
    index = t.get_device()
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != OK:
        _raise(st, what)


def _ids(t: torch.Tensor, what: str) -> tuple[torch.Tensor, int]:
    t = _device_tensor(t, what)
    kind = _INDEX_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")
    return t, kind


def _storage(t: torch.Tensor) -> int:
    code = _STORAGE_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return code


def _with(first: torch.Tensor, t: torch.Tensor, what: str) -> None:
    if t.device != first.device:
        raise ValueError(f"{what} must be on {first.device}, got {t.device}")


def _at(t) -> int | None:
    return None if t is None else t.data_ptr()


def _result(out, shape, like: torch.Tensor, what: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(out.shape) != tuple(shape) or out.dtype != like.dtype or out.device != like.device \
            or not out.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} tensor of {like.dtype} on {like.device}")
    return out


def embedding(ids: torch.Tensor, W: torch.Tensor, scale: float = 1.0,
              padding_idx: int | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * W[ids]: ids (...) int32/int64, W (V, d) -> (..., d) in W's dtype.
    Rows of padding_idx are zeros; an id outside [0, V) gives a row of NaN
    (nothing synchronises to raise)."""
    ids, ids_type = _ids(ids, "ids")
    W = _device_tensor(W, "W")
    if W.dim() != 2:
        raise ValueError("W must have shape (V, d)")
    _with(ids, W, "W")
    V, d = W.shape
    code = _storage(W)
    rows = _result(out, (*ids.shape, d), W, "out")
    _run("embedding", load().nrnn_embedding, W, ids.data_ptr(), ids_type, W.data_ptr(), code,
         ids.numel(), V, d, -1 if padding_idx is None else padding_idx, scale, rows.data_ptr())
    return rows


def embedding_backward(ids: torch.Tensor, g: torch.Tensor, num_rows: int, scale: float = 1.0,
                       padding_idx: int | None = None, out: torch.Tensor | None = None,
                       accumulate: bool = False, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dL/dW (num_rows, d) of embedding() from g = dL/drows (..., d), in g's
    dtype: fp32 sums in an order fixed by the ids.  With accumulate=True the
    sums are added to `out` (a weight shared with the vocabulary loss)."""
    ids, ids_type = _ids(ids, "ids")
    g = _device_tensor(g, "g")
    if g.dim() < 1 or tuple(g.shape[:-1]) != tuple(ids.shape):
        raise ValueError("g must have shape (*ids.shape, d)")
    _with(ids, g, "g")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    n, d, V = ids.numel(), g.shape[-1], int(num_rows)
    code = _storage(g)
    lib = load()
    nbytes = lib.nrnn_embedding_backward_workspace_bytes(n, V, d)
    if nbytes == 0:
        raise ValueError("num_rows and the width of g must be positive (and fit the library's limits)")
    gW = _result(out, (V, d), g, "out")
    ws = _space(workspace, nbytes, g.device)
    _run("embedding_backward", lib.nrnn_embedding_backward, g, ids.data_ptr(), ids_type, g.data_ptr(),
         code, n, V, d, -1 if padding_idx is None else padding_idx, scale, accumulate,
         gW.data_ptr(), ws.data_ptr(), nbytes)
    return gW


def _weight(t, d: int, x: torch.Tensor, what: str):
    if t is None:
        return None
    t = _device_tensor(t, what)
    if t.dim() != 1 or t.shape[0] != d or t.dtype != torch.float32 or t.device != x.device:
        raise ValueError(f"{what} must be a float32 vector of {d} values on {x.device}")
    return t


def _like(t, x: torch.Tensor, what: str):
    if t is None:
        return None
    t = _device_tensor(t, what)
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{what} must match x in shape, dtype and device")
    return t


def block_norm(x: torch.Tensor, h: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               w_post: torch.Tensor | None = None, scale: torch.Tensor | None = None,
               w_pre: torch.Tensor | None = None, eps: float = 1e-6, next_norm: bool = True,
               out: torch.Tensor | None = None):
    """The norms around a block with its gate and residual scale, in one pass:

        x_out = x + scale * (norm(h) * w_post * silu(gate));  u = norm(x_out) * w_pre

    with norm(v) = v / sqrt(mean(v^2) + eps) over the last axis.  x, h, gate
    (..., d); w_post, scale, w_pre float32 (d), None = ones; gate None: no gate.
    Returns (x_out, u).  h None: the norm before the first block, x_out is x.
    next_norm=False: the last block, u is None.  out (with h): x_out's tensor, may be x."""
    x = _device_tensor(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have shape (..., d)")
    d = x.shape[-1]
    if h is None and (gate is not None or not next_norm):
        raise ValueError("without h there is no gate, and u is the only result")
    h, gate = _like(h, x, "h"), _like(gate, x, "gate")
    w_post, scale = _weight(w_post, d, x, "w_post"), _weight(scale, d, x, "scale")
    w_pre = _weight(w_pre, d, x, "w_pre")
    if h is None and out is not None and out is not x:
        raise ValueError("without h x_out is x: there is nothing for out")
    code = _storage(x)
    x_out = x if h is None else torch.empty_like(x) if out is None else _result(out, x.shape, x, "out")
    u = torch.empty_like(x) if next_norm else None
    _run("block_norm", load().nrnn_block_norm_forward, x, x.data_ptr(), _at(h), _at(gate), _at(w_post),
         _at(scale), _at(w_pre), code, x.numel() // d if d else 0, d, eps,
         None if h is None else x_out.data_ptr(), _at(u))
    return x_out, u


class BlockNormGrads(NamedTuple):
    gx: torch.Tensor
    gh: torch.Tensor | None
    g_gate: torch.Tensor | None
    gw_post: torch.Tensor | None
    g_scale: torch.Tensor | None
    gw_pre: torch.Tensor | None


def block_norm_backward(x_out: torch.Tensor, h: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                        scale: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                        g_x: torch.Tensor | None = None, g_u: torch.Tensor | None = None,
                        eps: float = 1e-6, workspace: torch.Tensor | None = None) -> BlockNormGrads:
    """Gradients of block_norm() at its stored x_out (h None: x), from g_x =
    dL/dx_out (None: zeros) and g_u = dL/du (None: u took no part).  The
    weights' gradients are float32; those of parts that took no part are None."""
    x_out = _device_tensor(x_out, "x_out")
    if x_out.dim() < 1:
        raise ValueError("x_out must have shape (..., d)")
    d = x_out.shape[-1]
    if g_x is None and g_u is None:
        raise ValueError("give g_x, g_u or both")
    if h is None and (gate is not None or g_u is None):
        raise ValueError("without h there is no gate, and u is the only result")
    h, gate = _like(h, x_out, "h"), _like(gate, x_out, "gate")
    g_x, g_u = _like(g_x, x_out, "g_x"), _like(g_u, x_out, "g_u")
    w_post, scale = _weight(w_post, d, x_out, "w_post"), _weight(scale, d, x_out, "scale")
    w_pre = _weight(w_pre, d, x_out, "w_pre")
    code = _storage(x_out)
    rows = x_out.numel() // d if d else 0
    lib = load()
    nbytes = lib.nrnn_block_norm_backward_workspace_bytes(rows, d)
    if nbytes == 0:
        raise TypeError(f"block_norm_backward: unsupported width {d}")
    dev = x_out.device
    sums = torch.empty((3, d), dtype=torch.float32, device=dev)
    gx = torch.empty_like(x_out)
    gh = None if h is None else torch.empty_like(x_out)
    g_gate = None if gate is None else torch.empty_like(x_out)
    ws = _space(workspace, nbytes, dev)
    at = sums.data_ptr()
    _run("block_norm_backward", lib.nrnn_block_norm_backward, x_out, x_out.data_ptr(), _at(h),
         _at(gate), _at(w_post), _at(scale), _at(w_pre), _at(g_x), _at(g_u), code, rows, d, eps,
         gx.data_ptr(), _at(gh), _at(g_gate), at, at + 4 * d, at + 8 * d, ws.data_ptr(), nbytes)
    return BlockNormGrads(gx, gh, g_gate, None if h is None else sums[0],
                          None if h is None else sums[1], None if g_u is None else sums[2])


def _vocab_args(x, W, targets):
    x, W = _device_tensor(x, "x"), _device_tensor(W, "W")
    targets, kind = _ids(targets, "targets")
    if x.dim() < 1 or W.dim() != 2 or W.shape[1] != x.shape[-1]:
        raise ValueError("x must have shape (..., d) and W (V, d)")
    if x.dtype != W.dtype:
        raise TypeError("x and W must share a dtype")
    if targets.shape != x.shape[:-1]:
        raise ValueError("targets must have shape x.shape[:-1]")
    _with(x, W, "W")
    _with(x, targets, "targets")
    return x, W, targets, kind, _storage(x)


def vocab_loss(x: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, logit_scale: float = 1.0,
               ignore_index: int = -100, workspace: torch.Tensor | None = None):
    """Softmax cross entropy over the vocabulary with logits logit_scale * x W^T,
    which are not stored: x (..., d), W (V, d), targets (...) int32/int64.
    Returns (loss, lse), float32 (...): the loss of each row and the log of its
    normaliser, which vocab_loss_backward takes.  Rows whose target is
    ignore_index take no part (0 in both); any other target outside [0, V)
    gives NaN (nothing synchronises to raise)."""
    x, W, targets, kind, code = _vocab_args(x, W, targets)
    V, d = W.shape
    rows = targets.numel()
    lib = load()
    nbytes = lib.nrnn_vocab_loss_workspace_bytes(rows, d, V, code, 0)
    out = torch.empty((2, *targets.shape), dtype=torch.float32, device=x.device)
    loss, lse = out[0], out[1]
    ws = _space(workspace, nbytes, x.device)
    _run("vocab_loss", lib.nrnn_vocab_loss_forward, x, x.data_ptr(), W.data_ptr(), code, rows, d, V,
         targets.data_ptr(), kind, ignore_index, logit_scale, loss.data_ptr(), lse.data_ptr(),
         ws.data_ptr(), nbytes)
    return loss, lse


def vocab_loss_backward(x: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                        g_loss: torch.Tensor, logit_scale: float = 1.0, ignore_index: int = -100,
                        workspace: torch.Tensor | None = None):
    """(dL/dx, dL/dW) of vocab_loss() in x's dtype, from lse as it returned it
    and g_loss = dL/dloss, float32 (...) (for a mean over the kept rows: one
    over their number).  The logits are computed again, as much of the
    vocabulary at a time as 1 GiB of their gradient holds."""
    x, W, targets, kind, code = _vocab_args(x, W, targets)
    V, d = W.shape
    rows = targets.numel()
    both = []
    for t, what in ((lse, "lse"), (g_loss, "g_loss")):
        t = _device_tensor(t, what)
        if t.shape != targets.shape or t.dtype != torch.float32 or t.device != x.device:
            raise ValueError(f"{what} must be float32 of shape {tuple(targets.shape)} on {x.device}")
        both.append(t)
    lib = load()
    nbytes = lib.nrnn_vocab_loss_workspace_bytes(rows, d, V, code, 1)
    gx, gW = torch.empty_like(x), torch.empty_like(W)
    ws = _space(workspace, nbytes, x.device)
    _run("vocab_loss_backward", lib.nrnn_vocab_loss_backward, x, x.data_ptr(), W.data_ptr(), code, rows,
         d, V, targets.data_ptr(), kind, ignore_index, logit_scale, both[0].data_ptr(),
         both[1].data_ptr(), gx.data_ptr(), gW.data_ptr(), ws.data_ptr(), nbytes)
    return gx, gW
