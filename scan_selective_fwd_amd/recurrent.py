"""Operators of a recurrent block over token-major rows: thin PyTorch binding.

    residual_norm_*      the norm that opens a block, with the residual's addition;
                         its output in the activations' type or in 8 bits
    gated_recurrence_*   the gated linear recurrence: x, r, i, z (batch, L, dim),
                         A (dim,), states (batch, dim) or a pool (pool, dim)

Activations are float32 or bfloat16, all the same; x, r, i, z and the norm's x
and residual may be views of wider rows (their last dimension contiguous).
Weights and states are float32.  Gradients have the type of the tensor they
belong to, each rounded once from a float32 sum.  Every call only enqueues
kernels on the current stream of its tensors' device, so it may be captured into a
graph.  A backward through autograd is captured only once no eager graph of the same
leaves is alive: the leaves' accumulation would run on that graph's stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MambaScanError, _dtype_code, _first_order, _flags, _lib, _ptr, lib
from .heads import _dims, _gpu, _req, _slots, _stream, _view, _workspace

_F32 = torch.float32
_FP8 = torch.float8_e4m3fn
_current = torch._C._cuda_getDevice


@functools.lru_cache(maxsize=None)
def _function(name):
    return getattr(lib(), name)


def _call(name, dev, *args):
    """The library's call with `dev` the current device, whose stream it goes on."""
    if _current() == dev.index:
        st = _function(name)(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = _function(name)(*args, _stream(dev))
    if st:
        _lib.check(st, name)


@functools.lru_cache(maxsize=1024)
def _struct(*fields):
    """mamba_recurrence_shape of these fields, in their order, and a reference to
    it.  The calls only read it."""
    s = _lib.RecurrenceShape(*fields)
    return s, ctypes.byref(s)


@functools.lru_cache(maxsize=1024)
def _fwd_bytes(*fields):
    """The forward's workspace for these fields."""
    return _function("mamba_gated_recurrence_fwd_workspace_size")(_struct(*fields)[1])


@functools.lru_cache(maxsize=1024)
def _bwd_bytes(kept, *fields):
    return _function("mamba_gated_recurrence_bwd_workspace_size")(_struct(*fields)[1], kept)


def _new(like, dtype=None):
    """A dense tensor of `like`'s shape (empty_like costs half of empty, but keeps the
    order of a permuted tensor's dimensions)."""
    if like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(like.shape, dtype=dtype or like.dtype, device=like.device)


def _strides(t, name, dtype, shape, dev):
    """Checks a tensor that may be a view of wider rows; its strides but the last's."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev:
        st = t.stride()
        if st[-1] == 1:
            return st[:-1]
    return _view(t, name, dtype, shape, dev, len(shape) - 1)


# --------------------------------------------------------------------------- recurrence

def _shape(x, r, i, z):
    dev = _gpu(x, "x")
    shape = _dims(x, "x", 3)
    dt = x.dtype
    code = _dtype_code(x)
    fields = (*shape, *_strides(x, "x", dt, shape, dev), *_strides(r, "r", dt, shape, dev),
              *_strides(i, "i", dt, shape, dev),
              *((0, 0) if z is None else _strides(z, "z", dt, shape, dev)), code)
    return _struct(*fields)[1], fields, dev, shape


def _state_args(shape, A, h0, reset, dev):
    batch, L, dim = shape
    _req(A, "A", _F32, (dim,), dev)
    _req(h0, "h0", _F32, (batch, dim), dev)
    return _flags(reset, (batch, L), dev)


def _tiles(L):
    return -(-L // 64)


def gated_recurrence_checkpoint_shape(batch, L, dim):
    """Shape of the forward's checkpoints: the state entering every 64th step."""
    return (batch, _tiles(L), dim)


def _query(fn, batch, L, dim, dtype, *more):
    s = _lib.RecurrenceShape(batch=batch, seqlen=L, dim=dim,
                             dtype=0 if dtype == torch.float32 else 1)
    n = int(getattr(lib(), fn)(ctypes.byref(s), *more))
    if n >= 2 ** 63:
        raise MambaScanError(2 if min(batch, L, dim) <= 0 else 6, fn)
    return n


def gated_recurrence_fwd_workspace_bytes(batch, L, dim, dtype=torch.float32) -> int:
    return _query("mamba_gated_recurrence_fwd_workspace_size", batch, L, dim, dtype)


def gated_recurrence_bwd_workspace_bytes(batch, L, dim, dtype=torch.float32,
                                         with_checkpoints=True) -> int:
    return _query("mamba_gated_recurrence_bwd_workspace_size", batch, L, dim, dtype,
                  int(bool(with_checkpoints)))


def gated_recurrence_fwd(x, r, i, A, z=None, h0=None, *, reset=None, return_last_state=False,
                         out=None, last_state=None, checkpoints=None, workspace=None):
    """Gated linear recurrence over a prompt, with s(v) = 1 / (1 + exp(-v)):

        a_t = exp(A s(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t
        out_t = h_t  (h_t z_t s(z_t) with z),  A <= 0

    Returns out (batch, L, dim), or (out, last_state).  `last_state`: a tensor to
    receive it, h0 itself where the state is to step in place.  `reset`: (batch,
    L) uint8/bool flags of packed sequences: the state before a flagged step is
    left out.  `checkpoints`: a float32 tensor of
    gated_recurrence_checkpoint_shape that receives the state entering every
    64th step, for gated_recurrence_bwd.  `workspace`: a contiguous GPU tensor of
    at least gated_recurrence_fwd_workspace_bytes, reused across calls that follow
    one another on a stream (allocated when absent or smaller)."""
    ref, fields, dev, shape = _shape(x, r, i, z)
    reset = _state_args(shape, A, h0, reset, dev)
    batch, L, dim = shape
    if out is None:
        out = _new(x)
    else:
        _req(out, "out", x.dtype, shape, dev)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim), dtype=_F32, device=dev) if h0 is None \
            else torch.empty_like(h0)
    else:
        _req(last_state, "last_state", _F32, (batch, dim), dev)
    if checkpoints is not None:
        _req(checkpoints, "checkpoints", _F32, (batch, _tiles(L), dim), dev)
    n = _fwd_bytes(*fields)
    ws = _workspace(n, shape, "mamba_gated_recurrence_fwd", workspace, dev)
    _call("mamba_gated_recurrence_fwd", dev, ref, _ptr(x), _ptr(r), _ptr(i), _ptr(A), _ptr(z),
          _ptr(h0), _ptr(reset), _ptr(out), _ptr(last_state), _ptr(checkpoints),
          _ptr(ws) if n else None, n)
    return (out, last_state) if return_last_state else out


def gated_recurrence_bwd(x, r, i, A, z, dout, h0=None, *, dlast_state=None, reset=None,
                         checkpoints=None, workspace=None):
    """Backward of gated_recurrence_fwd for the gradient `dout` at out and,
    optionally, `dlast_state` at the last state.  `checkpoints`: those of the
    forward over the same inputs; absent, they are formed again.  Returns a
    dict: dx, dr, di (and dz) in their tensors' type, dA (and dh0) in
    float32."""
    ref, fields, dev, shape = _shape(x, r, i, z)
    reset = _state_args(shape, A, h0, reset, dev)
    batch, L, dim = shape
    _req(_need(dout, "dout"), "dout", x.dtype, shape, dev)
    _req(dlast_state, "dlast_state", _F32, (batch, dim), dev)
    if checkpoints is not None:
        _req(checkpoints, "checkpoints", _F32, (batch, _tiles(L), dim), dev)
    g = dict(dx=_new(x), dr=_new(x), di=_new(x), dA=_new(A))
    if z is not None:
        g["dz"] = _new(x)
    if h0 is not None:
        g["dh0"] = _new(h0)
    n = _bwd_bytes(int(checkpoints is not None), *fields)
    ws = _workspace(n, shape, "mamba_gated_recurrence_bwd", workspace, dev)
    _call("mamba_gated_recurrence_bwd", dev, ref, _ptr(x), _ptr(r), _ptr(i), _ptr(A), _ptr(z),
          _ptr(h0), _ptr(reset), _ptr(dout), _ptr(dlast_state), _ptr(checkpoints), _ptr(g["dx"]),
          _ptr(g["dr"]), _ptr(g["di"]), _ptr(g["dA"]), _ptr(g.get("dz")), _ptr(g.get("dh0")),
          _ptr(ws) if n else None, n)
    return g


def gated_recurrence_update(state, x, r, i, A, z=None, *, slots=None, out=None):
    """One step for a batch of sequences; `state` (pool, dim) float32 is updated
    in place.  x, r, i, z (batch, dim).  `slots` (batch,) int32: the state of each
    row (all different); a row whose slot lies outside the pool is left out and
    gives zeros.  Returns out (batch, dim)."""
    dev = _gpu(state, "state")
    _gpu(x, "x")
    shape = _dims(x, "x", 2)
    batch, dim = shape
    dt = x.dtype
    pool = _dims(state, "state", 2)[0]
    ref = _struct(batch, 1, dim, *_strides(x, "x", dt, shape, dev), 0,
                  *_strides(r, "r", dt, shape, dev), 0, *_strides(i, "i", dt, shape, dev), 0,
                  *((0,) if z is None else _strides(z, "z", dt, shape, dev)), 0,
                  _dtype_code(x))[1]
    _req(A, "A", _F32, (dim,), dev)
    _req(state, "state", _F32, (pool, dim), dev)
    slots = _slots(slots, batch, dev)
    if out is None:
        out = _new(x)
    else:
        _req(out, "out", dt, shape, dev)
    _call("mamba_gated_recurrence_update", dev, ref, _ptr(state), _ptr(slots), pool, _ptr(x),
          _ptr(r), _ptr(i), _ptr(A), _ptr(z), _ptr(out))
    return out


def _need(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


class _GatedRecurrenceFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, A, z, h0, reset):
        kept = torch.empty(gated_recurrence_checkpoint_shape(*_dims(_need(x, "x"), "x", 3)),
                           dtype=_F32, device=x.device)
        out, last = gated_recurrence_fwd(x, r, i, A, z, h0, reset=reset, return_last_state=True,
                                         checkpoints=kept)
        ctx.save_for_backward(x, r, i, A, z, h0, reset, kept)
        ctx.set_materialize_grads(False)
        return out, last

    @staticmethod
    @_first_order
    def backward(ctx, dout, dlast):
        x, r, i, A, z, h0, reset, kept = ctx.saved_tensors
        dout = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dout is None else dout
        g = gated_recurrence_bwd(x, r, i, A, z, dout.contiguous(), h0,
                                 dlast_state=None if dlast is None else dlast.contiguous(),
                                 reset=reset, checkpoints=kept)
        return g["dx"], g["dr"], g["di"], g["dA"], g.get("dz"), g.get("dh0"), None


def gated_recurrence(x, r, i, A, z=None, h0=None, *, reset=None, return_last_state=False):
    """gated_recurrence_fwd with gradients (through out and the last state)."""
    reset = reset if reset is None or reset.dtype != torch.bool else reset.to(torch.uint8)
    out, last = _GatedRecurrenceFn.apply(x, r, i, A, z, h0, reset)
    return (out, last) if return_last_state else out


# --------------------------------------------------------------------------- norm

def _residual_code(t, x):
    """The code of a residual stream's type: x's, or float32."""
    if t.dtype is not x.dtype and t.dtype is not _F32:
        raise TypeError(f"residual has dtype {t.dtype}, expected {x.dtype} or torch.float32")
    return _dtype_code(t)


def _row_strides(t, name):
    """Batch and row stride of a (..., dim) tensor, dense or a view: its rows are one run
    (the batch stride is None then), or one for each index of the first dimension, of
    whatever stride, a broadcast one's 0 too."""
    if t.is_contiguous():
        return None, t.shape[-1]
    for lead in (1, t.shape[0]):
        try:
            v = t.view(lead, -1, t.shape[-1])
        except RuntimeError:
            continue
        if t.shape[-1] == 1 or t.stride(-1) == 1:
            return (v.stride(0) if lead > 1 else None), (v.stride(1) if v.shape[1] > 1 else 0)
    raise ValueError(f"rows of {name} must be contiguous, and a step apart in each index of its "
                     "first dimension")


def _planes(t, a, b):
    """(batch, rows, dim) of t, one run of rows where the views are, and the views' batch
    and row strides among them."""
    dim = t.shape[-1]
    rows = t.numel() // dim if dim else 0
    (ab, ar), (bb, br) = a, b
    if ab is None and bb is None or not rows:
        return (1 if rows else 0, rows, dim), (0, ar), (0, br)
    batch = t.shape[0]
    rows //= batch
    return ((batch, rows, dim), (rows * ar if ab is None else ab, ar),
            (rows * br if bb is None else bb, br))


def _norm_args(x, residual, weight, residual_out):
    dev = _gpu(x, "x")
    dt, shape = x.dtype, x.shape
    code = rcode = _dtype_code(x)
    if not shape:
        raise ValueError("the norm needs at least one dimension")
    sx, sr = _row_strides(x, "x"), (None, 0)
    if residual is not None:
        if _gpu(residual, "residual") != dev:
            raise ValueError(f"residual is on {residual.device}, expected {dev}")
        if residual.dtype is not dt:
            rcode = _residual_code(residual, x)
        if residual.shape != shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}, expected "
                             f"{tuple(shape)}")
        sr = _row_strides(residual, "residual")
        if residual_out is None:
            residual_out = _new(residual)
        else:
            _req(residual_out, "residual_out", residual.dtype, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    sizes, sx, sr = _planes(x, sx, sr)
    _req(weight, "weight", _F32, sizes[2:], dev)
    return dev, code, rcode, sx, sr, sizes, residual_out


def residual_norm_fwd(x, residual=None, weight=None, *, eps=1e-5, out=None, residual_out=None):
    """The residual's addition and the root-mean-square norm of the sum:

        res = x + residual,  out = res / sqrt(mean(res^2) + eps) * weight

    over the last dimension of x (..., dim).  `residual`: x's type or float32;
    res is kept in it, and the norm is of what is kept.  Returns (out, res), out
    like x; without a residual res is x itself.  `residual_out`: a tensor to
    receive res, residual itself (dense) where the stream is carried in place."""
    dev, code, rcode, sx, sr, sizes, kept = _norm_args(x, residual, weight, residual_out)
    if out is None:
        out = _new(x)
    else:
        _req(out, "out", x.dtype, x.shape, dev)
    _call("mamba_residual_norm_fwd", dev, _ptr(x), *sx, _ptr(residual), *sr, _ptr(weight), *sizes,
          float(eps), code, rcode, _ptr(out), _ptr(kept))
    return out, x if kept is None else kept


def residual_norm_fp8(x, residual=None, weight=None, *, eps=1e-5, out=None, scale=None,
                      residual_out=None):
    """residual_norm_fwd with out in 8 bits: returns (out, scale, res), out
    torch.float8_e4m3fn like x, scale float32 of x's shape without its last
    dimension, max|out| / 448 of each row; out stands for out * scale."""
    dev, code, rcode, sx, sr, sizes, kept = _norm_args(x, residual, weight, residual_out)
    if out is None:
        out = _new(x, _FP8)
    else:
        _req(out, "out", _FP8, x.shape, dev)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    else:
        _req(scale, "scale", _F32, x.shape[:-1], dev)
    _call("mamba_residual_norm_fp8", dev, _ptr(x), *sx, _ptr(residual), *sr, _ptr(weight), *sizes,
          float(eps), code, rcode, _ptr(out), _ptr(scale), _ptr(kept))
    return out, scale, x if kept is None else kept


def residual_norm_bwd(res, weight, dout, dres=None, *, eps=1e-5, workspace=None):
    """Backward of residual_norm_fwd from the res that it returned: `dout` (x's
    type, dense) is the gradient at out, `dres` (res's type, dense) that which
    comes to res from the stream.  Returns a dict: dx in dout's type, dresidual
    in res's (dx itself where the types agree), and dweight float32 where weight
    is given."""
    dev = _gpu(res, "res")
    _gpu(dout, "dout")
    code, rcode = _dtype_code(dout), _residual_code(res, dout)
    if not res.shape:
        raise ValueError("the norm needs at least one dimension")
    (batch, rows, dim), sr, _ = _planes(res, _row_strides(res, "res"), (None, 0))
    _req(weight, "weight", _F32, (dim,), dev)
    _req(dout, "dout", dout.dtype, res.shape, dev)
    _req(dres, "dres", res.dtype, res.shape, dev)
    g = dict(dx=_new(dout))
    g["dresidual"] = g["dx"] if code == rcode else _new(res)
    if weight is not None:
        g["dweight"] = torch.empty((dim,), dtype=_F32, device=dev)
    n = _function("mamba_residual_norm_bwd_workspace_size")(batch * rows, dim)
    ws = _workspace(n, (rows, dim), "mamba_residual_norm_bwd", workspace, dev)
    _call("mamba_residual_norm_bwd", dev, _ptr(res), *sr, _ptr(weight), _ptr(dout), _ptr(dres),
          batch, rows, dim, float(eps), code, rcode, _ptr(g["dx"]),
          None if code == rcode else _ptr(g["dresidual"]), _ptr(g.get("dweight")), _ptr(ws), n)
    return g


class _ResidualNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        out, res = residual_norm_fwd(x, residual, weight, eps=eps)
        ctx.save_for_backward(res, weight)
        ctx.eps, ctx.alone, ctx.x_dtype = eps, residual is None, x.dtype
        ctx.set_materialize_grads(False)
        return out if residual is None else (out, res)

    @staticmethod
    @_first_order
    def backward(ctx, dout, dres=None):
        res, weight = ctx.saved_tensors
        if dout is None:      # out was not used: the stream's gradient goes through
            if dres is None:
                return None, None, None, None
            dout = torch.zeros(res.shape, dtype=ctx.x_dtype, device=res.device)
        g = residual_norm_bwd(res, weight, dout.contiguous(),
                              None if dres is None else dres.contiguous(), eps=ctx.eps)
        return g["dx"], None if ctx.alone else g["dresidual"], g.get("dweight"), None


def residual_norm(x, residual=None, weight=None, *, eps=1e-5):
    """residual_norm_fwd with gradients (through out and res)."""
    if residual is None:
        return _ResidualNormFn.apply(x, None, weight, eps), x
    return _ResidualNormFn.apply(x, residual, weight, eps)
