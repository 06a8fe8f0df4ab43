"""Multi-head operators over token-major rows: thin PyTorch binding.

The stages of a mixer whose scan has one decay a head, as a joined projection
writes its rows:

    conv1d_tokens_*    short causal convolution + SiLU, with a window carried
                       from prompt to decoding
    heads_scan_*       the scan: u (batch, L, heads, P), delta (batch, L,
                       heads), A, D, delta_bias (heads,), B, C (batch, L,
                       groups, N), states (batch, heads, P, N)
    gated_norm_*       the group norm of the scan's output under SiLU(z)

Sequence tensors are float32 or bfloat16, all the same; u, delta, B, C, x and
z may be views of wider rows (their last dimensions contiguous).  Weights and
states are float32.  Gradients have the type of the tensor they belong to,
each rounded once from a float32 sum.  Every call only enqueues kernels on the
current stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (MambaScanError, _disc_code, _dtype_code, _first_order, _flags, _lib, _own_workspace,
               _ptr, lib)
from . import _req as _refuse

_F32 = torch.float32


def _stream(dev):
    """The raw handle of the current stream (torch.cuda.current_stream makes an
    object around it first, which costs a small call a tenth of its time)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _req(t, name, dtype, shape, device):
    """The package's check of a dense tensor; _refuse words what is wrong."""
    if t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                     and t.is_contiguous() and t.device == device):
        return t
    return _refuse(t, name, dtype, shape, device)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    return t.device


def _view(t, name, dtype, shape, device, lead):
    """Checks a tensor that may be a view: its first `lead` dimensions may have
    any stride, the rest is contiguous.  Returns those strides in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    strides, run = t.stride(), 1
    for i in range(len(shape) - 1, lead - 1, -1):
        n = shape[i]
        if n != 1 and strides[i] != run:
            raise ValueError(f"the last {len(shape) - lead} dimensions of {name} must be "
                             "contiguous")
        run *= n
    if lead == 1:
        return (strides[0] if shape[0] > 1 else 0,)
    return (strides[0] if shape[0] > 1 else 0, strides[1] if shape[1] > 1 else 0)


@functools.lru_cache(maxsize=1024)
def _struct(*fields):
    """mamba_heads_shape of these fields, in their order, and a reference to it.
    The calls only read it."""
    s = _lib.HeadsShape(*fields)
    return s, ctypes.byref(s)


def _dims(t, name, n):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} has {len(shape)} dimensions, expected {n}")
    return shape


def _shape(u, delta, B, C, delta_softplus, disc, segments):
    """The mamba_heads_shape of these tensors, after checking them."""
    dev = _gpu(u, "u")
    for t, name in ((delta, "delta"), (B, "B"), (C, "C")):
        _gpu(t, name)
    batch, L, H, P = _dims(u, "u", 4)
    G, N = _dims(B, "B", 4)[2:]
    dt = u.dtype
    code = _dtype_code(u)
    s, ref = _struct(batch, L, H, P, G, N, *_view(u, "u", dt, (batch, L, H, P), dev, 2),
                     *_view(delta, "delta", dt, (batch, L, H), dev, 2),
                     *_view(B, "B", dt, (batch, L, G, N), dev, 2),
                     *_view(C, "C", dt, (batch, L, G, N), dev, 2),
                     1 if delta_softplus else 0, _disc_code(disc), code, int(segments))
    return s, ref, dev


def _head_args(s, A, D, delta_bias, h0, dev):
    f32, H = _F32, s.heads
    _req(A, "A", f32, (H,), dev)
    _req(D, "D", f32, (H,), dev)
    _req(delta_bias, "delta_bias", f32, (H,), dev)
    _req(h0, "h0", f32, (s.batch, H, s.headdim, s.dstate), dev)


def _workspace(nbytes, shape, where, workspace, dev):
    """A workspace of the queried size; the caller's own where it is large enough
    (a smaller one is left unused)."""
    if nbytes >= 2 ** 63:
        empty = min(shape) <= 0
        raise MambaScanError(2 if empty else 6, where)
    workspace = _own_workspace(workspace, dev)
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _sizes(s):
    return (s.batch, s.seqlen, s.heads, s.headdim, s.groups, s.dstate)


def _query(fn, batch, L, heads, P, groups, N, dtype, segments):
    s = _lib.HeadsShape(batch=batch, seqlen=L, heads=heads, headdim=P, groups=groups, dstate=N,
                        dtype=0 if dtype == torch.float32 else 1, segments=segments)
    n = int(getattr(lib(), fn)(ctypes.byref(s)))
    if n >= 2 ** 63:
        raise MambaScanError(2 if min(_sizes(s)) <= 0 else 6, fn)
    return n


def heads_fwd_workspace_bytes(batch, L, heads, P, groups, N, dtype=torch.float32,
                              segments=0) -> int:
    return _query("mamba_heads_scan_fwd_workspace_size", batch, L, heads, P, groups, N, dtype,
                  segments)


def heads_bwd_workspace_bytes(batch, L, heads, P, groups, N, dtype=torch.float32,
                              segments=0) -> int:
    return _query("mamba_heads_scan_bwd_workspace_size", batch, L, heads, P, groups, N, dtype,
                  segments)


def heads_scan_fwd(u, delta, A, B, C, D=None, delta_bias=None, h0=None, *, delta_softplus=True,
                   disc="zoh", reset=None, return_last_state=False, out=None, last_state=None,
                   segments=0, workspace=None):
    """Multi-head scan over a prompt.  Returns out (batch, L, heads, P), or
    (out, last_state).  `last_state`: a tensor to receive it, h0 itself where the
    state is to step in place.  `reset`: (batch, L) uint8/bool flags of packed
    sequences.  `segments`: pieces of the sequence run in parallel, 0 =
    automatic.  `workspace`: a contiguous GPU tensor of at least
    heads_fwd_workspace_bytes, reused across calls (allocated when absent or
    smaller)."""
    s, ref, dev = _shape(u, delta, B, C, delta_softplus, disc, segments)
    _head_args(s, A, D, delta_bias, h0, dev)
    reset = _flags(reset, (s.batch, s.seqlen), dev)
    if out is None:
        out = torch.empty(u.shape, dtype=u.dtype, device=dev)
    else:
        _req(out, "out", u.dtype, u.shape, dev)
    states = (s.batch, s.heads, s.headdim, s.dstate)
    if return_last_state and last_state is None:
        last_state = torch.empty(states, dtype=_F32, device=dev)
    else:
        _req(last_state, "last_state", _F32, states, dev)
    n = lib().mamba_heads_scan_fwd_workspace_size(ref)
    ws = _workspace(n, _sizes(s), "mamba_heads_scan_fwd", workspace, dev)
    st = lib().mamba_heads_scan_fwd(ref, _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(delta_bias), _ptr(h0), _ptr(reset), _ptr(out),
                                    _ptr(last_state), _ptr(ws) if n else None, n, _stream(dev))
    _lib.check(st, "mamba_heads_scan_fwd")
    return (out, last_state) if return_last_state else out


def heads_scan_bwd(u, delta, A, B, C, D, delta_bias, dout, h0=None, *, dlast_state=None,
                   delta_softplus=True, disc="zoh", reset=None, segments=0, workspace=None):
    """Backward of heads_scan_fwd for the gradient `dout` at out and, optionally,
    `dlast_state` at the last state.  Returns a dict: du, ddelta, dB, dC in
    their tensors' type, dA and (where the input is given) dD, ddelta_bias, dh0
    in float32."""
    s, ref, dev = _shape(u, delta, B, C, delta_softplus, disc, segments)
    _head_args(s, A, D, delta_bias, h0, dev)
    reset = _flags(reset, (s.batch, s.seqlen), dev)
    states = (s.batch, s.heads, s.headdim, s.dstate)
    _req(dout, "dout", u.dtype, u.shape, dev)
    _req(dlast_state, "dlast_state", torch.float32, states, dev)
    new = lambda like, dt=None: torch.empty(like.shape, dtype=dt or like.dtype, device=dev)  # noqa: E731
    g = dict(du=new(u), ddelta=new(delta), dA=new(A), dB=new(B), dC=new(C))
    if D is not None:
        g["dD"] = new(D)
    if delta_bias is not None:
        g["ddelta_bias"] = new(delta_bias)
    if h0 is not None:
        g["dh0"] = new(h0)
    n = lib().mamba_heads_scan_bwd_workspace_size(ref)
    ws = _workspace(n, _sizes(s), "mamba_heads_scan_bwd", workspace, dev)
    st = lib().mamba_heads_scan_bwd(ref, _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(delta_bias), _ptr(h0), _ptr(reset), _ptr(dout),
                                    _ptr(dlast_state), _ptr(g["du"]), _ptr(g["ddelta"]),
                                    _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
                                    _ptr(g.get("dD")), _ptr(g.get("ddelta_bias")),
                                    _ptr(g.get("dh0")), _ptr(ws) if n else None, n, _stream(dev))
    _lib.check(st, "mamba_heads_scan_bwd")
    return g


def _slots(slots, batch, dev):
    return _req(slots, "slots", torch.int32, (batch,), dev)


def heads_state_update(state, u, delta, A, B, C, D=None, delta_bias=None, *, slots=None,
                       delta_softplus=True, disc="zoh", out=None):
    """One step for a batch of sequences; `state` (pool, heads, P, N) float32 is
    updated in place.  u (batch, heads, P), delta (batch, heads), B, C (batch,
    groups, N).  `slots` (batch,) int32: the state of each row (all different);
    a row whose slot lies outside the pool is left out and gives zeros.
    Returns out (batch, heads, P)."""
    dev = _gpu(state, "state")
    _gpu(u, "u")
    batch, H, P = _dims(u, "u", 3)
    G, N = _dims(_checked(B, "B"), "B", 3)[1:]
    pool = state.shape[0]
    dt = u.dtype
    code = _dtype_code(u)
    s, ref = _struct(batch, 1, H, P, G, N, *_view(u, "u", dt, (batch, H, P), dev, 1), 0,
                     *_view(delta, "delta", dt, (batch, H), dev, 1), 0,
                     *_view(B, "B", dt, (batch, G, N), dev, 1), 0,
                     *_view(C, "C", dt, (batch, G, N), dev, 1), 0,
                     1 if delta_softplus else 0, _disc_code(disc), code, 0)
    _head_args(s, A, D, delta_bias, None, dev)
    _req(state, "state", _F32, (pool, H, P, N), dev)
    slots = _slots(slots, batch, dev)
    if out is None:
        out = torch.empty((batch, H, P), dtype=dt, device=dev)
    else:
        _req(out, "out", dt, (batch, H, P), dev)
    st = lib().mamba_heads_state_update(ref, _ptr(state), _ptr(slots), pool, _ptr(u),
                                        _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                        _ptr(delta_bias), _ptr(out), _stream(dev))
    _lib.check(st, "mamba_heads_state_update")
    return out


def _checked(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _conv_args(x, w, b, window, reset):
    dev = _gpu(x, "x")
    batch, L, dim = _dims(x, "x", 3)
    W = _dims(_checked(w, "w"), "w", 2)[1]
    strides = _view(x, "x", x.dtype, (batch, L, dim), dev, 2)
    _req(w, "w", torch.float32, (dim, W), dev)
    _req(b, "b", torch.float32, (dim,), dev)
    _req(window, "window", x.dtype, (batch, W - 1, dim), dev)
    return dev, batch, L, dim, W, strides, _flags(reset, (batch, L), dev)


def conv1d_tokens_fwd(x, w, b=None, *, window=None, reset=None, return_window=False, out=None):
    """Causal depthwise convolution (w (dim, W), 2 <= W <= 4) + SiLU of x
    (batch, L, dim).  `window` (batch, W - 1, dim): the inputs before x.  `out`
    may not be x.  Returns out, or (out, the window to continue from)."""
    dev, batch, L, dim, W, (sb, st_), reset = _conv_args(x, w, b, window, reset)
    if out is None:
        out = torch.empty((batch, L, dim), dtype=x.dtype, device=dev)
    else:
        _req(out, "out", x.dtype, (batch, L, dim), dev)
    after = torch.empty((batch, W - 1, dim), dtype=x.dtype, device=dev) if return_window else None
    st = lib().mamba_conv1d_tokens_fwd(_ptr(x), sb, st_, _ptr(w), _ptr(b), _ptr(window),
                                       _ptr(reset), W, _dtype_code(x), batch, dim, L, _ptr(out),
                                       _ptr(after), _stream(dev))
    _lib.check(st, "mamba_conv1d_tokens_fwd")
    return (out, after) if return_window else out


def conv1d_tokens_bwd(x, w, b, dout, *, window=None, reset=None, workspace=None):
    """Backward of conv1d_tokens_fwd's out.  Returns a dict: dx (and dwindow)
    in x's type, dw (and db) float32."""
    dev, batch, L, dim, W, (sb, st_), reset = _conv_args(x, w, b, window, reset)
    _req(dout, "dout", x.dtype, (batch, L, dim), dev)
    g = dict(dx=torch.empty((batch, L, dim), dtype=x.dtype, device=dev), dw=torch.empty_like(w))
    if b is not None:
        g["db"] = torch.empty_like(b)
    if window is not None:
        g["dwindow"] = torch.empty_like(window)
    n = lib().mamba_conv1d_tokens_bwd_workspace_size(batch, dim, L, W)
    ws = _workspace(n, (batch, dim, L), "mamba_conv1d_tokens_bwd", workspace, dev)
    st = lib().mamba_conv1d_tokens_bwd(_ptr(x), sb, st_, _ptr(w), _ptr(b), _ptr(window),
                                       _ptr(reset), _ptr(dout), W, _dtype_code(x), batch, dim, L,
                                       _ptr(g["dx"]), _ptr(g["dw"]), _ptr(g.get("db")),
                                       _ptr(g.get("dwindow")), _ptr(ws), n, _stream(dev))
    _lib.check(st, "mamba_conv1d_tokens_bwd")
    return g


def conv1d_tokens_update(x, window, w, b=None, *, slots=None, out=None):
    """One token: x (batch, dim), `window` (pool, W - 1, dim) of x's type
    updated in place, `slots` as for heads_state_update.  Returns out like x."""
    dev = _gpu(x, "x")
    batch, dim = _dims(x, "x", 2)
    W = _dims(_checked(w, "w"), "w", 2)[1]
    sb, = _view(x, "x", x.dtype, (batch, dim), dev, 1)
    _req(w, "w", torch.float32, (dim, W), dev)
    _req(b, "b", torch.float32, (dim,), dev)
    pool = _dims(_checked(window, "window"), "window", 3)[0]
    _req(window, "window", x.dtype, (pool, W - 1, dim), dev)
    slots = _slots(slots, batch, dev)
    if out is None:
        out = torch.empty((batch, dim), dtype=x.dtype, device=dev)
    else:
        _req(out, "out", x.dtype, (batch, dim), dev)
    st = lib().mamba_conv1d_tokens_update(_ptr(x), sb, _ptr(window), _ptr(slots), pool, _ptr(w),
                                          _ptr(b), W, _dtype_code(x), batch, dim, _ptr(out),
                                          _stream(dev))
    _lib.check(st, "mamba_conv1d_tokens_update")
    return out


def _rows(t):
    """A (..., dim) tensor as (rows, dim), without a copy."""
    if t.dim() < 1:
        raise ValueError("the norm needs at least one dimension")
    return t if t.dim() == 2 else t.view(-1, t.shape[-1])


def _norm_args(x, z, weight, groups):
    dev = _gpu(x, "x")
    x2 = _rows(x)
    rows, dim = x2.shape
    sx, = _view(x2, "x", x.dtype, (rows, dim), dev, 1)
    sz = 0
    if z is not None:
        _gpu(z, "z")
        if z.shape != x.shape:
            raise ValueError(f"z has shape {tuple(z.shape)}, expected {tuple(x.shape)}")
        z = _rows(z)
        sz, = _view(z, "z", x.dtype, (rows, dim), dev, 1)
    _req(weight, "weight", torch.float32, (dim,), dev)
    return dev, x2, sx, z, sz, rows, dim, int(groups)


def gated_norm_fwd(x, z=None, weight=None, *, groups=1, eps=1e-5, gate_first=True, out=None):
    """Group norm (root mean square over each of `groups` parts of the last
    dimension) of x under the gate SiLU(z): of x SiLU(z) when `gate_first`,
    else of x, times SiLU(z) after.  x, z (..., dim); returns out like x."""
    dev, x2, sx, z2, sz, rows, dim, groups = _norm_args(x, z, weight, groups)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _req(out, "out", x.dtype, x.shape, dev)
    st = lib().mamba_gated_norm_fwd(_ptr(x2), sx, _ptr(z2), sz, _ptr(weight), rows, dim, groups,
                                    float(eps), int(bool(gate_first)), _dtype_code(x), _ptr(out),
                                    _stream(dev))
    _lib.check(st, "mamba_gated_norm_fwd")
    return out


def gated_norm_bwd(x, z, weight, dout, *, groups=1, eps=1e-5, gate_first=True, workspace=None):
    """Backward of gated_norm_fwd: a dict with dx (and dz) in x's type and
    dweight float32, those whose input is given."""
    dev, x2, sx, z2, sz, rows, dim, groups = _norm_args(x, z, weight, groups)
    _req(dout, "dout", x.dtype, x.shape, dev)
    g = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=dev))
    if z is not None:
        g["dz"] = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if weight is not None:
        g["dweight"] = torch.empty_like(weight)
    n = lib().mamba_gated_norm_bwd_workspace_size(rows, dim, groups)
    ws = _workspace(n, (rows, dim, groups), "mamba_gated_norm_bwd", workspace, dev)
    st = lib().mamba_gated_norm_bwd(_ptr(x2), sx, _ptr(z2), sz, _ptr(weight), _ptr(dout), rows,
                                    dim, groups, float(eps), int(bool(gate_first)),
                                    _dtype_code(x), _ptr(g["dx"]), _ptr(g.get("dz")),
                                    _ptr(g.get("dweight")), _ptr(ws), n, _stream(dev))
    _lib.check(st, "mamba_gated_norm_bwd")
    return g


class _HeadsScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, delta_bias, h0, delta_softplus, disc, reset):
        out, last = heads_scan_fwd(u, delta, A, B, C, D, delta_bias, h0,
                                   delta_softplus=delta_softplus, disc=disc, reset=reset,
                                   return_last_state=True)
        ctx.save_for_backward(u, delta, A, B, C, D, delta_bias, h0, reset)
        ctx.flags = (delta_softplus, disc)
        ctx.set_materialize_grads(False)
        return out, last

    @staticmethod
    @_first_order
    def backward(ctx, dout, dlast):
        u, delta, A, B, C, D, delta_bias, h0, reset = ctx.saved_tensors
        sp, disc = ctx.flags
        dout = torch.zeros(u.shape, dtype=u.dtype, device=u.device) if dout is None else dout
        g = heads_scan_bwd(u, delta, A, B, C, D, delta_bias, dout.contiguous(), h0,
                           dlast_state=None if dlast is None else dlast.contiguous(),
                           delta_softplus=sp, disc=disc, reset=reset)
        return (g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"], g.get("dD"),
                g.get("ddelta_bias"), g.get("dh0"), None, None, None)


def heads_scan(u, delta, A, B, C, D=None, delta_bias=None, h0=None, *, delta_softplus=True,
               disc="zoh", reset=None, return_last_state=False):
    """heads_scan_fwd with gradients (through out and the last state)."""
    reset = reset if reset is None or reset.dtype != torch.bool else reset.to(torch.uint8)
    out, last = _HeadsScanFn.apply(u, delta, A, B, C, D, delta_bias, h0, delta_softplus, disc,
                                   reset)
    return (out, last) if return_last_state else out


class _Conv1dTokensFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, window, reset):
        ctx.save_for_backward(x, w, b, window, reset)
        return conv1d_tokens_fwd(x, w, b, window=window, reset=reset)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        x, w, b, window, reset = ctx.saved_tensors
        g = conv1d_tokens_bwd(x, w, b, dout.contiguous(), window=window, reset=reset)
        return g["dx"], g["dw"], g.get("db"), g.get("dwindow"), None


def conv1d_tokens(x, w, b=None, *, window=None, reset=None):
    """conv1d_tokens_fwd with gradients."""
    return _Conv1dTokensFn.apply(x, w, b, window, reset)


class _GatedNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, groups, eps, gate_first):
        ctx.save_for_backward(x, z, weight)
        ctx.flags = dict(groups=groups, eps=eps, gate_first=gate_first)
        return gated_norm_fwd(x, z, weight, **ctx.flags)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        x, z, weight = ctx.saved_tensors
        g = gated_norm_bwd(x, z, weight, dout.contiguous(), **ctx.flags)
        return g["dx"], g.get("dz"), g.get("dweight"), None, None, None


def gated_norm(x, z=None, weight=None, *, groups=1, eps=1e-5, gate_first=True):
    """gated_norm_fwd with gradients."""
    return _GatedNormFn.apply(x, z, weight, groups, eps, gate_first)
