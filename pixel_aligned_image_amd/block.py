"""Binding of include/p3d_block.h: the transformer block's operators.

Same rules as the package's other entry points: every function has the name
of its C entry point, checks its tensors and passes device pointers and
torch's current HIP stream; results go into tensors the caller gives.
``offsets`` are item tables, sequences of batch + 1 row numbers (or the ctypes
array ``make_offsets`` makes of one, for callers that reuse it). ``workspace``
is a uint8 device tensor of at least the matching ``*_workspace_size``, or
None for a fresh one (allocated by torch here, not by the library).
"""
import ctypes

import torch

from ._streams import fresh as _fresh, lends as _lends

__all__ = ["p3d_gated_norm", "p3d_gated_norm_backward", "p3d_gated_norm_workspace_size",
           "p3d_rotary", "p3d_rotary_backward", "p3d_rotary_workspace_size",
           "p3d_rotary_frequencies", "p3d_attention", "p3d_attention_backward",
           "p3d_attention_workspace_size", "p3d_attention_backward_workspace_size",
           "make_offsets", "NORM", "ROTARY_LAYOUT", "ROTARY_SCALING"]

NORM = {"none": 0, "layer": 1, "rms": 2}                                # p3d_norm_kind
ROTARY_LAYOUT = {"interleaved": 0, "half": 1}                           # p3d_rotary_layout
ROTARY_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}    # p3d_rotary_scaling

_vp, _i32, _i64, _f32, _f64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                               ctypes.c_double)
_size = ctypes.c_size_t


class p3d_norm_desc(ctypes.Structure):
    _fields_ = [("n", _i64), ("offsets", _vp), ("batch", _i32), ("dim", _i32),
                ("dtype", ctypes.c_int), ("pre", ctypes.c_int), ("post", ctypes.c_int),
                ("res_scale", _f32), ("eps", _f32), ("mod_stride", _i64), ("gate", _vp),
                ("scale", _vp), ("shift", _vp), ("weight", _vp), ("bias", _vp),
                ("post_weight", _vp)]


class p3d_rotary_desc(ctypes.Structure):
    _fields_ = [("n", _i64), ("heads", _i32), ("head_dim", _i32), ("dtype", ctypes.c_int),
                ("layout", ctypes.c_int), ("axes", _i32), ("pairs", _i32), ("pos_stride", _i32),
                ("magnitude", _f32), ("eps", _f32), ("positions", _vp), ("freqs", _vp),
                ("gamma", _vp)]


class p3d_attn_desc(ctypes.Structure):
    _fields_ = [("q_offsets", _vp), ("k_offsets", _vp), ("batch", _i32), ("heads", _i32),
                ("kv_heads", _i32), ("head_dim", _i32), ("dtype", ctypes.c_int),
                ("scale", _f32), ("causal", _i32)]


lib = None          # set by bind()
_core = None


def bind(core):
    """Declare the entry points on the loaded library (called on import)."""
    global lib, _core
    _core, lib = core, core.lib
    norm, rot, att = (ctypes.POINTER(t) for t in (p3d_norm_desc, p3d_rotary_desc, p3d_attn_desc))
    for name, res, args in [
            ("p3d_gated_norm", ctypes.c_int, [norm] + [_vp] * 5),
            ("p3d_gated_norm_workspace_size", _size, [norm]),
            ("p3d_gated_norm_backward", ctypes.c_int, [norm] + [_vp] * 13 + [_size, _vp]),
            ("p3d_rotary", ctypes.c_int, [rot, _vp, _i64, _vp, _i64, _vp]),
            ("p3d_rotary_workspace_size", _size, [rot]),
            ("p3d_rotary_backward", ctypes.c_int,
             [rot] + [_vp, _i64] * 3 + [_vp, _vp, _size, _vp]),
            ("p3d_rotary_frequencies", ctypes.c_int, [_f64, _i32, ctypes.c_int, _f64, _f64, _vp]),
            ("p3d_attention_workspace_size", _size, [att]),
            ("p3d_attention", ctypes.c_int, [att] + [_vp, _i64] * 4 + [_vp, _vp, _size, _vp]),
            ("p3d_attention_backward_workspace_size", _size, [att]),
            ("p3d_attention_backward", ctypes.c_int,
             [att] + [_vp, _i64] * 5 + [_vp] + [_vp, _i64] * 3 + [_vp, _size, _vp])]:
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ----------------------------------------------------------------- helpers ---
def make_offsets(offsets):
    """ctypes int64 array of an item table (batch + 1 row numbers). Only an
    int64 array is passed on as it is: the library reads 8 bytes an entry."""
    if isinstance(offsets, ctypes.Array) and offsets._type_ is _i64:
        return offsets
    return (_i64 * len(offsets))(*offsets)


def _dtype(t, name):
    dt = _core._DT.get(t.dtype)
    if dt is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return dt


def _ptr(t, name, dtype, shape):
    """Device pointer of an optional contiguous tensor. The smallest calls last
    a few microseconds, as long as ten tensors' checks: one line passes what is
    right, the package's own check words what is not."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    return _core._dev(t, name, dtype, shape)


def _stream(stream):
    """As the package's other calls: torch's current stream. Its handle alone
    costs 0.4 us, a torch.cuda.Stream of it 2.8 us."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _sized(size):
    if size == 0:
        raise _core.P3DError(_core.P3D_ERR_INVALID_ARG, _core.p3d_last_error())
    return int(size)


def _work(workspace, size, device, stream):
    """(pointer, bytes) of the caller's workspace, or of a fresh one. The
    tensor is returned too, so that it lives until the call is enqueued."""
    if workspace is None:
        workspace = _fresh(_sized(size()), device, stream)
    return workspace, _core._dev(workspace, "workspace", torch.uint8), workspace.numel()


def _heads(t, name, dtype, heads=None, head_dim=None, rows=None):
    """(pointer, token stride) of a [n, heads, head_dim] device tensor whose
    tokens may be strided (a view of a packed projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU, got %s" % (name, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 3 or (heads is not None and t.shape != (rows, heads, head_dim)):
        raise ValueError("%s must be [%s, %s, %s], got %s" % (
            name, "n" if rows is None else rows, "heads" if heads is None else heads,
            "head_dim" if head_dim is None else head_dim, tuple(t.shape)))
    n, h, d = t.shape
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError("%s must have contiguous heads, got strides %s" % (name, s))
    return t.data_ptr(), (s[0] if n > 1 else h * d)


# -------------------------------------------------------------- gated norm ---
def _norm(x, offsets, gate, scale, shift, pre, post, weight, bias, post_weight, res_scale, eps):
    if x.dim() != 2:
        raise ValueError("x must be [n, dim], got %s" % (tuple(x.shape),))
    dt = x.dtype
    n, dim = x.shape
    off = make_offsets((0, n) if offsets is None else offsets)
    batch = len(off) - 1
    d = p3d_norm_desc(n, ctypes.addressof(off), batch, dim, _dtype(x, "x"), NORM[pre],
                      NORM[post], res_scale, eps, dim)
    stride = None
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
        if t is None:
            continue
        # rows of a packed [batch, k, dim] modulation may be strided
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dt:
            raise TypeError("%s must be a %s tensor on the GPU" % (name, dt))
        if t.shape != (batch, dim) or (dim > 1 and t.stride(1) != 1):
            raise ValueError("%s must be [%d, %d] with contiguous rows, got %s, strides %s" % (
                name, batch, dim, tuple(t.shape), t.stride()))
        if batch > 1:
            if stride is not None and t.stride(0) != stride:
                raise ValueError("gate, scale and shift must have one row stride, got %d and %d"
                                 % (stride, t.stride(0)))
            stride = t.stride(0)
        setattr(d, name, t.data_ptr())
    if stride is not None:
        d.mod_stride = stride
    d.weight = _ptr(weight, "weight", dt, (dim,))
    d.bias = _ptr(bias, "bias", dt, (dim,))
    d.post_weight = _ptr(post_weight, "post_weight", dt, (dim,))
    return d, off


@_lends
def p3d_gated_norm(x, h, offsets=None, y=None, gate=None, scale=None, shift=None, r=None,
                   pre="layer", post="none", weight=None, bias=None, post_weight=None,
                   res_scale=1.0, eps=1e-6, stream=None):
    """Enqueue p3d_gated_norm: r = x + res_scale gate post(y) post_weight,
    h = (pre(r) weight + bias)(1 + scale) + shift. x, y, r, h: [n, dim], float32
    or bfloat16; gate, scale, shift: [batch, dim] (rows may be strided);
    weight, bias, post_weight: [dim]; offsets: the items' rows (None: one
    item)."""
    d, off = _norm(x, offsets, gate, scale, shift, pre, post, weight, bias, post_weight,
                   res_scale, eps)
    dt, shape = x.dtype, x.shape
    _core._check(lib.p3d_gated_norm(d, _ptr(x, "x", dt, shape), _ptr(y, "y", dt, shape),
                                    _ptr(r, "r", dt, shape), _ptr(h, "h", dt, shape),
                                    _stream(stream)))


def p3d_gated_norm_workspace_size(x, offsets=None):
    """Bytes of device workspace p3d_gated_norm_backward needs for rows like
    x's."""
    d, off = _norm(x, offsets, None, None, None, "layer", "none", None, None, None, 1.0, 1e-6)
    return _sized(lib.p3d_gated_norm_workspace_size(d))


@_lends
def p3d_gated_norm_backward(dh, x, dx, offsets=None, dr=None, y=None, dy=None, gate=None,
                            scale=None, pre="layer", post="none", weight=None, bias=None,
                            post_weight=None, res_scale=1.0, eps=1e-6, dgate=None, dscale=None,
                            dshift=None, dweight=None, dbias=None, dpost_weight=None,
                            workspace=None, stream=None):
    """Enqueue p3d_gated_norm_backward: dx (the whole gradient of r) and dy
    [n, dim] from dh and dr (the gradient that reaches r otherwise); float32
    parameter gradients dgate, dscale, dshift [batch, dim] and dweight, dbias,
    dpost_weight [dim], each None where it is not wanted."""
    d, off = _norm(x, offsets, gate, scale, None, pre, post, weight, bias, post_weight,
                   res_scale, eps)
    dev, dt, shape, f = _ptr, x.dtype, x.shape, torch.float32
    items, cols = (d.batch, d.dim), (d.dim,)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_gated_norm_workspace_size(d), x.device,
                             stream)
    _core._check(lib.p3d_gated_norm_backward(
        d, dev(dh, "dh", dt, shape), dev(dr, "dr", dt, shape), dev(x, "x", dt, shape),
        dev(y, "y", dt, shape), dev(dx, "dx", dt, shape), dev(dy, "dy", dt, shape),
        dev(dgate, "dgate", f, items), dev(dscale, "dscale", f, items),
        dev(dshift, "dshift", f, items), dev(dweight, "dweight", f, cols),
        dev(dbias, "dbias", f, cols), dev(dpost_weight, "dpost_weight", f, cols), ws, nbytes,
        _stream(stream)))


# ------------------------------------------------------------------ rotary ---
def _rotary(x, positions, freqs, layout, magnitude, gamma, eps):
    n, heads, hd = x.shape
    if not isinstance(positions, torch.Tensor) or not positions.is_cuda:
        raise TypeError("positions must be a torch.Tensor on the GPU")
    if positions.dtype is not torch.int32:
        raise TypeError("positions must be torch.int32, got %s" % positions.dtype)
    if positions.dim() != 2 or positions.shape[0] != n:
        raise ValueError("positions must be [%d, axes], got %s" % (n, tuple(positions.shape)))
    axes = positions.shape[1]
    pos_stride = positions.stride()
    if axes > 1 and pos_stride[1] != 1:
        raise ValueError("positions must have contiguous rows, got strides %s" % (pos_stride,))
    if n > 1 and pos_stride[0] >= 1 << 31:   # (ctypes would pass it on modulo 2^32)
        raise ValueError("positions must have rows less than 2^31 entries apart, got %d"
                         % pos_stride[0])
    if freqs.dim() != 1:
        raise ValueError("freqs must be [pairs], got %s" % (tuple(freqs.shape),))
    pairs = freqs.shape[0]
    return p3d_rotary_desc(n, heads, hd, _dtype(x, "x"), ROTARY_LAYOUT[layout], axes, pairs,
                           pos_stride[0] if n > 1 else axes, magnitude, eps,
                           positions.data_ptr(), _ptr(freqs, "freqs", torch.float32, (pairs,)),
                           _ptr(gamma, "gamma", x.dtype, (heads, hd)))


@_lends
def p3d_rotary(x, positions, freqs, out, layout="interleaved", magnitude=1.0, gamma=None,
               eps=1e-6, stream=None):
    """Enqueue p3d_rotary: the heads of x [n, heads, head_dim] (float32 or
    bfloat16; tokens may be strided), rms-normed with gamma [heads, head_dim]
    unless it is None, turned by positions (int32 [n, axes]; coords[:, 1:] is
    a grid cell's) times freqs (float32 [pairs]) into out, which may be x."""
    xp, xs = _heads(x, "x", x.dtype)
    d = _rotary(x, positions, freqs, layout, magnitude, gamma, eps)
    op, os = _heads(out, "out", x.dtype, x.shape[1], x.shape[2], x.shape[0])
    _core._check(lib.p3d_rotary(d, xp, xs, op, os, _stream(stream)))


def p3d_rotary_workspace_size(x, positions, freqs):
    """Bytes of device workspace p3d_rotary_backward needs with dgamma."""
    return _sized(lib.p3d_rotary_workspace_size(
        _rotary(x, positions, freqs, "interleaved", 1.0, None, 1e-6)))


@_lends
def p3d_rotary_backward(dout, positions, freqs, dx, layout="interleaved", magnitude=1.0,
                        gamma=None, eps=1e-6, x=None, dgamma=None, workspace=None, stream=None):
    """Enqueue p3d_rotary_backward: dx from dout [n, heads, head_dim]; with
    gamma, x is the forward call's input and dgamma (float32 [heads,
    head_dim]) is written unless it is None."""
    dp, ds = _heads(dout, "dout", dout.dtype)
    d = _rotary(dout, positions, freqs, layout, magnitude, gamma, eps)
    n, heads, hd = dout.shape
    xp, xs = (None, 0) if x is None else _heads(x, "x", dout.dtype, heads, hd, n)
    op, os = _heads(dx, "dx", dout.dtype, heads, hd, n)
    keep, ws, nbytes = None, None, 0
    if dgamma is not None:
        keep, ws, nbytes = _work(workspace, lambda: lib.p3d_rotary_workspace_size(d), dout.device,
                                 stream)
    _core._check(lib.p3d_rotary_backward(
        d, dp, ds, xp, xs, op, os, _ptr(dgamma, "dgamma", torch.float32, (heads, hd)), ws,
        nbytes, _stream(stream)))


def p3d_rotary_frequencies(base, pairs, scaling="plain", factor=1.0, trained=0.0):
    """The frequency table of one axis (p3d_rotary_frequencies; host-only) as
    a float32 CPU tensor: scaling "plain", "linear", "base" or "by_parts"."""
    freqs = torch.empty(max(0, int(pairs)), dtype=torch.float32)
    _core._check(lib.p3d_rotary_frequencies(float(base), int(pairs), ROTARY_SCALING[scaling],
                                            float(factor), float(trained), freqs.data_ptr()))
    return freqs


# --------------------------------------------------------------- attention ---
def _attention(q, k, q_offsets, k_offsets, scale, causal):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [n, heads, head_dim], got %s and %s"
                         % (tuple(q.shape), tuple(k.shape)))
    nq, heads, hd = q.shape
    nk, kv_heads = k.shape[:2]
    qo = make_offsets((0, nq) if q_offsets is None else q_offsets)
    ko = make_offsets((0, nk) if k_offsets is None else k_offsets)
    if len(qo) != len(ko):
        raise ValueError("q_offsets and k_offsets must have one length, got %d and %d"
                         % (len(qo), len(ko)))
    if qo[-1] != nq or ko[-1] != nk:
        raise ValueError("offsets must end at the rows of q and k (%d, %d), got %d and %d"
                         % (nq, nk, qo[-1], ko[-1]))
    return p3d_attn_desc(ctypes.addressof(qo), ctypes.addressof(ko), len(qo) - 1, heads,
                         kv_heads, hd, _dtype(q, "q"), hd ** -0.5 if scale is None else scale,
                         int(bool(causal))), (qo, ko)


def p3d_attention_workspace_size(q, k, q_offsets=None, k_offsets=None, causal=False):
    """Bytes of device workspace p3d_attention needs."""
    d, off = _attention(q, k, q_offsets, k_offsets, None, causal)
    return _sized(lib.p3d_attention_workspace_size(d))


@_lends
def p3d_attention(q, k, v, out, q_offsets=None, k_offsets=None, scale=None, causal=False,
                  lse=None, workspace=None, stream=None):
    """Enqueue p3d_attention: out [nq, heads, head_dim] from q, k, v ([n,
    heads or kv_heads, head_dim] bfloat16, tokens may be strided) per item of
    the offsets (None: one item); scale None: head_dim ** -0.5; lse: float32
    [nq, heads] or None."""
    d, off = _attention(q, k, q_offsets, k_offsets, scale, causal)
    dt = q.dtype
    nq, heads, hd = q.shape
    nk, kv_heads = k.shape[:2]
    qp, qs = _heads(q, "q", dt)
    kp, ks = _heads(k, "k", dt, kv_heads, hd, nk)
    vp, vs = _heads(v, "v", dt, kv_heads, hd, nk)
    op, os = _heads(out, "out", dt, heads, hd, nq)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_attention_workspace_size(d), q.device,
                             stream)
    _core._check(lib.p3d_attention(d, qp, qs, kp, ks, vp, vs, op, os,
                                   _ptr(lse, "lse", torch.float32, (nq, heads)), ws,
                                   nbytes, _stream(stream)))


def p3d_attention_backward_workspace_size(q, k, q_offsets=None, k_offsets=None, causal=False):
    """Bytes of device workspace p3d_attention_backward needs."""
    d, off = _attention(q, k, q_offsets, k_offsets, None, causal)
    return _sized(lib.p3d_attention_backward_workspace_size(d))


@_lends
def p3d_attention_backward(dout, q, k, v, out, lse, dq, dk, dv, q_offsets=None, k_offsets=None,
                           scale=None, causal=False, workspace=None, stream=None):
    """Enqueue p3d_attention_backward: dq, dk, dv (like q, k, v) from dout,
    and out and lse as p3d_attention wrote them."""
    d, off = _attention(q, k, q_offsets, k_offsets, scale, causal)
    dt = q.dtype
    nq, heads, hd = q.shape
    nk, kv_heads = k.shape[:2]
    args = []
    for name, t, n, h in (("dout", dout, nq, heads), ("q", q, nq, heads), ("k", k, nk, kv_heads),
                          ("v", v, nk, kv_heads), ("out", out, nq, heads)):
        args += _heads(t, name, dt, h, hd, n)
    args.append(_ptr(lse, "lse", torch.float32, (nq, heads)))
    for name, t, n, h in (("dq", dq, nq, heads), ("dk", dk, nk, kv_heads),
                          ("dv", dv, nk, kv_heads)):
        args += _heads(t, name, dt, h, hd, n)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_attention_backward_workspace_size(d),
                             q.device, stream)
    _core._check(lib.p3d_attention_backward(d, *args, ws, nbytes, _stream(stream)))
