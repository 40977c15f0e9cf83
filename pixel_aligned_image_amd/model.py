"""Binding of include/p3d_model.h: the model's operators around the block.

Same rules as block.py: every function has the name of its C entry point,
checks its tensors and passes device pointers and torch's current HIP stream;
results go into tensors the caller gives. Channels-last maps are passed as
rows: a [B, H, W, C] map's ``.view(-1, C)`` with the items' row numbers.
Tensors are on torch's current device.
"""
import ctypes

import torch

from . import block
from ._streams import lends as _lends

__all__ = ["p3d_group_norm", "p3d_group_norm_backward", "p3d_group_norm_workspace_size",
           "p3d_quantize_rows", "p3d_linear_i8", "p3d_adamw", "p3d_grad_norm",
           "p3d_grad_norm_workspace_size", "make_adamw_tensors", "ACT"]

ACT = {"none": 0, "silu": 1, "gelu": 2}                                 # p3d_act

_vp, _i32, _i64, _f32, _f64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                               ctypes.c_double)
_size = ctypes.c_size_t


class p3d_group_desc(ctypes.Structure):
    _fields_ = [("n", _i64), ("offsets", _vp), ("batch", _i32), ("channels", _i32),
                ("groups", _i32), ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", _f32),
                ("weight", _vp), ("bias", _vp)]


class p3d_linear_i8_desc(ctypes.Structure):
    _fields_ = [("n", _i64), ("in_dim", _i32), ("out_dim", _i32), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("weight", _vp), ("weight_scale", _vp), ("bias", _vp)]


class p3d_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("master", _vp), ("grad", _vp), ("m", _vp), ("v", _vp),
                ("m_scale", _vp), ("v_scale", _vp), ("size", _i64), ("weight_decay", _f32)]


class p3d_adamw_desc(ctypes.Structure):
    _fields_ = [("count", _i32), ("tensors", _vp), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("state_bits", _i32), ("lr", _f64), ("beta1", _f64),
                ("beta2", _f64), ("eps", _f64), ("step", _i64), ("seed", ctypes.c_uint64),
                ("grad_scale", _vp), ("device_lr", _vp), ("device_step", _vp)]


lib = None          # set by bind()
_core = None


def bind(core):
    """Declare the entry points on the loaded library (called on import)."""
    global lib, _core
    _core, lib = core, core.lib
    group, linear, adamw = (ctypes.POINTER(t) for t in (p3d_group_desc, p3d_linear_i8_desc,
                                                        p3d_adamw_desc))
    for name, res, args in [
            ("p3d_group_norm_workspace_size", _size, [group]),
            ("p3d_group_norm", ctypes.c_int,
             [group, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _size, _vp]),
            ("p3d_group_norm_backward", ctypes.c_int,
             [group] + [_vp, _i64] * 2 + [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _size, _vp]),
            ("p3d_quantize_rows", ctypes.c_int,
             [_vp, ctypes.c_int, _i64, _i32, _i64, _vp, _i64, _vp, _vp]),
            ("p3d_linear_i8", ctypes.c_int,
             [linear, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp]),
            ("p3d_adamw", ctypes.c_int, [adamw, _vp]),
            ("p3d_grad_norm_workspace_size", _size, [adamw]),
            ("p3d_grad_norm", ctypes.c_int, [adamw, _f32, _vp, _vp, _size, _vp])]:
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ----------------------------------------------------------------- helpers ---
# The smallest calls last a few microseconds, as long as the checks of ten
# tensors: one condition passes what is right, _refuse words what is not.
def _device():
    """The device that a call runs on (of no tensor, before there is one)."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _refuse(t, name, dtype, dev, wanted):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU, got %s" % (name, t.device))
    if t.get_device() != dev:
        raise ValueError("%s must be on torch's current device (%d), got %s"
                         % (name, dev, t.device))
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be %s, got %s, strides %s"
                     % (name, wanted, tuple(t.shape), t.stride()))


def _rows(t, name, dtype, dev, shape=None):
    """(pointer, row stride) of a [n, width] device tensor whose rows may be
    strided."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.dim() == 2 and (shape is None or t.shape == shape)):
        n, width = t.shape
        step, one = t.stride()
        if one == 1 or width <= 1:
            return t.data_ptr(), (step if n > 1 else width)
    _refuse(t, name, dtype, dev, "%s with contiguous rows" % (
        "[n, width]" if shape is None else list(shape)))


def _ptr(t, name, dtype, dev, shape):
    """Pointer of an optional contiguous tensor."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, dev, "%s and contiguous" % (list(shape),))


def _work(workspace, size, dev, stream):
    """As block._work, on the device that the call runs on."""
    if workspace is None:
        return block._work(None, size, torch.device("cuda", dev), stream)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        _refuse(workspace, "workspace", torch.uint8, dev, "a buffer of bytes")
    return block._work(workspace, size, None, stream)


def _choice(table, name, value):
    if value not in table:
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(table), value))
    return table[value]


# -------------------------------------------------------------- group norm ---
def _group(x, groups, offsets, weight, bias, act, eps, dev):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [n, channels], got %s" % (tuple(getattr(x, "shape", ())),))
    n, c = x.shape
    off = block.make_offsets((0, n) if offsets is None else offsets)
    dt = x.dtype
    d = p3d_group_desc(n, ctypes.addressof(off), len(off) - 1, c, int(groups),
                       block._dtype(x, "x"), _choice(ACT, "act", act), eps,
                       _ptr(weight, "weight", dt, dev, (c,)), _ptr(bias, "bias", dt, dev, (c,)))
    return d, off


def p3d_group_norm_workspace_size(x, groups, offsets=None):
    """Bytes of device workspace p3d_group_norm and p3d_group_norm_backward
    need for rows like x's."""
    d, off = _group(x, groups, offsets, None, None, "none", 1e-5, None)
    return block._sized(lib.p3d_group_norm_workspace_size(d))


@_lends
def p3d_group_norm(x, out, groups, offsets=None, weight=None, bias=None, act="none", eps=1e-5,
                   mean=None, rstd=None, workspace=None, stream=None):
    """Enqueue p3d_group_norm: out = act((x - mean) rstd weight + bias) with an
    item's mean and rstd over its rows and each of `groups` ranges of channels.
    x, out: [n, channels] float32 or bfloat16 (rows may be strided; out may be
    x); weight, bias: [channels]; act: "none", "silu" or "gelu" (its tanh form:
    torch's approximate="tanh"); mean, rstd: float32 [batch, groups], written
    unless None (the gradient needs them); offsets: the items' rows (None: one
    item)."""
    dev, f = _device(), torch.float32
    d, off = _group(x, groups, offsets, weight, bias, act, eps, dev)
    xp, xs = _rows(x, "x", x.dtype, dev)
    op, os = _rows(out, "out", x.dtype, dev, x.shape)
    stats = (d.batch, d.groups)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_group_norm_workspace_size(d), dev, stream)
    _core._check(lib.p3d_group_norm(d, xp, xs, op, os, _ptr(mean, "mean", f, dev, stats),
                                    _ptr(rstd, "rstd", f, dev, stats), ws, nbytes,
                                    block._stream(stream)))


@_lends
def p3d_group_norm_backward(dout, x, mean, rstd, dx, groups, offsets=None, weight=None, bias=None,
                            act="none", dweight=None, dbias=None, workspace=None, stream=None):
    """Enqueue p3d_group_norm_backward: dx (which may be dout or x) from dout,
    the forward call's x and the mean and rstd it wrote; float32 dweight and
    dbias [channels], each None where it is not wanted."""
    dev, dt, f = _device(), x.dtype, torch.float32
    d, off = _group(x, groups, offsets, weight, bias, act, 1e-5, dev)
    xp, xs = _rows(x, "x", dt, dev)
    dp, ds = _rows(dout, "dout", dt, dev, x.shape)
    op, os = _rows(dx, "dx", dt, dev, x.shape)
    stats, cols = (d.batch, d.groups), (d.channels,)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_group_norm_workspace_size(d), dev, stream)
    _core._check(lib.p3d_group_norm_backward(
        d, dp, ds, xp, xs, _ptr(mean, "mean", f, dev, stats), _ptr(rstd, "rstd", f, dev, stats),
        op, os, _ptr(dweight, "dweight", f, dev, cols), _ptr(dbias, "dbias", f, dev, cols), ws,
        nbytes, block._stream(stream)))


# ------------------------------------------------------------------ linear ---
@_lends
def p3d_quantize_rows(x, q, scale, stream=None):
    """Enqueue p3d_quantize_rows: q (int8, like x) and scale (float32 [n]) of
    the rows of x [n, width], float32 or bfloat16 (rows may be strided):
    tokens, or a weight [out, in]."""
    dev = _device()
    xp, xs = _rows(x, "x", x.dtype, dev)
    qp, qs = _rows(q, "q", torch.int8, dev, x.shape)
    n, width = x.shape
    _core._check(lib.p3d_quantize_rows(xp, block._dtype(x, "x"), n, width, xs, qp, qs,
                                       _ptr(scale, "scale", torch.float32, dev, (n,)),
                                       block._stream(stream)))


@_lends
def p3d_linear_i8(q, scale, weight, weight_scale, out, bias=None, act="none", residual=None,
                  stream=None):
    """Enqueue p3d_linear_i8: out = act(q weight^T scale weight_scale + bias) +
    residual. q: int8 [n, in] (rows may be strided) and scale: float32 [n] of
    p3d_quantize_rows; weight: int8 [out, in]; weight_scale: float32 [out];
    out, residual: [n, out] and bias: [out], float32 or bfloat16 (residual may
    be out); act: "none", "silu" or "gelu" (its tanh form)."""
    dev, dt, f = _device(), out.dtype, torch.float32
    qp, qs = _rows(q, "q", torch.int8, dev)
    n, k = q.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [out, in], got %s"
                         % (tuple(getattr(weight, "shape", ())),))
    m = weight.shape[0]
    op, os = _rows(out, "out", dt, dev, (n, m))
    rp, rs = (None, 0) if residual is None else _rows(residual, "residual", dt, dev, (n, m))
    d = p3d_linear_i8_desc(n, k, m, block._dtype(out, "out"), _choice(ACT, "act", act),
                           _ptr(weight, "weight", torch.int8, dev, (m, k)),
                           _ptr(weight_scale, "weight_scale", f, dev, (m,)),
                           _ptr(bias, "bias", dt, dev, (m,)))
    _core._check(lib.p3d_linear_i8(d, qp, qs, _ptr(scale, "scale", f, dev, (n,)), rp, rs, op, os,
                                   block._stream(stream)))


# ------------------------------------------------------------------- adamw ---
class AdamWTensors(tuple):
    """The tensors of p3d_adamw and their table (make_adamw_tensors)."""


def _flat(t, name, dtype, dev, size):
    """Pointer of a contiguous device tensor of `size` elements, of a type or
    one of several."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.numel() == size
            and (t.dtype is dtype or isinstance(dtype, tuple) and t.dtype in dtype)
            and t.is_contiguous()):
        return t.data_ptr() if size else None
    _refuse(t, name, dtype, dev, "%d contiguous elements" % size)


def make_adamw_tensors(params, grads, m, v, masters=None, m_scales=None, v_scales=None,
                       weight_decay=0.0):
    """The table of p3d_adamw and p3d_grad_norm, for callers to keep over the
    steps: lists of contiguous tensors, one entry a parameter (of any shape).
    params: float32 or bfloat16; grads: likewise; m, v: float32, or 8-bit
    (torch.float8_e4m3fn or uint8) with float32 m_scales and v_scales of
    (size + 255) // 256; masters: float32 copies of bfloat16 params, or None;
    weight_decay: a number or one for each. The table keeps the memory
    that the tensors have now: a gradient in another tensor, or a parameter whose
    .data was replaced, needs another table. (torch's zero_grad() drops the
    gradients, and the next backward makes others: a step with the old table would
    take the old ones. zero_grad(set_to_none=False) keeps them.) Making a
    table costs some 3 us a tensor."""
    params, grads, m, v = list(params), list(grads), list(m), list(v)
    n = len(params)
    lists = [("grads", grads), ("m", m), ("v", v)]
    masters, m_scales, v_scales = (None if x is None else list(x)
                                   for x in (masters, m_scales, v_scales))
    lists += [(k, x) for k, x in (("masters", masters), ("m_scales", m_scales),
                                  ("v_scales", v_scales)) if x is not None]
    decay = ([float(w) for w in weight_decay] if hasattr(weight_decay, "__len__")
             else [float(weight_decay)] * n)
    for name, x in lists + [("weight_decay", decay)]:
        if len(x) != n:
            raise ValueError("%s must have one entry for each of %d params, got %d"
                             % (name, n, len(x)))
    if (m_scales is None) != (v_scales is None):
        raise ValueError("m_scales and v_scales go together")
    pt, gt = (x[0].dtype if n else torch.float32 for x in (params, grads))
    for x, name in ((pt, "params"), (gt, "grads")):
        if x not in _core._DT:
            raise TypeError("%s must be float32 or bfloat16, got %s" % (name, x))
    bits = 32 if m_scales is None else 8
    st = torch.float32 if bits == 32 else (torch.float8_e4m3fn, torch.uint8)
    f = torch.float32
    rows, dev = (p3d_adamw_tensor * max(1, n))(), _device()
    for j in range(n):
        size, to = params[j].numel(), rows[j]
        blocks = (size + 255) // 256
        to.param = _flat(params[j], "params[%d]" % j, pt, dev, size)
        to.grad = _flat(grads[j], "grads[%d]" % j, gt, dev, size)
        to.m = _flat(m[j], "m[%d]" % j, st, dev, size)
        to.v = _flat(v[j], "v[%d]" % j, st, dev, size)
        if masters is not None:
            to.master = _flat(masters[j], "masters[%d]" % j, f, dev, size)
        if bits == 8:
            to.m_scale = _flat(m_scales[j], "m_scales[%d]" % j, f, dev, blocks)
            to.v_scale = _flat(v_scales[j], "v_scales[%d]" % j, f, dev, blocks)
        to.size, to.weight_decay = size, decay[j]
    # (aliases: a parameter whose .data is replaced leaves the old memory)
    table = AdamWTensors(t.detach() for t in params + grads + m + v + (masters or [])
                         + (m_scales or []) + (v_scales or []))
    table.rows, table.count, table.bits = rows, n, bits
    table.param_dtype, table.grad_dtype = _core._DT[pt], _core._DT[gt]
    table.index = dev
    return table


def _adamw(tensors):
    if not isinstance(tensors, AdamWTensors):
        raise TypeError("tensors must be a table of make_adamw_tensors")
    dev = _device()
    if tensors.index != dev:
        raise ValueError("tensors must be on torch's current device (%d), got %d"
                         % (dev, tensors.index))
    return dev, p3d_adamw_desc(tensors.count, ctypes.addressof(tensors.rows),
                               tensors.param_dtype, tensors.grad_dtype, tensors.bits)


@_lends
def p3d_adamw(tensors, lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, grad_scale=None,
              device_lr=None, device_step=None, stream=None):
    """Enqueue p3d_adamw: step `step` (from 1 on) on a table of
    make_adamw_tensors. grad_scale: float32 device tensor of one element (the
    second of p3d_grad_norm's result) or None; seed: of the random bits that
    8-bit states are rounded by, another for every step (a device_step is added
    to it); device_lr, device_step: float32 / int32 device tensors of one element
    that are read instead of lr and step when the work runs, or None. The weights
    are written as memory: their torch version counters stay, so a graph that was
    recorded before the step must not be differentiated after it (torch would not
    notice)."""
    dev, d = _adamw(tensors)
    d.lr, d.beta1, d.beta2, d.eps, d.step = lr, beta1, beta2, eps, step
    d.seed = seed & 0xffffffffffffffff
    f = torch.float32
    for name, t, dt in (("grad_scale", grad_scale, f), ("device_lr", device_lr, f),
                        ("device_step", device_step, torch.int32)):
        if t is not None:
            setattr(d, name, _flat(t, name, dt, dev, 1))
    _core._check(lib.p3d_adamw(d, block._stream(stream)))


def p3d_grad_norm_workspace_size(tensors):
    """Bytes of device workspace p3d_grad_norm needs."""
    return block._sized(lib.p3d_grad_norm_workspace_size(_adamw(tensors)[1]))


@_lends
def p3d_grad_norm(tensors, out, max_norm=float("inf"), workspace=None, stream=None):
    """Enqueue p3d_grad_norm: out (float32 [2]) = the norm over the table's
    gradients, and the factor that brings it to max_norm where it is above (NaN
    where it is not finite)."""
    dev, d = _adamw(tensors)
    keep, ws, nbytes = _work(workspace, lambda: lib.p3d_grad_norm_workspace_size(d), dev, stream)
    _core._check(lib.p3d_grad_norm(d, max_norm, _ptr(out, "out", torch.float32, dev, (2,)), ws,
                                   nbytes, block._stream(stream)))
