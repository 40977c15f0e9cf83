"""Plain 64-bit forms of the model's operators, from the formulas in
include/p3d_model.h: loops over items and groups and torch's elementary
operations on the CPU; group norm's gradients by torch's differentiation of
the forward form (checked against differences in test_model_ref.py). Test
infrastructure only; shares no code with the library."""
import math

import torch

F64 = torch.float64
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
U = 2.0 ** -24                                                  # one binary32 rounding


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def act(u, kind):
    if kind == "silu":
        return u * torch.sigmoid(u)
    if kind == "gelu":
        return u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))) / 2
    return u


# -------------------------------------------------------------- group norm ---
def group_stats(x, offsets, groups, eps):
    """mean, rstd [batch, groups]"""
    batch, c = len(offsets) - 1, x.shape[1]
    mean = torch.zeros(batch, groups, dtype=x.dtype)
    rstd = torch.full((batch, groups), eps ** -0.5, dtype=x.dtype)
    for b in range(batch):
        rows = x[offsets[b]:offsets[b + 1]].reshape(-1, groups, c // groups)
        if rows.shape[0]:
            mean[b] = rows.mean((0, 2))
            rstd[b] = ((rows - mean[b][:, None]) ** 2).mean((0, 2)).add(eps).rsqrt()
    return mean, rstd


def spread(v, offsets, channels):
    """[batch, groups] -> [n, channels]"""
    each = torch.tensor(offsets).diff()
    return v.repeat_interleave(channels // v.shape[1], 1).repeat_interleave(each, 0)


def group_norm(x, offsets, groups, weight=None, bias=None, kind="none", eps=1e-5):
    """(out, u): differentiable"""
    c = x.shape[1]
    outs = []
    for b in range(len(offsets) - 1):
        rows = x[offsets[b]:offsets[b + 1]].reshape(-1, groups, c // groups)
        if rows.shape[0] == 0:
            continue
        d = rows - rows.mean((0, 2), keepdim=True)
        outs.append((d / (d.square().mean((0, 2), keepdim=True) + eps).sqrt()).reshape(-1, c))
    u = torch.cat(outs) if outs else x * 1
    if weight is not None:
        u = u * weight
    if bias is not None:
        u = u + bias
    return act(u, kind), u


def group_norm_backward(dout, x, offsets, groups, weight=None, bias=None, kind="none", eps=1e-5):
    """{dx, dweight, dbias} by differentiation"""
    c = x.shape[1]
    leaves = {"x": x.clone(), "weight": torch.ones(c, dtype=x.dtype) if weight is None else
              weight.clone(), "bias": torch.zeros(c, dtype=x.dtype) if bias is None else
              bias.clone()}
    for t in leaves.values():
        t.requires_grad_(True)
    out, _ = group_norm(leaves["x"], offsets, groups, leaves["weight"], leaves["bias"], kind, eps)
    (out * dout).sum().backward()
    return {"d" + k if k != "x" else "dx": (t.grad if t.grad is not None else
                                            torch.zeros_like(t)).detach()
            for k, t in leaves.items()}


# ------------------------------------------------------------------ linear ---
def quantize(x):
    """(q, scale): the scale as binary32 holds it (the product of two of its
    numbers is exact here, and rounded once), the quotients exact."""
    top = x.abs().amax(1)
    scale = (top * (torch.ones(1) / 127).double()).float().double()
    scale[~torch.isfinite(top)] = math.nan
    by = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = (x / by).round().clamp(-127, 127)
    q[~(scale > 0)] = 0
    return q, scale


def linear(q, scale, weight, weight_scale, bias=None, kind="none", residual=None):
    """(out, how large the terms before the activation are)"""
    y = (q @ weight.t()) * scale[:, None] * weight_scale
    size = y.abs()
    if bias is not None:
        y, size = y + bias, size + bias.abs()
    out = act(y, kind)
    if residual is not None:
        out, size = out + residual, size + residual.abs()
    return out, size


# ------------------------------------------------------------------- adamw ---
def mix(x):
    m = 0xffffffff
    x ^= x >> 15
    x = x * 0xB504F335 & m
    x ^= x >> 13
    x = x * 0xDDB3D743 & m
    return x ^ x >> 16


def random_bits(first, count, number, seed):
    """The 32 bits of elements first .. first + count - 1 of tensor `number`."""
    m = 0xffffffff
    key = mix((number * 0x9E3779B1 & m) ^ mix(seed & m) ^ (seed >> 32 & m))
    return [mix((i * 0x9E3779B1 & m) ^ ((i >> 32) * 0xDDB3D743 & m) ^ key)
            for i in range(first, first + count)]


def encode(q, bits):
    """The e4m3 value that 16 random bits choose for each of q."""
    a = q.abs().clamp(max=448.0)
    exponent = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    # (log2 of a number just below a power of two may round up to it)
    exponent = torch.where(2.0 ** exponent > a.clamp(min=2.0 ** -6), exponent - 1, exponent)
    step = 2.0 ** (exponent - 3)
    return (torch.floor(a / step + bits / 65536) * step).clamp(max=448.0) * q.sign()


def blocks(x):
    return torch.cat([x, x.new_zeros(-x.numel() % 256)]).reshape(-1, 256)


def adamw(w, g, m, v, lr, beta1, beta2, eps, step, decay, grad_scale=1.0):
    """(w, m, v) of one tensor; v is the second moment itself."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = m / (1 - beta1 ** step) / ((v / (1 - beta2 ** step)).sqrt() + eps)
    return w - lr * decay * w - lr * update, m, v
