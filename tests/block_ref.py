"""Plain 64-bit forms of the transformer-block operators, from the formulas in
include/p3d_block.h: loops over items and heads and torch's elementary
operations on the CPU, gradients by torch's differentiation of the forward
form (checked against differences in test_block_ref.py). Test infrastructure
only; shares no code with the library."""
import math

import torch

F64 = torch.float64


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def uneven(total, items):
    """An item table with empty, short and long items."""
    weights = [(i * 7 + 3) % 5 for i in range(items)]
    if sum(weights) == 0:
        weights[0] = 1
    at, ends = 0, [0]
    for w in weights:
        at += w
        ends.append(total * at // sum(weights))
    return ends


# -------------------------------------------------------------- gated norm ---
def normed(v, kind, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v / (v.square().mean(1, keepdim=True) + eps).sqrt()


def gated_norm(x, offsets, y=None, gate=None, scale=None, shift=None, pre="layer", post="none",
               weight=None, bias=None, post_weight=None, res_scale=1.0, eps=1e-6):
    """(r, h)"""
    rs, hs = [], []
    for b in range(len(offsets) - 1):
        rows = slice(offsets[b], offsets[b + 1])
        r = x[rows]
        if y is not None:
            t = normed(y[rows], post, eps)
            if post_weight is not None:
                t = t * post_weight
            r = r + res_scale * (t * gate[b] if gate is not None else t)
        z = normed(r, pre, eps)
        if weight is not None:
            z = z * weight
        if bias is not None:
            z = z + bias
        if scale is not None:
            z = z * (1 + scale[b])
        if shift is not None:
            z = z + shift[b]
        rs.append(r)
        hs.append(z)
    return torch.cat(rs), torch.cat(hs)


# ------------------------------------------------------------------ rotary ---
def rotary(x, positions, freqs, layout, magnitude=1.0, gamma=None, eps=1e-6):
    """x [n, heads, head_dim]"""
    if gamma is not None:
        x = x / (x.square().mean(2, keepdim=True) + eps).sqrt() * gamma
    angle = (positions.to(F64)[:, :, None] * freqs.to(F64)).flatten(1)
    p = angle.shape[1]
    cos, sin = (magnitude * f(angle)[:, None] for f in (torch.cos, torch.sin))
    if layout == "half":
        u, w, rest = x[..., :p], x[..., p:2 * p], x[..., 2 * p:]
        return torch.cat([u * cos - w * sin, u * sin + w * cos, rest], 2)
    u, w, rest = x[..., 0:2 * p:2], x[..., 1:2 * p:2], x[..., 2 * p:]
    turned = torch.stack([u * cos - w * sin, u * sin + w * cos], 3).flatten(2)
    return torch.cat([turned, rest], 2)


# --------------------------------------------------------------- attention ---
def seen_by(nq, nk, causal):
    """Which keys each query sees [nq, nk]."""
    if not causal:
        return torch.ones(nq, nk, dtype=torch.bool)
    return torch.arange(nk)[None] <= torch.arange(nq)[:, None] + nk - nq


def attention_head(q, k, v, scale, causal):
    """(out, lse, P) of one head of one item."""
    s = scale * (q @ k.T)
    see = seen_by(q.shape[0], k.shape[0], causal)
    s = s.masked_fill(~see, -math.inf)
    top = s.detach().amax(1, keepdim=True) if s.shape[1] else s.new_full((s.shape[0], 1), 0.0)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = (s - top).exp()
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    return p @ v, (top + total.log())[:, 0], p


def attention(q, k, v, q_offsets, k_offsets, scale, causal):
    """(out, lse, reach): reach = sum_j P_ij |v_j|, the size that the rounding
    of the probabilities acts on."""
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    outs, lses, reaches = [], [], []
    for b in range(len(q_offsets) - 1):
        rows, keys = slice(*q_offsets[b:b + 2]), slice(*k_offsets[b:b + 2])
        per = [attention_head(q[rows, h], k[keys, h // group], v[keys, h // group], scale, causal)
               for h in range(heads)]
        outs.append(torch.stack([o for o, _, _ in per], 1))
        lses.append(torch.stack([l for _, l, _ in per], 1))
        reaches.append(torch.stack([p @ v[keys, h // group].abs()
                                    for h, (_, _, p) in enumerate(per)], 1))
    return torch.cat(outs), torch.cat(lses), torch.cat(reaches)


def attention_backward(dout, q, k, v, q_offsets, k_offsets, scale, causal):
    """dq, dk, dv by the formulas, and for each how far a result may be off
    when P and dS are rounded to bf16 (2^-8 of themselves: 8 significant bits),
    out (in D) and the results as well, and everything else is good to 2^-14 of the terms that it
    adds up."""
    group = q.shape[1] // k.shape[1]
    u, slack = 2.0 ** -8, 2.0 ** -14
    res = {n: torch.zeros_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    for b in range(len(q_offsets) - 1):
        rows, keys = slice(*q_offsets[b:b + 2]), slice(*k_offsets[b:b + 2])
        for h in range(q.shape[1]):
            qh, doh = q[rows, h], dout[rows, h]
            kh, vh = k[keys, h // group], v[keys, h // group]
            o, _, p = attention_head(qh, kh, vh, scale, causal)
            dp = doh @ vh.T
            d = (doh * o).sum(1, keepdim=True)
            ds = p * (dp - d)
            # out is off by 2 u sum p |v| at most (P rounded, out rounded)
            d_off = 2 * u * (doh.abs() * (p @ vh.abs())).sum(1, keepdim=True)
            sized = p * (doh.abs() @ vh.abs().T + d.abs())
            ds_off = u * ds.abs() + p * d_off + slack * sized
            res["dq"][rows, h] = scale * (ds @ kh)
            tol["dq"][rows, h] = scale * (ds_off @ kh.abs()) + u * res["dq"][rows, h].abs()
            res["dk"][keys, h // group] += scale * (ds.T @ qh)
            tol["dk"][keys, h // group] += scale * (ds_off.T @ qh.abs())
            res["dv"][keys, h // group] += p.T @ doh
            tol["dv"][keys, h // group] += (u + slack) * (p.T @ doh.abs())
    for n in ("dk", "dv"):
        tol[n] += u * res[n].abs()
    return res, tol


# --------------------------------------------------------------- tolerances ---
def off_by(got, want, tol):
    """The largest |got - want| / tol; entries that are not finite have to
    agree."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    assert torch.equal(got[bad & ~torch.isnan(want)], want[bad & ~torch.isnan(want)])
    if not got.numel():
        return 0.0
    d = torch.where(bad, torch.zeros_like(want), (got - want).abs())
    t = torch.as_tensor(tol, dtype=F64).expand_as(d)
    return float((d / (t + 1e-30)).max())


def rounded_once(want, dtype, sized=None):
    """Tolerance of a row-wise result [n, ..., d]: one rounding of the result
    (half an ulp: 2^-8 of bf16's 8 significant bits, taken as 2^-7.9 for results that a binary32
    error moves across a tie), and binary32 arithmetic good to 2^-17 of the
    row's root mean square `sized` (of the result itself where not given):
    sums of up to 8192 terms, in lane shares of at most 32 and a tree of 8
    levels, stay under 40 roundings of 2^-24 each, and a result passes a
    handful of such sums."""
    s = want if sized is None else sized
    rms = s.square().mean(-1, keepdim=True).sqrt()
    fine = 2.0 ** -17 * (rms + want.abs())
    return fine + (2.0 ** -7.9 * want.abs() if dtype == torch.bfloat16 else 0)


def rms_off(got, want):
    """The difference's 2-norm over the result's."""
    got, want = f64(got), f64(want)
    return float((got - want).norm() / want.norm())
