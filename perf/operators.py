"""Cases of the transformer-block operators: the gated norm, rotary positions
and attention, forward and with their gradients.

The sizes are this repository's own token budgets (a dense 16^3 grid, 7000
sparse tokens in two items, 100,000 and 200,000 sparse tokens), model widths
(1024 and 1536) and key counts (5 global tokens, 1029 image tokens), and
generic long contexts for single tokens.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # the five global tokens of one image between two blocks: latency
        {"name": "norm_global5", "op": "norm", "train": False, "dtype": BF16, "tokens": 5,
         "items": 1, "dim": 1536, "pre": "layer", "post": "none"},
        # one denoising step's modulated norm over a 100,000-token sparse shell
        {"name": "norm_shell100k", "op": "norm", "train": False, "dtype": BF16,
         "tokens": 100000, "items": 1, "dim": 1536, "pre": "layer", "post": "none"},
        # a training step in 32 bits on the dense 16^3 grid, sandwich norms
        {"name": "norm_train_dense16", "op": "norm", "train": True, "dtype": F32,
         "tokens": 4096, "items": 1, "dim": 1024, "pre": "rms", "post": "rms"},
        # a training step over two ragged items, 200,000 sparse tokens in all
        {"name": "norm_train_200k", "op": "norm", "train": True, "dtype": BF16,
         "tokens": 200000, "items": 2, "dim": 1536, "pre": "layer", "post": "none"},
        # seven new tokens of a long 1-D context (scaled), split-half layout
        {"name": "rotary_tokens7", "op": "rotary", "train": False, "dtype": BF16, "tokens": 7,
         "heads": 20, "head_dim": 128, "axes": 1, "pairs": 64, "layout": "half",
         "scaled": True, "norm": False},
        # q and k of a 100,000-token sparse shell: rms-normed, three grid axes
        {"name": "rotary_shell100k", "op": "rotary", "train": False, "dtype": BF16,
         "tokens": 100000, "heads": 24, "head_dim": 128, "axes": 3, "pairs": 21,
         "layout": "interleaved", "scaled": False, "norm": True},
        # a training step in 32 bits on the dense 16^3 grid, part of the head
        {"name": "rotary_train_dense16", "op": "rotary", "train": True, "dtype": F32,
         "tokens": 4096, "heads": 32, "head_dim": 64, "axes": 3, "pairs": 8, "layout": "half",
         "scaled": False, "norm": True},
        # single tokens of four requests over ragged contexts, shared heads
        {"name": "attn_single", "op": "attention", "train": False, "queries": 4, "keys": 40001,
         "items": 4, "heads": 16, "kv_heads": 4, "head_dim": 128, "causal": True},
        # cross-attention of 100,000 sparse tokens over the five global tokens
        {"name": "attn_global5", "op": "attention", "train": False, "queries": 100000, "keys": 5,
         "items": 1, "heads": 12, "kv_heads": 12, "head_dim": 128, "causal": False},
        # self-attention of a cascade's sparse tokens in one denoising step
        {"name": "attn_self12k", "op": "attention", "train": False, "queries": 12000,
         "keys": 12000, "items": 1, "heads": 12, "kv_heads": 12, "head_dim": 128,
         "causal": False},
        # a training step on two ragged items over 2 x 1029 image tokens
        {"name": "attn_train_image1029", "op": "attention", "train": True, "queries": 7000,
         "keys": 2058, "items": 2, "heads": 16, "kv_heads": 16, "head_dim": 64,
         "causal": False},
        # a causal training step over one long odd sequence with shared heads
        {"name": "attn_train_causal", "op": "attention", "train": True, "queries": 12289,
         "keys": 12289, "items": 1, "heads": 12, "kv_heads": 4, "head_dim": 128,
         "causal": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "attention"])
    train = rng.random() < 0.5
    if op == "norm":
        return {"op": op, "train": train, "dtype": rng.choice([BF16, F32]),
                "tokens": _log(rng, 1, 100000), "items": _log(rng, 1, 16),
                "dim": 8 * _log(rng, 16, 256), "pre": rng.choice(["layer", "rms"]),
                "post": rng.choice(["none", "layer", "rms"])}
    if op == "rotary":
        head_dim = 8 * rng.randint(4, 16)
        axes = rng.choice([1, 2, 3])
        return {"op": op, "train": train, "dtype": rng.choice([BF16, F32]),
                "tokens": _log(rng, 1, 60000), "heads": rng.randint(1, 32),
                "head_dim": head_dim, "axes": axes,
                "pairs": rng.randint(1, head_dim // 2 // axes),
                "layout": rng.choice(["interleaved", "half"]), "scaled": rng.random() < 0.5,
                "norm": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 3, 4, 6])
    heads = kv_heads * rng.choice([1, 1, 2, 4] if kv_heads <= 3 else [1, 1, 2])
    head_dim = rng.choice([64, 64, 80, 96, 128, 128])
    keys = _log(rng, 1, 10000)
    shape = rng.choice(["self", "cross", "single"])
    items = _log(rng, 1, 8)
    queries = keys if shape == "self" else _log(rng, 1, 10000) if shape == "cross" else items
    return {"op": op, "train": train and shape != "single", "queries": queries, "keys": keys,
            "items": items, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "causal": shape == "single" or rng.random() < 0.4}


# ------------------------------------------------------------------- sizes ---
def _offsets(total, items):
    """Row ranges of `items` uneven items (weights items, items + 1, ...)."""
    weights = [items + i for i in range(items)]
    at, ends, whole = 0, [0], sum(weights)
    for w in weights:
        at += w
        ends.append(total * at // whole)
    return ends


def _attention_offsets(case):
    items = case["items"]
    if case["queries"] == items:
        q_off = list(range(items + 1))
    else:
        q_off = _offsets(case["queries"], items)
    return q_off, _offsets(case["keys"], items)


def _pairs_seen(case):
    """Query-key pairs that the mask leaves, over all items (of one head)."""
    q_off, k_off = _attention_offsets(case)
    seen = 0
    for b in range(case["items"]):
        nq, nk = q_off[b + 1] - q_off[b], k_off[b + 1] - k_off[b]
        if not case["causal"]:
            seen += nq * nk
        elif nk >= nq:                       # query i sees nk - nq + i + 1 keys
            seen += nq * (nk - nq) + nq * (nq + 1) // 2
        else:                                # the first nq - nk queries see none
            seen += nk * (nk + 1) // 2
    return seen


def work(case):
    e = 4 if case.get("dtype") == F32 else 2
    if case["op"] == "norm":
        n, d, items = case["tokens"], case["dim"], case["items"]
        # x, y in; r, h out. With gradients: dh, dr in; dx, dy out
        planes = 8 if case["train"] else 4
        parameters = 3 * items * d + 3 * d
        return {"bytes": e * (planes * n * d + parameters)
                + (4 * (3 * items * d + 3 * d) if case["train"] else 0),
                "flops": (60 if case["train"] else 20) * n * d}
    if case["op"] == "rotary":
        n, w = case["tokens"], case["heads"] * case["head_dim"]
        planes = 4 if case["train"] else 2
        return {"bytes": e * planes * n * w + 4 * n * case["axes"] + 4 * case["pairs"]
                + (e * w if case["norm"] else 0)
                + (4 * w if case["norm"] and case["train"] else 0),
                "flops": (24 if case["train"] else 8) * n * w}
    nq, nk, hd = case["queries"], case["keys"], case["head_dim"]
    hq, hk = case["heads"], case["kv_heads"]
    q_plane, kv_plane = nq * hq * hd, nk * hk * hd
    # q, k, v in; out and lse out. With gradients: dout in; dq, dk, dv out
    data = 2 * (2 * q_plane + 2 * kv_plane) + 4 * nq * hq
    products = 2
    if case["train"]:
        data += 2 * (2 * q_plane + 2 * kv_plane)
        products = 7
    return {"bytes": data, "flops": 2 * products * hq * hd * _pairs_seen(case)}


# ------------------------------------------------------------------ inputs ---
def _type(name):
    return torch.float32 if name == F32 else torch.bfloat16


def _frequencies(case):
    """Frequencies of one axis's pairs; scaled: a context 8 times as long as
    the trained 4096 positions (slow pairs by interpolation, fast ones as
    they were, a ramp between 1 and 32 turns over the trained length)."""
    i = torch.arange(case["pairs"], dtype=torch.float64)
    f = BASE ** (-i / case["pairs"])
    if case["scaled"]:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / 8 * (1 - keep)
    return f.float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return (t * scale + mean).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        n, d, items, t = case["tokens"], case["dim"], case["items"], _type(case["dtype"])
        s["offsets"] = _offsets(n, items)
        # a residual stream with a few large columns, as trained models have
        columns = randn(d, scale=0.5, dtype=torch.float32).exp()
        s["x"] = (randn(n, d, dtype=torch.float32) * columns + 0.1).to(t)
        s["y"] = randn(n, d, scale=0.7, dtype=t)
        for k in ("gate", "scale", "shift"):
            s[k] = randn(items, d, scale=0.3, dtype=t)
        rms = case["pre"] == "rms"
        s["weight"] = randn(d, scale=0.2, mean=1.0, dtype=t) if rms else None
        s["post_weight"] = (randn(d, scale=0.2, mean=1.0, dtype=t)
                            if case["post"] != "none" else None)
        s["res_scale"] = 0.5 if case["post"] != "none" else 1.0
        s["r"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        if case["train"]:
            s["dh"], s["dr"] = randn(n, d, dtype=t), randn(n, d, dtype=t)
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            for k in ("dgate", "dscale", "dshift"):
                s[k] = torch.empty(items, d, device="cuda")
            s["dweight"] = torch.empty(d, device="cuda") if rms else None
            s["dpost_weight"] = (torch.empty(d, device="cuda") if case["post"] != "none"
                                 else None)
    elif case["op"] == "rotary":
        n, heads, hd, t = case["tokens"], case["heads"], case["head_dim"], _type(case["dtype"])
        s["x"] = randn(n, heads, hd, dtype=t)
        if case["axes"] == 1:
            # consecutive tokens of a context of up to 32768
            start = int(torch.randint(0, max(1, 32768 - n), (1,), generator=g, device="cuda"))
            s["positions"] = (start + torch.arange(n, device="cuda") % 32768).int()[:, None]
            s["positions"] = s["positions"].contiguous()
        else:
            s["positions"] = torch.randint(0, 1024, (n, case["axes"]), generator=g,
                                           device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(case).cuda()
        s["magnitude"] = 1 + 0.1 * math.log(8) if case["scaled"] else 1.0
        s["gamma"] = randn(heads, hd, scale=0.2, mean=1.0, dtype=t) if case["norm"] else None
        s["out"] = torch.empty_like(s["x"])
        if case["train"]:
            s["dout"] = randn(n, heads, hd, dtype=t)
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(heads, hd, device="cuda") if case["norm"] else None
    else:
        nq, nk, hd = case["queries"], case["keys"], case["head_dim"]
        hq, hk = case["heads"], case["kv_heads"]
        s["q_offsets"], s["k_offsets"] = _attention_offsets(case)
        s["q"] = randn(nq, hq, hd)
        packed = randn(nk, 2 * hk, hd)       # keys and values of one projection
        s["k"], s["v"] = packed[:, :hk], packed[:, hk:]
        s["scale"] = hd ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(nq, hq, device="cuda")
        if case["train"]:
            s["dout"] = randn(nq, hq, hd)
            s["dq"] = torch.empty_like(s["q"])
            s["dk"], s["dv"] = (torch.empty(nk, hk, hd, device="cuda", dtype=torch.bfloat16)
                                for _ in range(2))
    return s


# -------------------------------------------------------- the plain forms ---
def _row_items(offsets):
    """The item of every row."""
    lengths = torch.tensor(offsets, device="cuda").diff()
    return torch.repeat_interleave(torch.arange(len(offsets) - 1, device="cuda"), lengths)


def _normalise(x, kind):
    """x^ and the reciprocal deviation of every row."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    rstd = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    return x * rstd, rstd


def _normalise_backward(d, xn, rstd, kind):
    if kind == "none":
        return d
    g = d - xn * (d * xn).mean(1, keepdim=True)
    if kind == "layer":
        g = g - d.mean(1, keepdim=True)
    return g * rstd


def _item_sums(v, item, items):
    return torch.zeros(items, v.shape[1], device="cuda").index_add_(0, item, v)


def _norm_plain(s):
    t = s["x"].dtype
    item = _row_items(s["offsets"])
    x, y = s["x"].float(), s["y"].float()
    gate, scale, shift = (s[k].float() for k in ("gate", "scale", "shift"))
    yn, y_rstd = _normalise(y, s["post"])
    pw = s["post_weight"].float() if s["post_weight"] is not None else None
    tn = yn * pw if pw is not None else yn
    r = x + s["res_scale"] * gate[item] * tn
    rn, r_rstd = _normalise(r, s["pre"])
    w = s["weight"].float() if s["weight"] is not None else None
    z = rn * w if w is not None else rn
    h = z * (1 + scale[item]) + shift[item]
    out = {"r": r.to(t), "h": h.to(t)}
    if not s["train"]:
        return out
    items = len(s["offsets"]) - 1
    dh = s["dh"].float()
    dz = dh * (1 + scale[item])
    dn = dz * w if w is not None else dz
    dr = s["dr"].float() + _normalise_backward(dn, rn, r_rstd, s["pre"])
    dt = s["res_scale"] * gate[item] * dr
    dyn = dt * pw if pw is not None else dt
    out["dx"] = dr.to(t)
    out["dy"] = _normalise_backward(dyn, yn, y_rstd, s["post"]).to(t)
    out["dgate"] = _item_sums(s["res_scale"] * dr * tn, item, items)
    out["dscale"] = _item_sums(dh * z, item, items)
    out["dshift"] = _item_sums(dh, item, items)
    out["dweight"] = (dz * rn).sum(0) if w is not None else None
    out["dpost_weight"] = (dt * yn).sum(0) if pw is not None else None
    return out


def _phases(s):
    """cos and sin of every token's pairs [n, 1, axes * pairs]: the angle in
    48-bit fractions of a turn, so that no turn is lost to rounding."""
    turn = (s["frequencies"].double() / (2 * math.pi) * 2 ** 48).round().long()
    fraction = (s["positions"].long()[:, :, None] * turn) & (2 ** 48 - 1)
    angle = fraction.float() * (2 * math.pi / 2 ** 48)
    angle = angle.reshape(angle.shape[0], 1, -1)
    return angle.cos(), angle.sin()


def _turn(x, cos, sin, s):
    """The pairs of x rotated; the rest of the head as it is."""
    p = cos.shape[2]
    m = s["magnitude"]
    if s["layout"] == "half":
        u, w = x[..., :p], x[..., p:2 * p]
        a, b = m * (u * cos - w * sin), m * (u * sin + w * cos)
        return torch.cat([a, b, x[..., 2 * p:]], 2)
    u, w = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
    a, b = m * (u * cos - w * sin), m * (u * sin + w * cos)
    return torch.cat([torch.stack([a, b], 3).flatten(2), x[..., 2 * p:]], 2)


def _rotary_plain(s):
    t = s["x"].dtype
    x = s["x"].float()
    cos, sin = _phases(s)
    gamma = s["gamma"].float() if s["gamma"] is not None else None
    xn = x
    if gamma is not None:
        rstd = 1 / (x.square().mean(2, keepdim=True) + EPS).sqrt()
        xn = x * rstd
    out = {"out": _turn(xn * gamma if gamma is not None else x, cos, sin, s).to(t)}
    if not s["train"]:
        return out
    d = _turn(s["dout"].float(), cos, -sin, s)
    out["dgamma"] = None
    if gamma is not None:
        out["dgamma"] = (d * xn).sum(0)
        d = d * gamma
        d = rstd * (d - xn * (d * xn).mean(2, keepdim=True))
    out["dx"] = d.to(t)
    return out


def _padded(offsets):
    """Row of every (item, place), clamped, and whether it is one."""
    off = torch.tensor(offsets, device="cuda")
    lengths = off.diff()
    place = torch.arange(max(1, int(max(b - a for a, b in zip(offsets, offsets[1:])))),
                         device="cuda")
    there = place < lengths[:, None]
    return (off[:-1, None] + place).clamp(max=max(0, offsets[-1] - 1)), there, lengths


def _attention_plain(s):
    hq, hk, hd = s["heads"], s["kv_heads"], s["head_dim"]
    g = hq // hk
    qi, q_there, q_len = _padded(s["q_offsets"])
    ki, k_there, k_len = _padded(s["k_offsets"])
    items, lq = qi.shape

    def rows_of_heads(x):                    # [n, hq, hd] -> [items, hk, lq * g, hd]
        return (x[qi].float().reshape(items, lq, hk, g, hd).permute(0, 2, 1, 3, 4)
                .reshape(items, hk, lq * g, hd))

    def heads_of_rows(x):                    # and back
        d = x.shape[3]
        return x.reshape(items, hk, lq, g, d).permute(0, 2, 1, 3, 4).reshape(
            items, lq, hq, d)[q_there]

    q = rows_of_heads(s["q"])
    k, v = (s[x][ki].float().transpose(1, 2) for x in ("k", "v"))
    seen = k_there[:, None, :] & q_there[:, :, None]
    if s["causal"]:
        i = torch.arange(lq, device="cuda")[None, :, None]
        j = torch.arange(ki.shape[1], device="cuda")[None, None, :]
        seen = seen & (j <= i + (k_len - q_len)[:, None, None])
    seen = seen[:, None].repeat_interleave(g, 2)
    scores = (q @ k.transpose(2, 3)) * s["scale"]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp()
    del scores
    total = p.sum(3, keepdim=True)
    lse = top + total.log()                  # -inf where nothing is seen
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = p @ v
    out = {"out": heads_of_rows(o).to(torch.bfloat16), "lse": heads_of_rows(lse)[..., 0]}
    if not s["train"]:
        return out
    do = rows_of_heads(s["dout"]) * q_there[:, None, :, None].repeat_interleave(g, 2)
    out["dv"] = (p.transpose(2, 3) @ do).transpose(1, 2)[k_there].to(torch.bfloat16)
    ds = do @ v.transpose(2, 3)
    ds = p * (ds - (do * o).sum(3, keepdim=True)) * s["scale"]
    del p
    out["dq"] = heads_of_rows(ds @ k).to(torch.bfloat16)
    out["dk"] = (ds.transpose(2, 3) @ q).transpose(1, 2)[k_there].to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ passes ---
def _norm_own(s):
    import pixel_aligned_image_amd as p3d
    same = dict(offsets=s["offsets"], y=s["y"], gate=s["gate"], scale=s["scale"],
                shift=s["shift"], pre=s["pre"], post=s["post"], weight=s["weight"],
                post_weight=s["post_weight"], res_scale=s["res_scale"], eps=EPS)
    p3d.p3d_gated_norm(s["x"], s["h"], r=s["r"], **same)
    out = {"r": s["r"], "h": s["h"]}
    if s["train"]:
        del same["shift"]
        p3d.p3d_gated_norm_backward(
            s["dh"], s["x"], s["dx"], dr=s["dr"], dy=s["dy"], dgate=s["dgate"],
            dscale=s["dscale"], dshift=s["dshift"], dweight=s["dweight"],
            dpost_weight=s["dpost_weight"], **same)
        for k in ("dx", "dy", "dgate", "dscale", "dshift", "dweight", "dpost_weight"):
            out[k] = s[k]
    return out


def _rotary_own(s):
    import pixel_aligned_image_amd as p3d
    same = dict(layout=s["layout"], magnitude=s["magnitude"], gamma=s["gamma"], eps=EPS)
    p3d.p3d_rotary(s["x"], s["positions"], s["frequencies"], s["out"], **same)
    out = {"out": s["out"]}
    if s["train"]:
        p3d.p3d_rotary_backward(s["dout"], s["positions"], s["frequencies"], s["dx"],
                                x=s["x"] if s["gamma"] is not None else None,
                                dgamma=s["dgamma"], **same)
        out["dgamma"], out["dx"] = s["dgamma"], s["dx"]
    return out


def _attention_own(s):
    import pixel_aligned_image_amd as p3d
    same = dict(q_offsets=s["q_offsets"], k_offsets=s["k_offsets"], scale=s["scale"],
                causal=s["causal"])
    p3d.p3d_attention(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], **same)
    out = {"out": s["out"], "lse": s["lse"]}
    if s["train"]:
        p3d.p3d_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                   s["dq"], s["dk"], s["dv"], **same)
        out["dv"], out["dq"], out["dk"] = s["dv"], s["dq"], s["dk"]
    return out


def run(state):
    plain = {"norm": _norm_plain, "rotary": _rotary_plain, "attention": _attention_plain}
    kernels = {"norm": _norm_own, "rotary": _rotary_own, "attention": _attention_own}
    return (kernels if own else plain)[state["op"]](state)


# ------------------------------------------------------------ the exact values ---
def _exact_norm(s):
    out = {k: [] for k in ("r", "h", "dx", "dy", "dgate", "dscale", "dshift")}
    d = s["dim"]
    weight = s["weight"].double() if s["weight"] is not None else 1.0
    post_weight = s["post_weight"].double() if s["post_weight"] is not None else 1.0
    dweight, dpost = 0.0, 0.0
    for b in range(s["items"]):
        rows = slice(s["offsets"][b], s["offsets"][b + 1])
        x, y = s["x"][rows].double(), s["y"][rows].double()
        gate, scale, shift = (s[k][b].double() for k in ("gate", "scale", "shift"))
        leaves = {"x": x, "y": y}

        def moments(v, kind):
            mean = v.sum(1) / d if kind == "layer" else torch.zeros_like(v[:, 0])
            return mean[:, None], ((v - mean[:, None]).pow(2).sum(1) / d + EPS).rsqrt()[:, None]

        if s["post"] == "none":
            my, ry = 0.0, 1.0
        else:
            my, ry = moments(leaves["y"], s["post"])
        u = (leaves["y"] - my) * ry
        r = leaves["x"] + gate * (s["res_scale"] * post_weight) * u
        mr, rr = moments(r, s["pre"])
        v = (r - mr) * rr
        out["r"].append(r)
        out["h"].append(v * weight * (scale + 1) + shift)
        if not s["train"]:
            continue
        dh, dr = s["dh"][rows].double(), s["dr"][rows].double()
        dv = dh * (scale + 1) * weight
        # the derivative of (r - mean) / deviation, term by term
        dot = (dv * v).sum(1, keepdim=True) / d
        back = dv - v * dot
        if s["pre"] == "layer":
            back = back - dv.sum(1, keepdim=True) / d
        total = dr + back * rr
        du = total * gate * s["res_scale"] * post_weight
        if s["post"] == "none":
            dy = du
        else:
            dy = du - u * ((du * u).sum(1, keepdim=True) / d)
            if s["post"] == "layer":
                dy = dy - du.sum(1, keepdim=True) / d
            dy = dy * ry
        out["dx"].append(total)
        out["dy"].append(dy)
        out["dgate"].append((total * u).sum(0) * s["res_scale"] * post_weight)
        out["dscale"].append((dh * v).sum(0) * weight)
        out["dshift"].append(dh.sum(0))
        dweight = dweight + (dh * v).sum(0) * (scale + 1)
        dpost = dpost + (total * u).sum(0) * gate * s["res_scale"]
    got = {"r": torch.cat(out["r"]), "h": torch.cat(out["h"])}
    if s["train"]:
        got |= {k: torch.cat(out[k]) for k in ("dx", "dy")}
        got |= {k: torch.stack(out[k]) for k in ("dgate", "dscale", "dshift")}
        got["dweight"] = dweight if s["weight"] is not None else None
        got["dpost_weight"] = dpost if s["post_weight"] is not None else None
    return got


def _exact_rotary(s):
    p = s["axes"] * s["pairs"]
    angle = (s["positions"].double()[:, :, None] * s["frequencies"].double()).flatten(1)
    phase = s["magnitude"] * torch.polar(torch.ones_like(angle), angle)[:, None]
    if s["layout"] == "half":
        first = torch.arange(p, device="cuda")
        second = first + p
    else:
        first = 2 * torch.arange(p, device="cuda")
        second = first + 1

    def by(x, phase):
        x = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * phase
        x[..., first], x[..., second] = z.real, z.imag
        return x

    x = s["x"].double()
    if s["gamma"] is None:
        got = {"out": by(x, phase)}
        if s["train"]:
            got["dgamma"], got["dx"] = None, by(s["dout"].double(), phase.conj())
        return got
    gamma = s["gamma"].double()
    inv = (x.pow(2).sum(2, keepdim=True) / s["head_dim"] + EPS).pow(-0.5)
    got = {"out": by(x * inv * gamma, phase)}
    if s["train"]:
        back = by(s["dout"].double(), phase.conj())
        got["dgamma"] = (back * x * inv).sum(0)
        c = back * gamma
        got["dx"] = inv * c - x * inv.pow(3) * ((c * x).sum(2, keepdim=True) / s["head_dim"])
    return got


def _exact_attention(s):
    """One head of one item at a time, in blocks of 4096 queries."""
    group = s["heads"] // s["kv_heads"]
    names = ["out", "lse"] + (["dv", "dq", "dk"] if s["train"] else [])
    like = {"out": s["q"], "lse": s["lse"], "dq": s["q"], "dk": s["k"], "dv": s["v"]}
    got = {n: torch.zeros(like[n].shape, device="cuda", dtype=torch.float64) for n in names}
    got["lse"].fill_(-math.inf)
    for b in range(s["items"]):
        q0, q1 = s["q_offsets"][b:b + 2]
        k0, k1 = s["k_offsets"][b:b + 2]
        if k1 == k0:
            continue
        for h in range(s["heads"]):
            k, v = (s[x][k0:k1, h // group].double() for x in ("k", "v"))
            for a in range(q0, q1, 4096):
                z = min(q1, a + 4096)
                q = s["q"][a:z, h].double()
                x = torch.mm(q, k.t()) * s["scale"]
                live = torch.ones(z - a, dtype=torch.bool, device="cuda")
                if s["causal"]:
                    last = torch.arange(a - q0, z - q0, device="cuda") + (k1 - k0) - (q1 - q0)
                    x[torch.arange(k1 - k0, device="cuda") > last[:, None]] = -math.inf
                    live = last >= 0
                lse = torch.logsumexp(x, 1)
                p = (x - torch.where(live, lse, torch.zeros_like(lse))[:, None]).exp()
                o = torch.mm(p, v)
                got["out"][a:z, h], got["lse"][a:z, h] = o, lse
                if s["train"]:
                    do = s["dout"][a:z, h].double()
                    got["dv"][k0:k1, h // group] += torch.mm(p.t(), do)
                    ds = p * (torch.mm(do, v.t()) - (do * o).sum(1, keepdim=True))
                    got["dq"][a:z, h] = torch.mm(ds, k) * s["scale"]
                    got["dk"][k0:k1, h // group] += torch.mm(ds.t(), q) * s["scale"]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary,
            "attention": _exact_attention}[case["op"]](s)
