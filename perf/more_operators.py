"""Cases of the model's operators around the block: group norm with an
activation over channels-last maps, linear layers in 8-bit integers, and the
AdamW step with its gradient norm.

The sizes are this repository's own: maps of 16^3, 64 x 64, 512 x 512 and
200,000 sparse tokens, the block's widths (1024 and 1536) and its conditioning
channels (1024 and 2048), 5 global, 7000, 12,289 and 100,000 tokens, the
parameters of one to four transformer blocks.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-5                      # of the group norm
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.99, 1e-8, 1e-3, 0.1
MAX_NORM = 1.0
BLOCK = 256                     # elements that share a scale of an 8-bit state
TOP = 448.0                     # largest e4m3 number


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # the dense 16^3 grid inside the structure decoder, one image
        {"name": "group_dense16", "op": "group", "train": False, "dtype": BF16, "rows": 4096,
         "items": 1, "channels": 512, "groups": 32, "act": "silu"},
        # the upsampled half of a conditioning map, one image
        {"name": "group_map512", "op": "group", "train": False, "dtype": BF16, "rows": 262144,
         "items": 1, "channels": 1024, "groups": 32, "act": "silu"},
        # a training step in 32 bits over the patch maps of two images
        {"name": "group_train_map64", "op": "group", "train": True, "dtype": F32, "rows": 8192,
         "items": 2, "channels": 1024, "groups": 32, "act": "silu"},
        # a training step over two ragged items of a sparse decoder
        {"name": "group_train_200k", "op": "group", "train": True, "dtype": BF16,
         "rows": 200000, "items": 2, "channels": 256, "groups": 32, "act": "silu"},
        # the vectors of a few blocks' norms and gains, updated by themselves: latency
        {"name": "adamw_vectors", "op": "adamw", "bits": 32, "param": F32, "grad": F32,
         "master": False, "clip": False, "step": 100, "tensors": 24, "largest": 1536,
         "even": True, "width": 0, "channels": 0},
        # a mixed-precision training step of two blocks, gradients clipped
        {"name": "adamw_blocks2", "op": "adamw", "bits": 32, "param": BF16, "grad": BF16,
         "master": True, "clip": True, "step": 1000, "tensors": 2, "largest": 0, "even": False,
         "width": 1536, "channels": 2048},
        # one narrower block's first step in 32 bits, its states in 8
        {"name": "adamw8_block", "op": "adamw", "bits": 8, "param": F32, "grad": F32,
         "master": False, "clip": False, "step": 1, "tensors": 1, "largest": 0, "even": False,
         "width": 1024, "channels": 1024},
        # a training step of four blocks with little memory: bf16 weights, states in 8 bits
        {"name": "adamw8_blocks4", "op": "adamw", "bits": 8, "param": BF16, "grad": BF16,
         "master": False, "clip": True, "step": 1000, "tensors": 4, "largest": 0, "even": False,
         "width": 1536, "channels": 2048},
        # the five global tokens' projection: latency
        {"name": "linear_global5", "op": "linear", "dtype": BF16, "tokens": 5, "in": 1024,
         "out": 1536, "act": "none", "residual": False},
        # proj_linear of 7000 sparse tokens, added into the block's residual
        {"name": "linear_sparse7000", "op": "linear", "dtype": BF16, "tokens": 7000, "in": 2048,
         "out": 1536, "act": "none", "residual": True},
        # the first linear of a block's feed-forward part over one long odd sequence
        {"name": "linear_gelu12k", "op": "linear", "dtype": BF16, "tokens": 12289, "in": 1536,
         "out": 6144, "act": "gelu", "residual": False},
        # proj_linear of the 100,000-token sparse shell
        {"name": "linear_shell100k", "op": "linear", "dtype": BF16, "tokens": 100000,
         "in": 2048, "out": 1536, "act": "none", "residual": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "adamw", "linear"])
    if op == "group":
        groups = rng.choice([1, 4, 8, 16, 32, 32, 40])
        channels = groups * rng.randint(1, 1024 // groups)
        channels = max(8, channels // 8 * 8)
        groups = math.gcd(groups, channels)
        return {"op": op, "train": rng.random() < 0.5, "dtype": rng.choice([BF16, F32]),
                "rows": _log(rng, 1, 100000), "items": _log(rng, 1, 16), "channels": channels,
                "groups": groups, "act": rng.choice(["none", "silu", "silu", "gelu"])}
    if op == "adamw":
        param = rng.choice([BF16, F32])
        return {"op": op, "bits": rng.choice([8, 32]), "param": param,
                "grad": param if rng.random() < 0.7 else BF16,
                "master": param == BF16 and rng.random() < 0.5, "clip": rng.random() < 0.5,
                "step": _log(rng, 1, 100000), "tensors": _log(rng, 1, 200),
                "largest": _log(rng, 1, 400000), "even": rng.random() < 0.2, "width": 0,
                "channels": 0}
    return {"op": op, "dtype": rng.choice([BF16, BF16, F32]), "tokens": _log(rng, 1, 30000),
            "in": 16 * _log(rng, 4, 256), "out": 8 * _log(rng, 8, 512),
            "act": rng.choice(["none", "none", "silu", "gelu"]),
            "residual": rng.random() < 0.4}


# ------------------------------------------------------------------- sizes ---
def _offsets(total, items):
    """Row ranges of `items` uneven items (weights items, items + 1, ...)."""
    weights = [items + i for i in range(items)]
    at, ends, whole = 0, [0], sum(weights)
    for w in weights:
        at += w
        ends.append(total * at // whole)
    return ends


def _sizes(case):
    """Elements and weight decay of every tensor of an AdamW step: blocks of
    eight square matrices, the conditioning's, and four vectors; or tensors of
    uneven, mostly small, odd sizes."""
    if case["width"]:
        d, c = case["width"], case["channels"]
        block = [(d * d, DECAY)] * 8 + [(d * c, DECAY)] + [(d, 0.0)] * 4
        return block * case["tensors"]
    top = case["largest"]
    if case["even"]:                         # norm vectors, all of one width
        return [(top, 0.0)] * case["tensors"]
    return [(max(1, int(top * ((j * 0.618034 + 1) % 1.0 or 1.0) ** 3)), DECAY * (j % 3))
            for j in range(case["tensors"])]


def _padded(sizes):
    """The tensors' places in one buffer, each from a multiple of 256 on."""
    at, starts = 0, []
    for n, _ in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def work(case):
    if case["op"] == "group":
        e = 4 if case["dtype"] == F32 else 2
        plane = case["rows"] * case["channels"]
        # x in, out out. With gradients: dout in, dx out
        planes = 4 if case["train"] else 2
        small = 2 * e * case["channels"] + 8 * case["items"] * case["groups"]
        return {"bytes": e * planes * plane + small
                + (8 * case["channels"] if case["train"] else 0),
                "flops": (60 if case["train"] else 20) * plane}
    if case["op"] == "adamw":
        n = sum(s for s, _ in _sizes(case))
        p, g = (4 if case[k] == F32 else 2 for k in ("param", "grad"))
        # the gradient in; weights (their 32-bit copies) and two states in and out
        each = g + (8 + p if case["master"] else 2 * p)
        each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": each * n, "flops": (20 if case["bits"] == 32 else 60) * n}
    e = 4 if case["dtype"] == F32 else 2
    n, k, d = case["tokens"], case["in"], case["out"]
    # x, the weights and their scales and bias in; q, its scales and out out
    return {"bytes": e * n * k + n * k + 4 * n + d * k + (4 + e) * d
            + e * n * d * (2 if case["residual"] else 1), "flops": 2 * n * k * d}


# ------------------------------------------------------------------ inputs ---
def _type(name):
    return torch.float32 if name == F32 else torch.bfloat16


def _views(flat, sizes, starts):
    return [flat[a:a + n] for (n, _), a in zip(sizes, starts)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(mean).to(dtype)

    s = dict(case)
    if case["op"] == "group":
        n, c, items, t = case["rows"], case["channels"], case["items"], _type(case["dtype"])
        s["offsets"] = _offsets(n, items)
        # feature maps: channels with means and deviations of their own
        spread = randn(c, scale=0.5, dtype=torch.float32).exp()
        s["x"] = (randn(n, c, dtype=torch.float32).mul_(spread)
                  .add_(randn(c, scale=0.5, dtype=torch.float32)).to(t))
        s["weight"], s["bias"] = randn(c, scale=0.2, mean=1.0, dtype=t), randn(c, scale=0.2, dtype=t)
        s["out"] = torch.empty_like(s["x"])
        s["mean"], s["rstd"] = (torch.empty(items, case["groups"], device="cuda")
                                for _ in range(2))
        if case["train"]:
            s["dout"] = randn(n, c, dtype=t)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"], s["dbias"] = (torch.empty(c, device="cuda") for _ in range(2))
    elif case["op"] == "adamw":
        sizes = _sizes(case)
        starts, total = _padded(sizes)
        live = torch.zeros(total, device="cuda")
        for (n, _), a in zip(sizes, starts):
            live[a:a + n] = 1
        # gradients whose size differs from tensor to tensor and, less, within one
        size = torch.repeat_interleave(
            randn(len(sizes), dtype=torch.float32).exp() * 1e-3,
            torch.tensor([-(-n // BLOCK) * BLOCK for n, _ in sizes], device="cuda"))
        size = size * live
        s["grad"] = (randn(total, dtype=torch.float32) * size).to(_type(case["grad"]))
        weights = randn(total, scale=0.03, dtype=torch.float32) * live
        s["param"] = weights.to(_type(case["param"]))
        s["master"] = weights if case["master"] else None
        late = 0.0 if case["step"] == 1 else 1.0
        m = randn(total, dtype=torch.float32) * size * (0.3 * late)
        r = randn(total, scale=0.3, mean=1.0, dtype=torch.float32).abs_() * size * late
        if case["bits"] == 8:
            for name, x in (("m", m), ("r", r)):
                s[name + "_scale"] = x.reshape(-1, BLOCK).abs().amax(1) / TOP
                by = s[name + "_scale"].clamp(min=1e-30).repeat_interleave(BLOCK)
                s[name] = (x / by).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        else:
            s["m"], s["v"] = m, r.square()
        s["seed"] = seed & 0x7fffffff
        s["sizes"], s["starts"] = sizes, starts
        s["norm"] = torch.empty(2, device="cuda") if case["clip"] else None
        if own:
            s["tensors"] = _tensors(s)
    else:
        n, k, d, t = case["tokens"], case["in"], case["out"], _type(case["dtype"])
        # activations with a few large columns, as trained models have
        columns = randn(k, scale=0.7, dtype=torch.float32).exp()
        s["x"] = randn(n, k, dtype=torch.float32).mul_(columns).to(t)
        w = randn(d, k, scale=k ** -0.5, dtype=torch.float32)
        s["weight_scale"] = w.abs().amax(1) / 127
        s["weight"] = (w / s["weight_scale"][:, None]).round().to(torch.int8)
        s["bias"] = randn(d, scale=0.1, dtype=t)
        s["residual"] = randn(n, d, dtype=t) if case["residual"] else None
        s["q"] = torch.empty(n, k, dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(n, device="cuda")
        s["out"] = torch.empty(n, d, dtype=t, device="cuda")
    return s


def _tensors(s):
    """The table of tensors that a training program keeps over its steps."""
    import pixel_aligned_image_amd as p3d
    at = (s["sizes"], s["starts"])
    second = s["r"] if s["bits"] == 8 else s["v"]
    kw = {}
    if s["bits"] == 8:
        blocks = [(-(-n // BLOCK), 0) for n, _ in s["sizes"]]
        first = [a // BLOCK for a in s["starts"]]
        kw = dict(m_scales=_views(s["m_scale"], blocks, first),
                  v_scales=_views(s["r_scale"], blocks, first))
    return p3d.make_adamw_tensors(
        _views(s["param"], *at), _views(s["grad"], *at), _views(s["m"], *at),
        _views(second, *at), masters=_views(s["master"], *at) if s["master"] is not None else None,
        weight_decay=[w for _, w in s["sizes"]], **kw)


# -------------------------------------------------------- the plain forms ---
def _row_items(offsets):
    """The item of every row."""
    lengths = torch.tensor(offsets, device="cuda").diff()
    return torch.repeat_interleave(torch.arange(len(offsets) - 1, device="cuda"), lengths)


def _act(u, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1 / (1 + (-u).exp())
        return u * p, p * (1 + u * (1 - p))
    if kind == "gelu":                       # the tanh form, as a logistic
        z = 2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u)
        p = 1 / (1 + (-z).exp())
        dz = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u * u)
        return u * p, p + u * p * (1 - p) * dz
    return u, torch.ones_like(u)


def _group_sums(v, offsets, groups):
    """Sums [items, groups] over the rows of an item and a group's channels, the
    long ones in 64 bits."""
    rows = v.reshape(v.shape[0], groups, -1).sum(2)
    lengths = [b - a for a, b in zip(offsets, offsets[1:])]
    return torch.stack([r.sum(0, dtype=torch.float64) for r in rows.split(lengths)]).float()


def _group_plain(s):
    t, (n, c), groups = s["x"].dtype, s["x"].shape, s["groups"]
    offsets, each = s["offsets"], c // groups
    item = _row_items(offsets)
    count = (torch.tensor(offsets, device="cuda").diff() * each)[:, None].clamp(min=1)

    def wide(v):                             # [items, groups] -> one value an element
        return v.repeat_interleave(each, 1)[item]

    x = s["x"].float()
    mean = _group_sums(x, offsets, groups) / count
    centred = x - wide(mean)
    rstd = 1 / (_group_sums(centred.square(), offsets, groups) / count + EPS).sqrt()
    xn = centred * wide(rstd)
    del centred, x
    w, b = s["weight"].float(), s["bias"].float()
    y, slope = _act(xn * w + b, s["act"])
    out = {"out": y.to(t), "mean": mean, "rstd": rstd}
    if not s["train"]:
        return out
    du = s["dout"].float() * slope
    out["dbias"], out["dweight"] = du.sum(0), (du * xn).sum(0)
    dn = du * w
    a = wide(_group_sums(dn, offsets, groups) / count)
    e = wide(_group_sums(dn * xn, offsets, groups) / count)
    out["dx"] = (wide(rstd) * (dn - a - xn * e)).to(t)
    return out


MASK = 0xffffffff


def _mix(x):
    """32 bits from 32 bits, each depending on all (numbers or int64 tensors)."""
    x = x ^ (x >> 15)
    x = (x * 0xB504F335) & MASK
    x = x ^ (x >> 13)
    x = (x * 0xDDB3D743) & MASK
    return x ^ (x >> 16)


def _random(s):
    """The 32 random bits of every element, of the call's seed, the number of
    its tensor and its index there."""
    n = s["param"].numel()
    lengths = torch.tensor([-(-k // BLOCK) * BLOCK for k, _ in s["sizes"]], device="cuda")
    start = torch.tensor(s["starts"], device="cuda").repeat_interleave(lengths, output_size=n)
    key = _mix(((torch.arange(len(s["sizes"]), device="cuda") * 0x9E3779B1) & MASK)
               ^ _mix(s["seed"] & MASK) ^ (s["seed"] >> 32))
    index = torch.arange(n, device="cuda") - start
    x = ((index & MASK) * 0x9E3779B1) & MASK
    x = x ^ (((index >> 32) * 0xDDB3D743) & MASK)
    return _mix(x ^ key.repeat_interleave(lengths, output_size=n))


def _to_8_bits(x, random, least):
    """e4m3 codes and a scale for every 256 values; a value between two codes
    goes to the upper one where its 16 random bits say so."""
    blocks = x.reshape(-1, BLOCK)
    top = blocks.abs().amax(1, keepdim=True)
    top = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top)
    scale = top / TOP
    by = torch.where(top == 0, torch.zeros_like(top), TOP / top)
    q = (blocks * by).reshape(-1)
    a = q.abs().clamp(max=TOP)
    normal = ((a.view(torch.int32) + (random << 4).int()) >> 20) - 960
    small = (a * 512 + random.float() / 65536).floor().int()
    code = torch.where(a < 2.0 ** -6, small, normal)
    if least:                                # what is not 0 stays so
        code = torch.where((q > 0) & (code == 0), torch.ones_like(code), code)
    code = code | ((q < 0).int() << 7)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale.reshape(-1)


def _decay(s):
    lengths = torch.tensor([-(-n // BLOCK) * BLOCK for n, _ in s["sizes"]], device="cuda")
    return torch.tensor([w for _, w in s["sizes"]], device="cuda",
                        dtype=torch.float32).repeat_interleave(lengths,
                                                               output_size=s["param"].numel())


def _adamw_plain(s):
    g = s["grad"].float()
    out = {}
    if s["clip"]:
        norm = s["grad"].double().square().sum().sqrt()
        by = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)).float()
        out["norm"] = torch.stack([norm.float(), by])
        g = g * by
    if s["bits"] == 8:
        m = s["m"].float() * s["m_scale"].repeat_interleave(BLOCK)
        v = (s["r"].float() * s["r_scale"].repeat_interleave(BLOCK)).square()
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    r = v.sqrt()
    weights = s["master"] if s["master"] is not None else s["param"].float()
    c1, c2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    weights = (weights * (1 - LR * _decay(s))
               - (LR / c1) * m / (r / math.sqrt(c2) + ADAM_EPS))
    s["param"].copy_(weights)
    out["param"] = s["param"]
    if s["master"] is not None:
        s["master"].copy_(weights)
        out["master"] = s["master"]
    if s["bits"] == 8:
        random = _random(s)
        for name, x, bits in (("m", m, random & 0xffff), ("r", r, random >> 16)):
            code, scale = _to_8_bits(x, bits, name == "r")
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
            out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        out["m"], out["v"] = s["m"], s["v"]
    return out


def _linear_plain(s):
    t = s["x"].dtype
    x = s["x"].float()
    scale = x.abs().amax(1) / 127
    # values near the middle between two integers need more than 32 bits
    by = torch.where(scale == 0, torch.ones_like(scale), scale)[:, None].double()
    q = (x.double() / by).round()
    y = (q.float() @ s["weight"].float().t()) * (scale[:, None] * s["weight_scale"])
    y = _act(y + s["bias"].float(), s["act"])[0]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(t), "q": q.to(torch.int8), "scale": scale}


# ------------------------------------------------------------------ passes ---
def _group_own(s):
    import pixel_aligned_image_amd as p3d
    same = dict(offsets=s["offsets"], weight=s["weight"], bias=s["bias"], act=s["act"])
    p3d.p3d_group_norm(s["x"], s["out"], s["groups"], eps=EPS, mean=s["mean"], rstd=s["rstd"],
                       **same)
    out = {k: s[k] for k in ("out", "mean", "rstd")}
    if s["train"]:
        p3d.p3d_group_norm_backward(s["dout"], s["x"], s["mean"], s["rstd"], s["dx"],
                                    s["groups"], dweight=s["dweight"], dbias=s["dbias"], **same)
        out |= {k: s[k] for k in ("dbias", "dweight", "dx")}
    return out


def _adamw_own(s):
    import pixel_aligned_image_amd as p3d
    out = {"param": s["param"]}
    if s["clip"]:
        p3d.p3d_grad_norm(s["tensors"], s["norm"], MAX_NORM)
        out["norm"] = s["norm"]
    p3d.p3d_adamw(s["tensors"], LR, BETA1, BETA2, ADAM_EPS, s["step"], seed=s["seed"],
                  grad_scale=s["norm"][1:] if s["clip"] else None)
    if s["master"] is not None:
        out["master"] = s["master"]
    for name in ("m", "m_scale", "r", "r_scale") if s["bits"] == 8 else ("m", "v"):
        out[name] = s[name]
    return out


def _linear_own(s):
    import pixel_aligned_image_amd as p3d
    p3d.p3d_quantize_rows(s["x"], s["q"], s["scale"])
    p3d.p3d_linear_i8(s["q"], s["scale"], s["weight"], s["weight_scale"], s["out"],
                      bias=s["bias"], act=s["act"], residual=s["residual"])
    return {k: s[k] for k in ("out", "q", "scale")}


def run(state):
    plain = {"group": _group_plain, "adamw": _adamw_plain, "linear": _linear_plain}
    kernels = {"group": _group_own, "adamw": _adamw_own, "linear": _linear_own}
    return (kernels if own else plain)[state["op"]](state)


# ------------------------------------------------------------ the exact values ---
def _smooth(u, kind):
    if kind == "silu":
        return u * torch.sigmoid(u)
    if kind == "gelu":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u.pow(3))))
    return u


def _slope(u, kind):
    if kind == "silu":
        p = torch.sigmoid(u)
        return p + u * p * (1 - p)
    if kind == "gelu":
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * (u + 0.044715 * u.pow(3)))
        return 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * k * (1 + 3 * 0.044715 * u * u)
    return torch.ones_like(u)


def _exact_group(s):
    """One group of one item at a time."""
    c, groups, items = s["channels"], s["groups"], s["items"]
    each = c // groups
    f64 = dict(device="cuda", dtype=torch.float64)
    got = {"out": torch.empty(s["x"].shape, **f64), "mean": torch.zeros(items, groups, **f64),
           "rstd": torch.zeros(items, groups, **f64)}
    if s["train"]:
        got |= {"dx": torch.empty(s["x"].shape, **f64), "dbias": torch.zeros(c, **f64),
                "dweight": torch.zeros(c, **f64)}
    for b in range(items):
        rows = slice(s["offsets"][b], s["offsets"][b + 1])
        for j in range(groups):
            cols = slice(j * each, (j + 1) * each)
            x = s["x"][rows, cols].double()
            n = max(1, x.numel())
            mu = x.sum() / n
            inv = ((x - mu).pow(2).sum() / n + EPS).rsqrt()
            w, bias = s["weight"][cols].double(), s["bias"][cols].double()
            h = (x - mu) * inv
            u = h * w + bias
            got["out"][rows, cols] = _smooth(u, s["act"])
            got["mean"][b, j], got["rstd"][b, j] = mu, inv
            if s["train"]:
                d = s["dout"][rows, cols].double() * _slope(u, s["act"])
                got["dbias"][cols] += d.sum(0)
                got["dweight"][cols] += (d * h).sum(0)
                d = d * w
                got["dx"][rows, cols] = (d - d.sum() / n - h * ((d * h).sum() / n)) * inv
    return got


def _hash(index, number, seed):
    def mixed(x):
        x = x ^ x // 2 ** 15
        x = x * 0xB504F335 % 2 ** 32
        x = x ^ x // 2 ** 13
        x = x * 0xDDB3D743 % 2 ** 32
        return x ^ x // 2 ** 16

    key = mixed(number * 0x9E3779B1 % 2 ** 32 ^ mixed(seed % 2 ** 32) ^ seed // 2 ** 32)
    return mixed(index * 0x9E3779B1 % 2 ** 32 ^ key)


def _exact_8_bits(x, bits, least):
    """Values of the codes and scales of one tensor."""
    n = x.numel()
    x = torch.cat([x, x.new_zeros(-n % BLOCK)]).reshape(-1, BLOCK)
    bits = torch.cat([bits, bits.new_zeros(-n % BLOCK)]).reshape(-1, BLOCK)
    scale = x.abs().amax(1, keepdim=True) / TOP
    scale[scale < 2.0 ** -100 / TOP] = 0
    q = x / torch.where(scale == 0, torch.ones_like(scale), scale)
    q = torch.where(scale == 0, torch.zeros_like(q), q)
    step = torch.exp2((torch.frexp(q.abs())[1] - 1).clamp(min=-6).double() - 3)
    value = ((q.abs() / step + bits.double() / 65536).floor() * step).clamp(max=TOP)
    if least:
        value = torch.where((q > 0) & (value == 0), torch.full_like(value, 2.0 ** -9), value)
    return (value * q.sign()).reshape(-1)[:n], scale.reshape(-1)


def _exact_adamw(s):
    names = ["param", "m"] + (["r", "m_scale", "r_scale"] if s["bits"] == 8 else ["v"])
    got = {n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in names}
    by = 1.0
    if s["clip"]:
        norm = torch.linalg.vector_norm(s["grad"].double())
        by = MAX_NORM / norm if float(norm) > MAX_NORM else torch.ones_like(norm)
        got["norm"] = torch.stack([norm, by])
    if s["master"] is not None:
        got["master"] = torch.zeros_like(got["param"])
    for k, ((n, decay), a) in enumerate(zip(s["sizes"], s["starts"])):
        at, blocks = slice(a, a + n), slice(a // BLOCK, a // BLOCK + -(-n // BLOCK))
        g = s["grad"][at].double() * by
        if s["bits"] == 8:
            m, r = (s[x][at].double() * s[x + "_scale"][blocks].double()
                    .repeat_interleave(BLOCK)[:n] for x in ("m", "r"))
            v = r * r
        else:
            m, v = s["m"][at].double(), s["v"][at].double()
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g * g - v)
        r = v.sqrt()
        w = (s["master"] if s["master"] is not None else s["param"])[at].double()
        w = w - LR * decay * w
        w = w - LR * (m / (1 - BETA1 ** s["step"])) / ((v / (1 - BETA2 ** s["step"])).sqrt()
                                                       + ADAM_EPS)
        got["param"][at] = w
        if s["master"] is not None:
            got["master"][at] = w
        if s["bits"] == 8:
            bits = _hash(torch.arange(n, device="cuda"), k, s["seed"])
            got["m"][at], got["m_scale"][blocks] = _exact_8_bits(m, bits % 65536, False)
            got["r"][at], got["r_scale"][blocks] = _exact_8_bits(r, bits // 65536, True)
        else:
            got["m"][at], got["v"][at] = m, v
    return got


def _exact_linear(s):
    """The tokens as the call rounds them: their scales, in 32 bits, are part of
    what the integers mean."""
    x = s["x"].double()
    scale = (x.abs().amax(1) / 127).float().double()
    q = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
    y = torch.mm(q, s["weight"].double().t().contiguous())
    y = y * scale[:, None] * s["weight_scale"].double() + s["bias"].double()
    y = _smooth(y, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"out": y, "q": q.long(), "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    return {"group": _exact_group, "adamw": _exact_adamw, "linear": _exact_linear}[case["op"]](s)
