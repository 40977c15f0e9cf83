"""One block of a flow transformer over sparse 3-D tokens, on libp3d's
operators, forward and backward:

    h  = norm(x) (1 + scale1) + shift1             p3d_gated_norm
    q, k, v = Wq h, Wk h, Wv h                     p3d_proj_linear_grouped
    q, k = turn(rms(q) gq), turn(rms(k) gk)        p3d_rotary (by grid cell)
    y1 = Wo attention(q, k, v)                     p3d_attention, per item
    r1 = x + gate1 y1,  h2 = norm(r1) w + b        p3d_gated_norm
    y2 = Wo2 attention(Wq2 h2, Wk2 c, Wv2 c)       p3d_attention over the image's
         + Wp S                                    tokens c; S: p3d_proj_sample
    r2 = r1 + y2,  h3 = norm(r2) (1 + scale3) + shift3

bfloat16 tensors; x [n, D] in items of uneven lengths, c [m, D] likewise.

    python examples/flow_block.py [--tokens 7000] [--items 2] [--context 1029]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pixel_aligned_image_amd as p3d                                  # noqa: E402

LINEARS = ("q", "k", "v", "o", "q2", "k2", "v2", "o2", "p")


def linear(x, *weights):
    """W x for each weight, in one launch."""
    outs = [x.new_empty(x.shape[0], w.shape[0]) for w in weights]
    p3d.p3d_proj_linear_grouped(x, list(weights), outs)
    return outs[0] if len(outs) == 1 else outs


class FlowBlock:
    """params: matrices named as in LINEARS [out, in], norm weight and bias
    "w", "b" [D], head gains "gq", "gk" [heads, D / heads]."""

    def __init__(self, params, heads, freqs):
        self.p, self.heads, self.freqs = params, heads, freqs
        self.dim = params["o"].shape[0]

    def _heads(self, t):
        return t.view(t.shape[0], self.heads, -1)

    def forward(self, x, mod, context, samples, cells, items, context_items):
        """(r2, h3). mod: gate1, scale1, shift1, scale3, shift3, each [items,
        D]; samples: S [n, C]; cells: int32 [n, 3]; items, context_items: row
        tables of x and context."""
        p = self.p
        s = self.saved = dict(x=x, mod=mod, context=context, samples=samples, cells=cells,
                              items=p3d.make_offsets(items),
                              context_items=p3d.make_offsets(context_items))
        s["h"] = torch.empty_like(x)
        p3d.p3d_gated_norm(x, s["h"], s["items"], scale=mod["scale1"], shift=mod["shift1"])
        q, k, v = map(self._heads, linear(s["h"], p["q"], p["k"], p["v"]))
        s.update(q0=q, k0=k, v=v, q=torch.empty_like(q), k=torch.empty_like(k))
        p3d.p3d_rotary(q, cells, self.freqs, s["q"], gamma=p["gq"])
        p3d.p3d_rotary(k, cells, self.freqs, s["k"], gamma=p["gk"])
        s["a"], s["lse"] = self._attend(s["q"], s["k"], v, s["items"], s["items"])
        s["y1"] = linear(s["a"].flatten(1), p["o"])

        s["r1"], s["h2"] = torch.empty_like(x), torch.empty_like(x)
        p3d.p3d_gated_norm(x, s["h2"], s["items"], y=s["y1"], gate=mod["gate1"], r=s["r1"],
                           weight=p["w"], bias=p["b"])
        s["q2"] = self._heads(linear(s["h2"], p["q2"]))
        s["k2"], s["v2"] = map(self._heads, linear(context, p["k2"], p["v2"]))
        s["a2"], s["lse2"] = self._attend(s["q2"], s["k2"], s["v2"], s["items"],
                                          s["context_items"])
        y2 = linear(s["a2"].flatten(1), p["o2"])
        p3d.p3d_proj_linear_grouped(samples, [p["p"]], [y2], accumulate=True)
        s["y2"] = y2

        r2, h3 = torch.empty_like(x), torch.empty_like(x)
        p3d.p3d_gated_norm(s["r1"], h3, s["items"], y=y2, r=r2, scale=mod["scale3"],
                           shift=mod["shift3"])
        return r2, h3

    def _attend(self, q, k, v, items, key_items):
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        p3d.p3d_attention(q, k, v, out, items, key_items, lse=lse)
        return out, lse

    def backward(self, dr2, dh3):
        """Gradients by name: x, context, the modulations, and the parameters
        (linears', norms' and gains')."""
        s, p, mod = self.saved, self.p, self.saved["mod"]
        x, g = s["x"], {}
        f32 = dict(dtype=torch.float32, device=x.device)
        for name in ("gate1", "scale1", "shift1", "scale3", "shift3"):
            g[name] = torch.empty(mod["scale1"].shape, **f32)
        for name in ("w", "b"):
            g[name] = torch.empty(self.dim, **f32)
        for name in ("gq", "gk"):
            g[name] = torch.empty(p["gq"].shape, **f32)

        def through(dy, weight, given):      # a linear's input gradient; its weight's into g
            g[weight] = dy.t() @ given
            return dy @ p[weight]

        dr1, dy2 = torch.empty_like(x), torch.empty_like(x)
        p3d.p3d_gated_norm_backward(dh3, s["r1"], dr1, s["items"], dr=dr2, y=s["y2"], dy=dy2,
                                    scale=mod["scale3"], dscale=g["scale3"], dshift=g["shift3"])
        g["p"] = dy2.t() @ s["samples"]
        da2 = self._heads(through(dy2, "o2", s["a2"].flatten(1)))
        dq2, dk2, dv2 = (torch.empty_like(s[n]) for n in ("q2", "k2", "v2"))
        p3d.p3d_attention_backward(da2, s["q2"], s["k2"], s["v2"], s["a2"], s["lse2"], dq2, dk2,
                                   dv2, s["items"], s["context_items"])
        dh2 = through(dq2.flatten(1), "q2", s["h2"])
        g["context"] = (through(dk2.flatten(1), "k2", s["context"])
                        + through(dv2.flatten(1), "v2", s["context"]))

        dx, dy1 = torch.empty_like(x), torch.empty_like(x)
        p3d.p3d_gated_norm_backward(dh2, x, dx, s["items"], dr=dr1, y=s["y1"], dy=dy1,
                                    gate=mod["gate1"], weight=p["w"], bias=p["b"],
                                    dgate=g["gate1"], dweight=g["w"], dbias=g["b"])
        da = self._heads(through(dy1, "o", s["a"].flatten(1)))
        dq, dk, dv = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
        p3d.p3d_attention_backward(da, s["q"], s["k"], s["v"], s["a"], s["lse"], dq, dk, dv,
                                   s["items"], s["items"])
        p3d.p3d_rotary_backward(dq, s["cells"], self.freqs, dq, gamma=p["gq"], x=s["q0"],
                                dgamma=g["gq"])
        p3d.p3d_rotary_backward(dk, s["cells"], self.freqs, dk, gamma=p["gk"], x=s["k0"],
                                dgamma=g["gk"])
        dh = (through(dq.flatten(1), "q", s["h"]) + through(dk.flatten(1), "k", s["h"])
              + through(dv.flatten(1), "v", s["h"]))
        p3d.p3d_gated_norm_backward(dh, x, dx, s["items"], dr=dx, scale=mod["scale1"],
                                    dscale=g["scale1"], dshift=g["shift1"])
        g["x"] = dx
        return g


def make(tokens, items, context, dim, heads, channels, resolution=64, seed=1, device="cuda"):
    """(block, forward's arguments): random weights, tokens on random cells."""
    gen = torch.Generator().manual_seed(seed)

    def rand(*shape, by=1.0, base=0.0):
        return (torch.randn(*shape, generator=gen) * by + base).bfloat16().to(device)

    params = {n: rand(dim, channels if n == "p" else dim, by=dim ** -0.5) for n in LINEARS}
    params.update(w=rand(dim, by=0.1, base=1.0), b=rand(dim, by=0.1))
    head = (heads, dim // heads)
    params.update(gq=rand(*head, by=0.1, base=1.0), gk=rand(*head, by=0.1, base=1.0))
    mod = {n: rand(items, dim, by=0.2) for n in ("gate1", "scale1", "shift1", "scale3", "shift3")}
    # a third of a head's pairs for each of the cell's three axes
    freqs = p3d.p3d_rotary_frequencies(10000.0, dim // heads // 6).to(device)
    rows = [tokens * (b * b + b) // (items * items + items) for b in range(items + 1)]
    keys = [context * b for b in range(items + 1)]
    cells = torch.randint(0, resolution, (tokens, 3), generator=gen, dtype=torch.int32)
    item = torch.repeat_interleave(torch.arange(items), torch.tensor(rows).diff())
    coords = torch.cat([item[:, None].int(), cells], 1).contiguous().to(device)
    feat = rand(items, 32, 32, channels)
    samples = torch.empty(tokens, channels, dtype=torch.bfloat16, device=device)
    cams = [p3d.p3d_make_camera(40.0, p3d.p3d_distance_from_fov(40.0, 32, 0))] * items
    p3d.p3d_proj_sample(coords, tokens, resolution, cams, feat, samples)
    args = dict(x=rand(tokens, dim), mod=mod, context=rand(context * items, dim),
                samples=samples, cells=coords[:, 1:], items=rows, context_items=keys)
    return FlowBlock(params, heads, freqs), args


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 7000), ("items", 2), ("context", 1029), ("dim", 1024),
                        ("heads", 16), ("channels", 1024), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block, args = make(a.tokens, a.items, a.context, a.dim, a.heads, a.channels)
    dr2, dh3 = torch.randn_like(args["x"]), torch.randn_like(args["x"])

    def timed(call):
        for _ in range(2):
            call()
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            call()
        stop.record()
        stop.synchronize()
        return start.elapsed_time(stop) / a.steps

    forward = timed(lambda: block.forward(**args))
    both = timed(lambda: (block.forward(**args), block.backward(dr2, dh3)))
    grads = block.backward(dr2, dh3)
    assert all(bool(torch.isfinite(t).all()) for t in grads.values())
    print("%d tokens in %d items, width %d, %d heads, %d context tokens each: forward %.3f ms, "
          "forward and backward %.3f ms" % (a.tokens, a.items, a.dim, a.heads, a.context, forward,
                                            both))


if __name__ == "__main__":
    main()
