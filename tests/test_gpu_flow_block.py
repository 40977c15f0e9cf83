"""examples/flow_block.py, the operators together as a model uses them,
against the same block in 64 bits on the CPU with torch's differentiation."""
import os
import sys

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import flow_block

# A tensor rounded to bf16 is off by 2^-8 / sqrt(3) of itself at most, as a
# root mean square, and independent roundings add as squares. The longest
# forward path passes 11 rounded tensors (h, q, turned q, P, a, y1, h2, q2, P2,
# a2, y2) and the results' own; a gradient's passes those again in reverse,
# each with its tensor of the forward call (24 more).
FORWARD, BACKWARD = 12 ** 0.5 * 2 ** -8, 36 ** 0.5 * 2 ** -8


def block_in_64_bits(block, a, dr2, dh3):
    p = {n: ref.f64(t).requires_grad_() for n, t in block.p.items()}
    mod = {n: ref.f64(t).requires_grad_() for n, t in a["mod"].items()}
    x, c = (ref.f64(a[n]).requires_grad_() for n in ("x", "context"))
    samples, cells, freqs = ref.f64(a["samples"]), a["cells"].cpu(), ref.f64(block.freqs)
    items, keys = a["items"], a["context_items"]

    def heads(t):
        return t.view(t.shape[0], block.heads, -1)

    def attend(q, k, v, qi, ki):
        return ref.attention(q, k, v, qi, ki, q.shape[2] ** -0.5, False)[0].flatten(1)

    _, h = ref.gated_norm(x, items, scale=mod["scale1"], shift=mod["shift1"])
    q, k = (ref.rotary(heads(h @ p[n].T), cells, freqs, "interleaved", gamma=p["g" + n])
            for n in "qk")
    y1 = attend(q, k, heads(h @ p["v"].T), items, items) @ p["o"].T
    r1, h2 = ref.gated_norm(x, items, y=y1, gate=mod["gate1"], weight=p["w"], bias=p["b"])
    y2 = attend(heads(h2 @ p["q2"].T), heads(c @ p["k2"].T), heads(c @ p["v2"].T), items,
                keys) @ p["o2"].T + samples @ p["p"].T
    r2, h3 = ref.gated_norm(r1, items, y=y2, scale=mod["scale3"], shift=mod["shift3"])
    ((r2 * ref.f64(dr2)).sum() + (h3 * ref.f64(dh3)).sum()).backward()
    grads = {n: t.grad for n, t in [*p.items(), *mod.items(), ("x", x), ("context", c)]}
    return r2, h3, grads


@pytest.mark.parametrize("tokens,items,context,dim,heads", [
    (331, 2, 5, 192, 4), (700, 3, 97, 256, 2), (257, 1, 33, 384, 6)])
def test_block_against_64_bits(tokens, items, context, dim, heads):
    block, args = flow_block.make(tokens, items, context, dim, heads, 64)
    gen = torch.Generator().manual_seed(9)
    dr2, dh3 = (torch.randn(tokens, dim, generator=gen).bfloat16().cuda() for _ in range(2))
    r2, h3 = block.forward(**args)
    grads = block.backward(dr2, dh3)
    want_r2, want_h3, want = block_in_64_bits(block, args, dr2, dh3)
    assert ref.rms_off(r2, want_r2) < FORWARD
    assert ref.rms_off(h3, want_h3) < FORWARD
    assert set(grads) == set(want)
    off = {n: ref.rms_off(grads[n], want[n]) for n in want}
    print({n: "%.4f" % v for n, v in off.items()})
    assert max(off.values()) < BACKWARD, off


def test_block_gives_the_same_bits_twice():
    block, args = flow_block.make(1500, 2, 5, 256, 4, 64)
    dr2 = torch.randn_like(args["x"])
    first = [*block.forward(**args), *block.backward(dr2, dr2).values()]
    again = [*block.forward(**args), *block.backward(dr2, dr2).values()]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
