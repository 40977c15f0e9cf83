"""The 64-bit forms the GPU tests compare with, against themselves: the
gradients by formula and by torch's differentiation equal differences of the
forward forms; a planted mistake in each is caught. CPU only."""
import math

import pytest
import torch

import block_ref as ref

F64 = torch.float64


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, dtype=F64)


def difference(loss, x, u, eps=1e-5):
    return float((loss(x + eps * u) - loss(x - eps * u)) / (2 * eps))


def close(a, b):
    return abs(a - b) <= 1e-7 * (1 + abs(a) + abs(b))


@pytest.mark.parametrize("pre", ["layer", "rms"])
@pytest.mark.parametrize("post", ["none", "layer", "rms"])
def test_norm_gradients_are_differences(pre, post):
    g = torch.Generator().manual_seed(5)
    n, d, off = 11, 24, [0, 4, 4, 11]
    t = {k: rnd(g, n, d) for k in ("x", "y")}
    t |= {k: rnd(g, 3, d) for k in ("gate", "scale", "shift")}
    t |= {k: rnd(g, d) for k in ("weight", "bias")}
    if post != "none":
        t["post_weight"] = rnd(g, d)
    dr, dh = rnd(g, n, d), rnd(g, n, d)

    def loss(**kw):
        r, h = ref.gated_norm(offsets=off, pre=pre, post=post, res_scale=0.7, **(t | kw))
        return (r * dr).sum() + (h * dh).sum()

    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    grads = torch.autograd.grad(loss(**leaves), list(leaves.values()))
    for (k, v), grad in zip(t.items(), grads):
        u = rnd(g, *v.shape)
        assert close(float((grad * u).sum()), difference(lambda z: loss(**{k: z}), v, u)), k


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_gradients_are_differences(layout):
    g = torch.Generator().manual_seed(6)
    x, gamma, dout = rnd(g, 5, 2, 16), rnd(g, 2, 16), rnd(g, 5, 2, 16)
    pos = torch.randint(0, 50, (5, 2), generator=g)
    freqs = torch.tensor([1.0, 0.2, 0.05], dtype=F64)

    def loss(x, gamma):
        return (ref.rotary(x, pos, freqs, layout, 1.3, gamma) * dout).sum()

    a, b = x.clone().requires_grad_(), gamma.clone().requires_grad_()
    ga, gb = torch.autograd.grad(loss(a, b), (a, b))
    u = rnd(g, 5, 2, 16)
    assert close(float((ga * u).sum()), difference(lambda z: loss(z, gamma), x, u))
    u = rnd(g, 2, 16)
    assert close(float((gb * u).sum()), difference(lambda z: loss(x, z), gamma, u))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradients_are_differences(causal):
    g = torch.Generator().manual_seed(7)
    qo, ko = [0, 5, 5, 12], [0, 3, 6, 15]        # the first item's first queries see nothing
    t = {"q": rnd(g, 12, 4, 8), "k": rnd(g, 15, 2, 8), "v": rnd(g, 15, 2, 8)}
    dout = rnd(g, 12, 4, 8)

    def loss(**kw):
        out, _, _ = ref.attention(q_offsets=qo, k_offsets=ko, scale=0.4, causal=causal,
                                  **(t | kw))
        return (out * dout).sum()

    res, tol = ref.attention_backward(dout, t["q"], t["k"], t["v"], qo, ko, 0.4, causal)
    for k, v in t.items():
        u = rnd(g, *v.shape)
        got = float((res["d" + k] * u).sum())
        assert close(got, difference(lambda z: loss(**{k: z}), v, u)), k
        assert (tol["d" + k] >= 0).all()
    out, lse, _ = ref.attention(t["q"], t["k"], t["v"], qo, ko, 0.4, causal)
    if causal:
        assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
        assert torch.isfinite(lse[2:]).all()


def test_planted_mistakes_are_outside_the_tolerances():
    """Each tolerance is tight enough to see a wrong formula."""
    g = torch.Generator().manual_seed(8)
    q, k, v = rnd(g, 40, 2, 32), rnd(g, 50, 2, 32), rnd(g, 50, 2, 32)
    out, lse, reach = ref.attention(q, k, v, [0, 40], [0, 50], 0.2, False)
    less, _, _ = ref.attention(q, k[:-1], v[:-1], [0, 40], [0, 49], 0.2, False)   # a lost key
    assert ref.off_by(less, out, (2.0 ** -7 + 2.0 ** -13) * reach) > 1
    dout = rnd(g, 40, 2, 32)
    res, tol = ref.attention_backward(dout, q, k, v, [0, 40], [0, 50], 0.2, False)
    part, _ = ref.attention_backward(dout, q, k[:-1], v[:-1], [0, 40], [0, 49], 0.2, False)
    assert ref.off_by(part["dq"], res["dq"], tol["dq"]) > 1
    assert ref.off_by(res["dk"] + res["dq"].std(), res["dk"], tol["dk"]) > 1
    assert ref.rms_off(res["dk"] * 1.01, res["dk"]) > 2.0 ** -8
    x = rnd(g, 7, 64)
    _, h = ref.gated_norm(x, [0, 7])
    _, wrong = ref.gated_norm(x, [0, 7], eps=1e-2)
    assert ref.off_by(wrong, h, ref.rounded_once(h, torch.float32)) > 1


@pytest.mark.parametrize("causal", [False, True])
def test_the_two_forms_of_the_attention_gradients_agree(causal):
    """block_ref's, and the one of whole heads that the GPU tests of large
    launches use; a lost key shows in the latter."""
    import test_gpu_block_regimes as regimes
    g = torch.Generator().manual_seed(10)
    q, dout, k, v = rnd(g, 30, 2, 16), rnd(g, 30, 2, 16), rnd(g, 25, 1, 16), rnd(g, 25, 1, 16)
    want, tol = ref.attention_backward(dout, q, k, v, [0, 30], [0, 25], 0.3, causal)
    out, lse, reach = ref.attention(q, k, v, [0, 30], [0, 25], 0.3, causal)
    got = regimes.head_values(q, k[:, 0], v[:, 0], dout, 0.3, causal)
    for n, w, t in (("out", out, (2.0 ** -7 + 2.0 ** -13) * reach), ("dq", want["dq"], tol["dq"]),
                    ("dk", want["dk"][:, 0], tol["dk"][:, 0]),
                    ("dv", want["dv"][:, 0], tol["dv"][:, 0])):
        assert torch.allclose(got[n][0], w, rtol=1e-12, atol=1e-13), n
        assert torch.allclose(got[n][1], t, rtol=1e-12, atol=1e-13), n
    assert torch.allclose(got["lse"][0], lse, rtol=1e-13, atol=0)
    less = regimes.head_values(q, k[1:, 0], v[1:, 0], dout, 0.3, causal)
    for n in ("out", "dq"):
        assert ref.off_by(less[n][0], got[n][0], got[n][1]) > 1, n
