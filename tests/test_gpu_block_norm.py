"""p3d_gated_norm and its gradients against the 64-bit form."""
import pytest
import torch

import block_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(n, dim, items, dtype, seed, post="none", pre="layer", full=True):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * scale + mean).to(dtype)

    t = {"x": rnd(n, dim, scale=2.0, mean=0.3), "y": rnd(n, dim)}
    t |= {k: rnd(items, dim, scale=0.4) for k in ("gate", "scale", "shift")}
    if full:
        t |= {"weight": rnd(dim, scale=0.3, mean=1.0), "bias": rnd(dim, scale=0.3)}
    if post != "none":
        t["post_weight"] = rnd(dim, scale=0.3, mean=1.0)
    return t, {"dh": rnd(n, dim), "dr": rnd(n, dim)}


def forward(t, offsets, dtype, **kw):
    c = {k: v.cuda() for k, v in t.items()}
    x = c.pop("x")
    r, h = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    p3d.p3d_gated_norm(x, h, offsets=offsets, r=r, **c, **kw)
    return r, h


SIZES = [(1, 8, 1), (5, 1536, 1), (33, 128, 3), (67, 136, 5), (64, 264, 2), (130, 1024, 7),
         (41, 1544, 4), (19, 2048, 1), (9, 2056, 2), (6, 4096, 3), (5, 8192, 2), (300, 512, 256)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,dim,items", SIZES)
def test_forward(n, dim, items, dtype):
    for k, (pre, post) in enumerate([("layer", "none"), ("rms", "rms"), ("layer", "layer")]):
        t, _ = make(n, dim, items, dtype, seed=n + dim + k, pre=pre, post=post)
        off = ref.uneven(n, items)
        kw = dict(pre=pre, post=post, res_scale=0.6, eps=1e-5)
        r, h = forward(t, off, dtype, **kw)
        wr, wh = ref.gated_norm(offsets=off, **{a: ref.f64(b) for a, b in t.items()}, **kw)
        assert ref.off_by(r, wr, ref.rounded_once(wr, dtype)) <= 1
        assert ref.off_by(h, wh, ref.rounded_once(wh, dtype)) <= 1


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,dim,items", SIZES)
def test_backward(n, dim, items, dtype):
    for k, (pre, post) in enumerate([("layer", "none"), ("rms", "rms"), ("layer", "layer")]):
        t, d = make(n, dim, items, dtype, seed=2 * n + dim + k, pre=pre, post=post)
        off = ref.uneven(n, items)
        kw = dict(pre=pre, post=post, res_scale=0.6, eps=1e-5)
        leaves = {a: ref.f64(b).requires_grad_() for a, b in t.items()}
        r, h = ref.gated_norm(offsets=off, **leaves, **kw)
        loss = (r * ref.f64(d["dr"])).sum() + (h * ref.f64(d["dh"])).sum()
        want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))

        c = {a: b.cuda() for a, b in t.items() if a != "shift"}
        x = c.pop("x")
        dx, dy = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
        par = {a: torch.full(t[a].shape, float("nan"), device="cuda")
               for a in t if a not in ("x", "y")}
        p3d.p3d_gated_norm_backward(d["dh"].cuda(), x, dx, offsets=off, dr=d["dr"].cuda(), dy=dy,
                                    **c, **kw, **{"d" + a: v for a, v in par.items()})
        # a norm's gradient is rstd (d - n mean(d n) - mean d): its terms are
        # as large as rstd |d|, and x, y are near 1 in size
        big = {"x": want["x"].abs() + 2, "y": want["y"].abs() + 2}
        assert ref.off_by(dx, want["x"], ref.rounded_once(want["x"], dtype, big["x"])) <= 1
        assert ref.off_by(dy, want["y"], ref.rounded_once(want["y"], dtype, big["y"])) <= 1
        # sums over rows of products near 1: up to n roundings, bounded by
        # 2^-17 of sqrt(n) terms' size for these n
        for a, v in par.items():
            assert ref.off_by(v, want[a], 2.0 ** -17 * (8 * n ** 0.5 + want[a].abs())) <= 1, a


def test_gradient_against_differences():
    """The kernels' gradient in a random direction equals the difference of
    the kernels' own forward values (binary32, so 1e-3 of the size)."""
    t, d = make(40, 256, 2, F32, seed=3, pre="rms", post="layer")
    off = [0, 13, 40]
    kw = dict(pre="rms", post="layer", res_scale=0.6)
    g = torch.Generator().manual_seed(9)
    c = {a: b.cuda() for a, b in t.items()}
    grads = {a: torch.empty_like(b) for a, b in c.items()}
    p3d.p3d_gated_norm_backward(
        d["dh"].cuda(), c["x"], grads["x"], offsets=off, dr=d["dr"].cuda(), dy=grads["y"],
        **{a: b for a, b in c.items() if a not in ("x", "shift")}, **kw,
        **{"d" + a: v for a, v in grads.items() if a not in ("x", "y")})

    def loss(t):
        r, h = forward(t, off, F32, **kw)
        return float((ref.f64(r) * ref.f64(d["dr"])).sum() + (ref.f64(h) * ref.f64(d["dh"])).sum())

    for name in t:
        # along the gradient's own signs, so that the change is no small sum
        u = grads[name].cpu().sign() * torch.rand(t[name].shape, generator=g)
        eps = 2.0 ** -7
        diff = (loss(t | {name: t[name] + eps * u}) - loss(t | {name: t[name] - eps * u})) / (2 * eps)
        got = float((ref.f64(grads[name]) * ref.f64(u)).sum())
        assert abs(diff - got) <= 1e-2 * abs(got) + 1e-2, (name, diff, got)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_absent_parts_and_packed_modulation(dtype):
    n, dim, items = 37, 520, 3
    t, _ = make(n, dim, items, dtype, seed=1)
    off = [0, 10, 10, 37]
    # no y: r = x; no modulation, no weight
    x = t["x"].cuda()
    h = torch.full_like(x, float("nan"))
    p3d.p3d_gated_norm(x, h, offsets=off)
    _, wh = ref.gated_norm(ref.f64(t["x"]), off)
    assert ref.off_by(h, wh, ref.rounded_once(wh, dtype)) <= 1
    # gate, scale, shift as rows of one packed [items, 6, dim] tensor
    pack = torch.zeros(items, 6, dim, dtype=dtype)
    for i, k in ((1, "shift"), (3, "scale"), (5, "gate")):
        pack[:, i] = t[k]
    pack = pack.cuda()
    r = torch.full_like(x, float("nan"))
    p3d.p3d_gated_norm(x, h, offsets=off, y=t["y"].cuda(), r=r, gate=pack[:, 5],
                       scale=pack[:, 3], shift=pack[:, 1])
    del t["weight"], t["bias"]
    wr, wh = ref.gated_norm(offsets=off, **{a: ref.f64(b) for a, b in t.items()})
    assert ref.off_by(r, wr, ref.rounded_once(wr, dtype)) <= 1
    assert ref.off_by(h, wh, ref.rounded_once(wh, dtype)) <= 1


def test_in_place_and_no_rows():
    t, d = make(50, 1536, 2, BF16, seed=4)
    off = [0, 50, 50]
    r, h = forward(t, off, BF16)
    c = {a: b.cuda() for a, b in t.items()}
    x = c.pop("x")
    y = c["y"]
    p3d.p3d_gated_norm(x, y, offsets=off, r=x, **c)              # r over x, h over y
    assert torch.equal(x, r) and torch.equal(y, h)
    # gradients over their inputs; the empty item's are 0
    c = {a: b.cuda() for a, b in t.items() if a != "shift"}
    x = c.pop("x")
    dh, dr = d["dh"].cuda(), d["dr"].cuda()
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    dscale = torch.full((2, 1536), float("nan"), device="cuda")
    p3d.p3d_gated_norm_backward(dh, x, dx, offsets=off, dr=dr, dy=dy, dscale=dscale, **c)
    assert (dscale[1] == 0).all() and torch.isfinite(dscale[0]).all()
    p3d.p3d_gated_norm_backward(dh, x, dr, offsets=off, dr=dr, dy=c["y"], **c)
    assert torch.equal(dr, dx) and torch.equal(c["y"], dy)
    # no rows at all: the parameter gradients are written
    e = torch.empty(0, 1536, dtype=BF16, device="cuda")
    p3d.p3d_gated_norm(e, e.clone(), offsets=[0, 0])
    dw, ds = torch.full((1536,), 7.0, device="cuda"), torch.full((2, 1536), 7.0, device="cuda")
    p3d.p3d_gated_norm_backward(e, e, e.clone(), offsets=[0, 0, 0], dweight=dw, dshift=ds)
    assert (dw == 0).all() and (ds == 0).all()


def test_rows_that_are_constant_or_not_finite():
    """A constant row's deviation is eps alone; a row with an infinity or NaN
    gives NaN, its neighbours what they gave."""
    x = torch.randn(9, 1024, generator=torch.Generator().manual_seed(2))
    x[2] = 3.0
    x[4, 7] = float("inf")
    x[6, 1000] = float("nan")
    c, h = x.cuda(), torch.empty(9, 1024, device="cuda")
    p3d.p3d_gated_norm(c, h)
    _, want = ref.gated_norm(ref.f64(x), [0, 9])
    assert (h[2] == 0).all()
    for i in (0, 1, 3, 5, 7, 8):
        assert ref.off_by(h[i:i + 1], want[i:i + 1], ref.rounded_once(want[i:i + 1], F32)) <= 1
    assert torch.isnan(h[4]).any() and torch.isnan(h[6]).all()


def test_repeatable_and_on_another_stream():
    t, d = make(5000, 1536, 3, BF16, seed=6)
    off = [0, 1, 2600, 5000]
    c = {a: b.cuda() for a, b in t.items() if a != "shift"}
    x = c.pop("x")
    dh, dr = d["dh"].cuda(), d["dr"].cuda()

    def once(stream=None):
        dx, dy = torch.empty_like(x), torch.empty_like(x)
        par = {"d" + a: torch.empty(t[a].shape, device="cuda") for a in t if a not in ("x", "y")}
        ws = torch.empty(p3d.p3d_gated_norm_workspace_size(x, off), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        p3d.p3d_gated_norm_backward(dh, x, dx, offsets=off, dr=dr, dy=dy, workspace=ws,
                                    stream=stream, **par, **c)
        torch.cuda.synchronize()
        return [dx, dy, *par.values()]

    first = once()
    for got in (once(), once(torch.cuda.Stream())):
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_captured_in_a_graph():
    t, _ = make(700, 1536, 2, BF16, seed=8)
    c = {a: b.cuda() for a, b in t.items()}
    x = c.pop("x")
    r, h = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    p3d.p3d_gated_norm(x, h, offsets=[0, 300, 700], r=r, **c)
    with torch.cuda.graph(graph):
        p3d.p3d_gated_norm(x, h, offsets=[0, 300, 700], r=r, **c)
    for i in range(3):
        x.copy_(t["x"].cuda() * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        got = h.clone()
        h.zero_()
        p3d.p3d_gated_norm(x, h, offsets=[0, 300, 700], r=r, **c)
        assert torch.equal(got, h)


@pytest.mark.parametrize("over", ["x", "dh", "dr"])
def test_in_place_gradient_of_ragged_chunks(over):
    """dx over one of its inputs, chunks that do not fill their last turn, and
    a last row whose dx is not finite: the columns' sums are those of the call
    into a tensor of its own, and finite where dh and x are."""
    for n, dim in ((17, 64), (33, 256), (18, 1024), (1041, 128)):
        g = torch.Generator().manual_seed(n)
        t = {k: torch.randn(n, dim, generator=g).cuda() for k in ("x", "dh", "dr")}
        t["dr"][-1] = float("inf")

        def call(dx, **kw):
            sums = {k: torch.full((1, dim), float("nan"), device="cuda")
                    for k in ("dscale", "dshift")}
            a = t | kw
            p3d.p3d_gated_norm_backward(a["dh"], a["x"], dx, dr=a["dr"], pre="rms", **sums)
            return dx, sums

        want, sums = call(torch.empty_like(t["x"]))
        own = t[over].clone()
        got, again = call(own, **{over: own})
        assert torch.equal(got, want)
        for k in sums:
            assert torch.isfinite(sums[k]).all() and torch.equal(again[k], sums[k]), k
