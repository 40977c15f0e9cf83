"""p3d_rotary and its gradients against the 64-bit form."""
import pytest
import torch

import block_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# n, heads, head_dim, axes, pairs: whole heads, parts, odd pair counts, one lane
SIZES = [(1, 1, 8, 1, 4), (7, 20, 128, 1, 64), (33, 24, 128, 3, 21), (65, 16, 64, 3, 8),
         (40, 3, 80, 2, 19), (5, 2, 256, 1, 128), (19, 5, 96, 3, 1), (1000, 2, 24, 1, 5),
         (3, 33, 72, 3, 12), (130, 1, 16, 2, 3)]


def make(n, heads, hd, axes, pairs, dtype, seed, top=1024):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, hd, generator=g).to(dtype)
    dout = torch.randn(n, heads, hd, generator=g).to(dtype)
    gamma = (1 + 0.3 * torch.randn(heads, hd, generator=g)).to(dtype)
    pos = torch.randint(-3, top, (n, axes), generator=g, dtype=torch.int32)
    freqs = p3d.p3d_rotary_frequencies(10000.0, pairs)
    return x, dout, gamma, pos, freqs


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,heads,hd,axes,pairs", SIZES)
def test_forward_and_backward(n, heads, hd, axes, pairs, layout, dtype):
    x, dout, gamma, pos, freqs = make(n, heads, hd, axes, pairs, dtype, seed=n + hd)
    for gm, m in ((None, 1.0), (gamma, 1.25)):
        kw = dict(layout=layout, magnitude=m, eps=1e-5)
        gd = None if gm is None else gm.cuda()
        xd, pd, fd = x.cuda(), pos.cuda(), freqs.cuda()
        out = torch.full_like(xd, float("nan"))
        p3d.p3d_rotary(xd, pd, fd, out, gamma=gd, **kw)
        leaf = ref.f64(x).requires_grad_()
        gleaf = None if gm is None else ref.f64(gm).requires_grad_()
        want = ref.rotary(leaf, pos, freqs, gamma=gleaf, **kw)
        wd = want.detach()
        assert ref.off_by(out, wd, ref.rounded_once(wd, dtype)) <= 1

        loss = (want * ref.f64(dout)).sum()
        grads = torch.autograd.grad(loss, [leaf] + ([] if gm is None else [gleaf]))
        dx = torch.full_like(xd, float("nan"))
        dgamma = None if gm is None else torch.full((heads, hd), float("nan"), device="cuda")
        p3d.p3d_rotary_backward(dout.cuda(), pd, fd, dx, gamma=gd, x=None if gm is None else xd,
                                dgamma=dgamma, **kw)
        big = grads[0].abs() + 2                         # terms of dx cancel; x, dout near 1
        assert ref.off_by(dx, grads[0], ref.rounded_once(grads[0], dtype, big)) <= 1
        if gm is not None:
            # sums over n tokens of products near 1
            tol = 2.0 ** -17 * (8 * n ** 0.5 + grads[1].abs())
            assert ref.off_by(dgamma, grads[1], tol) <= 1


def test_gradient_against_differences():
    x, dout, gamma, pos, freqs = make(30, 4, 64, 3, 10, F32, seed=2)
    pd, fd = pos.cuda(), freqs.cuda()
    dx, dgamma = torch.empty_like(x).cuda(), torch.empty(4, 64, device="cuda")
    p3d.p3d_rotary_backward(dout.cuda(), pd, fd, dx, gamma=gamma.cuda(), x=x.cuda(),
                            dgamma=dgamma)

    def loss(x, gamma):
        out = torch.empty_like(x).cuda()
        p3d.p3d_rotary(x.cuda(), pd, fd, out, gamma=gamma.cuda())
        return float((ref.f64(out) * ref.f64(dout)).sum())

    eps = 2.0 ** -7
    for grad, at in ((dx, 0), (dgamma, 1)):
        args = [x, gamma]
        u = grad.cpu().sign()
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + eps * u, args[at] - eps * u
        diff = (loss(*hi) - loss(*lo)) / (2 * eps)
        got = float((ref.f64(grad) * ref.f64(u)).sum())
        assert abs(diff - got) <= 1e-2 * abs(got) + 1e-2


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_packed_in_place_and_grid_coords(layout):
    """q and k of a packed qkv in one call, in place, positions from the
    coords' last three columns; v and the rest of the buffer stay."""
    g = torch.Generator().manual_seed(4)
    n, heads, hd = 77, 4, 64
    qkv = torch.randn(n, 3 * heads, hd, generator=g).to(BF16).cuda()
    coords = torch.randint(0, 64, (n, 4), generator=g, dtype=torch.int32).cuda()
    freqs = p3d.p3d_rotary_frequencies(10000.0, 10).cuda()
    gamma = (1 + 0.2 * torch.randn(2 * heads, hd, generator=g)).to(BF16).cuda()
    before = qkv.clone()
    part = qkv[:, :2 * heads]
    p3d.p3d_rotary(part, coords[:, 1:], freqs, part, layout=layout, gamma=gamma)
    want = ref.rotary(ref.f64(before[:, :2 * heads]), coords[:, 1:].cpu(), freqs.cpu(), layout,
                      gamma=ref.f64(gamma))
    assert ref.off_by(part, want, ref.rounded_once(want, BF16)) <= 1
    assert torch.equal(qkv[:, 2 * heads:], before[:, 2 * heads:])
    # the gradient in place over dout
    dout = torch.randn(n, 3 * heads, hd, generator=g).to(BF16).cuda()
    dx = torch.empty(n, 2 * heads, hd, dtype=BF16, device="cuda")
    x = before[:, :2 * heads]
    p3d.p3d_rotary_backward(dout[:, :2 * heads], coords[:, 1:], freqs, dx, layout=layout,
                            gamma=gamma, x=x)
    p3d.p3d_rotary_backward(dout[:, :2 * heads], coords[:, 1:], freqs, dout[:, :2 * heads],
                            layout=layout, gamma=gamma, x=x)
    assert torch.equal(dout[:, :2 * heads], dx)


def test_long_contexts_keep_their_angles():
    """Positions up to the largest int32: the angle is the exact product."""
    pos = torch.tensor([[0], [1], [32767], [1 << 20], [(1 << 24) + 1], [2 ** 31 - 1],
                        [-(2 ** 31)]], dtype=torch.int32)
    x = torch.randn(7, 2, 64, generator=torch.Generator().manual_seed(1))
    freqs = p3d.p3d_rotary_frequencies(10000.0, 32, "by_parts", 8.0, 4096)
    out = torch.empty_like(x).cuda()
    p3d.p3d_rotary(x.cuda(), pos.cuda(), freqs.cuda(), out, layout="half")
    want = ref.rotary(ref.f64(x), pos, freqs, "half")
    # binary64 turns: 2^31 radians keep 2^-22 of a turn
    assert ref.off_by(out, want, ref.rounded_once(want, F32) + 2.0 ** -18) <= 1


def test_offsets_past_32_bits():
    """Tokens so far apart that the last ones lie past 2^32 elements."""
    n, stride = 5, 1 << 30
    buf = torch.empty(4 * stride + 256, dtype=BF16, device="cuda")
    x = buf.as_strided((n, 2, 128), (stride, 128, 1))
    g = torch.Generator().manual_seed(3)
    host = torch.randn(n, 2, 128, generator=g).to(BF16)
    x.copy_(host)
    pos = torch.arange(n, dtype=torch.int32)[:, None]
    freqs = p3d.p3d_rotary_frequencies(10000.0, 64)
    p3d.p3d_rotary(x, pos.cuda(), freqs.cuda(), x)
    want = ref.rotary(ref.f64(host), pos, freqs, "interleaved")
    assert ref.off_by(x, want, ref.rounded_once(want, BF16)) <= 1


def test_no_tokens_and_repeatable():
    freqs = p3d.p3d_rotary_frequencies(10000.0, 8).cuda()
    e = torch.empty(0, 3, 32, dtype=BF16, device="cuda")
    pos = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    gamma = torch.ones(3, 32, dtype=BF16, device="cuda")
    dgamma = torch.full((3, 32), 5.0, device="cuda")
    p3d.p3d_rotary(e, pos, freqs, e.clone(), gamma=gamma)
    p3d.p3d_rotary_backward(e, pos, freqs, e.clone(), gamma=gamma, x=e, dgamma=dgamma)
    assert (dgamma == 0).all()
    x, dout, gamma, pos, freqs = make(3000, 24, 128, 3, 21, BF16, seed=5)
    args = [dout.cuda(), pos.cuda(), freqs.cuda()]
    got = []
    for stream in (None, None, torch.cuda.Stream()):
        dx = torch.empty_like(args[0])
        dg = torch.empty(24, 128, device="cuda")
        ws = torch.empty(p3d.p3d_rotary_workspace_size(*args), dtype=torch.uint8, device="cuda")
        xd, gd = x.cuda(), gamma.cuda()
        torch.cuda.synchronize()
        p3d.p3d_rotary_backward(*args, dx, gamma=gd, x=xd, dgamma=dg, workspace=ws,
                                stream=stream)
        torch.cuda.synchronize()
        got.append((dx, dg))
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(got[0], g))


def test_positions_further_apart_than_the_descriptor_holds():
    """pos_stride is an int32: rows 2^32 + 1 entries apart, which would pass
    as 1, are refused by name."""
    x = torch.randn(2, 1, 8, device="cuda")
    far = torch.zeros((1 << 32) + 2, dtype=torch.int32, device="cuda").as_strided(
        (2, 1), ((1 << 32) + 1, 1))
    freqs = p3d.p3d_rotary_frequencies(10000.0, 4).cuda()
    with pytest.raises(ValueError, match="positions"):
        p3d.p3d_rotary(x, far, freqs, torch.empty_like(x))
