"""p3d_group_norm and its gradient on the GPU against 64 bits."""
import pytest
import torch

import model_ref as ref
import pixel_aligned_image_amd as p3d
from block_ref import uneven

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def made(n, c, dtype, seed, mean=0.5, by=1.5):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, scale=1.0, base=0.0):
        return (torch.randn(*shape, generator=g) * scale + base).to(dtype).cuda()

    x = randn(n, c, scale=by) + randn(c, scale=mean)
    return dict(x=x, w=randn(c, scale=0.3, base=1.0), b=randn(c, scale=0.5), dout=randn(n, c))


def strided(t, more):
    """The same rows in a wider buffer of NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + more), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, more // 2:more // 2 + t.shape[1]] = t
    return wide[:, more // 2:more // 2 + t.shape[1]], wide


def near(got, want, dtype, slack, what):
    """Within half a step of the type of the value, and `slack` of binary32's
    roundings before that (which the last rounding may carry over a step)."""
    got, want = got.double().cpu(), want
    assert got.shape == want.shape
    if got.numel() == 0:
        return
    bound = ref.HALF[dtype] * want.abs() + slack * (1 + 2 * ref.HALF[dtype]) + 1e-37
    off = (got - want).abs()
    assert bool((off <= bound).all()), (what, float((off / bound).max()),
                                        int((off / bound).argmax()))


def check(n, c, groups, dtype, kind, off=None, s=None, seed=0, affine=True, eps=1e-5, stride=0,
          in_place=False):
    off = [0, n] if off is None else off
    s = made(n, c, dtype, seed) if s is None else s
    w, b = (s["w"], s["b"]) if affine else (None, None)
    x64, w64, b64 = ref.f64(s["x"]), ref.f64(w), ref.f64(b)
    items = len(off) - 1
    mean, rstd = (torch.full((items, groups), float("nan"), device="cuda") for _ in range(2))
    x = s["x"].clone()
    out = x if in_place else torch.full_like(x, float("nan"))
    if stride:
        x, _ = strided(x, stride)
        out, wide = strided(out, 2 * stride)
    p3d.p3d_group_norm(x, out, groups, off, w, b, kind, eps, mean, rstd)
    torch.cuda.synchronize()
    want, u = ref.group_norm(x64, off, groups, w64, b64, kind, eps)
    m64, r64 = ref.group_stats(x64, off, groups, eps)
    # the statistics: a chunk's are sums of batches' own means, each good to a
    # few roundings of the largest value, 64 of them one after the other
    top = float(x64.abs().max()) if n else 0.0
    assert torch.all((mean.cpu().double() - m64).abs() <= 2 * ref.U * m64.abs() + 64 * ref.U * top)
    assert torch.all((rstd.cpu().double() - r64).abs() <= 64 * ref.U * r64 * (1 + r64 * top * 1e-2))
    # u: the mean's error times rstd and weight, and a few roundings of its terms;
    # the activation: |act'| <= 1.13, and a hardware exponential and reciprocal
    gain = ref.spread(r64, off, c) * (1 if w64 is None else w64.abs())
    size = u.abs() + (0 if b64 is None else b64.abs())
    slack = 1.2 * (64 * ref.U * top * gain + 80 * ref.U * size) + 4 * ref.U * want.abs() * (
        2 + 2 * u.abs())
    near(out, want, dtype, slack, "out")
    if stride:
        assert wide[:, :stride].isnan().all() and wide[:, stride + c:].isnan().all()

    grads = ref.group_norm_backward(ref.f64(s["dout"]), x64, off, groups, w64, b64, kind, eps)
    dweight, dbias = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
    x, dout = s["x"].clone(), s["dout"].clone()
    dx = dout if in_place else torch.full_like(x, float("nan"))
    if stride:
        x, _ = strided(x, stride)
        dout, _ = strided(dout, 3 * stride)
        dx, wide = strided(dx, 2 * stride)
    p3d.p3d_group_norm_backward(dout, x, mean, rstd, dx, groups, off, w, b, kind, dweight, dbias)
    torch.cuda.synchronize()
    # du carries the slope's error (hardware exponential and reciprocal of u,
    # and u's own), sums over rows a thread's serial roundings
    d64 = ref.f64(s["dout"]).abs() * 1.2
    du = d64 * (64 * ref.U * (2 + size) + 64 * ref.U * top * gain)
    xn = (x64 - ref.spread(m64, off, c)).abs() * ref.spread(r64, off, c)
    w1 = 1 if w64 is None else w64.abs()
    terms = d64 * w1

    def average(v):                          # over an item's group, back on its elements
        out = torch.zeros(items, groups, dtype=torch.float64)
        for i in range(items):
            r = v[off[i]:off[i + 1]]
            if r.shape[0]:
                out[i] = r.reshape(-1, groups, c // groups).mean((0, 2))
        return ref.spread(out, off, c)

    each = du * w1 + 128 * ref.U * terms
    slack = ref.spread(r64, off, c) * (each + average(each) + (xn + 1) * average(each * (xn + 1)))
    near(dx, grads["dx"], dtype, slack, "dx")
    sums = (du + 128 * ref.U * d64)
    near(dbias, grads["dbias"], torch.float32, sums.sum(0), "dbias")
    near(dweight, grads["dweight"], torch.float32, (sums * (xn + 1)).sum(0), "dweight")
    if stride:
        assert wide[:, :stride].isnan().all() and wide[:, stride + c:].isnan().all()


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,c,groups", [
    (1, 8, 1), (2, 8, 8), (3, 24, 3), (7, 40, 5), (5, 104, 13), (33, 64, 32), (100, 320, 32),
    (257, 96, 1), (1000, 512, 32), (64, 2056, 8), (130, 4096, 32), (9, 4096, 4096),
    (4097, 72, 9), (904, 72, 9), (2728, 72, 9), (2729, 72, 9), (4096, 512, 32), (4100, 512, 32),
    (9000, 104, 13), (33000, 8, 1), (33000, 8, 8), (5000, 2056, 8), (3000, 4096, 64),
    (2000, 4096, 4096), (20000, 40, 40)])
def test_sizes(n, c, groups, dtype, kind):
    check(n, c, groups, TYPES[dtype], kind, seed=n + c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,items", [(1, 3), (40, 7), (3000, 5), (20000, 17), (700, 256),
                                     (60000, 3), (90000, 20)])
def test_ragged_items(n, items, dtype):
    check(n, 64, 16, TYPES[dtype], "silu", uneven(n, items), seed=items)


def test_one_channel_a_group_and_no_affine():
    check(77, 12, 12, torch.float32, "gelu", affine=False)
    check(77, 24, 24, torch.bfloat16, "none", affine=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_keep_what_lies_between(dtype):
    check(301, 72, 9, TYPES[dtype], "silu", uneven(301, 4), stride=16)
    check(12000, 72, 9, TYPES[dtype], "silu", uneven(12000, 4), stride=16)


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(dtype):
    check(1500, 128, 8, TYPES[dtype], "silu", uneven(1500, 3), in_place=True)
    check(30000, 128, 8, TYPES[dtype], "silu", uneven(30000, 3), in_place=True)


def test_a_large_mean_keeps_the_digits():
    """Channels a thousand deviations from 0: the deviations come out as the
    input holds them."""
    for n in (500, 5000, 50000):
        s = made(n, 64, torch.float32, 5)
        s["x"] = (torch.randn(n, 64, generator=torch.Generator().manual_seed(6)) + 1000).cuda()
        check(n, 64, 8, torch.float32, "none", s=s)


@pytest.mark.parametrize("n", [500, 50000])
def test_constant_rows(n):
    """A variance of 0: out is act(bias), rstd is 1 / sqrt(eps)."""
    s = made(n, 32, torch.float32, 7)
    s["x"] = torch.full((n, 32), 3.25, device="cuda")
    out, mean, rstd = torch.empty_like(s["x"]), torch.empty(1, 4, device="cuda"), torch.empty(
        1, 4, device="cuda")
    p3d.p3d_group_norm(s["x"], out, 4, weight=s["w"], bias=s["b"], mean=mean, rstd=rstd)
    assert torch.equal(out, s["b"].expand(n, 32)) and (mean == 3.25).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("by", [1, 100])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_in_their_group(dtype, by):
    n, c, groups, off = 300 * by, 64, 8, [0, 100 * by, 250 * by, 300 * by]
    s = made(n, c, TYPES[dtype], 8)
    clean = torch.empty_like(s["x"])
    p3d.p3d_group_norm(s["x"], clean, groups, off, s["w"], s["b"], "silu")
    s["x"][120 * by, 10] = float("nan")
    s["x"][220 * by, 63] = float("inf")
    out = torch.empty_like(clean)
    p3d.p3d_group_norm(s["x"], out, groups, off, s["w"], s["b"], "silu")
    bad = torch.zeros(n, c, dtype=torch.bool, device="cuda")
    bad[100 * by:250 * by, 8:16] = True
    bad[100 * by:250 * by, 56:64] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


def test_no_rows():
    x = torch.empty(0, 32, device="cuda")
    mean, rstd = torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    p3d.p3d_group_norm(x, x.clone(), 4, [0, 0, 0], mean=mean, rstd=rstd)
    assert (mean == 0).all() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))
    dw, db = torch.full((32,), 7.0, device="cuda"), torch.full((32,), 7.0, device="cuda")
    p3d.p3d_group_norm_backward(x, x, mean, rstd, x.clone(), 4, [0, 0, 0], dweight=dw, dbias=db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("n,off", [(400, [0, 400]), (400, [0, 1, 399, 400]), (40000, [0, 40000]),
                                   (40000, [0, 1, 39999, 40000])])
def test_only_the_gradients_that_are_wanted(n, off):
    s = made(n, 64, torch.bfloat16, 9)
    mean, rstd = (torch.empty(len(off) - 1, 8, device="cuda") for _ in range(2))
    p3d.p3d_group_norm(s["x"], torch.empty_like(s["x"]), 8, off, mean=mean, rstd=rstd)
    got = []
    for dw, db in ((1, 1), (1, 0), (0, 1), (0, 0)):
        dx = torch.empty_like(s["x"])
        dw, db = (torch.empty(64, device="cuda") if k else None for k in (dw, db))
        p3d.p3d_group_norm_backward(s["dout"], s["x"], mean, rstd, dx, 8, off, dweight=dw,
                                    dbias=db)
        got.append((dx, dw, db))
    assert all(torch.equal(g[0], got[0][0]) for g in got)
    assert torch.equal(got[1][1], got[0][1]) and torch.equal(got[2][2], got[0][2])


@pytest.mark.parametrize("n", [300, 30000])
def test_the_same_call_gives_the_same_bytes(n):
    s = made(n, 256, torch.bfloat16, 10)
    off = uneven(n, 5)
    runs = []
    for _ in range(3):
        mean, rstd = torch.empty(5, 32, device="cuda"), torch.empty(5, 32, device="cuda")
        out, dx = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        dw, db = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
        p3d.p3d_group_norm(s["x"], out, 32, off, s["w"], s["b"], "silu", 1e-5, mean, rstd)
        p3d.p3d_group_norm_backward(s["dout"], s["x"], mean, rstd, dx, 32, off, s["w"], s["b"],
                                    "silu", dw, db)
        runs.append((out, mean, rstd, dx, dw, db))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_gradient_against_differences():
    """Central differences of the GPU's own forward results in binary32, summed
    in 64 bits: a difference's error is the results' over the step."""
    n, c, groups = 40, 16, 4
    s = made(n, c, torch.float32, 11)
    mean, rstd = torch.empty(1, groups, device="cuda"), torch.empty(1, groups, device="cuda")

    def loss(x):
        out = torch.empty_like(x)
        p3d.p3d_group_norm(x, out, groups, weight=s["w"], bias=s["b"], act="silu", mean=mean,
                           rstd=rstd)
        return float((out.double() * s["dout"].double()).sum())

    loss(s["x"])
    dx = torch.empty_like(s["x"])
    p3d.p3d_group_norm_backward(s["dout"], s["x"], mean, rstd, dx, groups, weight=s["w"],
                                bias=s["b"], act="silu")
    h = 2.0 ** -6
    for i in range(0, n * c, 37):
        ends = []
        for d in (h, -h):
            x = s["x"].clone()
            x.view(-1)[i] += d
            ends.append(loss(x))
        # (640 results of size 3 good to 2^-20, over 2 h; and h^2 / 6 of a third
        # derivative of a few units)
        assert abs((ends[0] - ends[1]) / (2 * h) - float(dx.view(-1)[i])) < 640 ** 0.5 * 3 * (
            2.0 ** -20) / h + 10 * h * h, i


@pytest.mark.parametrize("value", [0.1, 100.3, 12345.678, -3e5 - 1 / 3])
@pytest.mark.parametrize("n,c,groups", [
    (45, 32, 4), (500, 32, 1), (501, 24, 8), (5003, 16, 16), (50000, 32, 4),
    # (8 rows a thread and more)
    (20011, 1024, 32), (9001, 2048, 1), (20011, 1024, 1024), (30011, 320, 32)])
def test_constant_rows_whose_sums_are_rounded(n, c, groups, value):
    """A variance of 0 about a mean whose multiples binary32 does not hold: out is
    act(bias), rstd 1 / sqrt(eps), in the gradient's x^ nothing is left either."""
    s = made(n, c, torch.float32, 7)
    s["x"] = torch.full((n, c), value, device="cuda")
    out, mean, rstd = torch.empty_like(s["x"]), torch.empty(1, groups, device="cuda"), torch.empty(
        1, groups, device="cuda")
    p3d.p3d_group_norm(s["x"], out, groups, weight=s["w"], bias=s["b"], mean=mean, rstd=rstd)
    top = abs(float(s["x"][0, 0]))
    r = 1e-5 ** -0.5
    # Items in registers: the sum of at most 128 rows is off by 64 roundings (32 in a
    # thread, then a tree), so deviations are 64 U of the value at most, and their own
    # mean, taken off again, is off by as many roundings of that. Chunks: batches are
    # exact, 1023 of them are joined in binary64.
    left = 64 * ref.U * 64 * ref.U * top + 1100 * 2.0 ** -53 * top
    bound = left * r * s["w"].abs().double() + 2 * ref.U * s["b"].abs().double() + 1e-37
    assert torch.all((out.double() - s["b"].double()).abs() <= bound)
    assert (mean == s["x"][0, 0]).all()
    # (the variance: 64 roundings of the deviations' squares)
    var = 64 * ref.U * (64 * ref.U * top) ** 2 + left ** 2
    assert torch.all((rstd.double() / r - 1).abs() <= 4 * ref.U + var / 1e-5)
    dx, dw, db = torch.empty_like(out), *(torch.empty(c, device="cuda") for _ in range(2))
    p3d.p3d_group_norm_backward(s["dout"], s["x"], mean, rstd, dx, groups, weight=s["w"],
                                dweight=dw, dbias=db)
    assert not dw.any()
    assert torch.allclose(db.double(), s["dout"].double().sum(0),
                          atol=float(s["dout"].double().abs().sum(0).max()) * 64 * ref.U)


@pytest.mark.parametrize("value", [100.5, -3e5])
def test_constant_rows_in_bf16(value):
    n, c, groups = 20011, 1024, 32
    x = torch.full((n, c), value, dtype=torch.bfloat16, device="cuda")
    out, mean, rstd = torch.empty_like(x), *(torch.empty(1, groups, device="cuda") for _ in "ab")
    b = made(n, c, torch.bfloat16, 7)["b"]
    p3d.p3d_group_norm(x, out, groups, bias=b, mean=mean, rstd=rstd)
    assert torch.equal(out, b.expand(n, c)) and (mean == x[0, 0].float()).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


def check_group_by_group(n, c, groups, dtype, kind, off, stride=0, in_place=False, seed=0, eps=1e-5):
    """As check, of maps whose 64-bit form would not be quick on the CPU: a group
    at a time, on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, base=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + base).to(dtype)

    def buffer(t, more):
        wide = torch.full((n, c + more), float("nan"), dtype=dtype, device="cuda")
        wide[:, more // 2:more // 2 + c] = t
        return wide[:, more // 2:more // 2 + c]

    x = randn(n, c, scale=1.5) + randn(c, scale=0.5)
    dout, w, b = randn(n, c), randn(c, scale=0.3, base=1.0), randn(c, scale=0.5)
    items, per = len(off) - 1, c // groups
    mean, rstd = (torch.full((items, groups), float("nan"), device="cuda") for _ in range(2))
    keep, kept = x.clone(), dout.clone()
    if stride:
        x, dout = buffer(x, stride), buffer(dout, 3 * stride)
    out = x if in_place else buffer(torch.full_like(keep, float("nan")), 2 * stride)
    p3d.p3d_group_norm(x, out, groups, off, w, b, kind, eps, mean, rstd)
    out = out.clone()
    if in_place:
        x.copy_(keep)
    dx = dout if in_place else buffer(torch.full_like(keep, float("nan")), 2 * stride)
    dweight, dbias = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
    p3d.p3d_group_norm_backward(dout, x, mean, rstd, dx, groups, off, w, b, kind, dweight, dbias)
    lengths = torch.tensor(off, device="cuda").diff()
    item = torch.repeat_interleave(torch.arange(items, device="cuda"), lengths)
    count = (lengths * per).clamp(min=1).double()[:, None]

    def over(v):                             # [n, per] -> averages [items, 1]
        return torch.stack([v[i:k].sum() for i, k in zip(off, off[1:])])[:, None] / count

    def close(got, want, dtype, slack, what):
        bound = ref.HALF[dtype] * want.abs() + slack * (1 + 2 * ref.HALF[dtype]) + 1e-37
        off_ = (got.double() - want).abs()
        assert bool((off_ <= bound).all()), (what, float((off_ / bound).max()))

    for j in range(groups):
        cols = slice(j * per, (j + 1) * per)
        x64, d64, w64, b64 = (t[..., cols].double() for t in (keep, kept, w, b))
        m64 = over(x64)
        r64 = (over((x64 - m64[item]).square()) + eps).rsqrt()
        top = float(x64.abs().max())
        # (bounds as in check)
        assert torch.all((mean[:, j:j + 1] - m64).abs() <= 2 * ref.U * m64.abs() + 64 * ref.U * top)
        assert torch.all((rstd[:, j:j + 1] - r64).abs()
                         <= 64 * ref.U * r64 * (1 + r64 * top * 1e-2))
        xn = (x64 - m64[item]) * r64[item]
        u = (xn * w64 + b64).requires_grad_(True)
        want = ref.act(u, kind)
        slope, = torch.autograd.grad(want.sum(), u)
        u, want = u.detach(), want.detach()
        gain = r64[item] * w64.abs()
        size = u.abs() + b64.abs()
        slack = 1.2 * (64 * ref.U * top * gain + 80 * ref.U * size) + 4 * ref.U * want.abs() * (
            2 + 2 * u.abs())
        close(out[:, cols], want, dtype, slack, ("out", j))
        du64 = d64 * slope
        dn = du64 * w64
        dx64 = r64[item] * (dn - over(dn)[item] - xn * over(dn * xn)[item])
        big = d64.abs() * 1.2
        du = big * (64 * ref.U * (2 + size) + 64 * ref.U * top * gain)
        each = du * w64.abs() + 128 * ref.U * big * w64.abs()
        slack = r64[item] * (each + over(each)[item]
                             + (xn.abs() + 1) * over(each * (xn.abs() + 1))[item])
        close(dx[:, cols], dx64, dtype, slack, ("dx", j))
        sums = du + 128 * ref.U * big
        close(dbias[cols], du64.sum(0), torch.float32, sums.sum(0), ("dbias", j))
        close(dweight[cols], (du64 * xn).sum(0), torch.float32,
              (sums * (xn.abs() + 1)).sum(0), ("dweight", j))


@pytest.mark.parametrize("n,c,groups,dtype,items,kind,stride,in_place", [
    (110001, 1024, 32, "bf16", 1, "silu", 0, False), (110001, 1024, 32, "bf16", 3, "gelu", 16, False),
    (110001, 1024, 32, "bf16", 3, "silu", 0, True),
    # few groups, many items: the chunks of either fit the bound of joining them in place
    (110001, 1024, 1, "bf16", 1, "silu", 0, False), (110001, 1024, 2, "bf16", 1, "none", 0, True),
    (262144, 1024, 32, "bf16", 16, "silu", 0, False),
    # groups that straddle vectors, and one channel each
    (110001, 1000, 40, "bf16", 2, "silu", 16, False), (1700001, 64, 64, "bf16", 2, "silu", 0, False),
    (60001, 1024, 32, "f32", 2, "silu", 16, False), (60001, 1000, 200, "f32", 1, "gelu", 0, True)])
def test_maps_larger_than_the_caches(n, c, groups, dtype, items, kind, stride, in_place):
    check_group_by_group(n, c, groups, TYPES[dtype], kind, uneven(n, items), stride, in_place,
                         seed=n + groups)
