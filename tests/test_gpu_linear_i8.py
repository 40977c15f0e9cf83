"""p3d_quantize_rows and p3d_linear_i8 on the GPU: integers exactly, outputs
against 64 bits."""
import pytest
import torch

import model_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def quantized(x):
    q = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    s = torch.full((x.shape[0],), -1.0, device="cuda")
    p3d.p3d_quantize_rows(x, q, s)
    return q, s


def check_quantize(x):
    q, s = quantized(x)
    want, scale = ref.quantize(ref.f64(x))
    assert torch.equal(s.cpu().double().nan_to_num(-7), scale.nan_to_num(-7))
    off = (q.cpu().double() != want).nonzero()
    assert off.numel() == 0, (off[:5], x[off[0, 0], off[0, 1]], s[off[0, 0]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(1, 16), (3, 64), (5, 512), (7, 528), (130, 1024), (66, 1040),
                                 (33, 2048), (9, 2064), (5, 8192), (3, 8208), (2, 32768),
                                 (2, 32784), (3, 65536)])
def test_quantize_sizes(n, k, dtype):
    g = gen(n + k)
    x = torch.randn(n, k, generator=g) * torch.randn(k, generator=g).exp()
    check_quantize(x.to(TYPES[dtype]).cuda())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(32769, 1040), (16385, 2048), (8127, 2064), (2049, 8192)])
def test_quantize_many_rows(n, k, dtype):
    """More than 2^25 (from 2049 a row on: 2^24) elements, where a thread holds
    more of them: each row as it comes out among few."""
    few = torch.randn(100, k, generator=gen(k)).to(TYPES[dtype]).cuda()
    check_quantize(few)
    q, s = quantized(few)
    pick = torch.randint(0, 100, (n,), generator=gen(n)).cuda()
    many_q, many_s = quantized(few[pick])
    assert torch.equal(many_q, q[pick]) and torch.equal(many_s, s[pick])


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_between_two_integers(dtype):
    """Quotients at and next to the middle: the largest a multiple of 127 gives
    exact scales and ties, others quotients a rounding away from them."""
    k, rows = 256, []
    for top in (127.0, 254.0, 127.0 * 2 ** -20, 100.0, 3.0, 1.0, 0.1, 85.0):
        base = torch.arange(k, dtype=torch.float64) - k // 2
        row = (base + 0.5) / 127 * top
        row[0] = top
        for shift in (0.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -22):
            r = row * (1 + shift)
            r[0] = top
            rows.append(r.clamp(-top, top))
    x = torch.stack(rows).float().to(TYPES[dtype]).cuda()
    check_quantize(x)
    g = gen(1)
    halves = torch.randint(-127, 128, (64, 512), generator=g).float() / 2
    halves[:, 3] = 127.0
    check_quantize(halves.to(TYPES[dtype]).cuda())


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_edges(dtype):
    x = torch.zeros(7, 64)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[2, 6] = 1.0
    x[3, :] = torch.linspace(-1, 1, 64) * 1e-42           # scales below the normal numbers
    x[4, :] = torch.linspace(-1, 1, 64) * 3e38
    x[5, 0] = 1e-45                                       # a scale that rounds to 0
    x[6, :] = torch.linspace(-1, 1, 64) * 1e-31
    check_quantize(x.to(TYPES[dtype]).cuda())


def test_quantize_strided_rows():
    wide = torch.randn(50, 200, generator=gen(2)).bfloat16().cuda()
    out = torch.full((50, 160), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(50, device="cuda")
    p3d.p3d_quantize_rows(wide[:, 8:104], out[:, 16:112], s)
    want, _ = ref.quantize(ref.f64(wide[:, 8:104]))
    assert torch.equal(out[:, 16:112].cpu().double(), want)
    assert (out[:, :16] == 77).all() and (out[:, 112:] == 77).all()


def made(n, k, d, dtype, seed, bias=True, residual=False):
    g = gen(seed)
    return dict(q=torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8).cuda(),
                s=(torch.rand(n, generator=g) * 0.02 + 1e-3).cuda(),
                w=torch.randint(-128, 128, (d, k), generator=g, dtype=torch.int8).cuda(),
                t=(torch.rand(d, generator=g) * 2e-3 / k ** 0.5 + 1e-5).cuda(),
                b=torch.randn(d, generator=g).to(dtype).cuda() if bias else None,
                r=torch.randn(n, d, generator=g).to(dtype).cuda() if residual else None)


def check_out(out, s, dtype, kind):
    want, size = ref.linear(ref.f64(s["q"]), ref.f64(s["s"]), ref.f64(s["w"]), ref.f64(s["t"]),
                            ref.f64(s["b"]), kind, ref.f64(s["r"]))
    # conversion of the sum, two products, two sums; |act'| <= 1.13 and, with an
    # activation, a hardware exponential and reciprocal of an argument of that size
    slack = ref.U * size * (8 if kind == "none" else 8 + 8 * (2 + size))
    bound = ref.HALF[dtype] * want.abs() + slack * (1 + 2 * ref.HALF[dtype]) + 1e-37
    off = (out.cpu().double() - want).abs()
    assert bool((off <= bound).all()), (float((off / bound).max()), int((off / bound).argmax()))


def check(n, k, d, dtype, kind="none", bias=True, residual=False, seed=None):
    s = made(n, k, d, dtype, n + k + d if seed is None else seed, bias, residual)
    out = torch.full((n, d), float("nan"), dtype=dtype, device="cuda")
    p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], out, s["b"], kind, s["r"])
    check_out(out, s, dtype, kind)


SIZES = [(1, 16, 8), (1, 64, 24), (5, 1024, 1536), (16, 80, 16), (17, 528, 40), (32, 1040, 136),
         (33, 512, 64), (64, 4096, 72), (65, 16, 8), (66, 128, 64), (100, 144, 200),
         (129, 256, 136), (300, 1040, 520), (1000, 2048, 1536), (2100, 400, 1032),
         (4100, 272, 4104), (5000, 1536, 3080), (70, 8192, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k,d", SIZES)
def test_sizes(n, k, d, dtype):
    check(n, k, d, TYPES[dtype])


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_epilogues(dtype, bias, residual, kind):
    for n, k, d in ((3, 96, 48), (40, 96, 48), (200, 208, 296), (3000, 144, 2064)):
        check(n, k, d, TYPES[dtype], kind, bias, residual)


def test_sums_at_the_ends_of_the_integers():
    """-128 throughout over the longest rows: 2^14 * 65536 is 2^30."""
    for n, d in ((4, 16), (130, 136)):
        q = torch.full((n, 65536), -128, dtype=torch.int8, device="cuda")
        w = torch.full((d, 65536), -128, dtype=torch.int8, device="cuda")
        w[::2] = 127
        one = torch.ones
        out = torch.empty(n, d, device="cuda")
        p3d.p3d_linear_i8(q, one(n, device="cuda"), w, one(d, device="cuda"), out)
        assert (out[:, 1::2] == 2.0 ** 30).all() and (out[:, ::2] == -128.0 * 127 * 65536).all()


def test_scales_apply_one_after_the_other():
    """Scales whose product binary32 does not hold."""
    for n in (3, 200):
        q = torch.full((n, 64), 100, dtype=torch.int8, device="cuda")
        w = torch.full((16, 64), 100, dtype=torch.int8, device="cuda")
        out = torch.empty(n, 16, device="cuda")
        p3d.p3d_linear_i8(q, torch.full((n,), 2.0 ** -80, device="cuda"), w,
                          torch.full((16,), 2.0 ** -60, device="cuda"), out)
        assert (out == 640000 * 2.0 ** -140).all()


def test_a_row_that_is_not_finite_stays_alone():
    for n in (5, 500):
        x = torch.randn(n, 128, generator=gen(3)).cuda()
        x[2, 7] = float("inf")
        q, s = quantized(x)
        d = made(n, 128, 72, torch.float32, 4)
        out = torch.empty(n, 72, device="cuda")
        p3d.p3d_linear_i8(q, s, d["w"], d["t"], out, d["b"])
        assert out[2].isnan().all() and out.isnan().sum() == 72


@pytest.mark.parametrize("n", [9, 150, 3000])
def test_strided_tokens_and_outputs(n):
    k, d = 208, 264
    s = made(n, k, d, torch.bfloat16, 5, residual=True)
    wide = torch.full((n, k + 48), 111, dtype=torch.int8, device="cuda")
    wide[:, 32:32 + k] = s["q"]
    out = torch.full((n, d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    res = torch.full((n, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    res[:, :d] = s["r"]
    p3d.p3d_linear_i8(wide[:, 32:32 + k], s["s"], s["w"], s["t"], out[:, 8:8 + d], s["b"],
                      "silu", res[:, :d])
    check_out(out[:, 8:8 + d], s, torch.bfloat16, "silu")
    assert (out[:, :8] == 7).all() and (out[:, 8 + d:] == 7).all()


@pytest.mark.parametrize("n", [9, 150, 3000])
def test_added_into_the_residual(n):
    s = made(n, 320, 136, torch.bfloat16, 6, residual=True)
    out = s["r"].clone()
    p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], out, s["b"], residual=out)
    check_out(out, s, torch.bfloat16, "none")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(300, 1544), (1500, 1544), (3900, 1544), (6990, 1544),
                                 (15000, 1544), (20000, 1544), (2500, 6152), (600, 12296)])
def test_residuals_in_every_tile(n, d, dtype):
    """Each tile's shape, one and several rounds, bands of features, ragged at both
    ends: added in place and into another tensor, the same."""
    s = made(n, 80, d, TYPES[dtype], n + d, residual=True)
    out, other = s["r"].clone(), torch.full_like(s["r"], 9)
    p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], out, s["b"], "silu", residual=out)
    p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], other, s["b"], "silu", residual=s["r"])
    assert torch.equal(out, other)
    check_out(out, s, TYPES[dtype], "silu")


def test_the_same_call_gives_the_same_bytes():
    for n in (5, 1000, 20000):
        s = made(n, 1024, 520, torch.bfloat16, 7)
        outs = [torch.empty(n, 520, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        for o in outs:
            p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], o, s["b"], "gelu")
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_no_tokens():
    s = made(0, 64, 16, torch.float32, 8)
    p3d.p3d_linear_i8(s["q"], s["s"], s["w"], s["t"], torch.empty(0, 16, device="cuda"), s["b"])
    p3d.p3d_quantize_rows(torch.empty(0, 64, device="cuda"), s["q"], s["s"])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", [16, 48, 64, 112, 128, 176, 192, 240, 256, 320])
def test_several_tiles_of_few_stages(k, residual):
    """Rows of one stage to five, the last of every length, where a workgroup goes on
    to other tiles: the loads of the next stand beside the end of one."""
    for n, d in ((21000, 1544), (3000, 4104)):
        check(n, k, d, torch.bfloat16, "none", True, residual)
