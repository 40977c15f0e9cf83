"""p3d_adamw and p3d_grad_norm on the GPU against 64 bits."""
import math

import pytest
import torch

import model_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [1, 7, 255, 256, 257, 1536, 4096, 4097, 8191, 50000]
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)


class Model:
    """Tensors of the given sizes with guards around them, kept in 64 bits too."""

    def __init__(self, sizes, param="f32", grad="f32", master=False, bits=32, seed=0, late=True):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.bits = sizes, bits
        self.decay = [0.1 * (j % 3) for j in range(len(sizes))]
        self.guards = []

        def held(x, dtype):
            """x in the middle of a buffer whose other bytes are checked."""
            wide = torch.ones(x.numel() + 64, dtype=dtype, device="cuda")
            wide[32:32 + x.numel()] = x.to(dtype).cuda()
            self.guards.append((wide, x.numel()))
            return wide[32:32 + x.numel()]

        self.w, self.g, self.m, self.v, self.masters, self.ms, self.vs = ([] for _ in range(7))
        for n in sizes:
            size = float(torch.rand(1, generator=g)) * 1e-2 + 1e-4
            w = torch.randn(n, generator=g) * 0.1
            grad_ = torch.randn(n, generator=g) * size
            grad_[torch.rand(n, generator=g) < 0.05] = 0
            m = torch.randn(n, generator=g) * size * 0.3 * late
            r = (torch.randn(n, generator=g).abs() + 0.01) * size * late
            if master:
                self.masters.append(held(w, torch.float32))
            self.w.append(held(w, TYPES[param]))
            self.g.append(held(grad_, TYPES[grad]))
            if bits == 32:
                self.m.append(held(m, torch.float32))
                self.v.append(held(r * r, torch.float32))
            else:
                for x, codes, scales in ((m, self.m, self.ms), (r, self.v, self.vs)):
                    rows = ref.blocks(x)
                    s = rows.abs().amax(1) / 448
                    q = (rows / s.clamp(min=1e-30)[:, None]).reshape(-1)[:n]
                    codes.append(held(q.to(torch.float8_e4m3fn).view(torch.uint8).float(),
                                      torch.uint8).view(torch.float8_e4m3fn))
                    scales.append(held(s, torch.float32))
        self.table = p3d.make_adamw_tensors(
            self.w, self.g, self.m, self.v, masters=self.masters or None,
            m_scales=self.ms or None, v_scales=self.vs or None, weight_decay=self.decay)

    def states(self, j):
        """(w, m, v) of tensor j in 64 bits"""
        w = ref.f64((self.masters or self.w)[j])
        if self.bits == 32:
            return w, ref.f64(self.m[j]), ref.f64(self.v[j])
        n = self.sizes[j]
        m, r = (ref.f64(c[j].float()) * ref.f64(s[j]).repeat_interleave(256)[:n]
                for c, s in ((self.m, self.ms), (self.v, self.vs)))
        return w, m, r * r

    def check_guards(self):
        for wide, n in self.guards:
            assert (wide[:32].float() == 1).all() and (wide[32 + n:].float() == 1).all()


def check_codes(codes, scales, x, slack, bits, least, what):
    """Codes that the bits choose for the states x, each known to `slack`: a
    binary32 state is off by a few roundings, which may move it over a border."""
    n = x.numel()
    top = ref.blocks(x).abs().amax(1)
    off = ref.blocks(slack).amax(1)
    got_scale = ref.f64(scales)
    assert torch.all((got_scale - top / 448).abs() <= off / 448 + 3 * ref.U * top / 448), what
    by = torch.where(got_scale > 0, 1 / got_scale.clamp(min=1e-300), torch.zeros_like(top))
    by = by.repeat_interleave(256)[:n]
    got = ref.f64(codes.float())
    # (the scale's reciprocal and the product: 4 roundings)
    ends = [ref.encode((x + d * (slack + 4 * ref.U * x.abs())) * by, bits.double())
            for d in (-1, 1)]
    low, high = torch.minimum(*ends), torch.maximum(*ends)
    if least:
        low, high = (torch.where((x > 0) & (by > 0) & (e <= 0), torch.full_like(e, 2.0 ** -9), e)
                     for e in (low, high))
    assert torch.all((got >= low) & (got <= high)), (
        what, (~((got >= low) & (got <= high))).nonzero().flatten()[:5])


def step_and_check(model, step, scale=None, seed=0, hyper=None, **kw):
    hyper = hyper or HYPER
    before = [model.states(j) for j in range(len(model.sizes))]
    by = 1.0 if scale is None else float(scale)
    p3d.p3d_adamw(model.table, step=step, seed=seed, grad_scale=scale, **hyper, **kw)
    torch.cuda.synchronize()
    for j, n in enumerate(model.sizes):
        w, m, v = before[j]
        g = ref.f64(model.g[j])
        want, m1, v1 = ref.adamw(w, g, m, v, hyper["lr"], hyper["beta1"], hyper["beta2"],
                                 hyper["eps"], step, float(torch.tensor(model.decay[j])), by)
        # A dozen binary32 roundings of the update (the factors among them), two of
        # w. m = b1 m + c1 g is a sum of two terms that may cancel: its products, the
        # factors and the sum are off by 6 roundings of |b1 m| + |c1 g| and not of
        # |m|, which the update divides by the same denominator as m.
        size_m = hyper["beta1"] * m.abs() + (1 - hyper["beta1"]) * (g * by).abs()
        under = (v1 / (1 - hyper["beta2"] ** step)).sqrt() + hyper["eps"]
        slack = (24 * ref.U * ((want - w).abs() + hyper["lr"] * w.abs()) + 3 * ref.U * w.abs()
                 + 6 * ref.U * hyper["lr"] / (1 - hyper["beta1"] ** step) * size_m / under)
        own = (model.masters or model.w)[j]
        bound = ref.HALF[own.dtype] * want.abs() + 2 * slack + 1e-40
        assert torch.all((ref.f64(own) - want).abs() <= bound), ("w", j, n)
        if model.masters:
            assert torch.equal(model.w[j], model.masters[j].bfloat16()), ("param", j)
        if model.bits == 32:
            assert torch.all((ref.f64(model.m[j]) - m1).abs() <= 6 * ref.U * size_m + 1e-44), j
            assert torch.all((ref.f64(model.v[j]) - v1).abs() <= 8 * ref.U * v1 + 1e-44), j
        else:
            bits = torch.tensor(ref.random_bits(0, n, j, seed), dtype=torch.int64)
            check_codes(model.m[j], model.ms[j], m1, 6 * ref.U * size_m, bits & 0xffff, False,
                        ("m", j))
            r1 = v1.sqrt()
            check_codes(model.v[j], model.vs[j], r1, 8 * ref.U * r1, bits >> 16, True, ("v", j))
    model.check_guards()


KINDS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
         ("bf16", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", KINDS)
def test_types(param, grad, master, bits):
    model = Model(SIZES, param, grad, master, bits, seed=bits)
    step_and_check(model, 3, seed=11)
    step_and_check(model, 4, seed=12)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_empty_states(bits):
    model = Model(SIZES, bits=bits, late=False)
    step_and_check(model, 1, hyper=dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    sizes = [(j * 37) % 300 for j in range(173)]          # some of them empty
    step_and_check(Model(sizes, "bf16", "bf16", True, bits, seed=3), 7, seed=(5 << 32) + 6)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", TYPES)
def test_clipped(grad, bits):
    model = Model(SIZES + [200000], "f32", grad, bits=bits, seed=4)
    want = math.sqrt(sum(float(ref.f64(g).square().sum()) for g in model.g))
    out = torch.empty(2, device="cuda")
    for most in (want / 3, want * 3, math.inf):
        p3d.p3d_grad_norm(model.table, out, most)
        assert math.isclose(float(out[0]), want, rel_tol=2 * ref.U)
        assert math.isclose(float(out[1]), min(1.0, most / want), rel_tol=3 * ref.U)
    p3d.p3d_grad_norm(model.table, out, want / 3)
    step_and_check(model, 5, scale=out[1:], seed=9)


def test_norm_of_nothing_and_of_many():
    out = torch.full((2,), 9.0, device="cuda")
    p3d.p3d_grad_norm(Model([]).table, out, 1.0)
    assert out.tolist() == [0.0, 1.0]
    p3d.p3d_grad_norm(Model([0, 0]).table, out, 1.0)
    assert out.tolist() == [0.0, 1.0]
    model = Model([(j * 37) % 300 for j in range(173)], grad="bf16", seed=5)
    p3d.p3d_grad_norm(model.table, out, 1e-3)
    want = math.sqrt(sum(float(ref.f64(g).square().sum()) for g in model.g))
    assert math.isclose(float(out[0]), want, rel_tol=2 * ref.U)


def test_norms_that_squares_in_32_bits_would_lose():
    for size in (1e-30, 1e30):
        g = torch.full((5000,), size, device="cuda")
        w, m, v = (torch.zeros(5000, device="cuda") for _ in range(3))
        out = torch.empty(2, device="cuda")
        p3d.p3d_grad_norm(p3d.make_adamw_tensors([w], [g], [m], [v]), out, 1.0)
        assert math.isclose(float(out[0]), float(g[0]) * 5000 ** 0.5, rel_tol=1e-6)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_gradient_that_is_not_finite_leaves_the_step_out(value, bits):
    model = Model([300, 5000], bits=bits, seed=6)
    model.g[1][77] = value
    out = torch.empty(2, device="cuda")
    before = [t.clone() for t in model.table]
    p3d.p3d_grad_norm(model.table, out, 1.0)
    assert not math.isfinite(float(out[0])) and math.isnan(float(out[1]))
    p3d.p3d_adamw(model.table, step=2, grad_scale=out[1:], **HYPER)
    for a, b in zip(before, model.table):
        assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))


def test_a_gradient_that_is_not_finite_stays_in_its_element():
    model = Model([3000], bits=32, seed=7)
    model.g[0][77] = math.nan
    p3d.p3d_adamw(model.table, step=2, **HYPER)
    assert model.w[0].isnan().nonzero().flatten().tolist() == [77]
    model = Model([3000], bits=8, seed=7)
    model.g[0][777] = math.inf
    p3d.p3d_adamw(model.table, step=2, **HYPER)
    block = torch.arange(3000) // 256
    assert (~torch.isfinite(model.w[0])).nonzero().flatten().tolist() == [777]
    for codes, scales in ((model.m, model.ms), (model.v, model.vs)):
        value = codes[0].float() * scales[0].repeat_interleave(256)[:3000]
        assert torch.equal(~torch.isfinite(value).cpu(), block == 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_rate_on_the_device(bits):
    a, b = Model(SIZES, "bf16", "f32", True, bits, 8), Model(SIZES, "bf16", "f32", True, bits, 8)
    for step, lr in ((1, 1e-2), (2, 5e-3), (1000, 1e-4)):
        hyper = dict(lr=float(torch.tensor(lr)), beta1=0.9, beta2=0.999, eps=1e-8)
        p3d.p3d_adamw(a.table, step=step, seed=step, **hyper)
        # (the device's step is added to the seed)
        p3d.p3d_adamw(b.table, step=77, seed=0, **{**hyper, "lr": 3.0},
                      device_lr=torch.tensor([lr], device="cuda"),
                      device_step=torch.tensor([step], dtype=torch.int32, device="cuda"))
        for x, y in zip(a.table, b.table):
            # (factors in binary64 rounded once: equal but for a last place)
            assert torch.allclose(x.float(), y.float(), rtol=1e-6, atol=1e-12)
    c, d = Model([100], bits=bits), Model([100], bits=bits)
    p3d.p3d_adamw(c.table, step=1, **HYPER)
    p3d.p3d_adamw(d.table, step=5, **HYPER,
                  device_step=torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert torch.allclose(c.w[0], d.w[0], rtol=1e-6)


def test_a_table_keeps_the_memory_it_was_made_of():
    p = torch.nn.Parameter(torch.ones(5000, device="cuda"))
    g, m, v = (torch.ones(5000, device="cuda") for _ in range(3))
    table, old = p3d.make_adamw_tensors([p], [g], [m], [v]), p.data_ptr()
    p.data = torch.ones(5000, device="cuda")
    others = [torch.zeros(5000, device="cuda") for _ in range(8)]   # none of them the old one
    p3d.p3d_adamw(table, step=1, **HYPER)
    assert table[0].data_ptr() == old and bool((table[0] < 1).all())
    assert bool((p == 1).all()) and all(bool((x == 0).all()) for x in others)


def test_replays_of_a_captured_step_round_by_bits_of_their_own():
    """8-bit states in a graph: every replay is the call with the step's number
    added to the seed, over 2^32 as well."""
    a, b = Model(SIZES, "bf16", "f32", True, 8, 8), Model(SIZES, "bf16", "f32", True, 8, 8)
    seed, step = 2 ** 32 - 3, torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step += 1
        p3d.p3d_adamw(b.table, step=1, seed=seed, device_step=step, **HYPER)
    for t in (1, 2, 3, 4):
        graph.replay()
        p3d.p3d_adamw(a.table, step=t, seed=seed + t, **HYPER)
        torch.cuda.synchronize()
        assert int(step) == t
        for x, y in zip(a.m + a.v, b.m + b.v):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_eight_bit_states_keep_their_mean():
    """A second moment whose changes are far smaller than half a step of its
    numbers still follows: it falls from 1 to 1/4 by 0.4 % a step at most, where
    a number's neighbours are 6 to 12 % away."""
    n, steps, beta2 = 4096, 400, 0.99
    w, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
    m = torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda")
    r = torch.ones(n, device="cuda")
    g[::256] = r[::256] = 4.0                             # (the largest stays where it is)
    v = (r * 112).to(torch.float8_e4m3fn)
    ms, vs = torch.zeros(16, device="cuda"), torch.full((16,), 1 / 112.0, device="cuda")
    table = p3d.make_adamw_tensors([w], [g], [m], [v], m_scales=[ms], v_scales=[vs])
    for t in range(1, steps + 1):
        p3d.p3d_adamw(table, 0.0, 0.9, beta2, 1e-8, 1000 + t, seed=t)
    r = (v.float() * vs.repeat_interleave(256)).view(16, 256)
    assert torch.allclose(r[:, 0], torch.full((16,), 4.0, device="cuda"), rtol=1e-2)
    want = math.sqrt(0.25 + 0.75 * beta2 ** steps)
    rest = r[:, 1:] / want
    # A step that drifts by d between numbers s apart rounds with variance below
    # s d; s <= r / 8 and the drifts add up to log(1 / want) = 0.67, so the
    # variance stays below 0.084. v = r^2 gains as much: its mean is 8 % high at
    # most, r's 4, and a mean over 4080 is within 0.29 / 64 x 4 of that.
    assert -0.02 < float(rest.mean()) - 1 < 0.06 and float(rest.std()) < 0.3


def test_no_learning_rate_keeps_the_weights():
    model = Model([500], bits=32, seed=9)
    before = model.w[0].clone()
    p3d.p3d_adamw(model.table, 0.0, step=3)
    assert torch.equal(before, model.w[0])


def test_the_same_call_gives_the_same_bytes():
    runs = []
    for _ in range(2):
        model = Model(SIZES, "bf16", "bf16", False, 8, 10)
        out = torch.empty(2, device="cuda")
        p3d.p3d_grad_norm(model.table, out, 1e-2)
        p3d.p3d_adamw(model.table, step=3, seed=3, grad_scale=out[1:], **HYPER)
        runs.append([t.clone() for t in model.table] + [out])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*runs))


def test_a_tensor_whose_elements_pass_32_bits():
    """The random bits take the index's upper half, addresses pass 32 bits."""
    n = (1 << 32) + 700
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    tail = torch.randn(700, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    g[-700:] = tail
    table = p3d.make_adamw_tensors([w], [g], [m], [v], m_scales=[ms], v_scales=[vs])
    out = torch.empty(2, device="cuda")
    p3d.p3d_grad_norm(table, out)
    assert math.isclose(float(out[0]), float(ref.f64(tail).square().sum()) ** 0.5, rel_tol=1e-6)
    p3d.p3d_adamw(table, 1e-2, 0.9, 0.99, 1e-8, 1, seed=21)
    bits = torch.tensor(ref.random_bits(1 << 32, 700, 0, 21))
    want, m1, v1 = ref.adamw(torch.zeros(700).double(), ref.f64(tail), 0.0, 0.0, 1e-2, 0.9, 0.99,
                             1e-8, 1, 0.0)
    assert torch.all((ref.f64(w[-700:]) - want).abs() <= ref.HALF[torch.bfloat16] * want.abs()
                     + 1e-6 * want.abs())
    at = (1 << 32) // 256
    check_codes(m[-700:], ms[at:], m1, 6 * ref.U * m1.abs(), bits & 0xffff, False, "m")
    check_codes(v[-700:], vs[at:], v1.sqrt(), 8 * ref.U * v1.sqrt(), bits >> 16, True, "v")
    assert not w[:1 << 20].any() and not vs[:at].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1754942e-38, 1.1754944e-38, 1e-30])
def test_every_eps_that_binary32_holds(eps, bits):
    """An element without a gradient and without states keeps its weight (0 / eps
    is 0), however small eps is."""
    model = Model(SIZES, bits=bits, late=False, seed=11)
    assert any(bool((g == 0).any()) for g in model.g)
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=eps)
    step_and_check(model, 1, hyper=hyper)
    # a block, and a tensor, of which nothing has a gradient
    model = Model([700, 300], bits=bits, late=False, seed=12)
    model.g[0][256:512] = 0
    model.g[1].zero_()
    step_and_check(model, 1, hyper=hyper)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e30, 1e38])
def test_an_eps_beyond_the_reciprocals(eps, bits):
    """m / eps where 1 / eps is no normal number of binary32: m = 1e36 moves a
    weight of 0 by lr m / eps (of 0.9 m, as the gradient is 0)."""
    n = 600
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    if bits == 32:
        m, v = torch.full((n,), 1e36, device="cuda"), torch.zeros(n, device="cuda")
        table = p3d.make_adamw_tensors([w], [g], [m], [v])
    else:
        m, v = (torch.full((n,), x, device="cuda").to(torch.float8_e4m3fn) for x in (256.0, 0.0))
        ms, vs = torch.full((3,), 1e36 / 256, device="cuda"), torch.zeros(3, device="cuda")
        table = p3d.make_adamw_tensors([w], [g], [m], [v], m_scales=[ms], v_scales=[vs])
    p3d.p3d_adamw(table, 1.0, 0.9, 0.99, eps, 1000000)
    want = -0.9 * 1e36 / eps
    assert torch.all((w.double() - want).abs() <= 16 * ref.U * abs(want))


@pytest.mark.parametrize("most", [1.0, math.inf])
def test_a_norm_beyond_binary32_leaves_the_step_out(most):
    """Gradients that are finite, their norm 2^128 and more: the two results agree
    that it is none, and just below it that it is one."""
    n, out = 4096, torch.empty(2, device="cuda")
    g = torch.full((n,), 2.0 ** 122, device="cuda")              # norm 2^128
    w, m, v = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(
        n, device="cuda")
    table = p3d.make_adamw_tensors([w], [g], [m], [v])
    p3d.p3d_grad_norm(table, out, most)
    assert math.isinf(float(out[0])) and math.isnan(float(out[1]))
    p3d.p3d_adamw(table, grad_scale=out[1:], **HYPER)
    assert (w == 1).all() and not m.any() and not v.any()
    g[0] = 0
    p3d.p3d_grad_norm(table, out, most)
    norm = math.sqrt(4095) * 2.0 ** 122
    assert math.isclose(float(out[0]), norm, rel_tol=2 * ref.U)
    # (1 / norm is below the normal numbers: within half of their step)
    assert abs(float(out[1]) - min(1.0, most / norm)) <= 2.0 ** -150


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-40, 1e38])
def test_any_eps_with_step_and_rate_on_the_device(eps, bits):
    a, b = Model(SIZES, bits=bits, late=False, seed=13), Model(SIZES, bits=bits, late=False, seed=13)
    lr = torch.tensor([1e-3], device="cuda")
    hyper = dict(lr=float(lr), beta1=0.9, beta2=0.999, eps=eps)
    p3d.p3d_adamw(a.table, step=2, seed=2, **hyper)
    p3d.p3d_adamw(b.table, step=9, **{**hyper, "lr": 7.0}, device_lr=lr,
                  device_step=torch.tensor([2], dtype=torch.int32, device="cuda"))
    for x, y in zip(a.table, b.table):
        assert torch.isfinite(x.float()).all()
        assert torch.allclose(x.float(), y.float(), rtol=1e-6, atol=1e-12)
