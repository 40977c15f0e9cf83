"""The model's operators together, as a program uses them: a map is normalised,
gathered by the conditioning path and projected in 8-bit integers; its
gradients are taken, clipped and stepped on, and the new weights quantised
again. Against the same steps in 64 bits, on other streams, and captured."""
import ctypes

import pytest
import torch

import model_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu
ITEMS, SIDE, C, D, TOKENS, GROUPS = 2, 24, 64, 96, 700, 8
OFFSETS = [0, SIDE * SIDE, 2 * SIDE * SIDE]


class Model:
    """A normalised map, sampled at sparse tokens, through one linear layer."""

    def __init__(self, seed=0, bits=8):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, by=1.0, base=0.0, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g) * by + base).to(dtype).cuda()

        self.x = rand(ITEMS * SIDE * SIDE, C, by=2.0, base=0.3)
        self.dy = rand(ITEMS * SIDE * SIDE, C)
        self.dw = rand(D, C, by=0.01)
        self.w, self.b = rand(C, by=0.2, base=1.0), rand(C, by=0.2)
        self.matrix = rand(D, C, by=C ** -0.5)
        self.bias = rand(D, by=0.1)
        self.coords = torch.cat([
            torch.randint(0, ITEMS, (TOKENS, 1), generator=g),
            torch.randint(0, 64, (TOKENS, 3), generator=g)], 1).int().contiguous().cuda()
        self.cams = [p3d.p3d_make_camera(40.0, p3d.p3d_distance_from_fov(40.0, SIDE, 0))] * ITEMS
        e = torch.empty
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.mean, self.rstd = (e(ITEMS, GROUPS, device="cuda") for _ in range(2))
        self.gw, self.gb = e(C, device="cuda"), e(C, device="cuda")
        self.samples = e(TOKENS, C, dtype=torch.bfloat16, device="cuda")
        self.q = e(TOKENS, C, dtype=torch.int8, device="cuda")
        self.s = e(TOKENS, device="cuda")
        self.mq, self.ms = e(D, C, dtype=torch.int8, device="cuda"), e(D, device="cuda")
        self.out = e(TOKENS, D, dtype=torch.bfloat16, device="cuda")
        self.norm = e(2, device="cuda")
        self.step = torch.zeros(1, dtype=torch.int32, device="cuda")
        params = [self.matrix, self.w.float(), self.b.float()]
        self.fw, self.fb = params[1:]
        self.masters = [p.float().clone() for p in params]
        self.tables = []
        # the matrix: bf16 with a master, 8-bit states; the vectors: binary32
        z = torch.zeros
        n = self.matrix.numel()
        m, v = (z(n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        sm, sv = (z((n + 255) // 256, device="cuda") for _ in range(2))
        self.matrix_state = (m, v, sm, sv)
        self.tables.append(p3d.make_adamw_tensors(
            [self.matrix], [self.dw], [m], [v], masters=[self.masters[0]], m_scales=[sm],
            v_scales=[sv], weight_decay=0.1))
        vm, vv = ([z(C, device="cuda") for _ in range(2)] for _ in range(2))
        self.vector_state = (vm, vv)
        self.tables.append(p3d.make_adamw_tensors([self.fw, self.fb], [self.gw, self.gb], vm, vv))
        size = p3d.p3d_group_norm_workspace_size(self.x, GROUPS, OFFSETS)
        size = max([size] + [p3d.p3d_grad_norm_workspace_size(t) for t in self.tables])
        self.workspace = e(size, dtype=torch.uint8, device="cuda")
        self.offsets = p3d.make_offsets(OFFSETS)

    def run(self, stream=None, workspace=True):
        kw = dict(stream=stream)
        ws = dict(workspace=self.workspace if workspace else None, **kw)
        p3d.p3d_group_norm(self.x, self.y, GROUPS, self.offsets, self.w, self.b, "silu", 1e-5,
                           self.mean, self.rstd, **ws)
        p3d.p3d_proj_sample(self.coords, TOKENS, 64, self.cams,
                            self.y.view(ITEMS, SIDE, SIDE, C), self.samples, **kw)
        p3d.p3d_quantize_rows(self.matrix, self.mq, self.ms, **kw)
        p3d.p3d_quantize_rows(self.samples, self.q, self.s, **kw)
        p3d.p3d_linear_i8(self.q, self.s, self.mq, self.ms, self.out, self.bias, "gelu", **kw)
        p3d.p3d_group_norm_backward(self.dy, self.x, self.mean, self.rstd, self.dx, GROUPS,
                                    self.offsets, self.w, self.b, "silu", self.gw, self.gb, **ws)
        for k, t in enumerate(self.tables):
            p3d.p3d_grad_norm(t, self.norm, 0.5, **ws)
            p3d.p3d_adamw(t, 1e-2, 0.9, 0.95, 1e-8, 1, seed=77 + k, grad_scale=self.norm[1:],
                          device_step=self.step, **kw)

    def results(self):
        return [t.clone() for t in (
            self.y, self.mean, self.rstd, self.samples, self.mq, self.ms, self.q, self.s, self.out,
            self.dx, self.gw, self.gb, self.norm, self.matrix, *self.masters[:1],
            *(t.view(torch.uint8) for t in self.matrix_state[:2]), *self.matrix_state[2:],
            self.fw, self.fb, *self.vector_state[0], *self.vector_state[1])]


def test_against_64_bits():
    a = Model()
    x, w, b = ref.f64(a.x), ref.f64(a.w), ref.f64(a.b)
    matrix, master = ref.f64(a.matrix), ref.f64(a.masters[0])
    fw = ref.f64(a.fw)
    a.step += 1
    a.run()
    torch.cuda.synchronize()
    y, _ = ref.group_norm(x, OFFSETS, GROUPS, w, b, "silu")
    # bf16 results are half a step off at most; the sizes' own test bounds what
    # binary32 adds, far below a thousandth of that
    assert torch.all((ref.f64(a.y) - y).abs() <= 2.0 ** -8 * y.abs() * 1.01 + 2e-5)
    # from here on with the tensors as the calls before left them
    q, s = ref.quantize(ref.f64(a.samples))
    mq, ms = ref.quantize(matrix)
    assert torch.equal(ref.f64(a.q), q) and torch.equal(ref.f64(a.mq), mq)
    assert torch.equal(ref.f64(a.s), s) and torch.equal(ref.f64(a.ms), ms)
    out, size = ref.linear(q, s, mq, ms, ref.f64(a.bias), "gelu")
    assert torch.all((ref.f64(a.out) - out).abs() <= 2.0 ** -8 * out.abs() * 1.01
                     + 40 * ref.U * (1 + size) ** 2)
    # 8 bits stand for the product that bf16 would make: a token's and a weight's
    # entries are off by half of a 127th of their largest, independently, and K
    # products of both add up as squares
    real = ref.f64(a.samples) @ matrix.t() + ref.f64(a.bias)
    plain = (q @ mq.t()) * s[:, None] * ms + ref.f64(a.bias)
    sx, sw = (s[:, None] / 12 ** 0.5), (ms[None] / 12 ** 0.5)
    spread = ((sx * matrix.norm(dim=1)[None]) ** 2 + (sw * ref.f64(a.samples).norm(dim=1)[:, None])
              ** 2 + C * (sx * sw) ** 2).sqrt()
    assert torch.all((plain - real).abs() <= 7 * spread + 1e-12)    # (67,200 values: 7 deviations)
    grads = ref.group_norm_backward(ref.f64(a.dy), x, OFFSETS, GROUPS, w, b, "silu")
    assert torch.all((ref.f64(a.dx) - grads["dx"]).abs() <= 2.0 ** -8 * grads["dx"].abs() * 1.01
                     + 1e-4)
    for got, want in ((a.gw, grads["dweight"]), (a.gb, grads["dbias"])):
        assert torch.allclose(ref.f64(got), want, rtol=1e-5, atol=1e-4 * float(want.abs().max()))
    dw = ref.f64(a.dw)
    by = min(1.0, 0.5 / float(dw.norm()))
    want, m, v = ref.adamw(master.flatten(), dw.flatten(), 0.0, 0.0, 1e-2, 0.9, 0.95, 1e-8, 1, 0.1,
                           by)
    assert torch.allclose(ref.f64(a.masters[0]).flatten(), want, rtol=1e-5, atol=1e-7)
    assert torch.equal(a.matrix, a.masters[0].bfloat16())
    g = torch.cat([ref.f64(a.gw), ref.f64(a.gb)])
    assert abs(float(a.norm[0]) / float(g.norm()) - 1) < 1e-6
    want, _, _ = ref.adamw(fw, ref.f64(a.gw), 0.0, 0.0, 1e-2, 0.9, 0.95, 1e-8, 1, 0.0,
                           min(1.0, 0.5 / float(g.norm())))
    assert torch.allclose(ref.f64(a.fw), want, rtol=1e-5, atol=1e-6)


def test_on_another_stream_and_by_handle():
    a, b, c = Model(1), Model(1), Model(1)
    for m in (a, b, c):
        m.step += 1
    a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side, workspace=False)

    class Handle:
        cuda_stream = side.cuda_stream

    c.run(stream=Handle(), workspace=False)
    torch.cuda.synchronize()
    for x, y, z in zip(a.results(), b.results(), c.results()):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_two_streams_at_once():
    """Two models on two streams, each with a workspace of its own, write what
    they write one after the other."""
    pairs = [(Model(2), Model(3)) for _ in range(2)]
    for a, b in pairs:
        a.step += 1
        b.step += 1
    pairs[0][0].run()
    torch.cuda.synchronize()
    pairs[0][1].run()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    pairs[1][0].run(stream=one)
    pairs[1][1].run(stream=two)
    torch.cuda.synchronize()
    for x, y in zip(pairs[0], pairs[1]):
        for s, t in zip(x.results(), y.results()):
            assert torch.equal(s, t)


def test_captured_in_a_graph():
    """The steps captured once and replayed, the device's step going on between
    the replays, against the same steps run eagerly; a second graph of another
    model with its own workspace between them."""
    a, b, other = Model(4), Model(4), Model(5)
    graphs = []
    for m in (b, other):
        m.run()                              # (warm: nothing is allocated below)
    torch.cuda.synchronize()
    b, other = Model(4), Model(5)
    for m in (b, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.run()
        graphs.append(g)
    for t in range(1, 5):
        a.step += 1
        b.step += 1
        other.step += 1
        a.run()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for k, (x, y) in enumerate(zip(a.results(), b.results())):
            assert torch.equal(x, y), (t, k)


def test_item_table_arrays_are_taken_as_they_are():
    a = Model(6)
    table = (ctypes.c_int64 * 3)(*OFFSETS)
    p3d.p3d_group_norm(a.x, a.y, GROUPS, table, a.w, a.b)
    want = a.y.clone()
    p3d.p3d_group_norm(a.x, a.y, GROUPS, OFFSETS, a.w, a.b)
    assert torch.equal(want, a.y)


def test_binding_refuses_on_the_gpu():
    a = Model(7)
    x, out = a.x, a.y
    with pytest.raises(TypeError, match="out must be torch.bfloat16"):
        p3d.p3d_group_norm(x, out.float(), GROUPS)
    with pytest.raises(ValueError, match="out must be"):
        p3d.p3d_group_norm(x, out[:-1], GROUPS)
    with pytest.raises(ValueError, match="contiguous rows"):
        p3d.p3d_group_norm(x.t().contiguous().t(), out, GROUPS)
    with pytest.raises(ValueError, match="mean must be"):
        p3d.p3d_group_norm(x, out, GROUPS, mean=a.mean)
    with pytest.raises(p3d.P3DError, match="groups must divide"):
        p3d.p3d_group_norm(x, out, 7)
    with pytest.raises(p3d.P3DError, match="must not overlap"):
        p3d.p3d_group_norm(x[1:], x[:-1], GROUPS)
    with pytest.raises(p3d.P3DError, match="workspace"):
        p3d.p3d_group_norm(x, out, GROUPS, workspace=a.workspace[:16])
    with pytest.raises(TypeError, match="weight must be torch.int8"):
        p3d.p3d_linear_i8(a.q, a.s, a.matrix, a.ms, a.out)
    with pytest.raises(ValueError, match="weight must be"):
        p3d.p3d_linear_i8(a.q, a.s, a.mq[:, :32], a.ms, a.out)
    with pytest.raises(p3d.P3DError, match="in_dim"):
        p3d.p3d_linear_i8(a.q[:, :40], a.s, a.mq[:, :40].contiguous(), a.ms, a.out)
    t = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError, match=r"grads\[0\] must be 100 contiguous elements"):
        p3d.make_adamw_tensors([t], [torch.zeros(200, device="cuda")[::2]], [t], [t])
    with pytest.raises(p3d.P3DError, match="must not overlap"):
        p3d.p3d_adamw(p3d.make_adamw_tensors([t], [t.clone()], [t.clone()], [t]), 1e-3)
    with pytest.raises(p3d.P3DError, match="must not overlap"):
        s = [t.clone() for _ in range(4)]
        p3d.p3d_adamw(p3d.make_adamw_tensors([s[0]] * 2, [s[1]] * 2, [s[2]] * 2, [s[3]] * 2), 1e-3)
    with pytest.raises(ValueError, match="grad_scale must be 1 contiguous"):
        p3d.p3d_adamw(a.tables[1], 1e-3, grad_scale=a.norm)
