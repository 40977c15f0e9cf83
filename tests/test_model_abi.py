"""The entry points of include/p3d_model.h on the CPU: every one is exported,
every argument check answers with its status and names the argument, workspace
sizes hold what the kernels write. No call here reaches a launch."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "p3d_model.h")
INVALID, SHAPE, DTYPE, UNSUPPORTED = 1, 2, 3, 4
FAKE = 0x100000          # never dereferenced: every call below fails validation first
MB = 1 << 20

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="host-only checks (the GPU tests run the calls)")


@pytest.fixture(scope="module")
def p3d():
    import pixel_aligned_image_amd
    return pixel_aligned_image_amd


def refused(p3d, status, want, needle, fn):
    msg = p3d.p3d_last_error()
    assert status == want, (status, msg)
    assert msg.startswith(fn + ":") and needle in msg, msg


def test_every_declared_function_is_exported(p3d):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(p3d_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 8, names
    lib = ctypes.CDLL(p3d.LIB_PATH)
    for name in names:
        assert getattr(lib, name)
        assert name in p3d.__all__


# -------------------------------------------------------------- group norm ---
def group(p3d, off=(0, 10, 16), **kw):
    table = (ctypes.c_int64 * len(off))(*off)
    d = p3d.model.p3d_group_desc(off[-1], ctypes.addressof(table), len(off) - 1, 64, 8, p3d.P3D_BF16,
                                 1, 1e-5, FAKE, FAKE)
    d.keep = table
    for k, v in kw.items():
        setattr(d, k, v)
    return d


GROUP_CHECKS = [
    (dict(dtype=2), DTYPE, "dtype"), (dict(act=3), INVALID, "act"), (dict(n=-1), INVALID, "n must"),
    (dict(n=1 << 30), INVALID, "n must"), (dict(batch=0), INVALID, "batch"),
    (dict(batch=257), INVALID, "batch"), (dict(offsets=None), INVALID, "offsets is NULL"),
    (dict(n=17), SHAPE, "offsets[2]"), (dict(channels=0), INVALID, "channels"),
    (dict(channels=60), UNSUPPORTED, "channels"), (dict(channels=4104), UNSUPPORTED, "channels"),
    (dict(groups=0), SHAPE, "groups"), (dict(groups=7), SHAPE, "groups"),
    (dict(groups=128), SHAPE, "groups"), (dict(eps=0.0), INVALID, "eps"),
    (dict(eps=math.nan), INVALID, "eps"), (dict(eps=math.inf), INVALID, "eps"),
    (dict(weight=FAKE + 8), UNSUPPORTED, "weight"), (dict(bias=FAKE + 2), UNSUPPORTED, "bias")]


@pytest.mark.parametrize("kw,status,needle", GROUP_CHECKS)
def test_group_desc_checks(p3d, kw, status, needle):
    d = group(p3d, **kw)
    X, O, W = FAKE, FAKE + MB, FAKE + 2 * MB
    for fn, args in (("p3d_group_norm", (X, 64, O, 64, None, None, W, MB, None)),
                     ("p3d_group_norm_backward",
                      (X, 64, X, 64, FAKE, FAKE, O, 64, None, None, W, MB, None))):
        refused(p3d, getattr(p3d.lib, fn)(d, *args), status, needle, fn)
    fn = "p3d_group_norm_workspace_size"
    assert p3d.lib.p3d_group_norm_workspace_size(d) == 0
    assert p3d.p3d_last_error().startswith(fn + ":")


def test_group_offsets(p3d):
    for off, needle in (((1, 10, 16), "offsets[0]"), ((0, 20, 16), "must not decrease")):
        assert p3d.lib.p3d_group_norm_workspace_size(group(p3d, off)) == 0
        assert needle in p3d.p3d_last_error()


def test_group_tensor_checks(p3d):
    d = group(p3d, bias=FAKE + 4096)
    X, O, W = FAKE, FAKE + MB, FAKE + 2 * MB

    def forward(want, needle, x=X, xs=64, out=O, os=64, mean=None, rstd=None, ws=W, size=MB):
        refused(p3d, p3d.lib.p3d_group_norm(d, x, xs, out, os, mean, rstd, ws, size, None), want,
                needle, "p3d_group_norm")

    forward(INVALID, "x is NULL", x=None)
    forward(INVALID, "out is NULL", out=None)
    forward(UNSUPPORTED, "x must be", x=X + 8)
    forward(UNSUPPORTED, "out must be", out=O + 4)
    forward(SHAPE, "x_stride", xs=56)
    forward(UNSUPPORTED, "x_stride", xs=68)
    forward(UNSUPPORTED, "out_stride", os=(1 << 30) + 8)
    forward(UNSUPPORTED, "mean", mean=FAKE + 2)
    forward(UNSUPPORTED, "rstd", rstd=FAKE + 1)
    forward(INVALID, "mean must not overlap rstd", mean=FAKE + MB // 2, rstd=FAKE + MB // 2)
    forward(INVALID, "workspace", ws=None)
    forward(INVALID, "workspace", size=16)
    forward(UNSUPPORTED, "256-byte", ws=W + 16)
    forward(SHAPE, "in place", out=X, os=72)
    forward(INVALID, "out must not overlap x", out=X + 64)
    forward(INVALID, "out must not overlap x", out=X + 15 * 128)

    def backward(want, needle, dout=X, ds=64, x=X + MB // 2, xs=64, mean=FAKE, rstd=FAKE, dx=O,
                 dxs=64, dw=None, db=None, ws=W, size=MB):
        refused(p3d, p3d.lib.p3d_group_norm_backward(d, dout, ds, x, xs, mean, rstd, dx, dxs, dw,
                                                     db, ws, size, None), want, needle,
                "p3d_group_norm_backward")

    backward(INVALID, "dout is NULL", dout=None)
    backward(INVALID, "x is NULL", x=None)
    backward(INVALID, "mean is NULL", mean=None)
    backward(INVALID, "rstd is NULL", rstd=None)
    backward(INVALID, "dx is NULL", dx=None)
    backward(SHAPE, "dout_stride", ds=8)
    backward(SHAPE, "x_stride", xs=0)
    backward(UNSUPPORTED, "dx_stride", dxs=70)
    backward(UNSUPPORTED, "dweight", dw=FAKE + 1)
    backward(UNSUPPORTED, "dbias", db=FAKE + 3)
    backward(INVALID, "dweight must not overlap dbias", dw=O + MB // 2, db=O + MB // 2)
    backward(INVALID, "workspace", size=255)
    backward(INVALID, "dx must not overlap dout", dx=X + 128)
    backward(INVALID, "dx must not overlap x", dx=X + MB // 2 + 128)
    backward(SHAPE, "in place", dx=X, dxs=128)
    # results over what other workgroups still read, or over each other
    forward(INVALID, "out must not overlap mean", mean=O + 4)
    forward(INVALID, "out must not overlap weight", out=FAKE - 1024, x=X + 2 * MB)
    forward(INVALID, "mean must not overlap rstd", mean=O + MB // 2, rstd=O + MB // 2 + 32)
    forward(INVALID, "mean must not overlap bias", mean=FAKE + 4104, x=X + 2 * MB)
    forward(INVALID, "rstd must not overlap x", rstd=X + 2 * MB + 200, x=X + 2 * MB, xs=128)
    backward(INVALID, "dx must not overlap mean", mean=O + 15 * 128 + 124)
    backward(INVALID, "dx must not overlap weight", dx=FAKE - 1024, x=X + 3 * MB, dout=X + 2 * MB,
             mean=O, rstd=O)
    backward(INVALID, "dx must not overlap dbias", db=O + 64, mean=O + MB // 2, rstd=O + MB // 2)
    backward(INVALID, "dweight must not overlap dbias", dw=W - 512, db=W - 260)
    backward(INVALID, "dweight must not overlap bias", dw=FAKE + 4096 - 128, x=X + 3 * MB, dout=X + 2 * MB,
             mean=O + MB // 2, rstd=O + MB // 2)
    backward(INVALID, "dweight must not overlap dout", dw=X + 512, mean=O + MB // 2,
             rstd=O + MB // 2, x=X + MB // 2)
    backward(INVALID, "dbias must not overlap x", db=X + MB // 2, mean=O + MB // 2,
             rstd=O + MB // 2)
    # rows that are differently far apart: between each other's, and not
    forward(INVALID, "out must not overlap x", x=O, xs=128, out=O + 3 * 64, os=256)
    forward(INVALID, "workspace", x=O, xs=256, out=O + 128, os=512, size=16)
    # every item has a mean and an rstd, also one without rows
    d = group(p3d, (0, 0, 0))
    backward(INVALID, "mean is NULL", dout=None, x=None, dx=None, mean=None)
    backward(INVALID, "rstd is NULL", dout=None, x=None, dx=None, rstd=None)


def test_group_workspace_holds_the_partial_sums(p3d):
    """Both directions' partials of the chunks the header's rule makes: at most
    4 workgroups a CU and one more an item, 8 bytes a group or a channel."""
    for n, items, c, groups in ((1, 1, 8, 1), (100000, 1, 1024, 32), (100000, 256, 64, 64),
                                (262144, 3, 4096, 4096)):
        off = [n * i // items for i in range(items + 1)]
        size = p3d.lib.p3d_group_norm_workspace_size(
            group(p3d, off, channels=c, groups=groups))
        assert size % 256 == 0
        chunks = min(n, 1)
        assert size >= (chunks + items) * 2 * c * 4
        assert size <= (1024 + 2 * items) * 2 * c * 4 + 16 * items * groups + 1024


# ------------------------------------------------------------------ linear ---
def test_quantize_checks(p3d):
    X, Q, S = FAKE, FAKE + MB, FAKE + 2 * MB

    def call(want, needle, x=X, dt=1, n=16, k=64, xs=64, q=Q, qs=64, s=S):
        refused(p3d, p3d.lib.p3d_quantize_rows(x, dt, n, k, xs, q, qs, s, None), want, needle,
                "p3d_quantize_rows")

    call(DTYPE, "dtype", dt=5)
    call(INVALID, "n must", n=-1)
    call(INVALID, "n must", n=1 << 30)
    call(INVALID, "width", k=0)
    call(UNSUPPORTED, "width", k=24)
    call(UNSUPPORTED, "width", k=65552)
    call(INVALID, "x is NULL", x=None)
    call(INVALID, "q is NULL", q=None)
    call(INVALID, "scale is NULL", s=None)
    call(UNSUPPORTED, "x must be", x=X + 8)
    call(UNSUPPORTED, "q must be", q=Q + 8)
    call(UNSUPPORTED, "scale must be", s=S + 2)
    call(SHAPE, "x_stride", xs=48)
    call(UNSUPPORTED, "x_stride", xs=68)
    call(SHAPE, "q_stride", qs=48)
    call(UNSUPPORTED, "q_stride", qs=72)
    call(INVALID, "q must not overlap x", q=X)
    call(INVALID, "q must not overlap x", q=X + 16, n=1)
    call(INVALID, "scale must not overlap x", s=X)
    call(INVALID, "scale must not overlap x", s=X + 2044)
    call(INVALID, "scale must not overlap x", s=X - 4)
    call(INVALID, "q must not overlap scale", s=Q + 1020)
    call(INVALID, "q must not overlap x", q=X + 16 * 128 - 16)
    call(INVALID, "q must not overlap x", q=X + 128 + 64, xs=128, qs=192)
    call(INVALID, "q must not overlap scale", s=Q)
    assert p3d.lib.p3d_quantize_rows(None, 1, 0, 64, 64, None, 64, None, None) == 0


def test_linear_checks(p3d):
    Q, S, R, O, W, T, B = (FAKE + i * MB for i in range(7))

    def call(want, needle, q=Q, qs=64, s=S, r=None, rs=0, out=O, os=128, **kw):
        d = p3d.model.p3d_linear_i8_desc(16, 64, 128, p3d.P3D_BF16, 0, W, T, B)
        for k, v in kw.items():
            setattr(d, k, v)
        refused(p3d, p3d.lib.p3d_linear_i8(d, q, qs, s, r, rs, out, os, None), want, needle,
                "p3d_linear_i8")

    refused(p3d, p3d.lib.p3d_linear_i8(None, Q, 64, S, None, 0, O, 128, None), INVALID, "desc",
            "p3d_linear_i8")
    call(DTYPE, "dtype", dtype=7)
    call(INVALID, "act", act=-1)
    call(INVALID, "n must", n=-3)
    call(INVALID, "in_dim", in_dim=-16)
    call(UNSUPPORTED, "in_dim", in_dim=40)
    call(UNSUPPORTED, "in_dim", in_dim=1 << 17)
    call(INVALID, "out_dim", out_dim=0)
    call(UNSUPPORTED, "out_dim", out_dim=12)
    call(UNSUPPORTED, "below 2^36", n=1 << 20, out_dim=1 << 16, os=1 << 16)
    call(INVALID, "weight is NULL", weight=None)
    call(INVALID, "weight_scale is NULL", weight_scale=None)
    call(INVALID, "q is NULL", q=None)
    call(INVALID, "scale is NULL", s=None)
    call(INVALID, "out is NULL", out=None)
    for k, v in (("weight", W + 8), ("weight_scale", T + 2), ("bias", B + 8)):
        call(UNSUPPORTED, k, **{k: v})
    call(UNSUPPORTED, "q must be", q=Q + 4)
    call(UNSUPPORTED, "residual must be", r=R + 8, rs=128)
    call(UNSUPPORTED, "out must be", out=O + 8)
    call(SHAPE, "q_stride", qs=48)
    call(UNSUPPORTED, "q_stride", qs=72)
    call(UNSUPPORTED, "q_stride", qs=(1 << 22) + 16)
    call(SHAPE, "out_stride", os=120)
    call(UNSUPPORTED, "out_stride", os=132)
    call(SHAPE, "residual_stride", r=R, rs=64)
    call(UNSUPPORTED, "residual_stride", r=R, rs=129)
    call(INVALID, "out must not overlap q", out=Q)
    call(INVALID, "out must not overlap weight", out=W)
    call(INVALID, "out must not overlap scale", out=S)
    call(INVALID, "out must not overlap weight_scale", out=T)
    call(INVALID, "out must not overlap bias", out=B)
    call(SHAPE, "in place", r=O, rs=256)
    call(INVALID, "out must not overlap residual", r=O + 256, rs=128)


def test_linear_sizes(p3d):
    """Both sides of the limit on tokens times features, each in 64s: the next
    check refuses what this one takes."""
    def call(n, out_dim, needle):
        d = p3d.model.p3d_linear_i8_desc(n, 64, out_dim, p3d.P3D_BF16, 0, None, None, None)
        refused(p3d, p3d.lib.p3d_linear_i8(d, None, 64, None, None, 0, None, out_dim, None),
                INVALID if "NULL" in needle else UNSUPPORTED, needle, "p3d_linear_i8")

    big = 1 << 30
    for n, out_dim in ((1, big - 64), (64, big - 64), (65, big // 2 - 64), (big - 64, 8),
                       (1 << 20, (1 << 16) - 64)):
        call(n, out_dim, "weight is NULL")
    for n, out_dim in ((1, big - 56), (1, big - 8), (65, big // 2 - 56), (big - 63, 8),
                       (big - 1, 64), ((1 << 20) - 63, 1 << 16)):
        call(n, out_dim, "each rounded up to a multiple of 64, must be below 2^36")


# ------------------------------------------------------------------- adamw ---
def table(p3d, count=3, bits=32, master=False, **kw):
    """count tensors of 1000 elements, a megabyte apart."""
    rows = (p3d.model.p3d_adamw_tensor * max(1, count))()
    for j in range(count):
        at = FAKE + j * 8 * MB
        rows[j].param, rows[j].grad = at, at + MB
        rows[j].m, rows[j].v = at + 2 * MB, at + 3 * MB
        rows[j].master = at + 4 * MB if master else None
        if bits == 8:
            rows[j].m_scale, rows[j].v_scale = at + 5 * MB, at + 6 * MB
        rows[j].size = 1000
    d = p3d.model.p3d_adamw_desc(count, ctypes.addressof(rows), 1, 1, bits, 1e-3, 0.9, 0.99, 1e-8,
                                 1, 0, None, None, None)
    d.keep = rows
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status,needle", [
    (dict(count=-1), INVALID, "count"), (dict(count=65537), INVALID, "count"),
    (dict(tensors=None), INVALID, "tensors is NULL"), (dict(grad_dtype=3), DTYPE, "grad_dtype"),
    (dict(param_dtype=2), DTYPE, "param_dtype"), (dict(state_bits=16), INVALID, "state_bits"),
    (dict(lr=-1.0), INVALID, "lr"), (dict(lr=math.inf), INVALID, "lr"),
    (dict(beta1=1.0), INVALID, "beta1"), (dict(beta1=math.nan), INVALID, "beta1"),
    (dict(beta2=-0.1), INVALID, "beta2"), (dict(eps=0.0), INVALID, "eps"),
    (dict(eps=1e-60), INVALID, "eps"), (dict(eps=1e300), INVALID, "eps"),
    (dict(step=0), INVALID, "step"),
    (dict(grad_scale=FAKE + 2), UNSUPPORTED, "grad_scale"),
    (dict(device_lr=FAKE + 1), UNSUPPORTED, "device_lr"),
    (dict(device_step=FAKE + 3), UNSUPPORTED, "device_step")])
def test_adamw_desc_checks(p3d, kw, status, needle):
    refused(p3d, p3d.lib.p3d_adamw(table(p3d, **kw), None), status, needle, "p3d_adamw")


def test_adamw_tensor_checks(p3d):
    def call(want, needle, bits=32, master=False, **kw):
        d = table(p3d, bits=bits, master=master)
        for k, v in kw.items():
            setattr(d.keep[1], k, v)
        refused(p3d, p3d.lib.p3d_adamw(d, None), want, "tensors[1]" if want != SHAPE else needle,
                "p3d_adamw")
        assert needle in p3d.p3d_last_error()

    for name in ("param", "grad", "m", "v"):
        call(INVALID, name + " is NULL", **{name: None})
        call(UNSUPPORTED, name + " is not aligned", **{name: FAKE + 9 * MB + 8})
    d = table(p3d, master=True)
    d.keep[1].master = None
    refused(p3d, p3d.lib.p3d_adamw(d, None), INVALID, "tensors[1].master is NULL", "p3d_adamw")
    for name in ("m_scale", "v_scale"):
        call(INVALID, name + " is NULL", bits=8, **{name: None})
        call(UNSUPPORTED, name + " is not aligned", bits=8, **{name: FAKE + 2})
        call(INVALID, "has scales", **{name: FAKE})
    call(INVALID, "size", size=-1)
    call(INVALID, "size", size=1 << 34)
    call(INVALID, "weight_decay", weight_decay=math.nan)
    d = table(p3d, master=True, param_dtype=0)
    refused(p3d, p3d.lib.p3d_adamw(d, None), INVALID, "masters", "p3d_adamw")


def test_adamw_overlaps(p3d):
    """What a step writes is written once, and is no gradient: the same tensor
    twice, a state in the next tensor's weights, a range inside a longer one."""
    def call(needle, change, bits=32):
        d = table(p3d, bits=bits)
        change(d.keep)
        refused(p3d, p3d.lib.p3d_adamw(d, None), INVALID, needle, "p3d_adamw")

    def put(j, name, value):
        return lambda rows: setattr(rows[j], name, value)

    call("must not overlap", put(1, "param", FAKE))
    call("must not overlap", put(2, "m", FAKE + 3 * MB + 992 * 4))
    call("must not overlap", put(0, "v", FAKE + 2 * MB))
    call("must not overlap", put(0, "grad", FAKE))
    call("must not overlap", put(2, "grad", FAKE + 2 * MB + 16))
    call("must not overlap", put(1, "v_scale", FAKE + 8 * MB + 5 * MB + 12), bits=8)

    def inside(rows):
        rows[0].size = 4 * MB                # its param passes over its own gradient
    call("must not overlap", inside)
    # the rate that every workgroup reads, inside what they write
    for name in ("grad_scale", "device_lr", "device_step"):
        d = table(p3d)
        setattr(d, name, FAKE + 16)
        refused(p3d, p3d.lib.p3d_adamw(d, None), INVALID, "overlap", "p3d_adamw")
        assert name in p3d.p3d_last_error() and "tensors[0].param" in p3d.p3d_last_error()
    # gradients may be shared: only the size of the step is refused then
    d = table(p3d, step=0)
    d.keep[1].grad = FAKE + MB
    refused(p3d, p3d.lib.p3d_adamw(d, None), INVALID, "step", "p3d_adamw")


def test_empty_tables_enqueue_nothing(p3d):
    d = table(p3d, count=0, tensors=None)
    assert p3d.lib.p3d_adamw(d, None) == 0
    d = table(p3d, count=2)
    for r in d.keep:
        r.size = 0
        r.param = r.grad = r.m = r.v = None
    assert p3d.lib.p3d_adamw(d, None) == 0


def test_grad_norm_checks(p3d):
    fn = "p3d_grad_norm"

    def call(want, needle, d=None, most=1.0, out=FAKE, ws=FAKE + 256 * MB, size=MB):
        refused(p3d, p3d.lib.p3d_grad_norm(d or table(p3d), most, out, ws, size, None), want,
                needle, fn)

    call(INVALID, "count", table(p3d, count=-2))
    call(DTYPE, "grad_dtype", table(p3d, grad_dtype=9))
    for most in (0.0, -1.0, math.nan):
        call(INVALID, "max_norm", most=most)
    call(INVALID, "out is NULL", out=None)
    call(UNSUPPORTED, "out must be", out=FAKE + 2)
    call(INVALID, "out must not overlap tensors[1].grad", out=table(p3d).keep[1].grad - 4)
    call(INVALID, "workspace", ws=None)
    call(INVALID, "workspace", size=8)
    call(UNSUPPORTED, "256-byte", ws=FAKE + 16)
    d = table(p3d)
    d.keep[2].grad = None
    call(INVALID, "tensors[2].grad", d)
    d = table(p3d)
    d.keep[0].size = 1 << 33
    size = p3d.lib.p3d_grad_norm_workspace_size(d)
    assert size >= 1536 * 8 and size % 256 == 0          # a part for each of 1536 workgroups
    assert p3d.lib.p3d_grad_norm_workspace_size(table(p3d, grad_dtype=4)) == 0
    assert "grad_dtype" in p3d.p3d_last_error()


# ----------------------------------------------------------------- binding ---
def test_binding_checks(p3d):
    """The binding refuses CPU tensors, wrong types and shapes by name."""
    x, q = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        p3d.p3d_group_norm(x, x, 8)
    with pytest.raises(ValueError, match=r"x must be \[n, channels\]"):
        p3d.p3d_group_norm(x[None], x, 8)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        p3d.p3d_group_norm(x.half(), x, 8)
    with pytest.raises(ValueError, match="act must be one of none, silu, gelu"):
        p3d.p3d_group_norm(x, x, 8, act="relu")
    with pytest.raises(ValueError, match="weight must be on the GPU"):
        p3d.p3d_group_norm(x, x, 8, weight=x[0])
    with pytest.raises(ValueError, match="x must be on the GPU"):
        p3d.p3d_group_norm_backward(x, x, s, s, x, 8)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        p3d.p3d_quantize_rows(x, q, s)
    with pytest.raises(ValueError, match="q must be on the GPU"):
        p3d.p3d_linear_i8(q, s, q, s, x)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        p3d.p3d_quantize_rows(_Shaped(), q, s)
    with pytest.raises(TypeError, match="table of make_adamw_tensors"):
        p3d.p3d_adamw([x], 1e-3)
    with pytest.raises(ValueError, match="grads must have one entry for each of 1 params"):
        p3d.make_adamw_tensors([s], [], [s], [s])
    with pytest.raises(ValueError, match="m_scales and v_scales go together"):
        p3d.make_adamw_tensors([s], [s], [s], [s], m_scales=[s])
    with pytest.raises(TypeError, match="params must be float32 or bfloat16"):
        p3d.make_adamw_tensors([s.half()], [s], [s], [s])
    with pytest.raises(ValueError, match=r"params\[0\] must be on the GPU"):
        p3d.make_adamw_tensors([s], [s], [s], [s])


class _Shaped:
    dtype = torch.bfloat16


def test_group_workspace_size_through_the_binding(p3d):
    x = torch.zeros(100, 64)
    assert p3d.p3d_group_norm_workspace_size(x, 8) == p3d.p3d_group_norm_workspace_size(
        x, 8, [0, 100])
    with pytest.raises(p3d.P3DError, match="groups"):
        p3d.p3d_group_norm_workspace_size(x, 7)


class _On(torch.Tensor):
    """A tensor that says of itself that it is on a GPU."""
    at = 0
    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


def test_a_workspace_on_another_device_is_refused(p3d, monkeypatch):
    def on(t, at):
        t = t.as_subclass(_On)
        t.at = at
        return t

    def reached(*a):
        raise AssertionError("the library is not called")

    monkeypatch.setattr(p3d.model, "_device", lambda: 0)
    x, s = (on(torch.zeros(shape), 0) for shape in ((4, 64), (1, 8)))
    v = on(torch.zeros(100), 0)
    table = p3d.make_adamw_tensors([v], [v], [v], [v])
    for name in ("p3d_group_norm", "p3d_group_norm_backward", "p3d_grad_norm"):
        monkeypatch.setattr(p3d.model.lib, name, reached)
    for workspace, error, words in (
            (on(torch.zeros(1 << 20, dtype=torch.uint8), 1), ValueError, "current device"),
            (torch.zeros(1 << 20, dtype=torch.uint8), ValueError, "on the GPU"),
            (bytearray(1 << 20), TypeError, "a torch.Tensor")):
        for call in (lambda: p3d.p3d_group_norm(x, x, 8, workspace=workspace),
                     lambda: p3d.p3d_group_norm_backward(x, x, s, s, x, 8, workspace=workspace),
                     lambda: p3d.p3d_grad_norm(table, s, workspace=workspace)):
            with pytest.raises(error, match="workspace must be.*" + words):
                call()
