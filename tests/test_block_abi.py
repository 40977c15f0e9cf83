"""The entry points of include/p3d_block.h on the CPU: every one is exported,
every argument check answers with its status and names the argument, workspace
sizes and frequency tables are right. No call here reaches a launch."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "p3d_block.h")
INVALID, SHAPE, DTYPE, UNSUPPORTED = 1, 2, 3, 4
FAKE = 0x100000          # never dereferenced: every call below fails validation first

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="host-only checks (the GPU tests run the calls)")


@pytest.fixture(scope="module")
def p3d():
    import pixel_aligned_image_amd
    return pixel_aligned_image_amd


def offsets(*v):
    return (ctypes.c_int64 * len(v))(*v)


def norm_desc(p3d, off=None, **kw):
    off = offsets(0, 10, 16) if off is None else off
    d = p3d.block.p3d_norm_desc(16, ctypes.addressof(off), len(off) - 1, 64, p3d.P3D_BF16, 1, 0,
                                1.0, 1e-6, 64)
    d.keep = off
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def rotary_desc(p3d, **kw):
    d = p3d.block.p3d_rotary_desc(16, 4, 64, p3d.P3D_BF16, 0, 3, 10, 4, 1.0, 1e-6, FAKE, FAKE,
                                  FAKE)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def attn_desc(p3d, q=None, k=None, **kw):
    q = offsets(0, 10, 16) if q is None else q
    k = offsets(0, 5, 20) if k is None else k
    d = p3d.block.p3d_attn_desc(ctypes.addressof(q), ctypes.addressof(k), len(q) - 1, 8, 2, 64,
                                p3d.P3D_BF16, 0.125, 0)
    d.keep = (q, k)
    for a, b in kw.items():
        setattr(d, a, b)
    return d


def refused(p3d, status, want, needle, fn):
    msg = p3d.p3d_last_error()
    assert status == want, (status, msg)
    assert msg.startswith(fn + ":") and needle in msg, msg


def test_every_declared_function_is_exported(p3d):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(p3d_[a-z_]+)\s*\(", text)))
    assert len(names) == 11, names
    lib = ctypes.CDLL(p3d.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(p3d, name)), name
        assert name in p3d.__all__


NORM_CASES = [
    (dict(n=-1), INVALID, "n must be"), (dict(n=17), SHAPE, "offsets[2] must be n = 17"),
    (dict(off=offsets(1, 10, 16)), INVALID, "offsets[0] must be 0"),
    (dict(off=offsets(0, 12, 10)), INVALID, "must not decrease"),
    (dict(batch=0), INVALID, "batch"), (dict(batch=257), INVALID, "batch"),
    (dict(offsets=None), INVALID, "offsets is NULL"),
    (dict(off=offsets(0, 1 << 31), n=1 << 30), UNSUPPORTED, "offsets[1]"),
    (dict(dtype=5), DTYPE, "dtype"), (dict(dim=0), INVALID, "dim"),
    (dict(dim=60), UNSUPPORTED, "multiple of 8"), (dict(dim=8200), UNSUPPORTED, "8192"),
    (dict(dtype=0, dim=62), UNSUPPORTED, "multiple of 4"), (dict(pre=0), INVALID, "pre"),
    (dict(pre=7), INVALID, "pre"), (dict(post=3), INVALID, "post"),
    (dict(eps=0.0), INVALID, "eps"), (dict(eps=math.nan), INVALID, "eps"),
    (dict(res_scale=math.inf), INVALID, "res_scale"),
    (dict(post_weight=FAKE), INVALID, "post_weight"),
    (dict(gate=FAKE, mod_stride=32), SHAPE, "mod_stride"),
    (dict(gate=FAKE, mod_stride=68), UNSUPPORTED, "mod_stride"),
    (dict(gate=FAKE + 8), UNSUPPORTED, "gate must be 16-byte"),
    (dict(scale=FAKE + 8), UNSUPPORTED, "scale must be 16-byte"),
    (dict(weight=FAKE + 2), UNSUPPORTED, "weight must be 16-byte"),
]


@pytest.mark.parametrize("kw,status,needle", NORM_CASES, ids=lambda v: str(v)[:30])
def test_norm_desc_checks(p3d, kw, status, needle):
    d = norm_desc(p3d, **kw)
    st = p3d.lib.p3d_gated_norm(d, FAKE, FAKE, FAKE, FAKE * 2, None)
    refused(p3d, st, status, needle, "p3d_gated_norm")
    assert p3d.lib.p3d_gated_norm_workspace_size(d) == 0
    assert needle in p3d.p3d_last_error()
    st = p3d.lib.p3d_gated_norm_backward(d, FAKE, None, FAKE, FAKE, FAKE, FAKE * 2, *[None] * 6,
                                         FAKE, 1 << 40, None)
    refused(p3d, st, status, needle, "p3d_gated_norm_backward")


def test_norm_tensor_checks(p3d):
    lib, d = p3d.lib, norm_desc(p3d)
    fn = "p3d_gated_norm"
    refused(p3d, lib.p3d_gated_norm(None, FAKE, None, None, FAKE, None), INVALID, "desc", fn)
    refused(p3d, lib.p3d_gated_norm(d, None, None, None, FAKE, None), INVALID, "x is NULL", fn)
    refused(p3d, lib.p3d_gated_norm(d, FAKE, None, None, None, None), INVALID, "h is NULL", fn)
    refused(p3d, lib.p3d_gated_norm(d, FAKE, FAKE + 4, None, FAKE, None), UNSUPPORTED, "y", fn)
    refused(p3d, lib.p3d_gated_norm(d, FAKE, None, FAKE, FAKE, None), INVALID, "r and h", fn)
    fn += "_backward"
    need = lib.p3d_gated_norm_workspace_size(d)
    assert need >= (2 + 2) * 3 * 64 * 4 and need % 256 == 0

    def back(dh=FAKE, dr=None, x=FAKE, y=FAKE, dx=FAKE, dy=FAKE * 2, grads=(None,) * 6, ws=FAKE,
             size=need):
        return lib.p3d_gated_norm_backward(d, dh, dr, x, y, dx, dy, *grads, ws, size, None)

    refused(p3d, back(dh=None), INVALID, "dh is NULL", fn)
    refused(p3d, back(dx=None), INVALID, "dx is NULL", fn)
    refused(p3d, back(y=None), INVALID, "need y", fn)
    refused(p3d, back(y=None, dy=None, grads=(FAKE,) + (None,) * 5), INVALID, "need y", fn)
    refused(p3d, back(dy=FAKE), INVALID, "dx and dy", fn)
    refused(p3d, back(grads=(None, FAKE + 2, None, None, None, None)), UNSUPPORTED, "dscale", fn)
    refused(p3d, back(ws=None), INVALID, "workspace", fn)
    refused(p3d, back(size=need - 1), INVALID, str(need), fn)
    refused(p3d, back(ws=FAKE + 16), UNSUPPORTED, "256-byte", fn)
    empty = norm_desc(p3d, off=offsets(0, 0, 0), n=0)
    assert lib.p3d_gated_norm(empty, None, None, None, None, None) == 0


ROTARY_CASES = [
    (dict(n=-1), INVALID, "n must be"), (dict(dtype=3), DTYPE, "dtype"),
    (dict(heads=0), INVALID, "heads"), (dict(heads=1025), INVALID, "heads"),
    (dict(head_dim=60), UNSUPPORTED, "head_dim"), (dict(head_dim=264), UNSUPPORTED, "head_dim"),
    (dict(layout=2), INVALID, "layout"), (dict(axes=0), INVALID, "axes"),
    (dict(axes=4, pos_stride=4), INVALID, "axes"), (dict(pairs=0), SHAPE, "pairs"),
    (dict(pairs=11), SHAPE, "3 axes x 11 pairs in a head of 64"),
    (dict(pos_stride=2), SHAPE, "pos_stride"), (dict(magnitude=math.inf), INVALID, "magnitude"),
    (dict(eps=-1.0), INVALID, "eps"), (dict(positions=None), INVALID, "positions is NULL"),
    (dict(positions=FAKE + 2), UNSUPPORTED, "positions"),
    (dict(freqs=None), INVALID, "freqs is NULL"), (dict(gamma=FAKE + 4), UNSUPPORTED, "gamma"),
]


@pytest.mark.parametrize("kw,status,needle", ROTARY_CASES, ids=lambda v: str(v)[:30])
def test_rotary_desc_checks(p3d, kw, status, needle):
    d = rotary_desc(p3d, **kw)
    refused(p3d, p3d.lib.p3d_rotary(d, FAKE, 4096, FAKE, 4096, None), status, needle,
            "p3d_rotary")
    assert p3d.lib.p3d_rotary_workspace_size(d) == 0
    st = p3d.lib.p3d_rotary_backward(d, FAKE, 4096, FAKE, 4096, FAKE, 4096, FAKE, FAKE, 1 << 30,
                                     None)
    refused(p3d, st, status, needle, "p3d_rotary_backward")


def test_rotary_tensor_checks(p3d):
    lib, d = p3d.lib, rotary_desc(p3d)
    fn = "p3d_rotary"
    refused(p3d, lib.p3d_rotary(None, FAKE, 256, FAKE, 256, None), INVALID, "desc", fn)
    refused(p3d, lib.p3d_rotary(d, None, 256, FAKE, 256, None), INVALID, "x is NULL", fn)
    refused(p3d, lib.p3d_rotary(d, FAKE, 248, FAKE, 256, None), SHAPE, "x_stride", fn)
    refused(p3d, lib.p3d_rotary(d, FAKE, 256, FAKE, 260, None), UNSUPPORTED, "out_stride", fn)
    refused(p3d, lib.p3d_rotary(d, FAKE, 256, FAKE, 264, None), SHAPE, "in place", fn)
    fn += "_backward"
    need = lib.p3d_rotary_workspace_size(d)

    def back(d=d, dout=FAKE, x=FAKE, xs=256, dx=FAKE * 2, dxs=256, dg=FAKE, ws=FAKE, size=need):
        return lib.p3d_rotary_backward(d, dout, 256, x, xs, dx, dxs, dg, ws, size, None)

    refused(p3d, back(dout=None), INVALID, "dout is NULL", fn)
    refused(p3d, back(x=None), INVALID, "x is NULL", fn)
    refused(p3d, back(xs=128), SHAPE, "x_stride", fn)
    refused(p3d, back(dx=FAKE, dxs=512), SHAPE, "in place", fn)
    refused(p3d, back(dg=FAKE + 2), UNSUPPORTED, "dgamma", fn)
    refused(p3d, back(ws=None), INVALID, "workspace", fn)
    refused(p3d, back(size=need - 1), INVALID, str(need), fn)
    refused(p3d, back(d=rotary_desc(p3d, gamma=None)), INVALID, "without gamma", fn)
    empty = rotary_desc(p3d, n=0, positions=None, freqs=None)
    assert lib.p3d_rotary(empty, None, 256, None, 256, None) == 0


def test_frequencies(p3d):
    base, pairs = 10000.0, 24
    plain = [base ** (-i / pairs) for i in range(pairs)]

    def table(*a):
        return p3d.p3d_rotary_frequencies(base, pairs, *a).double().tolist()

    def near(a, b):
        return all(abs(x - y) <= 2.0 ** -24 * abs(y) for x, y in zip(a, b))

    assert near(table(), plain)
    assert near(table("linear", 4.0), [f / 4 for f in plain])
    scaled = table("base", 8.0)
    assert scaled[0] == 1.0 and abs(scaled[-1] / (plain[-1] / 8) - 1) < 1e-6
    assert all(b <= a * (1 + 1e-7) for a, b in zip(plain, scaled))
    parts = table("by_parts", 8.0, 4096.0)
    for f, got in zip(plain, parts):
        w = 4096 * f / (2 * math.pi)
        k = min(max((w - 1) / 31, 0.0), 1.0)
        assert abs(got / (f * k + f / 8 * (1 - k)) - 1) < 1e-6
    assert parts[0] == 1.0 and abs(parts[-1] / (plain[-1] / 8) - 1) < 1e-6
    lib, buf = p3d.lib, (ctypes.c_float * 128)()
    for args, needle in [((1.0, 8, 0, 1.0, 0.0), "base"), ((math.inf, 8, 0, 1.0, 0.0), "base"),
                         ((1e4, 0, 0, 1.0, 0.0), "pairs"), ((1e4, 129, 0, 1.0, 0.0), "pairs"),
                         ((1e4, 8, 4, 1.0, 0.0), "scaling"), ((1e4, 8, 1, 0.5, 0.0), "factor"),
                         ((1e4, 1, 2, 2.0, 0.0), "2 pairs"), ((1e4, 8, 3, 2.0, 0.0), "trained")]:
        refused(p3d, lib.p3d_rotary_frequencies(*args, ctypes.addressof(buf)), INVALID, needle,
                "p3d_rotary_frequencies")
    refused(p3d, lib.p3d_rotary_frequencies(1e4, 8, 0, 1.0, 0.0, None), INVALID, "freqs",
            "p3d_rotary_frequencies")


ATTN_CASES = [
    (dict(dtype=9), DTYPE, "dtype"), (dict(dtype=0), UNSUPPORTED, "BF16"),
    (dict(kv_heads=0), INVALID, "kv_heads"), (dict(heads=1), INVALID, "kv_heads"),
    (dict(heads=1026), INVALID, "1024"), (dict(kv_heads=3), SHAPE, "multiple of kv_heads"),
    (dict(head_dim=60), UNSUPPORTED, "head_dim"), (dict(head_dim=136), UNSUPPORTED, "head_dim"),
    (dict(scale=0.0), INVALID, "scale"), (dict(scale=math.nan), INVALID, "scale"),
    (dict(causal=2), INVALID, "causal"), (dict(batch=0), INVALID, "batch"),
    (dict(q=offsets(0, 9, 8)), INVALID, "q_offsets must not decrease"),
    (dict(k=offsets(2, 9, 20)), INVALID, "k_offsets[0]"),
    (dict(q_offsets=None), INVALID, "q_offsets is NULL"),
    (dict(q=offsets(0, 1, 1 << 28)), UNSUPPORTED, "2^30"),
    (dict(k=offsets(0, 1, 1 << 29)), UNSUPPORTED, "2^30"),
]


@pytest.mark.parametrize("kw,status,needle", ATTN_CASES, ids=lambda v: str(v)[:30])
def test_attention_desc_checks(p3d, kw, status, needle):
    d = attn_desc(p3d, **kw)
    st = p3d.lib.p3d_attention(d, *[FAKE, 1 << 20] * 4, None, FAKE, 1 << 40, None)
    refused(p3d, st, status, needle, "p3d_attention")
    assert p3d.lib.p3d_attention_workspace_size(d) == 0
    assert p3d.lib.p3d_attention_backward_workspace_size(d) == 0
    st = p3d.lib.p3d_attention_backward(d, *[FAKE, 1 << 20] * 5, FAKE, *[FAKE, 1 << 20] * 3, FAKE,
                                        1 << 40, None)
    refused(p3d, st, status, needle, "p3d_attention_backward")


def test_attention_tensor_checks(p3d):
    lib, d = p3d.lib, attn_desc(p3d)
    names, widths = ["q", "k", "v", "out"], [512, 128, 128, 512]
    need = lib.p3d_attention_workspace_size(d)
    assert need >= 256 and need % 256 == 0
    fn = "p3d_attention"

    def fwd(ws=FAKE, size=need, **kw):
        args = []
        for n, w in zip(names, widths):
            args += [kw.get(n, FAKE), kw.get(n + "_stride", w)]
        return lib.p3d_attention(d, *args, kw.get("lse"), ws, size, None)

    refused(p3d, lib.p3d_attention(None, *[FAKE, 512] * 4, None, FAKE, need, None), INVALID,
            "desc", fn)
    for n, w in zip(names, widths):
        refused(p3d, fwd(**{n: None}), INVALID, n + " is NULL", fn)
        refused(p3d, fwd(**{n: FAKE + 8}), UNSUPPORTED, n + " must be 16-byte", fn)
        refused(p3d, fwd(**{n + "_stride": w - 8}), SHAPE, n + "_stride", fn)
        refused(p3d, fwd(**{n + "_stride": w + 4}), UNSUPPORTED, n + "_stride", fn)
    refused(p3d, fwd(lse=FAKE + 2), UNSUPPORTED, "lse", fn)
    refused(p3d, fwd(out_stride=1024), SHAPE, "in place", fn)
    refused(p3d, fwd(ws=None), INVALID, "workspace", fn)
    refused(p3d, fwd(size=need - 1), INVALID, str(need), fn)
    refused(p3d, fwd(ws=FAKE + 64), UNSUPPORTED, "256-byte", fn)
    fn += "_backward"
    need_b = lib.p3d_attention_backward_workspace_size(d)
    assert need_b >= 2 * 4 * 16 * 8
    back_names = [("dout", 512), ("q", 512), ("k", 128), ("v", 128), ("out", 512), ("dq", 512),
                  ("dk", 128), ("dv", 128)]

    def back(ws=FAKE, size=need_b, lse=FAKE, **kw):
        args = []
        for n, w in back_names:
            args += [kw.get(n, FAKE), kw.get(n + "_stride", w)]
        return lib.p3d_attention_backward(d, *args[:10], lse, *args[10:], ws, size, None)

    for n, w in back_names:
        refused(p3d, back(**{n: None}), INVALID, n + " is NULL", fn)
        refused(p3d, back(**{n + "_stride": w - 8}), SHAPE, n + "_stride", fn)
    refused(p3d, back(lse=None), INVALID, "lse is NULL", fn)
    refused(p3d, back(size=need_b - 1), INVALID, str(need_b), fn)
    refused(p3d, back(ws=FAKE + 64), UNSUPPORTED, "256-byte", fn)
    empty = attn_desc(p3d, q=offsets(0, 0, 0), k=offsets(0, 0, 0))
    assert lib.p3d_attention(empty, *[None, 512] * 4, None, FAKE, 256, None) == 0


def test_split_workspaces_hold_every_part(p3d):
    """One query over many keys: the parts' binary32 rows fit the size."""
    d = attn_desc(p3d, q=offsets(0, 1), k=offsets(0, 100000))
    one = p3d.lib.p3d_attention_workspace_size(d)
    assert one >= 100 * 8 * (64 + 2) * 4         # 2 key heads: 128 parts wanted
    d = attn_desc(p3d, q=offsets(0, 100000), k=offsets(0, 5))
    assert p3d.lib.p3d_attention_workspace_size(d) == 256
    # 5 keys x 2 heads: the rows are cut for dk and dv
    assert p3d.lib.p3d_attention_backward_workspace_size(d) > 2 * 4 * 100000 * 8 + \
        2 * 100 * 5 * 2 * 64 * 4


def test_binding_checks(p3d):
    """The binding refuses CPU tensors, wrong types and shapes by name."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        p3d.p3d_gated_norm(x, x)
    with pytest.raises(ValueError, match=r"x must be \[n, dim\]"):
        p3d.p3d_gated_norm(x[None], x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        p3d.p3d_gated_norm(x.half(), x)
    with pytest.raises(TypeError, match="gate must be"):
        p3d.p3d_gated_norm(x, x, gate=x[:1])
    h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        p3d.p3d_rotary(h, None, None, h)
    with pytest.raises(ValueError, match="q must be on the GPU"):
        p3d.p3d_attention(h, h, h, h)
    with pytest.raises(ValueError, match="end at the rows"):
        p3d.p3d_attention(h, h, h, h, [0, 3], [0, 4])
    with pytest.raises(ValueError, match="one length"):
        p3d.p3d_attention(h, h, h, h, [0, 4], [0, 2, 4])
    with pytest.raises(KeyError):
        p3d.p3d_gated_norm(x, x, pre="batch")


def test_item_tables_of_other_types(p3d):
    """The library reads int64 entries: an array of another type is converted,
    one that holds no integers refused, an int64 array reused."""
    table = offsets(0, 0, 4)
    assert p3d.make_offsets(table) is table
    for kind in (ctypes.c_int32, ctypes.c_uint32, ctypes.c_int16):
        made = p3d.make_offsets((kind * 3)(0, 0, 4))
        assert made._type_ is ctypes.c_int64 and list(made) == [0, 0, 4]
    with pytest.raises(TypeError):
        p3d.make_offsets((ctypes.c_double * 2)(0.0, 4.0))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    # 12 bytes, of which int64 entries would be read past the end
    assert p3d.p3d_gated_norm_workspace_size(x, (ctypes.c_int32 * 3)(0, 0, 4)) == \
        p3d.p3d_gated_norm_workspace_size(x, [0, 0, 4])


def test_attention_results_do_not_overlap(p3d):
    """Results over an input or over each other: equal tensors, views of one
    packed buffer whose columns or rows meet, a single row inside another
    tensor."""
    lib, d = p3d.lib, attn_desc(p3d)         # 16 queries of 8 heads, 20 keys of 2, heads of 64
    step = 1 << 20
    fn = "p3d_attention_backward"
    need = lib.p3d_attention_backward_workspace_size(d)
    names = ["dout", "q", "k", "v", "out", "dq", "dk", "dv"]
    wide = {"dout": 512, "q": 512, "k": 128, "v": 128, "out": 512, "dq": 512, "dk": 128,
            "dv": 128}
    apart = {n: FAKE + (i + 1) * step for i, n in enumerate(names)}
    lse = FAKE + 20 * step

    def back(d=d, need=need, lse=lse, stride=None, **at):
        args = []
        for n in names:
            args += [at.get(n, apart[n]), stride or wide[n]]
        return lib.p3d_attention_backward(d, *args[:10], lse, *args[10:], FAKE, need, None)

    for n in ("dq", "dk", "dv"):
        for other in names:
            if n != other:
                refused(p3d, back(**{n: apart[other]}), INVALID, "must not overlap", fn)
        refused(p3d, back(**{n: lse}), INVALID, n + " must not overlap lse", fn)
    # one packed buffer of 1600 columns: 2 * 128 of dk from column 512 on
    base = FAKE + 64 * step
    for at in (512 - 8, 512 + 8, 512, 512 - 120, 512 + 120):
        refused(p3d, back(stride=1600, dk=base + 2 * 512, dv=base + 2 * at), INVALID,
                "dk must not overlap dv", fn)
    # a row further down, and one that runs on into the next row's first columns
    refused(p3d, back(stride=1600, dk=base, dv=base + 2 * (1600 * 19 + 64)), INVALID,
            "dk must not overlap dv", fn)
    refused(p3d, back(stride=1600, dk=base, dv=base + 2 * (1600 - 64)), INVALID,
            "dk must not overlap dv", fn)
    refused(p3d, back(stride=1600, dv=base, dk=base + 2 * (1600 - 64)), INVALID,
            "dk must not overlap dv", fn)
    # one query's row of 512 over the keys' rows of 128: inside, from before, at the end
    one = attn_desc(p3d, q=offsets(0, 1, 1))
    need_one = lib.p3d_attention_backward_workspace_size(one)
    for at in (128 * 3, -504, 128 * 20 - 8):
        refused(p3d, back(d=one, need=need_one, dq=apart["dk"] + 2 * at), INVALID,
                "dq must not overlap dk", fn)
        refused(p3d, back(d=one, need=need_one, dk=apart["q"] - 2 * at), INVALID,
                "dk must not overlap q", fn)

    fn = "p3d_attention"
    need_f = lib.p3d_attention_workspace_size(d)

    def fwd(q=apart["q"], k=apart["k"], v=apart["v"], out=apart["out"], stride=None):
        args = []
        for n, p in (("q", q), ("k", k), ("v", v), ("out", out)):
            args += [p, stride or wide[n]]
        return lib.p3d_attention(d, *args, None, FAKE, need_f, None)

    refused(p3d, fwd(out=apart["k"]), INVALID, "out must not overlap k", fn)
    refused(p3d, fwd(out=apart["v"]), INVALID, "out must not overlap v", fn)
    refused(p3d, fwd(stride=1600, q=base, out=base + 2 * 8), INVALID, "out must not overlap q", fn)
    refused(p3d, fwd(stride=1600, q=base, out=base + 2 * 1600), INVALID, "out must not overlap q",
            fn)


def test_attention_scales_at_the_ends_of_binary32(p3d):
    """scale log2(e) and, in the gradient, lse / scale have to be finite: past
    that the answers were NaN for scores of 0, and gradients of 0."""
    lib = p3d.lib
    f32 = ctypes.c_float
    assert math.isinf(f32(2.0 ** 127 * 1.5 * math.log2(math.e)).value)
    assert math.isinf(f32(math.log(20) / 2.0 ** -127).value)
    d = attn_desc(p3d, scale=2.0 ** 127 * 1.5)
    args = [FAKE, 1 << 20] * 4, [FAKE, 1 << 20] * 5, [FAKE, 1 << 20] * 3
    refused(p3d, lib.p3d_attention(d, *args[0], None, FAKE, 1 << 40, None), UNSUPPORTED, "2^127",
            "p3d_attention")
    assert lib.p3d_attention_workspace_size(d) == 0
    d = attn_desc(p3d, scale=2.0 ** -101)
    assert lib.p3d_attention_workspace_size(d) > 0
    assert lib.p3d_attention_backward_workspace_size(d) == 0
    refused(p3d, lib.p3d_attention_backward(d, *args[1], FAKE, *args[2], FAKE, 1 << 40, None),
            UNSUPPORTED, "2^-100", "p3d_attention_backward")
    for scale in (2.0 ** 127, 2.0 ** -100):
        assert lib.p3d_attention_backward_workspace_size(attn_desc(p3d, scale=scale)) > 0
