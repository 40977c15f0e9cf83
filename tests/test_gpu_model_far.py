"""The model's operators on rows so far apart that offsets pass 32 bits: column
ranges of one wide buffer, compared with the same call on tensors of their own."""
import pytest
import torch

import pixel_aligned_image_amd as p3d
from block_ref import uneven

pytestmark = pytest.mark.gpu
N, WIDE = 70000, 65536                  # 4.6e9 elements


def randn(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("items,c,groups", [(1, 64, 8), (7, 72, 9), (200, 64, 8)])
def test_group_norm(items, c, groups):
    wide = torch.empty(N, WIDE, dtype=torch.bfloat16, device="cuda")
    x, dout, out, dx = (wide[:, at:at + c] for at in (0, 128, 20000, WIDE - c))
    x.copy_(randn(N, c, seed=1))
    dout.copy_(randn(N, c, seed=2))
    w, b, off = randn(c, seed=3), randn(c, seed=4), uneven(N, items)
    got = []
    for t in ((x, dout, out, dx), tuple(t.clone() for t in (x, dout, x, x))):
        mean, rstd = (torch.empty(items, groups, device="cuda") for _ in range(2))
        dw, db = (torch.empty(c, device="cuda") for _ in range(2))
        p3d.p3d_group_norm(t[0], t[2], groups, off, w, b, "silu", 1e-5, mean, rstd)
        p3d.p3d_group_norm_backward(t[1], t[0], mean, rstd, t[3], groups, off, w, b, "silu", dw,
                                    db)
        got.append((t[2].clone(), t[3].clone(), mean, rstd, dw, db))
    for near, far in zip(*got):
        assert torch.equal(near, far) and not far.float().isnan().any()


@pytest.mark.parametrize("k,d,few", [(128, 136, 0), (528, 72, 0), (4096, 64, 5)])
def test_linear(k, d, few):
    x = torch.empty(N, WIDE, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(N, WIDE, dtype=torch.int8, device="cuda")
    # (few tokens: the last ones of the buffer)
    rows = slice(N - few, N) if few else slice(0, N)
    a, qs = x[rows, 8000:8000 + k], q[rows, WIDE - k:]
    out, res = x[rows, 16:16 + d], x[rows, WIDE - d:]
    a.copy_(randn(*a.shape, seed=5))
    res.copy_(randn(*res.shape, seed=6))
    weight = torch.randint(-127, 128, (d, k), device="cuda").to(torch.int8)
    t = torch.full((d,), 1e-3, device="cuda")
    got = []
    for y in ((a, qs, res, out), (a.clone(), torch.empty(a.shape, dtype=torch.int8, device="cuda"),
                                  res.clone(), torch.empty_like(out))):
        scale = torch.empty(a.shape[0], device="cuda")
        p3d.p3d_quantize_rows(y[0], y[1], scale)
        p3d.p3d_linear_i8(y[1], scale, weight, t, y[3], act="gelu", residual=y[2])
        got.append((y[1].clone(), scale, y[3].clone()))
    for near, far in zip(*got):
        assert torch.equal(near, far)
    assert bool(got[0][0].any()) and not got[0][2].float().isnan().any()
