"""The block operators at the sizes where a launch is cut another way: more
units than the chip holds at once (some of them cut along the keys, some
whole), single tokens over long contexts, gradients of many tiles, results
that go past the caches, scores far from 0."""
import math

import pytest
import torch

import block_ref as ref
import pixel_aligned_image_amd as p3d
from test_gpu_attention import backward, forward, make

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -8                                # bf16 keeps 8 significant bits


def head_values(q, k, v, dout, scale, causal, score_off=0.0):
    """One key head of one item in 64 bits on the GPU: q, dout [nq, group, hd],
    k, v [nk, hd] -> {name: (value, tolerance)}, tolerances as in
    block_ref.attention_backward. score_off: how far a score less its row's
    lse may be off, which is the relative error of a probability."""
    nq, group, hd = q.shape
    slack = 2.0 ** -14
    k, v = k.to(F64), v.to(F64)
    res = {n: [] for n in ("out", "lse", "dq")}
    dk, dv, dk_tol, dv_tol = (torch.zeros_like(k) for _ in range(4))
    hidden = torch.zeros(nq, k.shape[0], dtype=torch.bool, device=k.device)
    if causal:
        at = torch.arange(nq, device=k.device)[:, None] + k.shape[0] - nq
        hidden = torch.arange(k.shape[0], device=k.device)[None] > at
    for m in range(group):
        x, do = q[:, m].to(F64), dout[:, m].to(F64)
        s = (scale * (x @ k.T)).masked_fill(hidden, -math.inf)
        lse = torch.logsumexp(s, 1)
        p = (s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None]).exp()
        reach = p @ v.abs()
        o = p @ v
        res["out"].append((o, (2 * U + 2.0 ** -13 + 2 * score_off) * reach))
        res["lse"].append((lse, 2.0 ** -16 + score_off))
        dp = do @ v.T
        d = (do * o).sum(1, keepdim=True)
        ds = p * (dp - d)
        d_off = (2 * U + 2 * score_off) * (do.abs() * reach).sum(1, keepdim=True)
        sized = p * (do.abs() @ v.abs().T + d.abs())
        ds_off = U * ds.abs() + p * d_off + (slack + score_off) * sized
        dq = scale * (ds @ k)
        res["dq"].append((dq, scale * (ds_off @ k.abs()) + U * dq.abs()))
        dk += scale * (ds.T @ x)
        dk_tol += scale * (ds_off.T @ x.abs())
        dv += p.T @ do
        dv_tol += (U + slack + score_off) * (p.T @ do.abs())
    got = {n: tuple(torch.stack([torch.as_tensor(t[i], device=k.device, dtype=F64).expand(
        t[0].shape) for t in res[n]], 1) for i in (0, 1)) for n in res}
    got["dk"] = dk, dk_tol + U * dk.abs()
    got["dv"] = dv, dv_tol + U * dv.abs()
    return got


def check_head(got, q, k, v, dout, qo, ko, scale, causal, item, kv_head, **kw):
    """The results of one key head of one item, those of `got` that are there."""
    group = q.shape[1] // k.shape[1]
    rows, keys = slice(*qo[item:item + 2]), slice(*ko[item:item + 2])
    heads = slice(kv_head * group, (kv_head + 1) * group)
    want = head_values(q[rows, heads], k[keys, kv_head], v[keys, kv_head], dout[rows, heads],
                       scale, causal, **kw)
    for n, t in got.items():
        mine = t[keys, kv_head] if n in ("dk", "dv") else t[rows, heads]
        w, tol = (x.cpu() for x in want[n])
        assert ref.off_by(mine, w, tol) <= 1, (n, item, kv_head)


# Units are 128-row tiles times key heads; the chip takes 512 at once for heads
# above 64 and 768 for narrower ones. nq, nk, q table, k table, heads, kv_heads,
# hd, units cut along the keys, their parts
CUT = [
    (4224, 600, None, None, 16, 16, 128, 16, 2), (2112, 600, None, None, 32, 16, 128, 16, 2),
    (6272, 600, None, None, 16, 16, 64, 16, 2), (4288, 1400, [0, 1100, 4288], [0, 100, 1400], 16,
                                                 16, 96, 32, 5),
    (4200, 5000, None, None, 16, 16, 104, 16, 19)]


@pytest.mark.parametrize("nq,nk,qo,ko,heads,kv_heads,hd,cut,parts", CUT)
def test_whole_units_beside_cut_ones(nq, nk, qo, ko, heads, kv_heads, hd, cut, parts):
    qo, ko = qo or [0, nq], ko or [0, nk]
    q, k, v, dout = (t.cuda() for t in make(nq, nk, heads, kv_heads, hd, seed=nq + hd))
    size = p3d.p3d_attention_workspace_size(q, k, qo, ko)
    assert size == (256 + cut * parts * 128 * (hd * 4 + 8) + 255) // 256 * 256
    out, lse = forward(q, k, v, qo, ko, hd ** -0.5, False)
    for item in range(len(qo) - 1):
        for head in (0, 7, kv_heads - 1):
            check_head({"out": out, "lse": lse}, q, k, v, dout, qo, ko, hd ** -0.5, False, item,
                       head)


# blocks of the gradient's launches: at least 1024 (uncut), 256 to 1023 (cut
# where the other axis is long), fewer
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("nq,nk,heads,kv_heads,hd", [
    (4224, 4224, 16, 16, 128), (4100, 2500, 32, 16, 64), (8300, 8193, 16, 16, 64),
    (700, 9000, 8, 2, 96), (9000, 700, 8, 2, 128), (3000, 4100, 6, 3, 80)])
def test_launches_of_more_than_a_round(nq, nk, heads, kv_heads, hd, causal):
    q, k, v, dout = (t.cuda() for t in make(nq, nk, heads, kv_heads, hd, seed=nq + nk))
    off, scale = ([0, nq], [0, nk]), hd ** -0.5
    out, lse = forward(q, k, v, *off, scale, causal)
    got = backward(dout, q, k, v, out, lse, *off, scale, causal) | {"out": out, "lse": lse}
    for head in (0, kv_heads - 1):
        check_head(got, q, k, v, dout, *off, scale, causal, 0, head)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_ragged_items_of_more_than_a_round(causal):
    qo, ko = [0, 2300, 2300, 2301, 5000], [0, 2600, 2700, 2990, 5600]
    q, k, v, dout = (t.cuda() for t in make(5000, 5600, 16, 16, 64, seed=21))
    out, lse = forward(q, k, v, qo, ko, 0.125, causal)
    got = backward(dout, q, k, v, out, lse, qo, ko, 0.125, causal) | {"out": out, "lse": lse}
    for item in range(4):
        for head in (0, 15):
            check_head(got, q, k, v, dout, qo, ko, 0.125, causal, item, head)


@pytest.mark.parametrize("keys,heads,kv_heads,hd", [
    ([40001], 8, 2, 128), ([40001], 8, 8, 64), ([0, 33000, 70, 5, 9001], 16, 4, 128),
    ([700] * 30 + [9000, 0, 1, 4000], 4, 4, 80), ([100001], 1, 1, 128)])
def test_single_tokens_over_long_contexts(keys, heads, kv_heads, hd):
    """Keys cut into up to 64 parts of equal size over the items, one workgroup
    a CU at most, or as many as there are items and heads."""
    items = len(keys)
    qo = list(range(items + 1))
    ko = [sum(keys[:b]) for b in range(items + 1)]
    q, k, v, dout = (t.cuda() for t in make(items, ko[-1], heads, kv_heads, hd, seed=items))
    parts = p3d.p3d_attention_workspace_size(q, k, qo, ko) // (32 * (hd * 4 + 8))
    assert 16 * kv_heads <= parts <= max(256, items * kv_heads)
    for causal in (False, True):
        out, lse = forward(q, k, v, qo, ko, 0.1, causal)
        for item in range(items):
            for head in (0, kv_heads - 1):
                check_head({"out": out, "lse": lse}, q, k, v, dout, qo, ko, 0.1, causal, item,
                           head)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("spread", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("nq,nk,hd", [(150, 500, 64), (300, 260, 128)])
def test_gradients_of_flat_and_peaked_rows(nq, nk, hd, spread, causal):
    """The gradient starts a score's sum at -lse / scale. With scores of size s
    (up to some thousand) that sum of up to 128 products passes values of 2 s /
    scale, each rounding 2^-24 of them: together under 2^-16 s; lse is good to
    2^-16 (1 + s). A probability is off by as much of itself."""
    q, k, v, dout = (t.cuda() for t in make(nq, nk, 2, 1, hd, seed=3, spread=spread))
    scale = hd ** -0.5
    size = scale * float(q.double().norm(dim=2).max() * k.double().norm(dim=2).max())
    off = [0, nq], [0, nk]
    out, lse = forward(q, k, v, *off, scale, causal)
    got = backward(dout, q, k, v, out, lse, *off, scale, causal) | {"out": out, "lse": lse}
    check_head(got, q, k, v, dout, *off, scale, causal, 0, 0, score_off=2.0 ** -15 * (1 + size))


# Results of calls whose tensors pass 256 MB are stored past the caches; the
# same rows in calls of half the size are not, and every row is on its own.
PAST = 1 << 28


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_norm_rows_past_the_caches(dtype):
    e, dim = dtype.itemsize, 1536
    n = PAST // (4 * dim * e) + 101
    cut = n // 2 - 3
    g = torch.Generator(device="cuda").manual_seed(1)
    t = {a: torch.randn(n, dim, generator=g, device="cuda").to(dtype)
         for a in ("x", "y", "dh", "dr")}
    mod = {a: torch.randn(2, dim, generator=g, device="cuda").to(dtype)
           for a in ("gate", "scale", "shift")}
    assert n * dim * 4 * e > PAST > max(cut, n - cut) * dim * 6 * e

    def call(rows, items, offsets):
        a = {name: x[rows] for name, x in t.items()}
        m = {name: x[items].contiguous() for name, x in mod.items()}
        r, h, dx, dy = (torch.full_like(a["x"], float("nan")) for _ in range(4))
        p3d.p3d_gated_norm(a["x"], h, offsets, y=a["y"], r=r, **m)
        del m["shift"]
        p3d.p3d_gated_norm_backward(a["dh"], a["x"], dx, offsets, dr=a["dr"], y=a["y"], dy=dy,
                                    **m)
        return r, h, dx, dy

    whole = call(slice(0, n), slice(0, 2), [0, cut, n])
    for rows, item in ((slice(0, cut), 0), (slice(cut, n), 1)):
        part = call(rows, slice(item, item + 1), [0, rows.stop - rows.start])
        assert all(torch.equal(w[rows], p) for w, p in zip(whole, part))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_rotary_rows_past_the_caches(dtype, layout):
    e, heads, hd = dtype.itemsize, 24, 128
    n = PAST // (2 * heads * hd * e) + 77
    cut = n // 2 - 5
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dout = (torch.randn(n, heads, hd, generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = torch.randn(heads, hd, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1024, (n, 3), generator=g, device="cuda", dtype=torch.int32)
    freqs = p3d.p3d_rotary_frequencies(10000.0, 21).cuda()
    assert n * heads * hd * 2 * e > PAST > (n - cut) * heads * hd * 3 * e

    def call(rows):
        out, dx, turned = (torch.full_like(x[rows], float("nan")) for _ in range(3))
        p3d.p3d_rotary(x[rows], pos[rows], freqs, out, layout=layout, gamma=gamma)
        p3d.p3d_rotary_backward(dout[rows], pos[rows], freqs, dx, layout=layout, gamma=gamma,
                                x=x[rows])
        p3d.p3d_rotary_backward(dout[rows], pos[rows], freqs, turned, layout=layout)
        return out, dx, turned

    whole = call(slice(0, n))
    for rows in (slice(0, cut), slice(cut, n)):
        assert all(torch.equal(w[rows], p) for w, p in zip(whole, call(rows)))


@pytest.mark.parametrize("nk,heads,hd", [(5, 12, 128), (40, 24, 64), (64, 16, 96)])
def test_few_keys_past_the_caches(nk, heads, hd):
    n = PAST // (4 * heads * hd) + 33
    cut = n // 2 - 7
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(n, heads, hd, generator=g, device="cuda").to(BF16)
    k, v = (torch.randn(nk, heads, hd, generator=g, device="cuda").to(BF16) for _ in range(2))
    assert n * heads * hd * 4 > PAST > (n - cut) * heads * hd * 4
    out, lse = forward(q, k, v, [0, n], [0, nk], 0.1, False)
    for rows in (slice(0, cut), slice(cut, n)):
        o, l = forward(q[rows], k, v, [0, rows.stop - rows.start], [0, nk], 0.1, False)
        assert torch.equal(out[rows], o) and torch.equal(lse[rows], l)
    some = slice(n - 300, n)
    check_head({"out": out[some], "lse": lse[some]}, q[some], k, v, q[some], [0, 300], [0, nk],
               0.1, False, 0, heads - 1)
