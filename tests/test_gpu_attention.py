"""p3d_attention and its gradients against the 64-bit form."""
import math

import pytest
import torch

import block_ref as ref
import pixel_aligned_image_amd as p3d

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def make(nq, nk, heads, kv_heads, hd, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(BF16)

    return (rnd(nq, heads, hd, scale=spread), rnd(nk, kv_heads, hd), rnd(nk, kv_heads, hd),
            rnd(nq, heads, hd))


def forward(q, k, v, qo, ko, scale, causal, **kw):
    out = torch.full(q.shape, float("nan"), dtype=BF16, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    p3d.p3d_attention(q, k, v, out, qo, ko, scale=scale, causal=causal, lse=lse, **kw)
    return out, lse


def check_forward(out, lse, q, k, v, qo, ko, scale, causal):
    wo, wl, reach = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), qo, ko, scale, causal)
    # P rounded (2^-8), out rounded (2^-8), binary32 sums and exponentials
    assert ref.off_by(out, wo, (2.0 ** -7 + 2.0 ** -13) * reach) <= 1
    # a score's sum of up to 128 products, log and exp: 2^-16 of the scores' size
    size = scale * float(ref.f64(q).norm(dim=2).max() if q.numel() else 0) * \
        float(ref.f64(k).norm(dim=2).max() if k.numel() else 0)
    assert ref.off_by(lse, wl, 2.0 ** -16 * (1 + size)) <= 1
    return wo


def backward(dout, q, k, v, out, lse, qo, ko, scale, causal, **kw):
    nan = float("nan")
    dq = torch.full(q.shape, nan, dtype=BF16, device="cuda")
    dk, dv = (torch.full(k.shape, nan, dtype=BF16, device="cuda") for _ in range(2))
    p3d.p3d_attention_backward(dout, q, k, v, out, lse, dq, dk, dv, qo, ko, scale=scale,
                               causal=causal, **kw)
    return {"dq": dq, "dk": dk, "dv": dv}


def check_backward(got, dout, q, k, v, qo, ko, scale, causal):
    want, tol = ref.attention_backward(ref.f64(dout), ref.f64(q), ref.f64(k), ref.f64(v), qo, ko,
                                       scale, causal)
    for n in got:
        assert ref.off_by(got[n], want[n], tol[n]) <= 1, n


# nq, nk, items, heads, kv_heads, head_dim
SIZES = [
    (1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 1, 128), (3, 5, 1, 2, 2, 128), (200, 5, 1, 3, 3, 128),
    (129, 65, 1, 2, 1, 64), (64, 64, 1, 1, 1, 8), (33, 31, 1, 4, 2, 24), (130, 257, 1, 2, 2, 80),
    (127, 191, 1, 2, 2, 96), (100, 100, 3, 2, 2, 104), (300, 310, 4, 4, 2, 128),
    (40, 200, 7, 6, 2, 72), (256, 128, 1, 1, 1, 128), (1, 700, 1, 8, 2, 128),
    (4, 1300, 4, 16, 4, 128), (5, 900, 2, 5, 1, 64), (60, 2100, 1, 2, 1, 128),
    (700, 40, 2, 2, 2, 64),
]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("nq,nk,items,heads,kv_heads,hd", SIZES)
def test_forward_and_backward(nq, nk, items, heads, kv_heads, hd, causal):
    q, k, v, dout = (t.cuda() for t in make(nq, nk, heads, kv_heads, hd, seed=nq + nk + hd))
    qo, ko = ref.uneven(nq, items), ref.uneven(nk, items)
    if items == nq:
        qo = list(range(nq + 1))
    scale = hd ** -0.5
    out, lse = forward(q, k, v, qo, ko, scale, causal)
    check_forward(out, lse, q, k, v, qo, ko, scale, causal)
    got = backward(dout, q, k, v, out, lse, qo, ko, scale, causal)
    check_backward(got, dout, q, k, v, qo, ko, scale, causal)


def test_errors_on_the_whole():
    """Over many random rows the roundings are independent: a result sees at
    most three (a factor's, out's through D, its own), each of relative size
    2^-8 / sqrt(3) at most, so its error's 2-norm is under 2^-8 of its own."""
    for causal in (False, True):
        q, k, v, dout = (t.cuda() for t in make(600, 700, 4, 2, 128, seed=11))
        off = ([0, 200, 600], [0, 250, 700])
        out, lse = forward(q, k, v, *off, 0.088, causal)
        wo, _, _ = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), *off, 0.088, causal)
        assert ref.rms_off(out, wo) < 2.0 ** -8
        got = backward(dout, q, k, v, out, lse, *off, 0.088, causal)
        want, _ = ref.attention_backward(ref.f64(dout), ref.f64(q), ref.f64(k), ref.f64(v), *off,
                                         0.088, causal)
        for n in got:
            assert ref.rms_off(got[n], want[n]) < 2.0 ** -8, n


@pytest.mark.parametrize("hd", [64, 96, 128])
def test_errors_over_few_keys(hd):
    """Rows of three keys: dq is off by its own rounding alone (dS is taken in
    two factors, D from the same probabilities), 2^-8 / sqrt(3) at most, and
    2^-6 of that for everything else."""
    items = 60
    q, k, v, dout = (t.cuda() for t in make(20 * items, 3 * items, 4, 4, hd, seed=hd))
    off = [20 * b for b in range(items + 1)], [3 * b for b in range(items + 1)]
    out, lse = forward(q, k, v, *off, hd ** -0.5, False)
    got = backward(dout, q, k, v, out, lse, *off, hd ** -0.5, False)
    want, _ = ref.attention_backward(ref.f64(dout), ref.f64(q), ref.f64(k), ref.f64(v), *off,
                                     hd ** -0.5, False)
    assert ref.rms_off(got["dq"], want["dq"]) < 2.0 ** -8 / 3 ** 0.5 * (1 + 2.0 ** -6)


def test_rows_of_one_key():
    """Their probability is 1 whatever the score: dq is 0, and dk of a key
    that nothing else sees; also beside items that are cut into parts."""
    for nq, nk, hd, causal in (([9], [1], 64, False), ([9], [1], 128, True),
                               ([2, 700, 1], [1, 2500, 1], 128, False),
                               ([1, 40], [1, 3000], 96, True)):
        qo = [sum(nq[:b]) for b in range(len(nq) + 1)]
        ko = [sum(nk[:b]) for b in range(len(nk) + 1)]
        q, k, v, dout = (t.cuda() for t in make(qo[-1], ko[-1], 4, 2, hd, seed=hd))
        out, lse = forward(q, k, v, qo, ko, 0.1, causal)
        got = backward(dout, q, k, v, out, lse, qo, ko, 0.1, causal)
        check_backward(got, dout, q, k, v, qo, ko, 0.1, causal)
        for b, keys in enumerate(nk):
            if keys == 1:
                assert (got["dq"][qo[b]:qo[b + 1]] == 0).all()
                assert (got["dk"][ko[b]:ko[b + 1]] == 0).all()


def test_items_without_queries_or_keys():
    """Rows without keys give 0 and -inf, keys without queries gradient 0."""
    qo, ko = [0, 40, 40, 75, 90], [0, 0, 33, 70, 170]
    q, k, v, dout = (t.cuda() for t in make(90, 170, 4, 2, 64, seed=1))
    for causal in (False, True):
        out, lse = forward(q, k, v, qo, ko, 0.125, causal)
        assert (out[:40] == 0).all() and (lse[:40] == -math.inf).all()
        check_forward(out, lse, q, k, v, qo, ko, 0.125, causal)
        got = backward(dout, q, k, v, out, lse, qo, ko, 0.125, causal)
        assert (got["dq"][:40] == 0).all() and (got["dk"][:33] == 0).all()
        assert (got["dv"][:33] == 0).all()
        check_backward(got, dout, q, k, v, qo, ko, 0.125, causal)


def test_causal_rows_that_see_nothing():
    """More queries than keys: the first ones see no key."""
    for nq, nk, hd in ((50, 7, 128), (300, 130, 64), (20, 19, 96)):
        q, k, v, dout = (t.cuda() for t in make(nq, nk, 2, 1, hd, seed=nq))
        out, lse = forward(q, k, v, [0, nq], [0, nk], 0.1, True)
        assert (out[:nq - nk] == 0).all() and (lse[:nq - nk] == -math.inf).all()
        check_forward(out, lse, q, k, v, [0, nq], [0, nk], 0.1, True)
        got = backward(dout, q, k, v, out, lse, [0, nq], [0, nk], 0.1, True)
        assert (got["dq"][:nq - nk] == 0).all()
        check_backward(got, dout, q, k, v, [0, nq], [0, nk], 0.1, True)


def test_nothing_at_all():
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    q = torch.randn(3, 2, 64, device="cuda").to(BF16)
    out, lse = forward(e, e, e, [0, 0], [0, 0], 1.0, False)
    out, lse = forward(q, e, e, [0, 3], [0, 0], 1.0, False)
    assert (out == 0).all() and (lse == -math.inf).all()
    got = backward(q, q, e, e, out, lse, [0, 3], [0, 0], 1.0, False)
    assert (got["dq"] == 0).all()
    out, lse = forward(e, q, q, [0, 0], [0, 3], 1.0, False)
    got = backward(e, e, q, q, out, lse, [0, 0], [0, 3], 1.0, False)
    assert (got["dk"] == 0).all() and (got["dv"] == 0).all()


@pytest.mark.parametrize("spread", [0.0, 30.0, 200.0])
def test_flat_and_peaked_rows(spread):
    """All scores equal, and scores so far apart that one key takes all (the
    running maximum rises many times)."""
    q, k, v, dout = (t.cuda() for t in make(150, 500, 2, 2, 64, seed=3, spread=spread))
    out, lse = forward(q, k, v, [0, 150], [0, 500], 0.125, False)
    wo, wl, reach = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), [0, 150], [0, 500], 0.125,
                                  False)
    # a score of size s is good to 2^-20 s, and so is its probability
    size = 0.125 * float((ref.f64(q).norm(dim=2).max() * ref.f64(k).norm(dim=2).max()))
    assert ref.off_by(out, wo, (2.0 ** -7 + 2.0 ** -13 + 2.0 ** -19 * size) * reach) <= 1
    assert ref.off_by(lse, wl, 2.0 ** -16 * (1 + size)) <= 1


def test_neighbours_are_not_read():
    """NaN in other items' rows, past the last row and in a padded buffer's
    other heads stays where it is."""
    nan = float("nan")
    q0, k0, v0, d0 = make(70, 90, 2, 2, 80, seed=5)
    big_k, big_v = (torch.full((200, 5, 80), nan, dtype=BF16, device="cuda") for _ in range(2))
    k, v = big_k[:90, 1:3], big_v[:90, 2:4]
    k.copy_(k0)
    v.copy_(v0)
    qo, ko = [0, 30, 70], [0, 33, 90]
    for causal in (False, True):
        out, lse = forward(q0.cuda(), k, v, qo, ko, 0.11, causal)
        check_forward(out, lse, q0, k0, v0, qo, ko, 0.11, causal)
        got = backward(d0.cuda(), q0.cuda(), k, v, out, lse, qo, ko, 0.11, causal)
        check_backward(got, d0, q0, k0, v0, qo, ko, 0.11, causal)
        # one item's NaN leaves the other item's results alone
        kn = k0.clone()
        kn[40] = nan
        o2, l2 = forward(q0.cuda(), kn.cuda(), v0.cuda(), qo, ko, 0.11, causal)
        assert torch.equal(o2[:30], out[:30]) and torch.equal(l2[:30], lse[:30])


def test_packed_projection_and_in_place():
    """q, k, v as views of one packed buffer, gradients into one packed
    buffer, out over q."""
    g = torch.Generator().manual_seed(6)
    n, heads, hd = 333, 4, 128
    qkv = torch.randn(n, 3 * heads, hd, generator=g).to(BF16).cuda()
    q, k, v = qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    dout = torch.randn(n, heads, hd, generator=g).to(BF16).cuda()
    off = [0, 100, 333]
    out, lse = forward(q, k, v, off, off, 0.09, False)
    check_forward(out, lse, q, k, v, off, off, 0.09, False)
    d = torch.full_like(qkv, float("nan"))
    p3d.p3d_attention_backward(dout, q, k, v, out, lse, d[:, :heads], d[:, heads:2 * heads],
                               d[:, 2 * heads:], off, off, scale=0.09)
    check_backward({"dq": d[:, :heads], "dk": d[:, heads:2 * heads], "dv": d[:, 2 * heads:]},
                   dout, q, k, v, off, off, 0.09, False)
    p3d.p3d_attention(q, k, v, q, off, off, scale=0.09)
    assert torch.equal(q, out)


def test_gradient_against_differences():
    """The kernels' gradients in the direction of their own signs against
    differences of the 64-bit form."""
    q, k, v, dout = make(90, 120, 4, 2, 64, seed=7)
    off = ([0, 90], [0, 120])
    out, lse = forward(q.cuda(), k.cuda(), v.cuda(), *off, 0.125, True)
    got = backward(dout.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, *off, 0.125, True)
    t = {"q": ref.f64(q), "k": ref.f64(k), "v": ref.f64(v)}

    def loss(**kw):
        return float((ref.attention(q_offsets=off[0], k_offsets=off[1], scale=0.125, causal=True,
                                    **(t | kw))[0] * ref.f64(dout)).sum())

    for n in t:
        grad = ref.f64(got["d" + n])
        u = grad.sign()
        diff = (loss(**{n: t[n] + 1e-4 * u}) - loss(**{n: t[n] - 1e-4 * u})) / 2e-4
        assert abs(diff - float((grad * u).sum())) <= 2.0 ** -7 * abs(diff)


def test_offsets_past_32_bits():
    """A cache whose tokens lie 2^24 elements apart: the last past 2^32."""
    n, stride = 260, 1 << 24
    buf = torch.empty((n - 1) * stride + 512, dtype=BF16, device="cuda")
    k = buf.as_strided((n, 2, 64), (stride, 64, 1))
    v = buf[128:].as_strided((n, 2, 64), (stride, 64, 1))
    q, k0, v0, dout = make(70, n, 2, 2, 64, seed=8)
    k.copy_(k0)
    v.copy_(v0)
    off = ([0, 70], [0, n])
    out, lse = forward(q.cuda(), k, v, *off, 0.125, True)
    check_forward(out, lse, q, k0, v0, *off, 0.125, True)
    got = backward(dout.cuda(), q.cuda(), k, v, out, lse, *off, 0.125, True)
    check_backward(got, dout, q, k0, v0, *off, 0.125, True)
    one, l1 = forward(q[:1].cuda(), k, v, [0, 1], [0, n], 0.125, True)
    check_forward(one, l1, q[:1], k0, v0, [0, 1], [0, n], 0.125, True)


def test_single_tokens_match_the_last_rows():
    """A causal prefill's last row and the same token alone over the cache
    differ by roundings of P and out only."""
    q, k, v, _ = (t.cuda() for t in make(500, 500, 8, 2, 128, seed=9))
    off = [0, 500]
    out, lse = forward(q, k, v, off, off, 0.09, True)
    one, l1 = forward(q[-1:], k, v, [0, 1], off, 0.09, True)
    reach = ref.attention(ref.f64(q[-1:]), ref.f64(k), ref.f64(v), [0, 1], off, 0.09, True)[2]
    assert ref.off_by(one, out[-1:], (2.0 ** -6 + 2.0 ** -12) * reach) <= 1
    assert ref.off_by(l1, lse[-1:], 2.0 ** -14) <= 1


def test_repeatable_on_another_stream_and_in_a_graph():
    q, k, v, dout = (t.cuda() for t in make(900, 1500, 4, 2, 128, seed=10))
    qo, ko = [0, 3, 900], [0, 1400, 1500]

    def once(stream=None):
        out, lse = torch.empty_like(q), torch.empty(900, 4, device="cuda")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(p3d.p3d_attention_workspace_size(q, k, qo, ko), dtype=torch.uint8,
                         device="cuda")
        wb = torch.empty(p3d.p3d_attention_backward_workspace_size(q, k, qo, ko),
                         dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        p3d.p3d_attention(q, k, v, out, qo, ko, lse=lse, workspace=ws, stream=stream)
        p3d.p3d_attention_backward(dout, q, k, v, out, lse, dq, dk, dv, qo, ko, workspace=wb,
                                   stream=stream)
        torch.cuda.synchronize()
        return out, lse, dq, dk, dv

    first = once()
    for got in (once(), once(torch.cuda.Stream())):
        assert all(torch.equal(a, b) for a, b in zip(first, got))

    out, lse = torch.empty_like(q), torch.empty(900, 4, device="cuda")
    grads = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(p3d.p3d_attention_workspace_size(q, k, qo, ko), dtype=torch.uint8,
                     device="cuda")
    wb = torch.empty(p3d.p3d_attention_backward_workspace_size(q, k, qo, ko), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p3d.p3d_attention(q, k, v, out, qo, ko, lse=lse, workspace=ws)
        p3d.p3d_attention_backward(dout, q, k, v, out, lse, *grads, qo, ko, workspace=wb)
    for _ in range(3):
        for t in (out, lse, *grads):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (out, lse, *grads)))
        once()                                   # eager work between the replays


@pytest.mark.parametrize("hd", [64, 128])
def test_two_factors_reach_every_row_of_few_keys(hd):
    """Rows that see 130 to 256 keys, in a launch whose tile of rows ends on
    257 and in one whose tile ends on 256: dq takes dS as two factors in both,
    so the same rows get the same bits."""
    nq, nk, heads = 256, 257, 2
    q, k, v, dout = (t.cuda() for t in make(nq, nk, heads, heads, hd, seed=12))
    out, lse = forward(q, k, v, [0, nq], [0, nk], 0.1, True)
    whole = backward(dout, q, k, v, out, lse, [0, nq], [0, nk], 0.1, True)["dq"]
    rows = slice(128, 255)
    part = backward(dout[rows], q[rows], k[:256], v[:256], out[rows], lse[rows], [0, 127],
                    [0, 256], 0.1, True)["dq"]
    assert torch.equal(whole[rows], part)


@pytest.mark.parametrize("hd", [64, 128])
def test_roundings_do_not_depend_on_the_parts(hd):
    """512 keys walked whole and in two parts; the second half's probabilities
    are 0, so that the parts' sums add nothing: the same rows get the same
    bits, however many parts the launch has."""
    few, many, nk = 64, 32768, 512
    q, k, v, dout = (t.cuda() for t in make(many, nk, 1, 1, hd, seed=13))
    q[:, 0, 0], k[:256, 0, 0], k[256:, 0, 0] = 64, 0, -64
    off = [0, few], [0, nk]
    # the parts' workspace shows that one launch is cut and the other is not
    stats = 256 + 2 * 512
    assert p3d.p3d_attention_backward_workspace_size(q[:few], k, *off) >= stats + \
        2 * few * (hd + 1) * 4
    out, lse = forward(q, k, v, [0, many], [0, nk], 0.125, False)
    whole = backward(dout, q, k, v, out, lse, [0, many], [0, nk], 0.125, False)["dq"]
    part = backward(dout[:few], q[:few], k, v, out[:few], lse[:few], *off, 0.125, False)["dq"]
    assert torch.equal(whole[:few], part)


@pytest.mark.parametrize("keys", [40, 500, 5000])
@pytest.mark.parametrize("rows", [1, 40])
def test_rows_of_nan_say_so(rows, keys):
    """A query of NaN gives NaN in out and in lse (-inf is what a query that
    sees no key gets), for single tokens and for many, and its neighbours what
    they gave without it."""
    q, k, v, _ = (t.cuda() for t in make(rows * 2, keys, 2, 1, 128, seed=14))
    off = [0, rows, 2 * rows], [0, keys // 2, keys]
    want, lse_want = forward(q, k, v, *off, 0.1, False)
    q[0] = float("nan")
    out, lse = forward(q, k, v, *off, 0.1, False)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[rows:], want[rows:]) and torch.equal(lse[rows:], lse_want[rows:])
