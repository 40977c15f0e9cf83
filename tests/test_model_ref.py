"""The plain forms of tests/model_ref.py on the CPU: group norm against torch's
own, its gradients against differences, the random bits and the 8-bit rounding
they choose."""
import math

import pytest
import torch

import model_ref as ref


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_group_norm_is_torchs(kind):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 24, 5, 7, generator=g, dtype=torch.float64) * 3 + 1
    w, b = (torch.randn(24, generator=g, dtype=torch.float64) for _ in range(2))
    want = ref.act(torch.nn.functional.group_norm(x, 6, w, b, 1e-3), kind)
    rows = x.permute(0, 2, 3, 1).reshape(-1, 24)
    got, _ = ref.group_norm(rows, [0, 35, 70], 6, w, b, kind, 1e-3)
    got = got.reshape(2, 5, 7, 24).permute(0, 3, 1, 2)
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_group_norm_gradients_are_the_differences(kind):
    g = torch.Generator().manual_seed(4)
    off, groups = [0, 5, 5, 9], 3
    x = torch.randn(9, 12, generator=g, dtype=torch.float64) * 2 + 0.5
    w, b = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(2))
    dout = torch.randn(9, 12, generator=g, dtype=torch.float64)
    got = ref.group_norm_backward(dout, x, off, groups, w, b, kind)
    h = 1e-6
    for name, leaf in (("dx", x), ("dweight", w), ("dbias", b)):
        for i in torch.randperm(leaf.numel(), generator=g)[:20].tolist():
            keep = leaf.view(-1)[i].item()
            ends = []
            for d in (h, -h):
                leaf.view(-1)[i] = keep + d
                ends.append((ref.group_norm(x, off, groups, w, b, kind)[0] * dout).sum().item())
            leaf.view(-1)[i] = keep
            assert math.isclose((ends[0] - ends[1]) / (2 * h), got[name].view(-1)[i].item(),
                                rel_tol=1e-6, abs_tol=1e-6), (name, i)


def test_random_bits_are_even():
    """Every bit is set about half the time, and seeds, tensors and neighbours
    are unlike: 5 standard deviations of a fair coin's count."""
    n = 20000
    runs = [torch.tensor(ref.random_bits(0, n, j, s)) for j, s in
            ((0, 0), (1, 0), (0, 1), (0, 1 << 32))]
    bound = 5 * 0.5 * n ** 0.5
    for r in runs:
        for k in range(32):
            assert abs(int((r >> k & 1).sum()) - n / 2) < bound, k
        for k in range(32):
            assert abs(int(((r[1:] ^ r[:-1]) >> k & 1).sum()) - n / 2) < bound, k
    for i in range(4):
        for j in range(i):
            for k in range(32):
                assert abs(int(((runs[i] ^ runs[j]) >> k & 1).sum()) - n / 2) < bound, (i, j, k)


def test_encode_keeps_the_mean():
    codes = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    n = 4096
    bits = torch.arange(0, 65536, 65536 // n, dtype=torch.float64)
    for q in [1e-5, 0.001, 0.0019, 0.01, 0.0156, 0.3, 1.0, 17.3, 300.0, 447.9, 448.0]:
        got = ref.encode(torch.full((n,), q, dtype=torch.float64), bits)
        assert torch.isin(got, codes).all()
        low = codes[codes <= q].max()
        high = codes[codes >= q].min()
        assert got.min() >= low and got.max() <= high
        # the bits are evenly spaced, so the mean misses by a step of theirs at most
        assert abs(got.mean().item() - q) <= (high - low).item() / n + 1e-12
    assert (ref.encode(torch.tensor([-3.0, 1e9], dtype=torch.float64), torch.zeros(2))
            == torch.tensor([-3.0, 448.0])).all()


def test_quantize_ties_and_edges():
    x = torch.tensor([[254.0, 1.0, 3.0, -1.0, -3.0], [0.0] * 5, [1.0, float("nan"), 0, 0, 0],
                      [float("inf"), 1.0, 0, 0, 0]], dtype=torch.float64)
    q, s = ref.quantize(x)
    assert s[0] == 2 and q[0].tolist() == [127, 0, 2, 0, -2]    # ties to even
    assert s[1] == 0 and not q[1].any()
    assert s[2:].isnan().all() and not q[2:].any()
