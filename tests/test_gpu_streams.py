"""Calls on a stream of their own: a tensor that the caller drops while the
call still waits for its turn is not handed out again before it has run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import pixel_aligned_image_amd as p3d

N, DIM = 4096, 512
SPIN = 20_000_000


def gated_norm(s):
    x = torch.randn(N, DIM, device="cuda")
    p3d.p3d_gated_norm(x, torch.empty_like(x), stream=s)


def norm_backward(s):
    x = torch.randn(N, DIM, device="cuda")
    p3d.p3d_gated_norm_backward(x, x, torch.empty_like(x), stream=s,
                                dweight=torch.empty(DIM, device="cuda"))


def rotary(s):
    x = torch.randn(N, 4, 128, device="cuda")
    p3d.p3d_rotary(x, torch.zeros(N, 1, dtype=torch.int32, device="cuda"),
                   torch.ones(64, device="cuda"), torch.empty_like(x), stream=s)


def attention(s):
    q = torch.randn(N, 8, 128, device="cuda").bfloat16()
    k = torch.randn(8 * N, 1, 128, device="cuda").bfloat16()
    p3d.p3d_attention(q[:8], k, k, torch.empty_like(q[:8]), stream=s)


def sample(s):
    feat = torch.randn(1, 32, 32, DIM, device="cuda")
    p3d.p3d_bilinear_sample(feat, torch.zeros(N, 2, device="cuda"),
                            torch.empty(N, DIM, device="cuda"), stream=s)


def token_order(s):
    coords = torch.zeros(N, 4, dtype=torch.int32, device="cuda")
    p3d.p3d_token_order(coords, N, 64, [(1.0, 2.0)], 32, 32,
                        torch.empty(N, dtype=torch.int32, device="cuda"), stream=s)


@pytest.mark.parametrize("call", [gated_norm, norm_backward, rotary, attention, sample,
                                  token_order], ids=lambda f: f.__name__)
def test_dropped_tensors_wait_for_the_stream(call):
    own = torch.cuda.Stream()
    call(own)                                # kernels loaded, workspaces' sizes cached
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        torch.cuda._sleep(SPIN)
    own.wait_stream(torch.cuda.current_stream())
    call(own)
    assert not own.query()
    # whatever the allocator gives out now keeps its values
    taken = [torch.full((size,), 7, dtype=torch.uint8, device="cuda")
             for size in (512, 1 << 12, 1 << 14, 1 << 16, 1 << 18, 1 << 20, N * DIM * 2,
                          N * DIM * 4) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in taken)


def test_fresh_workspaces_are_no_blocks_in_use_elsewhere():
    """Blocks freed on the current stream while work that writes them waits
    there: a call on another stream, which does not wait for that work, gets
    none of them as its workspace, and its results are those of a call alone."""
    own = torch.cuda.Stream()
    q = torch.randn(8, 8, 128, device="cuda").bfloat16()
    k = torch.randn(8 * N, 1, 128, device="cuda").bfloat16()
    x = torch.randn(N, DIM, device="cuda")
    size = p3d.p3d_attention_workspace_size(q, k)
    assert size > 1 << 20                    # the keys are split

    def calls(stream):
        out, dx, dw = torch.empty_like(q), torch.empty_like(x), torch.empty(DIM, device="cuda")
        own.wait_stream(torch.cuda.current_stream())

        def run():
            p3d.p3d_attention(q, k, k, out, stream=stream)
            p3d.p3d_gated_norm_backward(x, x, dx, dweight=dw, stream=stream)
            return out, dx, dw

        return run

    alone = calls(None)()
    torch.cuda.synchronize()
    run = calls(own)                         # own waits for nothing after this
    sizes = [size, p3d.p3d_gated_norm_workspace_size(x)]
    taken = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in taken]
    torch.cuda._sleep(SPIN // 10)
    for _ in range(20):
        for t in taken:
            t.fill_(255)                     # NaN, were it read as sums
    del taken, t
    from pixel_aligned_image_amd import _streams
    for s in sizes:
        at = _streams.fresh(s, "cuda", own).data_ptr()
        assert not any(a < at + s and at < b for a, b in spans)
    got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))


class Handle:
    """A stream of another library: a handle and nothing else."""

    def __init__(self, stream):
        self.cuda_stream, self.keep = stream.cuda_stream, stream


@pytest.mark.parametrize("call", [gated_norm, norm_backward, rotary, attention, sample,
                                  token_order], ids=lambda f: f.__name__)
def test_any_object_with_a_handle_is_a_stream(call):
    """The calls read no more of a stream than its handle; tensors dropped
    after such a call wait for it, too."""
    own = torch.cuda.Stream()
    call(Handle(own))
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        torch.cuda._sleep(SPIN)
    own.wait_stream(torch.cuda.current_stream())
    call(Handle(own))
    assert not own.query()
    taken = [torch.full((size,), 7, dtype=torch.uint8, device="cuda")
             for size in (512, 1 << 14, 1 << 18, N * DIM * 2, N * DIM * 4) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in taken)


def test_cameras_as_a_cpu_tensor_on_a_stream():
    coords = torch.zeros(N, 4, dtype=torch.int32, device="cuda")
    order = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    own = torch.cuda.Stream()
    own.wait_stream(torch.cuda.current_stream())
    p3d.p3d_token_order(coords, N, 64, torch.tensor([[1.0, 2.0]]), 32, 32, order, stream=own)
    torch.cuda.synchronize()
    assert torch.equal(order.sort().values, torch.arange(N, dtype=torch.int32, device="cuda"))
