"""Graphs that captured tf_kv_attend, replayed after other calls on their stream: the
library's workspace for the stream stays where it was, whatever is called there."""
import ctypes

import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV
from tests.test_gpu_attend import filled

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def new_stream():
    """A stream that nothing has run on (torch hands its own out in turn)."""
    handle = ctypes.c_void_p(0)
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
    return torch.cuda.ExternalStream(handle.value)


def capture(cache, x, batch, out, **how):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.current_stream()):
        cache.attend(x, batch, out=out, **how)
    return graph


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_graph_outlives_larger_calls_on_its_stream(dim):
    # Single tokens (split over CTAs) are captured; then calls that need more of the workspace, with both kernels; then
    # whatever memory they might have freed is taken and filled; then the replay.
    lens = [3000, 700]
    q = filled(lens, 2, dim, 64, 30)
    long = filled([6000] * 6, 2, dim, 64, 31)
    with torch.cuda.stream(torch.cuda.Stream()):
        x = torch.randn((2, 4 * dim), device=DEV).to(BF16)
        b = q.batch(lens, [1, 1])
        out = torch.zeros_like(x)
        want = q.cache.attend(x, b).clone()
        graph = capture(q.cache, x, b, out)
        rows = torch.randn((6 * 700, 4 * dim), device=DEV).to(BF16)
        for kernel in (tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES):
            long.cache.attend(rows, long.batch([6000] * 6, [700] * 6), kernel=kernel)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        taken = [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(64)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert all(bool(torch.all(t == 7.0)) for t in taken)
        assert torch.equal(q.cache.attend(x, b), want)
        tf.tf_device_status()


@pytest.mark.parametrize("kernel", [tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])
def test_graphs_of_growing_batches_on_one_stream(kernel):
    # A graph a batch size, the larger ones captured later: each gives the direct call's bits, in any order of replays.
    sizes = [1, 3, 8, 20]
    q = filled([2000] * 20, 2, 128, 64, 32)
    with torch.cuda.stream(torch.cuda.Stream()):
        steps = []
        for n in sizes:
            x = torch.randn((n, 8 * 128), device=DEV).to(BF16)
            b = q.batch([2000 - 7 * i for i in range(n)], [1] * n)
            want = q.cache.attend(x, b, kernel=kernel).clone()
            out = torch.zeros_like(x)
            steps.append((capture(q.cache, x, b, out, kernel=kernel), out, want, x, b))
        for i in (0, 3, 1, 0, 2, 3, 0):
            graph, out, want = steps[i][:3]
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        tf.tf_device_status()


def test_a_first_call_inside_a_capture_is_refused():
    q = filled([300], 2, 64, 16, 33)
    x = torch.randn((1, 256), device=DEV).to(BF16)
    b, out = q.batch([300], [1]), torch.zeros((1, 256), dtype=BF16, device=DEV)
    want = q.cache.attend(x, b).clone()
    torch.cuda.synchronize()
    stream = new_stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out.fill_(2.0)
        with pytest.raises(tf.TfError) as e:
            q.cache.attend(x, b, out=out)
        assert e.value.rc == -10 and "precede" in str(e.value)
        out.add_(1.0)
    graph.replay()                                    # the capture went on
    torch.cuda.synchronize()
    assert torch.all(out == 3.0)
    with torch.cuda.stream(stream):
        assert torch.equal(q.cache.attend(x, b), want)
    torch.cuda.synchronize()

