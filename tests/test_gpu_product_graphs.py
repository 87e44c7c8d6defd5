"""Graphs that captured products, replayed after larger products on their stream: the
workspace that a graph uses stays allocated."""
import pytest
import torch

import synth
import mlx_affine_bit_gb300 as tf
from tests.gpu_util import DEV, DevMatrix, dev, run_qmm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def outlives(call, small, large, y):
    """call(x) into y, captured with `small`; then with `large`, and what that may have freed taken and filled."""
    stream = torch.cuda.current_stream()
    call(small)
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(small)
    for x in large:
        call(x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    taken = [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(32)]
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all(bool(torch.all(t == 7.0)) for t in taken)
    tf.tf_device_status()


def test_split_k_product():
    # 2048 x 12288 splits K: a row's partials are 48 KB, 16 rows' 768 KB.
    dm = DevMatrix(synth.make_matrix(2048, 12288, 4, 64, 500, 0.001, 0.03))
    with torch.cuda.stream(torch.cuda.Stream()):
        y = torch.zeros((16, 2048), dtype=torch.float32, device=DEV)
        outlives(lambda x: run_qmm(dm, x, y=y), dev(synth.make_x(1, 12288, 501)),
                 [dev(synth.make_x(n, 12288, 502)) for n in (2, 5, 16)], y)


def test_prompt_product():
    m = synth.make_matrix(300, 4096, 6, 32, 510, 0.001, 0.03)
    dm = DevMatrix(m)
    with torch.cuda.stream(torch.cuda.Stream()):
        y = torch.zeros((400, 300), dtype=torch.float32, device=DEV)
        outlives(lambda x: tf.tf_qmm_prompt(x, x.shape[0], m.K, dm.W, dm.s, dm.b, m.N, m.bits, m.group, y, 300),
                 dev(synth.make_x(20, 4096, 511)), [dev(synth.make_x(n, 4096, 512)) for n in (64, 130, 400)], y)
