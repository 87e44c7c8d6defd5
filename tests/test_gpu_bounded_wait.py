"""Failure detection without a GPU fault: a withheld stage makes the kernel's
bounded wait run out; the kernel records it in the device status word and
completes, the host reads TF_EDEVICE, and the next call is correct again."""
import pytest
import torch

import synth
import mlx_affine_bit_gb300 as tf
from tests.gpu_util import DevMatrix, dev, oracle_check, run_qmm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("N,K,bits,group", [(256, 1024, 4, 64), (40, 96, 3, 32)])
def test_bounded_wait_runs_out_and_is_reported(N, K, bits, group):
    m = synth.make_matrix(N, K, bits, group, 160, 0.001, 0.03)
    dm = DevMatrix(m)
    x = synth.make_x(2, K, 161)
    xd = dev(x)
    torch.cuda.synchronize()
    tf.tf_device_status()                      # starts clean
    tf.tf_inject_stall()
    run_qmm(dm, xd)                            # its first stage never arrives: about 2 s
    torch.cuda.synchronize()
    with pytest.raises(tf.TfError) as e:
        tf.tf_device_status()
    assert e.value.rc == -11
    tf.tf_device_status()                      # reading cleared it
    y = run_qmm(dm, xd)                        # the context is usable and the next call right
    torch.cuda.synchronize()
    tf.tf_device_status()
    oracle_check(m, x, y.cpu().numpy())


@pytest.mark.parametrize("kernel", [tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 1), (128, 20), (256, 5)])
def test_attention_is_correct_again_after_a_wait_ran_out(kernel, dim, rows):
    # Items that several CTAs share and CTAs with several items: parts that never came must not be counted later.
    import numpy as np
    from tests.test_gpu_attend import filled
    rng = np.random.default_rng(dim + rows)
    lens = rng.integers(rows, 2500, 120).tolist()
    few = [9000, 40]
    q, p = filled(lens, 4, dim, 64, 40), filled(few, 1, dim, 64, 41)
    b, c = q.batch(lens, [rows] * 120), p.batch(few, [rows] * 2)
    x = torch.randn((120 * rows, 8 * dim), device=q.cache.k.device).to(torch.bfloat16)
    want = [q.cache.attend(x, b, kernel=kernel).clone(), p.cache.attend(x[:2 * rows], c, kernel=kernel).clone()]
    torch.cuda.synchronize()
    tf.tf_device_status()
    for one in (True, False):
        tf.tf_inject_stall()
        q.cache.attend(x, b, kernel=kernel) if one else p.cache.attend(x[:2 * rows], c, kernel=kernel)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -11
        for _ in range(2):
            assert torch.equal(q.cache.attend(x, b, kernel=kernel), want[0])
            assert torch.equal(p.cache.attend(x[:2 * rows], c, kernel=kernel), want[1])
        torch.cuda.synchronize()
        tf.tf_device_status()
