"""Every test of tf_kv_attend again, with each of its two kernels for every call:
the one for few rows on prompts, the one for prompts on single tokens."""
import pytest

import mlx_affine_bit_gb300 as tf
from tests.test_gpu_attend import *  # noqa: F401,F403  (the tests themselves)
from tests.test_gpu_attend import DEV, filled, pytestmark  # noqa: F401
import numpy as np
import torch


@pytest.fixture(autouse=True, params=[tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])
def kernel(request, monkeypatch):
    attend = tf.KvCache.attend
    monkeypatch.setattr(tf.KvCache, "attend", lambda self, *a, **k: attend(self, *a, kernel=request.param, **k))
    return request.param


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (8, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("window", [0, 900])
def test_shares_that_end_anywhere(heads, kv_heads, dim, window):
    # Many sequences of many lengths: items begin and end, and are cut, in the middle of a CTA's share.
    from tests.test_gpu_attend import run
    rng = np.random.default_rng(dim + window)
    lens = rng.integers(1, 2500, 40).tolist()
    rows = [int(min(n, rng.choice([0, 1, 3, 40, 300], p=[0.1, 0.3, 0.3, 0.2, 0.1]))) for n in lens]
    run(filled(lens, kv_heads, dim, 64, 20), lens, rows, heads, window=window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_long_sequence_in_many_parts(dim):
    from tests.test_gpu_attend import run
    run(filled([40000], 1, dim, 128, 21), [40000], [5], 3)


def test_both_kernels_refuse_to_be_both(kernel):
    q = filled([10], 1, 64, 16, 1)
    x = torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(tf.TfError) as e:
        tf.tf_kv_attend(q.cache.c, q.batch([10], [1]).c, x, 64, 1, x, 64, 1.0, 0, tf.TF_KV_BY_ROWS | tf.TF_KV_BY_TILES)
    assert e.value.rc == -12
