"""tf_kv_attend, by either kernel, where outputs are small: checked relative to what they are made of alone
(decode_oracle.attend's bound on the same values times 2^100)."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV, attend
from tests.test_gpu_attend import filled, queries

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
kernels = pytest.mark.parametrize("kernel", [tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def positive(q):
    """No value below 0, so that what a token adds is not made up for by others."""
    q.cache.v.copy_(q.cache.v.to(torch.int16).abs().clamp(max=127).to(torch.int8))
    return q


def run_small(q, lens, rows, heads, kernel, x, by=100):
    got = q.cache.attend(torch.from_numpy(x.reshape(sum(rows), -1)).to(DEV).to(BF16), q.batch(lens, rows), kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    got = got.double().cpu().numpy().reshape(sum(rows), heads, q.d) * 2.0 ** by
    at = 0
    for s, (n, r) in enumerate(zip(lens, rows)):
        k, v = q.values(s, n)
        vs = q.value_scales(s, n) * 2.0 ** by
        want, bound = attend(x[at:at + r], k, v.astype(np.float64) * 2.0 ** by, vs, q.d ** -0.5, r, True, 0, False)
        # (A bf16 output below 2^-126 is half of 2^-133 off at most, and a weight that fp32 holds no more is below 2^-126.)
        bound += 2.0 ** (by - 134) + n * 2.0 ** -126 * 128 * vs.max()
        err = np.abs(got[at:at + r] - want) / bound
        assert np.all(np.isfinite(err)) and err.max() <= 1, "sequence %d: %.3f of the bound" % (s, err.max())
        at += r


@kernels
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ahead", [60.0, 74.0])
def test_the_largest_scores_belong_to_zeros(dim, ahead, kernel):
    # All pages hold zeros but three, whose tokens' scores lie `ahead` below the largest.  So many sequences that a CTA takes
    # several steps of one; by rows, a warp that takes token 101 takes some of the others, too.
    lens = [333] * 160
    q = positive(filled(lens, 1, dim, 16, 43))
    x = np.abs(queries(np.random.default_rng(44), 160, 1, dim, BF16))
    q.cache.k_scale *= 0.01
    page = torch.from_numpy(q.table[:, 6]).to(DEV).long()
    codes = torch.zeros((16, dim), dtype=torch.int8, device=DEV)
    codes[5] = 127
    q.cache.k[page, 0] = codes
    q.cache.k_scale[page, 0] = torch.from_numpy(ahead / (127 * dim ** -0.5 * x.sum((1, 2)))).to(DEV).float()
    size = torch.zeros((q.n_blocks, 1))
    size[q.table[:, [2, 7, 14]].ravel().tolist()] = 1.0
    q.cache.v_scale *= size.to(DEV)
    run_small(q, lens, [1] * 160, 1, kernel, x)


@kernels
@pytest.mark.parametrize("dim,length,size", [(64, 5000, 1e-30), (64, 5000, 1e-33), (128, 5000, 1e-35), (256, 5000, 1e-35), (64, 200000, 1e-35)])
def test_small_values_of_many_tokens_alike(dim, length, size, kernel):
    # Outputs near bf16's smallest normal number, of a large sum of weights.
    q = positive(filled([length], 1, dim, 128, 45))
    q.cache.v_scale *= size
    run_small(q, [length], [2], 1, kernel, queries(np.random.default_rng(46), 2, 1, dim, BF16, spread=0.02))
