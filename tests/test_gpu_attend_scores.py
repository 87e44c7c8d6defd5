"""tf_kv_attend where scores are large: fp32 holds scores of 10^6 to a sixteenth of a
power of two only, and what it holds has to be all that is lost.

The rows tested are those that one key wins by far more than that, or several exactly
alike (pages with the same keys and key scale, other values): their result is the mean of
the winners' values.  Its bound: the rounding to bf16 (2^-8), the weights' to fp16
(2^-11), and 2^-10 for the exponents, whose sums of terms up to 2^13 (where the scores
are below 2^12; larger ones are subtracted from one another first) are rounded to 2^-11
of a power of two at most, in the weight and in the sum; and what the others add, e^-40
of a value each."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV, bf16
from tests.test_gpu_attend import filled

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def winners(q, x, n, heads, scale, causal):
    """Per row and head: (the mean of the winners' values, its bound), NaN where tokens near the winner leave it open."""
    kc, ks, vc, vs = q.stored(0, n)
    per = lambda s: np.repeat(s, q.b, axis=0)[:n].astype(np.float64)          # noqa: E731
    ks, v = per(ks), vc.astype(np.float64) * per(vs)[:, :, None]
    rows, g = x.shape[0], heads // q.h
    want, bound = np.full((rows, heads, q.d), np.nan), np.full((rows, heads, q.d), np.nan)
    for h in range(heads):
        k, qq = kc[:, h // g].astype(np.float64), x[:, h].astype(np.float64)
        raw = qq @ k.T                                   # (exact: few bits, sums below 2^53 of their last)
        s = raw * ks[:, h // g] * scale
        mag = (np.abs(qq) @ np.abs(k).T) * ks[:, h // g] * abs(scale) + np.abs(qq).sum(1)[:, None] * 128 * ks[:, h // g] * abs(scale)
        for i in range(rows):
            seen = n - rows + i + 1 if causal else n
            top = s[i, :seen].max()
            at = np.nonzero(s[i, :seen] == top)[0]
            # Rounding of a score: dim products in fp32 sums, and its scaling.
            err = mag[i, :seen].max() * q.d * 2.0 ** -23 + abs(top) * 2.0 ** -21
            rest = np.delete(s[i, :seen], at)
            if rest.size and rest.max() > top - 2 * err - 40:
                continue
            want[i, h] = v[at, h // g].mean(0)
            bound[i, h] = 2.0 ** -8 * np.abs(want[i, h]) + (1.01 * 2.0 ** -11 + 2.0 ** -10) * np.abs(v[at, h // g]).mean(0) + \
                n * np.exp(-40) * np.abs(v[:seen, h // g]).max()
    return want, bound


@pytest.mark.parametrize("kernel", [tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("size", [2e3, 1e4, 3e5, 2e6, 3e7, 1e30])
@pytest.mark.parametrize("rows,causal,scale,n", [(1, True, 1.0, 700), (5, False, -1.0, 646), (150, True, 0.125, 700), (140, False, 1.0, 775)])
def test_winning_keys(kernel, dim, block, size, rows, causal, scale, n):
    heads = 4
    q = filled([n], 2, dim, block, 50 + dim)
    pages = torch.from_numpy(q.table[0].astype(np.int64)).to(DEV)
    # Some pages hold the same keys with the same scale.
    for a, b in ((1, 3), (1, 8), (4, 9)):
        q.cache.k[pages[b]] = q.cache.k[pages[a]]
        q.cache.k_scale[pages[b]] = q.cache.k_scale[pages[a]]
    rng = np.random.default_rng(dim + rows)
    x = rng.integers(-128, 129, (rows, heads, dim)).astype(np.float64)        # (bf16's bits: any sum of products is exact)
    kc, ks, _, _ = q.stored(0, n)
    k = kc.astype(np.float64) * np.repeat(ks, block, axis=0)[:n, :, None].astype(np.float64)
    for h in range(heads):                                # the largest score of each row: about `size`
        top = np.abs(x[:, h] @ k[:, h // 2].T * scale).max(1)
        x[:, h] *= 2.0 ** np.round(np.log2(size / top))[:, None]
    x = bf16(x)
    m = torch.from_numpy(x.reshape(rows, -1)).to(DEV).to(BF16)
    got = q.cache.attend(m, q.batch([n], [rows]), scale=scale, causal=causal, kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    got = got.float().cpu().numpy().reshape(x.shape).astype(np.float64)
    want, bound = winners(q, x, n, heads, scale, causal)
    sure = ~np.isnan(want[:, :, 0])
    assert sure.mean() > 0.25 and np.all(np.isfinite(got))
    off = np.abs(got - want)[sure] / bound[sure]
    assert off.max() <= 1, "%.2f of the bound" % off.max()
    # What a row gives stays within the values that it sees.
    assert np.all(np.abs(got) <= 1.01 * np.abs(q.values(0, n)[1]).max())


@pytest.mark.parametrize("kernel", [tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES], ids=["rows", "tiles"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("spread", [30.0, 1000.0, 30000.0])
def test_scores_that_grow_along_a_sequence(kernel, dim, spread):
    # Key scales over six decades: small scores, then large ones, in one row and step; cut between CTAs anywhere, with and
    # without a window, sequences that end within a few tokens of a step.
    from tests.test_gpu_attend import queries, run
    lens, rows = [1300, 129, 400, 2570, 641], [200, 3, 130, 5, 60]
    q = filled(lens, 2, dim, 16, 60 + dim)
    gen = torch.Generator(device=DEV).manual_seed(dim)
    q.cache.k_scale.copy_(10.0 ** (torch.rand(q.cache.k_scale.shape, generator=gen, device=DEV) * 6 - 6))
    q.cache.k_scale[::7] = 0
    x = queries(np.random.default_rng(dim), sum(rows), 4, dim, BF16, spread)
    attend = tf.KvCache.attend
    for window in (0, 300):
        with pytest.MonkeyPatch.context() as mp:
            mp.setattr(tf.KvCache, "attend", lambda self, *a, **k: attend(self, *a, kernel=kernel, **k))
            run(q, lens, rows, 4, x=x, window=window)
