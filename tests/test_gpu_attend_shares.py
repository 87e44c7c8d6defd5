"""Attention by tiles where the beginning of a CTA's share is found by any lane of its first warp, which
then takes the CTA's tensor memory as a whole: one lane has searched, the others have waited."""
import numpy as np
import pytest

import mlx_affine_bit_gb300 as tf
from tests import test_gpu_attend, test_gpu_attend4

pytestmark = pytest.mark.gpu
TILES = tf.TF_KV_BY_TILES


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("seqs,dim", [(1, 128), (7, 64), (33, 256), (700, 64)])
def test_shares_that_any_lane_finds(seqs, dim, bits, monkeypatch):
    # 512 threads look through the sequences and their tiles: of 700 sequences a thread of the first warp has two, of fewer one or
    # none.  Lengths and rows differ, so that the lanes' loops do, too.
    rng = np.random.default_rng(seqs)
    lens = rng.integers(1, 300, seqs).tolist()
    rows = [int(min(n, rng.integers(0, 200))) for n in lens]
    rows[0] = max(rows[0], 1)
    if bits == 4:
        test_gpu_attend4.run(test_gpu_attend4.filled4(lens, 1, dim, 16, 50), lens, rows, 2, kernel=TILES)
    else:
        attend = tf.KvCache.attend
        monkeypatch.setattr(tf.KvCache, "attend", lambda self, *a, **k: attend(self, *a, kernel=TILES, **k))
        test_gpu_attend.run(test_gpu_attend.filled(lens, 1, dim, 16, 50), lens, rows, 2)
