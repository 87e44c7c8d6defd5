"""tf_kv_attend on the GPU against fp64 softmax attention over the values that the
cache holds, within the bound that decode_oracle.attend derives."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV, Sequences, attend, bf16

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def queries(rng, rows, heads, dim, dtype, spread=2.0):
    x = rng.standard_normal((rows, heads, dim)) * spread * np.exp(rng.standard_normal((rows, heads, 1)))
    return bf16(x) if dtype == BF16 else x.astype(np.float32)


def filled(lens, kv_heads, dim, block, seed):
    """A cache with random pages (any codes past a sequence's end)."""
    q = Sequences(lens, kv_heads, dim, block, BF16, seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    for pool, scale in ((q.cache.k, q.cache.k_scale), (q.cache.v, q.cache.v_scale)):
        pool.copy_(torch.randint(-128, 128, pool.shape, generator=gen, device=DEV, dtype=torch.int8))
        scale.copy_(torch.exp(torch.randn(scale.shape, generator=gen, device=DEV)) * 0.01)
    return q


def run(q, lens, rows, heads, dtype=BF16, causal=True, window=0, scale=None, seed=0, pad=0, shift=0, x=None):
    """Attends and checks every row; the worst error over its bound."""
    rng = np.random.default_rng(seed)
    total = sum(rows)
    x = queries(rng, total, heads, q.d, dtype) if x is None else x
    width = heads * q.d
    m = torch.zeros(total * (width + pad) + shift, dtype=dtype, device=DEV)[shift:].view(total, width + pad)[:, :width]
    m.copy_(torch.from_numpy(x.reshape(total, width)).to(DEV))
    o = torch.full((total * (width + pad) + shift,), 3.0, dtype=BF16, device=DEV)[shift:].view(total, width + pad)
    q.cache.attend(m, q.batch(lens, rows), out=o[:, :width], scale=scale, causal=causal, window=window)
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(o[:, width:] == 3.0)
    got = o[:, :width].float().cpu().numpy().reshape(total, heads, q.d).astype(np.float64)
    at, worst = 0, 0.0
    for s, (n, r) in enumerate(zip(lens, rows)):
        if r:
            k, v = q.values(s, n)
            want, bound = attend(x[at:at + r], k, v, q.value_scales(s, n), q.d ** -0.5 if scale is None else scale, r, causal, window,
                                 dtype == F32)
            err = np.abs(got[at:at + r] - want) / np.where(bound == 0, 1e-30, bound)
            assert np.all(np.isfinite(err)) and err.max() <= 1, "sequence %d: %.3f of the bound" % (s, err.max())
            worst = max(worst, err.max())
        at += r
    return worst


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv_heads,dim,block", [
    (8, 8, 64, 16), (32, 8, 128, 64), (16, 2, 256, 64), (12, 1, 64, 32), (7, 1, 128, 16), (6, 2, 256, 128), (40, 2, 64, 128)])
def test_single_tokens(heads, kv_heads, dim, block, dtype):
    lens = [1, 15, 16, 17, block, 2 * block + 3, 700]
    q = filled(lens, kv_heads, dim, block, heads + dim)
    run(q, lens, [1] * len(lens), heads, dtype)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 20), (True, 300)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (4, 1, 128), (8, 1, 256)])
def test_several_tokens(heads, kv_heads, dim, causal, window):
    lens, rows = [5, 33, 400, 129, 1000], [5, 1, 3, 17, 8]
    q = filled(lens, kv_heads, dim, 16, 3)
    run(q, lens, rows, heads, causal=causal, window=window)


@pytest.mark.parametrize("heads,kv_heads,dim,block", [(8, 2, 64, 16), (4, 1, 128, 64), (16, 2, 256, 32), (9, 3, 128, 128), (5, 5, 64, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
def test_prompts(heads, kv_heads, dim, block, causal, window):
    lens, rows = [190, 300, 129, 257], [190, 65, 128, 0]
    q = filled(lens, kv_heads, dim, block, 4)
    run(q, lens, rows, heads, causal=causal, window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_prompt(dtype):
    lens, rows = [1500, 900], [1500, 333]
    q = filled(lens, 1, 128, 64, 5)
    run(q, lens, rows, 2, dtype)


@pytest.mark.parametrize("rows", [1, 40])
def test_long_sequence(rows):
    lens = [20011, 3]
    q = filled(lens, 2, 128, 64, 6)
    run(q, lens, [rows, 3], 4)
    run(q, lens, [rows, 3], 4, window=9001)


@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [[1, 1], [30, 2], [150, 90]])
def test_strides_and_alignment(dtype, pad, shift, rows):
    lens = [200, 90]
    q = filled(lens, 2, 64, 32, 7)
    run(q, lens, rows, 4, dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("rows", [[4, 6, 2], [160, 200, 3]])
def test_rows_that_see_nothing(rows):
    # Sequences shorter than their rows: the rows before the first token, and a sequence of length 0, get zeros.
    lens = [2, 0, rows[2]]
    q = filled([max(n, 1) for n in lens], 2, 64, 16, 8)
    width = 4 * 64
    m = torch.randn((sum(rows), width), device=DEV).to(BF16)
    o = torch.full((sum(rows), width), 5.0, dtype=BF16, device=DEV)
    q.cache.attend(m, q.batch(lens, rows), out=o)
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(o[:rows[0] - 2] == 0) and torch.all(o[rows[0]:rows[0] + rows[1]] == 0)
    x = m.float().cpu().numpy().reshape(-1, 4, 64)
    k, v = q.values(0, 2)
    want, bound = attend(x[rows[0] - 2:rows[0]], k, v, q.value_scales(0, 2), 0.125, 2, True, 0, False)
    got = o[rows[0] - 2:rows[0]].float().cpu().numpy().reshape(2, 4, 64)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("rows", [2, 140])
def test_large_and_bad_queries_stay_in_their_rows(rows):
    # Scores of thousands, queries of 1e-30 and 1e30 (finite scores), NaN and infinities: the other rows keep theirs.
    lens = [300]
    q = filled(lens, 1, 64, 16, 9)
    rng = np.random.default_rng(1)
    x = queries(rng, rows, 2, 64, F32, spread=300.0)
    x[0, 1] *= np.float32(1e-30)
    run(q, lens, [rows], 2, F32, x=x)
    clean = q.cache.attend(torch.from_numpy(x.reshape(rows, -1)).to(DEV), q.batch(lens, [rows]))
    for bad in (np.nan, np.inf, -np.inf):
        y = x.copy()
        y[1, 0, 7] = bad
        got = q.cache.attend(torch.from_numpy(y.reshape(rows, -1)).to(DEV), q.batch(lens, [rows]))
        assert torch.all(torch.isnan(got[1, :64]))
        got[1, :64] = clean[1, :64]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("rows", [1, 150])
def test_scales_far_apart(rows):
    # Value scales over 12 decades, zero among them: blocks with small values count where their keys win.
    lens = [330]
    q = filled(lens, 2, 64, 16, 10)
    n = q.cache.v_scale.numel()
    q.cache.v_scale.view(-1)[:] = 10.0 ** torch.linspace(-6, 3, n, device=DEV)
    q.cache.v_scale[3] = 0
    q.cache.k_scale[5] = 0
    run(q, lens, [rows], 4)


def test_a_token_far_above_the_others():
    # One key wins by 2^60: its value comes out, however many others there are.
    lens = [4096]
    q = filled(lens, 1, 64, 16, 11)
    x = queries(np.random.default_rng(2), 1, 1, 64, BF16)
    k, v = q.values(0, 4096)
    x *= 300 / np.abs(k[:, 0].astype(np.float64) @ x[0, 0]).max()
    run(q, lens, [1], 1, x=bf16(x), scale=1.0)


def test_batch_of_many(seqs=150):
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 500, seqs).tolist()
    rows = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    q = filled(lens, 2, 64, 32, 12)
    run(q, lens, rows, 8)


@pytest.mark.parametrize("rows", [1, 200])
def test_offsets_past_32_bits(rows):
    q = Sequences([300], 8, 128, 64, BF16, 13, n_blocks=73000)
    assert q.cache.k.numel() > 1 << 32
    q.append([(0, 300)])
    run(q, [300], [rows], 8)


@pytest.mark.parametrize("rows", [1, 200])
def test_numbers_that_do_not_fit_are_reported(rows):
    lens = [300, 300]
    q = filled(lens, 2, 64, 16, 14)
    x = torch.randn((2 * rows, 256), device=DEV).to(BF16)
    ok = q.cache.attend(x, q.batch(lens, [rows, rows]))
    for wrong in ("page", "length"):
        b = q.batch(lens, [rows, rows])
        if wrong == "page":
            b._keep[1][0, 3] = -5
        else:
            b._keep[0][0] = 301
        got = q.cache.attend(x, b)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
        assert torch.equal(got[rows:], ok[rows:])
        if wrong == "length":
            assert torch.all(got[:rows] == 0)
        else:
            assert torch.all(torch.isfinite(got))


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_again_and_on_other_streams(rows):
    # The same bits on every call, whatever ran before (another shape, another stream).
    lens = [3000, 700]
    q = filled(lens, 2, 128, 64, 15)
    x = torch.randn((2 * rows, 4 * 128), device=DEV).to(BF16)
    b = q.batch(lens, [rows, rows])
    first = q.cache.attend(x, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        q.cache.attend(x[:1], q.batch([77], [1], seqs=[0]))
        assert torch.equal(q.cache.attend(x, b), first)
        out = torch.empty_like(first)
        q.cache.attend(x, b, out=out, stream=side)
        side.synchronize()
        assert torch.equal(out, first)


def test_captured_decode_step():
    # append + attend in a CUDA graph, replayed with lengths that move on the device.
    q = Sequences([90, 40], 2, 64, 16, BF16, 16)
    q.append([(0, 60), (0, 10)])
    i32 = dict(dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([60, 10], **i32)
    b = tf.KvBatch(kv_len, torch.from_numpy(q.table).to(DEV), 90)
    k, v = (torch.zeros((2, 128), dtype=BF16, device=DEV) for _ in range(2))
    x = torch.zeros((2, 256), dtype=BF16, device=DEV)
    out = torch.zeros((2, 256), dtype=BF16, device=DEV)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q.cache.attend(x, b, out=out)           # the stream's workspace, before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kv_len.add_(1)
            q.cache.append(k, v, b)
            q.cache.attend(x, b, out=out)
    rng = np.random.default_rng(4)
    for i in range(30):
        for s, n in enumerate((60 + i, 10 + i)):
            k[s] = torch.from_numpy(q.k[s][n].reshape(-1)).to(DEV)
            v[s] = torch.from_numpy(q.v[s][n].reshape(-1)).to(DEV)
        xs = queries(rng, 2, 4, 64, BF16)
        x.copy_(torch.from_numpy(xs.reshape(2, -1)))
        graph.replay()
        torch.cuda.synchronize()
        got = out.float().cpu().numpy().reshape(2, 4, 64)
        for s, n in enumerate((61 + i, 11 + i)):
            kk, vv = q.values(s, n)
            want, bound = attend(xs[s:s + 1], kk, vv, q.value_scales(s, n), 0.125, 1, True, 0, False)
            assert np.all(np.abs(got[s] - want[0]) <= bound[0])
    tf.tf_device_status()
    q.check(0, 90)
    q.check(1, 40)


@pytest.mark.parametrize("rows", [[6, 1, 9], [160, 2, 300]])
def test_windows_of_any_size(rows):
    # As large as a window can be given: every token is seen, also by sequences that have fewer tokens than rows.
    lens = [2, 300, 7]
    q = filled(lens, 2, 64, 16, 17)
    x = torch.randn((sum(rows), 256), device=DEV).to(BF16)
    b = q.batch(lens, rows)
    want = q.cache.attend(x, b)
    for window in (300, 301, 1 << 20, 2 ** 31 - 300, 2 ** 31 - 2, 2 ** 31 - 1):
        assert torch.equal(q.cache.attend(x, b, window=window), want), window
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(torch.any(want[rows[0] - 2:rows[0]] != 0, dim=1))
