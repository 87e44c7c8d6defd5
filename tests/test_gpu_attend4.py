"""tf_kv4_attend on the GPU, with its own choice of the kernel and with each of the
two, against fp64 softmax attention over the values that the cache holds, within the
bound that serve_oracle.attend4 derives.  Whatever no sequence holds is NaN, infinite or
any other bits (serve_oracle.filled4)."""
import ctypes

import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import bf16
from tests.serve_oracle import DEV, Sequences4, attend4, filled4

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROWS, TILES = tf.TF_KV_BY_ROWS, tf.TF_KV_BY_TILES
kernels = pytest.mark.parametrize("kernel", [ROWS, TILES], ids=["rows", "tiles"])


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def queries(rng, rows, heads, dim, dtype, spread=1.0):
    x = rng.standard_normal((rows, heads, dim)) * spread * np.exp(rng.standard_normal((rows, heads, 1)))
    return bf16(x) if dtype == BF16 else x.astype(np.float32)


def run(q, lens, rows, heads, dtype=BF16, causal=True, window=0, scale=None, seed=0, pad=0, shift=0, x=None, kernel=0):
    """Attends and checks every row; the worst error over its bound."""
    total = sum(rows)
    x = queries(np.random.default_rng(seed), total, heads, q.d, dtype) if x is None else x
    width = heads * q.d
    m = torch.zeros(total * (width + pad) + shift, dtype=dtype, device=DEV)[shift:].view(total, width + pad)[:, :width]
    m.copy_(torch.from_numpy(x.reshape(total, width)).to(DEV))
    o = torch.full((total * (width + pad) + shift,), 3.0, dtype=BF16, device=DEV)[shift:].view(total, width + pad)
    q.cache.attend(m, q.batch(lens, rows), out=o[:, :width], scale=scale, causal=causal, window=window, kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(o[:, width:] == 3.0)
    got = o[:, :width].float().cpu().numpy().reshape(total, heads, q.d).astype(np.float64)
    at, worst = 0, 0.0
    for s, (n, r) in enumerate(zip(lens, rows)):
        if r:
            want, bound = attend4(x[at:at + r], *q.stored(s, n), q.d ** -0.5 if scale is None else scale, causal, window, dtype == F32)
            err = np.abs(got[at:at + r] - want) / np.where(bound == 0, 1e-30, bound)
            assert np.all(np.isfinite(err)) and err.max() <= 1, "sequence %d: %.3f of the bound" % (s, err.max())
            worst = max(worst, err.max())
        at += r
    return worst


@kernels
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv_heads,dim,block", [
    (8, 8, 64, 16), (32, 8, 128, 64), (16, 2, 256, 64), (12, 1, 64, 32), (7, 1, 128, 16), (6, 2, 256, 128), (40, 2, 64, 128), (4, 1, 256, 16)])
def test_single_tokens(heads, kv_heads, dim, block, dtype, kernel):
    lens = [1, 15, 16, 17, block, 2 * block + 3, 700]
    q = filled4(lens, kv_heads, dim, block, heads + dim)
    run(q, lens, [1] * len(lens), heads, dtype, kernel=kernel)


@kernels
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 20), (True, 300)])
@pytest.mark.parametrize("heads,kv_heads,dim,block", [(8, 2, 64, 16), (4, 1, 128, 16), (8, 1, 256, 32), (8, 2, 128, 64)])
def test_several_tokens(heads, kv_heads, dim, block, causal, window, kernel):
    lens, rows = [5, 33, 400, 129, 1000], [5, 1, 3, 17, 8]
    q = filled4(lens, kv_heads, dim, block, 3)
    run(q, lens, rows, heads, causal=causal, window=window, kernel=kernel)


@kernels
@pytest.mark.parametrize("heads,kv_heads,dim,block", [(8, 2, 64, 16), (4, 1, 128, 64), (16, 2, 256, 32), (9, 3, 128, 128), (5, 5, 64, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
def test_prompts(heads, kv_heads, dim, block, causal, window, kernel):
    lens, rows = [190, 300, 129, 257], [190, 65, 128, 0]
    q = filled4(lens, kv_heads, dim, block, 4)
    run(q, lens, rows, heads, causal=causal, window=window, kernel=kernel)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_prompt(dim, dtype):
    lens, rows = [1500, 900], [1500, 333]
    run(filled4(lens, 1, dim, 64, 5), lens, rows, 2, dtype)


@pytest.mark.parametrize("rows", [1, 40])
def test_long_sequence(rows):
    lens = [20011, 3]
    q = filled4(lens, 2, 128, 64, 6)
    run(q, lens, [rows, 3], 4)
    run(q, lens, [rows, 3], 4, window=9001)


@kernels
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_long_sequence_in_many_parts(dim, kernel):
    run(filled4([40000], 1, dim, 128, 21), [40000], [5], 3, kernel=kernel)


@kernels
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (8, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("window", [0, 900])
def test_shares_that_end_anywhere(heads, kv_heads, dim, window, kernel):
    rng = np.random.default_rng(dim + window)
    lens = rng.integers(1, 2500, 24).tolist()
    rows = [int(min(n, rng.choice([0, 1, 3, 40, 300], p=[0.1, 0.3, 0.3, 0.2, 0.1]))) for n in lens]
    run(filled4(lens, kv_heads, dim, 64, 20), lens, rows, heads, window=window, kernel=kernel)


@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [[1, 1], [30, 2], [150, 90]])
def test_strides_and_alignment(dtype, pad, shift, rows):
    lens = [200, 90]
    run(filled4(lens, 2, 64, 32, 7), lens, rows, 4, dtype, pad=pad, shift=shift)


@kernels
@pytest.mark.parametrize("rows", [[4, 6, 2], [160, 200, 3]])
def test_rows_that_see_nothing(rows, kernel):
    # Sequences shorter than their rows: the rows before the first token, and a sequence of length 0, get zeros; rows behind
    # the last sequence stay as they are.
    lens = [2, 0, rows[2]]
    q = filled4([max(n, 1) for n in lens], 2, 64, 16, 8)
    m = torch.randn((sum(rows) + 3, 4 * 64), device=DEV).to(BF16)
    o = torch.full((sum(rows) + 3, 4 * 64), 5.0, dtype=BF16, device=DEV)
    b = q.batch(lens, rows)
    b.rows = b.c.rows = sum(rows) + 3
    q.cache.attend(m, b, out=o, kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(o[:rows[0] - 2] == 0) and torch.all(o[rows[0]:rows[0] + rows[1]] == 0) and torch.all(o[-3:] == 5.0)
    x = m.float().cpu().numpy().reshape(-1, 4, 64)
    want, bound = attend4(x[rows[0] - 2:rows[0]], *q.stored(0, 2), 0.125, True, 0, False)
    assert np.all(np.abs(o[rows[0] - 2:rows[0]].float().cpu().numpy().reshape(2, 4, 64) - want) <= bound)


@kernels
@pytest.mark.parametrize("rows", [2, 140])
def test_large_and_bad_queries_stay_in_their_rows(rows, kernel):
    lens = [300]
    q = filled4(lens, 1, 64, 16, 9)
    x = queries(np.random.default_rng(1), rows, 2, 64, F32, spread=300.0)
    x[0, 1] *= np.float32(1e-30)
    run(q, lens, [rows], 2, F32, x=x, kernel=kernel)
    clean = q.cache.attend(torch.from_numpy(x.reshape(rows, -1)).to(DEV), q.batch(lens, [rows]), kernel=kernel)
    for bad in (np.nan, np.inf, -np.inf):
        y = x.copy()
        y[1, 0, 7] = bad
        got = q.cache.attend(torch.from_numpy(y.reshape(rows, -1)).to(DEV), q.batch(lens, [rows]), kernel=kernel)
        assert torch.all(torch.isnan(got[1, :64]))
        got[1, :64] = clean[1, :64]
        assert torch.equal(got, clean)


@kernels
@pytest.mark.parametrize("rows", [1, 150])
def test_scales_far_apart(rows, kernel):
    # Values over 12 decades from block to block, groups of one value only (scale 0) and of zeros among them.
    lens = [330]
    q = filled4(lens, 2, 64, 16, 10)
    n = q.n_blocks
    q.cache.v_affine *= (10.0 ** torch.linspace(-6, 3, n, device=DEV)).view(n, 1, 1, 1, 1).to(BF16)
    pages = torch.from_numpy(q.table[0]).to(DEV).long()
    q.cache.v_affine[pages[2], :, 3:9, :, 0] = 0
    q.cache.v_affine[pages[4]] = 0
    q.cache.k_affine[pages[5], :, ::2, :, 0] = 0
    q.cache.k_affine[pages[7]] = 0
    run(q, lens, [rows], 4, kernel=kernel)


@kernels
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_values_of_any_size(size, kernel):
    # The values' range is that of bf16 scales (the outputs' too), the keys' is made up for by the scale of scores.
    lens, rows = [200, 70], [3, 1]
    q = filled4(lens, 2, 128, 32, 22)
    held = torch.zeros(q.n_blocks * 32, dtype=torch.bool, device=DEV)
    held[q.slots([(0, n) for n in lens])] = True
    held = held.view(-1, 1, 32, 1, 1)
    for t in (q.cache.k_affine, q.cache.v_affine):
        t.copy_(torch.where(held, (t.float() * size).to(BF16), t))
    run(q, lens, rows, 4, scale=128 ** -0.5 / size, kernel=kernel)


@kernels
def test_a_token_far_above_the_others(kernel):
    lens = [4096]
    q = filled4(lens, 1, 64, 16, 11)
    x = queries(np.random.default_rng(2), 1, 1, 64, BF16)
    c, s, b = q.stored(0, 4096)[0]
    k = c[:, 0] * s[:, 0] + b[:, 0]
    x *= 300 / np.abs(k.astype(np.float64) @ x[0, 0]).max()
    run(q, lens, [1], 1, x=bf16(x), scale=1.0, kernel=kernel)


@kernels
@pytest.mark.parametrize("top", [1e3, 1e6])
def test_large_scores(top, kernel):
    # Scores far past what an exponent's fused sum could hold: told apart as well as fp32 scores can be.
    lens = [700]
    q = filled4(lens, 1, 128, 16, 23)
    x = queries(np.random.default_rng(3), 40, 2, 128, BF16)
    c, s, b = q.stored(0, 700)[0]
    k = (c[:, 0].reshape(700, 2, 64) * s[:, 0, :, None] + b[:, 0, :, None]).reshape(700, 128).astype(np.float64)
    size = np.abs(x.reshape(-1, 128) @ k.T).max(1).reshape(40, 2, 1)
    got = run_large(q, bf16(x * top / size), kernel)
    assert np.all(np.isfinite(got))


def run_large(q, x, kernel):
    """Where a row's largest score is ahead of the next by more than the bound of its error, the output is that token's value."""
    n, heads = x.shape[:2]
    m = torch.from_numpy(x.reshape(n, -1)).to(DEV).to(BF16)
    got = q.cache.attend(m, q.batch([700], [n]), scale=1.0, causal=False, kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    got = got.float().cpu().numpy().reshape(n, heads, 128)
    (kc, ks, kb), (vc, vs, vb) = q.stored(0, 700)
    wide = lambda t: np.repeat(t[:, 0].astype(np.float64), 64, axis=1)   # noqa: E731
    k, v = wide(ks) * kc[:, 0] + wide(kb), wide(vs) * vc[:, 0] + wide(vb)
    k_size = wide(ks) * kc[:, 0] + np.abs(wide(kb))
    sure = 0
    for i in range(n):
        for h in range(heads):
            s, err = k @ x[i, h].astype(np.float64), k_size @ np.abs(x[i, h]) * (2.0 ** -11 + 128 * 2.0 ** -23)
            order = np.argsort(-s)
            if s[order[0]] - err[order[0]] > np.max((s + err)[order[1:]]) + 40:
                sure += 1
                # (2^-11 of the value and its bias in the second product, 2^-11 of the value as fp16, 2^-8 of the result)
                far = 2.0 ** -11 * (np.abs(v) + 2 * np.abs(wide(vb)) + 15 * wide(vs))[order[0]] + 2.0 ** -8 * np.abs(v[order[0]]) + \
                    2.0 ** -20 * np.abs(v).max()
                assert np.all(np.abs(got[i, h] - v[order[0]]) <= far)
    assert sure > 0
    return got


def test_batch_of_many(seqs=150):
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 500, seqs).tolist()
    rows = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    run(filled4(lens, 2, 64, 32, 12), lens, rows, 8)


@pytest.mark.parametrize("rows", [1, 200])
def test_offsets_past_32_bits(rows):
    q = Sequences4([300], 8, 128, 64, BF16, 13, n_blocks=140000)
    assert q.cache.k.numel() > 1 << 32
    q.append([(0, 300)])
    run(q, [300], [rows], 8)


@pytest.mark.parametrize("rows", [1, 200])
def test_numbers_that_do_not_fit_are_reported(rows):
    lens = [300, 300]
    q = filled4(lens, 2, 64, 16, 14)
    x = torch.randn((2 * rows, 256), device=DEV).to(BF16)
    ok = q.cache.attend(x, q.batch(lens, [rows, rows]))
    for wrong in ("page", "length", "starts"):
        b = q.batch(lens, [rows, rows])
        if wrong == "page":
            b._keep[1][0, 3] = -5
        elif wrong == "length":
            b._keep[0][0] = 301
        else:
            b._keep[2][0] = -2 ** 31
        got = q.cache.attend(x, b)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
        assert torch.equal(got[rows:], ok[rows:])
        if wrong == "length":
            assert torch.all(got[:rows] == 0)
        elif wrong == "page":
            assert torch.all(torch.isfinite(got))


@kernels
def test_pages_before_the_window_may_be_gone(kernel):
    # A window's sequence whose earlier pages have been given away (or left out of the table): the same bits.
    lens, rows, window = [1000], [5], 100
    q = filled4(lens, 2, 64, 16, 15)
    x = torch.randn((5, 256), device=DEV).to(BF16)
    want = q.cache.attend(x, q.batch(lens, rows), window=window, kernel=kernel).clone()
    gone = torch.from_numpy(q.table[0, :(1000 - 5 - window + 1) // 16]).to(DEV).long()
    for t in (q.cache.k_affine, q.cache.v_affine):
        t[gone] = float("nan")
    assert torch.equal(q.cache.attend(x, q.batch(lens, rows), window=window, kernel=kernel), want)
    tf.tf_device_status()


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_again_and_on_other_streams(rows):
    # The same bits on every call, whatever ran before (another shape, the 8-bit cache's attention, another stream).
    from tests.test_gpu_attend import filled
    lens = [3000, 700]
    q, other = filled4(lens, 2, 128, 64, 16), filled(lens, 2, 128, 64, 16)
    x = torch.randn((2 * rows, 4 * 128), device=DEV).to(BF16)
    b = q.batch(lens, [rows, rows])
    first = q.cache.attend(x, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        q.cache.attend(x[:1], q.batch([77], [1], seqs=[0]))
        other.cache.attend(x, other.batch(lens, [rows, rows]))
        assert torch.equal(q.cache.attend(x, b), first)
        out = torch.empty_like(first)
        q.cache.attend(x, b, out=out, stream=side)
        side.synchronize()
        assert torch.equal(out, first)
    tf.tf_device_status()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_graphs_of_both_caches_on_one_stream(dim):
    # They share the stream's workspace: replays after one another, in any order, and after larger calls.
    from tests.test_gpu_attend import filled
    lens = [3000, 700]
    q, other = filled4(lens, 2, dim, 64, 30), filled(lens, 2, dim, 64, 31)
    with torch.cuda.stream(torch.cuda.Stream()):
        x = torch.randn((2, 4 * dim), device=DEV).to(BF16)
        steps = []
        for s in (q, other):
            b, out = s.batch(lens, [1, 1]), torch.zeros_like(x)
            want = s.cache.attend(x, b).clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.current_stream()):
                s.cache.attend(x, b, out=out)
            steps.append((graph, out, want, b))          # (the graph reads the batch's tensors)
        long = torch.randn((900, 4 * dim), device=DEV).to(BF16)
        for kernel in (ROWS, TILES):
            q.cache.attend(long, q.batch(lens, [600, 300]), kernel=kernel)
        for i in (0, 1, 1, 0, 0, 1):
            graph, out, want = steps[i][:3]
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        tf.tf_device_status()


def test_a_first_call_inside_a_capture_is_refused():
    q = filled4([300], 2, 64, 16, 33)
    x = torch.randn((1, 256), device=DEV).to(BF16)
    b, out = q.batch([300], [1]), torch.zeros((1, 256), dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    handle = ctypes.c_void_p(0)
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.ExternalStream(handle.value)):
        out.fill_(2.0)
        with pytest.raises(tf.TfError) as e:
            q.cache.attend(x, b, out=out)
        assert e.value.rc == -10
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(out == 2.0)


@kernels
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 20), (256, 5)])
def test_correct_again_after_a_wait_ran_out(kernel, dim, rows):
    rng = np.random.default_rng(dim + rows)
    lens = rng.integers(rows, 2500, 60).tolist()
    q = filled4(lens, 4, dim, 64, 40)
    b = q.batch(lens, [rows] * 60)
    x = torch.randn((60 * rows, 8 * dim), device=DEV).to(BF16)
    want = q.cache.attend(x, b, kernel=kernel).clone()
    torch.cuda.synchronize()
    tf.tf_device_status()
    tf.tf_inject_stall()
    q.cache.attend(x, b, kernel=kernel)
    torch.cuda.synchronize()
    with pytest.raises(tf.TfError) as e:
        tf.tf_device_status()
    assert e.value.rc == -11
    for _ in range(2):
        assert torch.equal(q.cache.attend(x, b, kernel=kernel), want)
    tf.tf_device_status()


@pytest.mark.parametrize("rows", [[6, 1, 9], [160, 2, 300]])
def test_windows_of_any_size(rows):
    lens = [2, 300, 7]
    q = filled4(lens, 2, 64, 16, 17)
    x = torch.randn((sum(rows), 256), device=DEV).to(BF16)
    b = q.batch(lens, rows)
    want = q.cache.attend(x, b)
    for window in (300, 301, 1 << 20, 2 ** 31 - 300, 2 ** 31 - 1):
        assert torch.equal(q.cache.attend(x, b, window=window), want), window
    torch.cuda.synchronize()
    tf.tf_device_status()


def run_small(q, lens, rows, heads, kernel, by=100, x=None, scale=None):
    """run(), against the same values times 2^by: the outputs are checked relative to what they are made of alone.  (What a
    bf16 output below 2^-126 rounds to is half of 2^-133 off at most, and a weight that fp32 holds no more is below 2^-126.)"""
    x = queries(np.random.default_rng(0), sum(rows), heads, q.d, BF16) if x is None else x
    got = q.cache.attend(torch.from_numpy(x.reshape(sum(rows), -1)).to(DEV).to(BF16), q.batch(lens, rows), scale=scale, kernel=kernel)
    torch.cuda.synchronize()
    tf.tf_device_status()
    got = got.double().cpu().numpy().reshape(sum(rows), heads, q.d) * 2.0 ** by
    at = 0
    for s, (n, r) in enumerate(zip(lens, rows)):
        k, (c, vs, vb) = q.stored(s, n)
        up = [t.astype(np.float64) * 2.0 ** by for t in (vs, vb)]
        want, bound = attend4(x[at:at + r], k, (c, *up), q.d ** -0.5 if scale is None else scale, True, 0, False)
        bound += 2.0 ** (by - 134) + n * 2.0 ** -126 * max(15 * np.abs(up[0]).max(), np.abs(up[1]).max())
        err = np.abs(got[at:at + r] - want) / bound
        assert np.all(np.isfinite(err)) and err.max() <= 1, "sequence %d: %.3f of the bound" % (s, err.max())
        at += r


def shrink_values(q, lens, size):
    """The held tokens' values times `size`, a number or one for each page of the pool; none below 0, so that what a token
    adds is not made up for by others."""
    held = torch.zeros(q.n_blocks * q.b, dtype=torch.bool, device=DEV)
    held[q.slots([(0, n) for n in lens])] = True
    size = torch.as_tensor(size, dtype=torch.float32, device=DEV).reshape(-1, 1, 1, 1, 1)
    t = q.cache.v_affine
    t.copy_(torch.where(held.view(-1, 1, q.b, 1, 1), (t.float().abs() * size).to(BF16), t))


@kernels
@pytest.mark.parametrize("size", [1e-28, 1e-30, 1e-31, 1e-33])
@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(4, 2, 64, [3, 1]), (8, 2, 128, [1, 2]), (2, 1, 256, [4, 6])])
def test_small_values(heads, kv_heads, dim, rows, size, kernel):
    lens = [200, 70]
    q = filled4(lens, kv_heads, dim, 32, 41)
    shrink_values(q, lens, size)
    run_small(q, lens, rows, heads, kernel)


@kernels
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_small_values_of_many_sizes(dim, kernel):
    # Tokens of different steps, warps and parts on both sides of 2^-97, each of which counts.
    lens = [9000]
    q = filled4(lens, 1, dim, 64, 42)
    shrink_values(q, lens, 2.0 ** torch.linspace(-101, -94, q.n_blocks)[torch.randperm(q.n_blocks, generator=torch.Generator().manual_seed(1))])
    run_small(q, lens, [3], 3, kernel)


@kernels
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ahead", [60.0, 74.0])
def test_the_largest_scores_belong_to_zeros(dim, ahead, kernel):
    # All pages hold zeros but three, whose tokens' scores lie `ahead` below the largest.  So many sequences that a CTA takes
    # several steps of one; by rows, a warp that takes token 101 takes some of the others, too.
    lens = [333] * 160
    q = filled4(lens, 1, dim, 16, 43)
    x = np.abs(queries(np.random.default_rng(44), 160, 1, dim, BF16))
    q.cache.k_affine *= 0.01
    page = torch.from_numpy(q.table[:, 6]).to(DEV).long()
    q.cache.k_affine[page, 0, 5, :, 0] = 0
    q.cache.k_affine[page, 0, 5, :, 1] = torch.from_numpy(ahead / (dim ** -0.5 * x.sum((1, 2)))).to(DEV).to(BF16)[:, None]
    size = torch.zeros(q.n_blocks)
    size[q.table[:, [2, 7, 14]].ravel().tolist()] = 1.0
    shrink_values(q, lens, size)
    run_small(q, lens, [1] * 160, 1, kernel, x=x)


@kernels
@pytest.mark.parametrize("dim,length,size", [(64, 5000, 1e-33), (128, 5000, 1e-36), (256, 5000, 1e-36), (64, 200000, 1e-36)])
def test_small_values_of_many_tokens_alike(dim, length, size, kernel):
    # Outputs near bf16's smallest normal number, of a large sum of weights.
    q = filled4([length], 1, dim, 128, 45)
    shrink_values(q, [length], size)
    run_small(q, [length], [2], 1, kernel, x=queries(np.random.default_rng(46), 2, 1, dim, BF16, spread=0.02))
