"""The 8-bit cache on the GPU: what tf_kv_append holds is, code for code, the
header's fp32 arithmetic on each page's tokens, however calls cut a sequence."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV, Sequences, bf16, cache_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def status_clean():
    torch.cuda.synchronize()
    tf.tf_device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,dim,heads", [(16, 64, 3), (32, 128, 2), (64, 256, 1), (128, 256, 2), (128, 64, 1), (64, 128, 8)])
def test_whole_prompts(dtype, block, dim, heads):
    lens = [1, block - 1, block, block + 1, 3 * block + 5, 0]
    q = Sequences(lens, heads, dim, block, dtype, 1)
    q.append([(0, n) for n in lens])
    status_clean()
    for s, n in enumerate(lens):
        if n:
            q.check(s, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,dim", [(16, 64), (32, 256), (64, 128)])
def test_any_cut_gives_the_same_cache(dtype, block, dim):
    # Token by token, in random pieces (from one token to several pages) and at once.
    n = 5 * block + 3
    rng = np.random.default_rng(block)
    q = Sequences([n, n, n], 2, dim, block, dtype, 2)
    for a in (q.k, q.v):
        a[1][:] = a[0]
        a[2][:] = a[0]
    for i in range(n):
        q.append([(i, i + 1)], seqs=[0])
    at = 0
    while at < n:
        step = int(rng.choice([1, 2, block // 2, block, 2 * block + 1, 3 * block]))
        q.append([(at, min(n, at + step))], seqs=[1])
        at = min(n, at + step)
    q.append([(0, n)], seqs=[2])
    status_clean()
    for s in range(3):
        q.check(s, n)
    # The open rings hold the last two pages' originals, whatever the cut.
    first = (n - 1) // block * block - block
    for ring, x in ((q.cache.open_k, q.k[0]), (q.cache.open_v, q.v[0])):
        for p in range(first, n):
            want = torch.from_numpy(x[p]).to(DEV).to(dtype)
            for s in range(3):
                assert torch.equal(ring[s, :, p % (2 * block)], want)


@pytest.mark.parametrize("start", [1, 7, 15])
@pytest.mark.parametrize("more", [16, 17, 31, 32, 33, 48, 49, 50, 80])
def test_begun_page_then_a_long_call(start, more):
    # The long call's last pages go where the begun page's originals are; the page's scale grows with the call.
    q = Sequences([start + more], 2, 64, 16, BF16, 3)
    for a in (q.k, q.v):
        a[0][start:] *= 8
    q.append([(0, start)])
    q.append([(start, start + more)])
    q.append([(start + more - 1, start + more)])      # and the last token once more
    status_clean()
    q.check(0, start + more)


def test_rewound_tokens_leave_no_trace():
    # Rejected drafts (large ones, over a page's end) are written over; up to a page back.
    block, n = 16, 60
    q = Sequences([n], 2, 64, block, BF16, 4)
    good = [a[0].copy() for a in (q.k, q.v)]
    at = 0
    rng = np.random.default_rng(5)
    while at < n:
        draft = min(n, at + int(rng.integers(1, block + 1)))
        for a in (q.k, q.v):
            a[0][at:draft] = bf16(100 * rng.standard_normal(a[0][at:draft].shape))
        q.append([(at, draft)])
        for a, g in zip((q.k, q.v), good):
            a[0][at:draft] = g[at:draft]
        take = int(rng.integers(1, draft - at + 1))
        q.append([(at, at + take)])
        at += take
    status_clean()
    q.check(0, n)


@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 3), (64, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(dtype, pad, shift):
    lens = [5, 37, 16]
    q = Sequences(lens, 3, 64, 16, dtype, 6)
    q.append([(0, n) for n in lens], pad, shift)
    for s, n in enumerate(lens):
        q.check(s, n)
    # Reading back into strided, unaligned rows leaves the gaps alone.
    b = q.batch(lens, lens)
    width = 3 * 64
    out = [torch.full((b.rows * (width + pad) + shift,), 7.0, dtype=F32, device=DEV)[shift:].view(b.rows, width + pad)
           for _ in range(2)]
    q.cache.read(b, k_out=out[0][:, :width], v_out=out[1][:, :width])
    status_clean()
    want = [np.concatenate(x).reshape(-1, width) for x in zip(*[q.values(s, n) for s, n in enumerate(lens)])]
    for o, x in zip(out, want):
        assert np.array_equal(o[:, :width].cpu().numpy(), x)
        assert torch.all(o[:, width:] == 7.0)


@pytest.mark.parametrize("block,dim", [(16, 64), (64, 128), (128, 256)])
def test_read_back_some(block, dim):
    lens, rows = [3 * block + 1, block, 2 * block - 1], [block + 9, 1, 0]
    q = Sequences(lens, 2, dim, block, F32, 7, slots=[4, 0, 2])
    q.append([(0, n) for n in lens])
    b = q.batch(lens, rows)
    want = [np.concatenate(x).reshape(-1, 2 * dim) for x in zip(*[[a[n - r:] for a in q.values(s, n)] for s, (n, r) in enumerate(zip(lens, rows))])]
    for got, x in zip(q.cache.read(b), want):
        assert np.array_equal(got.cpu().numpy(), x)
    for got, x in zip(q.cache.read(b, BF16), want):
        assert np.array_equal(got.float().cpu().numpy(), bf16(x))
    # Half a step is the most that a value moves (and fp32 rounding of scale and value).
    for x, c in ((q.k, 0), (q.v, 1)):
        for s, n in enumerate(lens):
            step = np.repeat(cache_of(x[s], block)[1], block, axis=0)[:n, :, None]
            assert np.all(np.abs(q.values(s, n)[c] - x[s]) <= step * (0.5 + 2.0 ** -15))
    status_clean()


def test_values_that_are_not_finite():
    q = Sequences([40], 2, 64, 16, BF16, 8)
    k, v = q.k[0], q.v[0]
    k[3, 0, 5], k[20, 1, 0], v[0, 0, 0], v[39, 1, 63] = np.nan, np.inf, -np.inf, np.nan
    k[16:32, 0] = 0                        # a page of zeros
    v[32:, 0] = 1e-40                      # subnormal
    v[32:, 1, :62] = 3e38                  # near the largest
    q.k[0], q.v[0] = bf16(k), bf16(v)
    q.append([(0, 40)])
    status_clean()
    q.check(0, 40)
    got = q.values(0, 40)
    assert all(np.all(np.isfinite(x)) for x in got)
    assert got[0][3, 0, 5] == 0 and np.all(got[0][16:32, 0] == 0)
    for i in range(40):                    # one token at a time: the same
        q.append([(i, i + 1)])
    q.check(0, 40)


def test_offsets_past_32_bits():
    # Pages at the end of pools of 4.8 GB each.
    q = Sequences([150], 8, 128, 64, BF16, 9, n_blocks=73000)
    assert q.cache.k.numel() > 1 << 32
    q.append([(0, 100)])
    q.append([(100, 150)])
    status_clean()
    q.check(0, 150)
    for got, x in zip(q.cache.read(q.batch([150], [150]), F32), q.values(0, 150)):
        assert np.array_equal(got.cpu().numpy(), x.reshape(150, -1))


def test_numbers_that_do_not_fit_are_reported():
    # A page outside the pool, a length past max_len, a slot outside the ring: skipped, reported once; the
    # other sequence is written.
    for wrong in ("page", "length", "slot", "rows"):
        q = Sequences([20, 20], 1, 64, 16, BF16, 10)
        b = q.batch([20, 20], [20, 20])
        kv_len, table, row_start, _ = b._keep
        slots = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        if wrong == "page":
            table[0, :] = q.n_blocks
        if wrong == "length":
            kv_len[0] = 21
        if wrong == "slot":
            slots[0] = -1
        if wrong == "rows":
            row_start[0] = -1
        b = tf.KvBatch(kv_len, table, 20, row_start, 40, 20, slots)
        q.cache.append(q.rows(q.k), q.rows(q.v), b)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
        tf.tf_device_status()
        q.check(1, 20)
        assert torch.all(q.cache.k[torch.from_numpy(q.table[0].astype(np.int64)).to(DEV)] == 0)


def test_another_stream():
    q = Sequences([70], 2, 64, 16, BF16, 11)
    k, v, b = q.rows(q.k), q.rows(q.v), q.batch([70], [70])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.cache.append(k, v, b, stream=side)
    side.synchronize()
    q.check(0, 70)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("amax", [127.0, 1.0, 0.3, 3e-4, 1e-28, 3e-31, 5e36])
def test_values_in_the_middle_of_two_codes(dtype, amax):
    # (c + 1/2) scale, and its neighbours some fp32 steps away: nearest, even in the middle, of the rounded quotient.
    q = Sequences([64 + 20], 1, 128, 64, dtype, 10)
    scale = np.float32(amax) * (np.float32(1) / np.float32(127))
    rng = np.random.default_rng(11)
    for a in (q.k, q.v):
        with np.errstate(under="ignore"):
            x = (rng.integers(-126, 126, a[0].shape) + 0.5).astype(np.float32) * scale
        steps = rng.integers(-40, 41, x.shape)
        x = (x.view(np.int32) + np.where(x == 0, 0, steps).astype(np.int32)).view(np.float32)
        x[0, 0, 0] = x[64, 0, 3] = amax
        a[0] = bf16(x) if dtype == BF16 else x
    q.append([(0, 70)])
    q.append([(70, 84)])
    status_clean()
    q.check(0, 84)


@pytest.mark.parametrize("wrong", [(2 ** 31 - 1, -2 ** 31, -2 ** 31 + 5), (0, 2 ** 31 - 1, -2 ** 31 + 3), (-2 ** 31, 2 ** 31 - 1, 20)])
def test_row_starts_that_wrap_around_are_reported(wrong):
    # Starts far outside whose 32-bit difference looks like a few rows: nothing is read or written there.
    q = Sequences([20, 20], 1, 64, 16, BF16, 12)
    b = q.batch([20, 20], [10, 10])
    b._keep[2].copy_(torch.tensor(wrong, dtype=torch.int32))
    x = torch.ones((20, 64), dtype=BF16, device=DEV)
    out = [torch.full((20, 64), 3.0, dtype=BF16, device=DEV) for _ in range(2)]
    for call in (lambda: q.cache.append(x, x, b), lambda: q.cache.read(b, k_out=out[0], v_out=out[1]),
                 lambda: q.cache.attend(x, b, out=out[0], kernel=tf.TF_KV_BY_ROWS),
                 lambda: q.cache.attend(x, b, out=out[0], kernel=tf.TF_KV_BY_TILES)):
        call()
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
    assert torch.all(q.cache.k == 0) and torch.all(out[0] == 3.0) and torch.all(out[1] == 3.0)


@pytest.mark.parametrize("block,dtype", [(16, BF16), (32, F32)])
def test_rewinding_again_and_again_leaves_no_trace(block, dtype):
    # Back and forth between the longest length and a page before it, drafts of any size in between; every kept token in
    # the end is the one written last.
    n = 6 * block + 5
    q = Sequences([n], 2, 64, block, dtype, 13)
    good = [a[0].copy() for a in (q.k, q.v)]
    rng = np.random.default_rng(block)
    longest = length = 0
    while length < n:
        for _ in range(4):
            start = int(rng.integers(max(0, longest - block), length + 1))
            end = min(n, start + int(rng.integers(1, block + 1)))
            for a in (q.k, q.v):
                a[0][start:end] = bf16(100 * rng.standard_normal(a[0][start:end].shape))
            q.append([(start, end)])
            longest, length = max(longest, end), end
        # What is kept: from the lowest place that may be gone on from.
        start = max(0, longest - block) if longest < n else max(0, min(length, n - block))
        for a, g in zip((q.k, q.v), good):
            a[0][start:] = g[start:]
        end = min(n, start + block + 1)
        q.append([(start, end)])
        longest, length = max(longest, end), end
        q.check(0, length)
    # And to a page's first token, from anywhere.
    for a, g in zip((q.k, q.v), good):
        a[0][:] = bf16(0.01 * g)
    q.append([(block, n - 3)])
    for a, g in zip((q.k, q.v), good):
        a[0][2 * block:] = g[2 * block:]
    q.append([(2 * block, n)])
    q.append([(n - 7, n)])
    status_clean()
    kc, ks, vc, vs = q.stored(0, n)
    for x, c, sc in ((q.k[0], kc, ks), (q.v[0], vc, vs)):
        want_c, want_s = cache_of(x[block:], block)
        assert np.array_equal(c[block:], want_c) and np.array_equal(sc[1:], want_s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("small", [0.0, 1e-45, 7e-44, 8e-44])
def test_pages_of_scale_zero_hold_zeros(dtype, small):
    # Nothing but zeros (or what max / 127 rounds to 0: up to 63 of the smallest subnormals) beside infinities and NaN.
    q = Sequences([40], 2, 64, 16, dtype, 14)
    for a in (q.k, q.v):
        x = np.full(a[0].shape, np.float32(small), np.float32)
        x[::2] *= -1
        x[3, 0, 5], x[20, 1, 0], x[17, 1, 63], x[36, 0, 1] = np.inf, -np.inf, np.nan, np.inf
        a[0] = bf16(x) if dtype == BF16 else x
    amax = np.max(np.abs(q.k[0][np.isfinite(q.k[0])]))
    scale = np.float32(amax) * (np.float32(1) / np.float32(127))
    q.append([(0, 30)])
    q.append([(30, 40)])
    status_clean()
    kc, ks, vc, vs = q.stored(0, 40)
    assert np.all(ks == scale) and np.all(vs == scale)
    if scale == 0:
        assert np.all(kc == 0) and np.all(vc == 0)
    else:
        assert kc[3, 0, 5] == 127 and kc[20, 1, 0] == -127 and kc[17, 1, 63] == 0
    for x in q.values(0, 40):
        assert np.all(np.isfinite(x))


@pytest.mark.parametrize("wrong", ["length", "rows"])
def test_sequences_without_rows_are_checked_too(wrong):
    # Each call reports numbers that do not fit, also of a sequence that has nothing to write or read; the other is served.
    q = Sequences([20, 20], 1, 64, 16, BF16, 15)
    b = q.batch([20, 20], [20, 0])
    if wrong == "length":
        b._keep[0][1] = 21
    else:
        b._keep[2][2] = 41
    x, y = q.rows([q.k[0]]), q.rows([q.v[0]])
    calls = [lambda: q.cache.append(x, y, b), lambda: q.cache.read(b), lambda: q.cache.attend(x, b)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
    q.check(0, 20)
    # A slot stands for nothing where there is nothing to write.
    c = tf.KvBatch(*b._keep[:2], 20, torch.tensor([0, 20, 20], dtype=torch.int32, device=DEV), 20, 20,
                   torch.tensor([0, -1], dtype=torch.int32, device=DEV))
    c._keep[0][1] = 20
    q.cache.append(x, y, c)
    status_clean()
