"""The 4-bit cache on the GPU: what tf_kv4_append holds is, code for code and to the
bit of scales and biases, the header's definition in 64-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.serve_oracle import DEV, Sequences4, quantise4, values4

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def status_clean():
    torch.cuda.synchronize()
    tf.tf_device_status()


def held(x, dtype=F32, block=16):
    """What a cache holds of rows x [rows][heads][dim]: (codes, scales, biases) of keys, after an append to slots 0, 1, ..."""
    rows, heads, dim = x.shape
    cache = tf.Kv4Cache.empty(-(-rows // block), heads, dim, block, DEV)
    m = torch.from_numpy(np.ascontiguousarray(x.reshape(rows, -1), dtype=np.float32)).to(DEV).to(dtype)
    cache.append(m, m, torch.arange(rows, device=DEV))
    status_clean()
    out = []
    for pool, pair in ((cache.k, cache.k_affine), (cache.v, cache.v_affine)):
        c, a = (np.moveaxis(t.cpu().numpy(), 1, 2).reshape(-1, heads, *t.shape[3:])[:rows] for t in (pool, pair.float()))
        out.append((np.stack([c & 15, c >> 4], -1).reshape(x.shape), a[..., 0], a[..., 1]))
    assert all(np.array_equal(a, b) for a, b in zip(*out))
    return out[0]


def exact(x, dtype=F32):
    for got, want, name in zip(held(x, dtype), quantise4(x.astype(np.float32)), ("codes", "scales", "biases")):
        wrong = np.argwhere(got != want)
        assert wrong.size == 0, (name, len(wrong), wrong[0], got[tuple(wrong[0])], want[tuple(wrong[0])])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,dim,heads", [(16, 64, 3), (32, 128, 2), (64, 256, 1), (128, 256, 2), (128, 64, 1), (64, 128, 8), (16, 64, 1)])
def test_whole_prompts_and_what_is_read_back(dtype, block, dim, heads):
    lens = [1, block - 1, block, block + 1, 3 * block + 5]
    q = Sequences4(lens, heads, dim, block, dtype, 1)
    q.append([(0, n) for n in lens])
    status_clean()
    for s, n in enumerate(lens):
        q.check(s, n)
    # The last tokens of each sequence, in both types; one output alone.
    rows = [1, 3, 0, block + 1, 2 * block + 7]
    b = q.batch(lens, rows)
    want = [np.concatenate([values4(*q.stored(s, n)[i])[n - r:] for s, (n, r) in enumerate(zip(lens, rows))]).reshape(sum(rows), -1) for i in (0, 1)]
    for got, w in zip(q.cache.read(b, dtype=F32), want):
        assert np.array_equal(got.cpu().numpy(), w)
    for got, w in zip(q.cache.read(b), want):
        assert torch.equal(got.cpu(), torch.from_numpy(w).to(BF16))
    out = torch.zeros((sum(rows), heads * dim), device=DEV)
    tf.tf_kv4_read(q.cache.c, b.c, None, 0, out, heads * dim)
    status_clean()
    assert np.array_equal(out.cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_cut_gives_the_same_cache(dtype):
    n, rng = 150, np.random.default_rng(2)
    q = Sequences4([n, n], 2, 128, 32, dtype, 2)
    at = 0
    while at < n:
        to = min(n, at + int(rng.choice([1, 2, 17, 64])))
        q.append([(at, to), (0, 0)])
        at = to
    q.append([(0, 0), (0, n)])
    q.append([(n - 20, n), (0, 1)])                      # and some again
    status_clean()
    q.check(0, n)
    q.check(1, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_prompts(dtype):
    # Two vectors a thread; every code, scale and bias of some four million values.
    q = Sequences4([2100, 700], 8, 128, 64, dtype, 3)
    q.append([(0, 2100), (0, 700)])
    status_clean()
    q.check(0, 2100)
    q.check(1, 700)


def test_values_in_the_middle_of_two_codes():
    # Multiples of half a scale from the bias on, one unit of the last place to either side, and odd multiples of a 15th of the scale.
    rng = np.random.default_rng(4)
    x = np.zeros((400, 1, 64), np.float32)
    for i in range(400):
        scale = np.float32(2.0 ** rng.integers(-20, 20)) * np.float32(rng.integers(128, 256)) / 128
        bias = np.float32(np.float32(rng.integers(-255, 256)) / 16 * scale)
        bias = torch.tensor(bias).to(BF16).float().item()
        y = bias + scale * (rng.integers(0, 31, 64) / 2)
        y[0], y[1] = bias, bias + 15 * scale
        y = y.astype(np.float32)
        y[2:] = np.nextafter(y[2:], np.float32(rng.choice([-1, 1]) * np.inf)) if i % 3 else y[2:]
        x[i, 0] = np.clip(y, min(y[0], y[1]), max(y[0], y[1]))
    exact(x)


@pytest.mark.parametrize("size", [1e-45, 1e-41, 1e-38, 1e-33, 1e-30, 1e-25, 1e-18, 1e18, 1e30, 8e37])
def test_small_and_large_values(size):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 2, 64)) * size * np.exp(3 * rng.standard_normal((40, 2, 1)))).clip(-3.4e38, 3.4e38).astype(np.float32)
    exact(x)
    # Around a value far from 0, and the same value throughout.
    exact((np.float32(size) + x * np.float32(1e-4)).astype(np.float32))
    exact(np.broadcast_to(x[:, :, :1], x.shape).copy())


def test_ends_of_the_range():
    # A group's smallest and largest value a unit of the last place from a bf16 number, and where 15 scales just reach or just do not.
    rng = np.random.default_rng(6)
    x = rng.random((600, 1, 64)).astype(np.float32)
    for i in range(600):
        scale = np.float32(rng.integers(128, 256)) * np.float32(2.0 ** rng.integers(-12, 12))
        bias = torch.tensor(float(rng.standard_normal() * 100 * scale)).to(BF16).float().numpy()
        lo, hi = np.float32(bias), np.float32(bias + np.float32(15) * scale)
        step = [lambda v: v, lambda v: np.nextafter(v, np.float32(np.inf)), lambda v: np.nextafter(v, np.float32(-np.inf))]
        lo, hi = step[i % 3](lo), step[i // 3 % 3](hi)
        x[i, 0] = np.clip(lo + x[i, 0] * (hi - lo), lo, hi)
        x[i, 0, 5], x[i, 0, 6] = lo, hi
    exact(x)
    exact(x.astype(np.float32), F32)


def test_infinities_nan_and_zeros():
    x = np.random.default_rng(7).standard_normal((12, 1, 128)).astype(np.float32)
    x[0, 0, 3] = np.inf
    x[1, 0, 3] = -np.inf
    x[2, 0, 70] = np.nan
    x[3] = np.nan
    x[4] = np.inf
    x[5, 0, :64] = 0
    x[6, 0, :64] = -0.0
    x[7, 0, 9], x[7, 0, 10], x[7, 0, 11] = np.inf, -np.inf, np.nan
    x[8, 0, :64] = 5.0
    x[8, 0, 7] = -np.inf
    x[9, 0, 0], x[9, 0, 1] = 3.4e38, -3.4e38
    exact(x)
    codes, scales, biases = held(x)
    assert np.all(np.isfinite(scales)) and np.all(np.isfinite(biases)) and not np.any(np.signbit(biases[5:7, 0, 0]))
    assert codes[0, 0, 3] == 15 and codes[1, 0, 3] == 0
    assert np.all(scales[3] == 0) and np.all(biases[4] == 0)
    # The others of the group are held as without the bad value.
    y = np.delete(x[0, 0, :64], 3)
    v = values4(codes[0, 0, :64], scales[0, 0, :1], biases[0, 0, :1])
    assert np.all(np.abs(np.delete(v, 3) - y) <= scales[0, 0, 0] / 2 * (1 + 1e-6))


def test_no_value_is_off_by_more_than_half_a_scale():
    x = (np.random.default_rng(8).standard_normal((200, 4, 64)) * np.array([1e-3, 1, 30, 1e4]).reshape(1, 4, 1)).astype(np.float32)
    codes, scales, biases = held(x)
    v = codes * scales.astype(np.float64) + biases
    assert np.all(np.abs(v - x) <= scales.astype(np.float64) / 2)


@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(dtype, pad, shift):
    q = Sequences4([70, 9], 2, 64, 32, dtype, 9)
    q.append([(0, 70), (0, 9)], pad, shift)
    status_clean()
    q.check(0, 70)
    q.check(1, 9)
    for out in (BF16, F32):
        o = torch.full((79 * (128 + pad) + shift,), 3.0, dtype=out, device=DEV)[shift:].view(79, 128 + pad)
        k, v = q.cache.read(q.batch([70, 9], [70, 9]), k_out=o[:, :128])
        status_clean()
        assert k.data_ptr() == o.data_ptr() and torch.all(o[:, 128:] == 3.0)
        assert torch.equal(k, q.cache.read(q.batch([70, 9], [70, 9]), dtype=out)[0]) and v.dtype == out


def test_rows_without_a_slot_are_left_out_and_bad_slots_reported():
    q = Sequences4([40], 2, 64, 16, BF16, 10)
    k = q.rows([q.k[0]])
    slots = q.slots([(0, 40)])
    slots[::2] = -1
    q.cache.append(k, k, slots)
    status_clean()
    kept = (q.cache.k_affine[..., 0, 0] != 0).sum()
    assert int(kept) == 20 * 2
    before = [t.clone() for t in (q.cache.k, q.cache.v, q.cache.k_affine, q.cache.v_affine)]
    for bad in (-2, q.n_blocks * 16, 2 ** 40, -2 ** 63):
        slots[:] = -1
        slots[7] = bad
        q.cache.append(k, k, slots)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
        assert all(torch.equal(a, b) for a, b in zip(before, (q.cache.k, q.cache.v, q.cache.k_affine, q.cache.v_affine)))


def test_reading_what_does_not_fit_is_reported():
    q = Sequences4([40, 20], 2, 64, 16, BF16, 11)
    q.append([(0, 40), (0, 20)])
    b = q.batch([40, 20], [40, 20])
    want = q.cache.read(b)[0]
    for wrong in ("page", "length", "rows"):
        b = q.batch([40, 20], [40, 20])
        if wrong == "page":
            b._keep[1][0, 1] = q.n_blocks
        elif wrong == "length":
            b._keep[0][0] = 41
        else:
            b._keep[0][0] = 39                            # fewer tokens than rows
        out = torch.full((60, 128), 9.0, dtype=BF16, device=DEV)
        q.cache.read(b, k_out=out)
        torch.cuda.synchronize()
        with pytest.raises(tf.TfError) as e:
            tf.tf_device_status()
        assert e.value.rc == -14
        assert torch.equal(out[40:], want[40:])
        assert torch.all(out[16:32] == 9.0) if wrong == "page" else torch.all(out[:40] == 9.0)


def test_offsets_past_32_bits():
    q = Sequences4([300], 8, 128, 64, BF16, 12, n_blocks=140000)
    assert q.cache.k.numel() > 1 << 32
    q.append([(0, 300)])
    status_clean()
    q.check(0, 300)
    k, _ = q.cache.read(q.batch([300], [300]), dtype=F32)
    assert np.array_equal(k.cpu().numpy().reshape(300, 8, 128), values4(*q.stored(0, 300)[0]))


def test_captured_append_and_read_on_another_stream():
    q = Sequences4([64], 2, 128, 16, BF16, 13)
    k, v, slot = torch.zeros((1, 256), dtype=BF16, device=DEV), torch.zeros((1, 256), dtype=BF16, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = tf.KvBatch(n, torch.from_numpy(q.table).to(DEV), 64)
    out = torch.zeros((1, 256), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            n.add_(1)
            q.cache.append(k, v, slot)
            q.cache.read(b, k_out=out)
    side.synchronize()
    slots = q.slots([(0, 64)])
    for i in range(64):
        k.copy_(torch.from_numpy(q.k[0][i].reshape(1, -1)))
        v.copy_(torch.from_numpy(q.v[0][i].reshape(1, -1)))
        slot.copy_(slots[i:i + 1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy().reshape(2, 128), values4(*quantise4(q.k[0][i])))
    status_clean()
    q.check(0, 64)
    assert not math.isnan(float(out.sum()))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_groups_of_one_bf16_value(dtype):
    # Scale 0 and codes 0, at any size; beside them groups of the same size that are not constant, and constant but for an
    # infinity or a NaN, which a scale of 0 holds as the value itself.
    sizes = [0.0, 2.0 ** -133, 2.0 ** -126, 1.0, 1.5, 2.0 ** 63, 2.0 ** 64, 1.25 * 2.0 ** 64, 2.0 ** 70, 2.0 ** 100, 2.0 ** 126]
    x = np.array(sizes + [-s for s in sizes[1:]], np.float32)[:, None, None] * np.ones((1, 1, 256), np.float32)
    x[:, 0, 64 + 7] *= 2
    x[:, 0, 128 + 9], x[:, 0, 192 + 60] = np.inf, np.nan
    exact(x.clip(-2.0 ** 126, np.inf), dtype)
    codes, scales, _ = held(x, dtype)
    assert np.all(codes[:, 0, :64] == 0) and np.all(scales[:, 0, 0] == 0)
