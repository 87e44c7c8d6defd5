"""tf_rope on the GPU against fp64.

The bound: an angle is off by the 2^-32 of a turn that its product is cut to and by the rounding of at most an
eighth of a turn to fp32 (2^-24 of it), cosine and sine by one unit of 2^-23 in fp32 and their product with the
factor by 2^-24; two products and a sum are rounded, 3 2^-24; all of |a| + |b|.  Then the rounding to bf16, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import bf16
from tests.serve_oracle import DEV, rope

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EDGE = 2 * math.pi * 2.0 ** -32 + math.pi / 4 * 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -24 + 3 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def matrix(x, dtype, pad, shift):
    rows, width = x.shape
    m = torch.full((rows * (width + pad) + shift,), 3.0, dtype=dtype, device=DEV)[shift:].view(rows, width + pad)
    m[:, :width] = torch.from_numpy(x).to(DEV).to(dtype)
    return m


def check(turn, x, positions, src=BF16, dst=F32, inverse=False, pad=0, shift=0, in_place=False):
    rows, heads, dim = x.shape
    x = bf16(x) if src == BF16 else x.astype(np.float32)
    m = matrix(x.reshape(rows, -1), src, pad, shift)
    o = m if in_place else matrix(np.full((rows, heads * dim), 5.0, np.float32), dst, pad, shift)
    p = torch.tensor(positions, dtype=torch.int32, device=DEV)
    got = turn(m[:, :heads * dim], p, out=o[:, :heads * dim], inverse=inverse)
    torch.cuda.synchronize()
    tf.tf_device_status()
    assert torch.all(o[:, heads * dim:] == 3.0)
    got = got.float().cpu().numpy().reshape(x.shape).astype(np.float64)
    turns = [t % 2 ** 64 for t in turn.turns.cpu().tolist()]
    y, size = rope(x, [max(i, 0) for i in positions], turns, turn.factor, turn.rot_dim, turn.interleaved, inverse)
    live = np.array(positions) >= 0
    bound = size * turn.factor * EDGE + (2.0 ** -8 * np.abs(y) if o.dtype == BF16 else 0) + 1e-30
    bound *= 1 + 2.0 ** -8                       # (the rounding is of the value that is already off)
    assert np.all(np.abs(got - y)[live] <= bound[live]), float((np.abs(got - y) / bound)[live].max())
    rest = got[live][..., turn.rot_dim:]
    want = x[live][..., turn.rot_dim:]
    assert np.array_equal(rest, bf16(want) if o.dtype == BF16 else want)
    assert np.array_equal(got[~live], x[~live] if in_place else np.full(x[~live].shape, 5.0))


def draw(rows, heads, dim, seed=0):
    return np.random.default_rng(seed).standard_normal((rows, heads, dim)) * 3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,dst", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("heads,dim,rot", [(1, 64, 64), (3, 128, 64), (40, 128, 128), (18, 256, 64), (2, 80, 32), (5, 6, 4), (1, 2, 2), (2, 1024, 1024)])
def test_shapes(heads, dim, rot, src, dst, interleaved):
    turn = tf.Rope(dim, rot, interleaved=interleaved)
    rng = np.random.default_rng(dim)
    check(turn, draw(7, heads, dim), rng.integers(0, 100000, 7).tolist(), src, dst)
    check(turn, draw(1, heads, dim), [3], src, dst, inverse=True)


@pytest.mark.parametrize("rows", [4863, 4864, 6001])
@pytest.mark.parametrize("heads,dim,rot,interleaved", [(3, 64, 64, True), (2, 128, 32, False), (1, 6, 4, True)])
def test_many_short_rows(rows, heads, dim, rot, interleaved):
    # Eight rows a CTA, the last of them not whole, and rows of no position among them.
    positions = np.random.default_rng(rows).integers(-50, 9000, rows).tolist()
    check(tf.Rope(dim, rot, interleaved=interleaved), draw(rows, heads, dim), positions, BF16, BF16, pad=8)
    check(tf.Rope(dim, rot, interleaved=interleaved), draw(rows, heads, dim), positions, F32, F32, pad=3, shift=1, in_place=True)


@pytest.mark.parametrize("rows", [1, 151, 1215, 1216, 1219, 2500])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows(rows, interleaved):
    # One row a CTA and four, with rows that have no position.
    rng = np.random.default_rng(rows)
    positions = np.where(rng.random(rows) < 0.3, -1, rng.integers(0, 5000, rows))
    positions[rng.integers(rows)] = 5
    check(tf.Rope(64, 32, interleaved=interleaved), draw(rows, 2, 64), positions.tolist(), BF16, BF16)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (1, 4), (4, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_alignment_and_in_place(dtype, pad, shift, in_place):
    for interleaved in (False, True):
        check(tf.Rope(128, 64, interleaved=interleaved), draw(9, 3, 128), [4, -1, 0, 70000, 2, 9, -5, 1, 8], dtype, dtype, False,
              pad, shift, in_place)


@pytest.mark.parametrize("position", [0, 1, 2 ** 20 + 1, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(position):
    check(tf.Rope(128, base=5e5), draw(3, 2, 128), [position, max(position - 1, 0), position // 3], F32, F32)


@pytest.mark.parametrize("scaling", [dict(type="linear", factor=4.0), dict(type="ntk", factor=8.0),
                                     dict(type="bands", factor=8.0, low=1.0, high=4.0, original=8192),
                                     dict(type="yarn", factor=16.0, original=4096)])
def test_scaled(scaling):
    check(tf.Rope(128, 64, base=1e6, scaling=scaling), draw(5, 4, 128), [0, 7, 4096, 60000, 131071], F32, F32)


def test_turned_back():
    # The inverse is the gradient: <turn(x), g> = <x, back(g)>, and back(turn(x)) = x where factor is 1.
    turn = tf.Rope(128, 96, interleaved=True)
    x, g = (torch.randn((50, 4 * 128), device=DEV, dtype=F32) for _ in range(2))
    p = torch.arange(50, dtype=torch.int32, device=DEV) * 1237
    y = turn(x, p)
    back = turn(g, p, inverse=True)
    left, right = (y.double() * g.double()).sum(), (x.double() * back.double()).sum()
    # (Each side is off by EDGE times the sum of (|a| + |b|) |g|.)
    assert abs(float(left - right)) <= 4 * EDGE * float(x.double().abs().sum() * g.abs().max())
    again = turn(y, p, inverse=True)
    assert float((again - x).abs().max()) <= 4 * EDGE * 2 * float(x.abs().max())


def test_gradient_by_differences():
    # d <turn(x), g> / dx in the direction d, by a difference of two calls (the turn is linear: exact but for rounding).
    turn = tf.Rope(64, 64)
    x, g, d = (torch.randn((6, 2 * 64), device=DEV, dtype=F32) for _ in range(3))
    p = torch.tensor([0, 1, 900, 5, 77, 100000], dtype=torch.int32, device=DEV)
    f = lambda t: (turn(t, p).double() * g.double()).sum()               # noqa: E731
    slope = float(f(x + d) - f(x - d)) / 2
    want = float((turn(g, p, inverse=True).double() * d.double()).sum())
    # (Two calls, halved, and the rounding of x + d and x - d; and the gradient.)
    assert abs(slope - want) <= 5 * EDGE * float((x.abs() + d.abs()).double().sum() * g.abs().max())


def test_infinities_and_nan_stay_in_their_pairs():
    turn = tf.Rope(64)
    x = torch.randn((3, 64), device=DEV)
    p = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    clean = turn(x, p)
    x[1, 3], x[2, 40] = math.inf, math.nan
    got = turn(x, p)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[1, [3, 35]] = keep[2, [8, 40]] = False
    assert torch.equal(got[keep], clean[keep]) and not torch.any(torch.isfinite(got[~keep]))


def test_columns_of_one_matrix():
    # Queries turned into other columns of the rows they come from; overlaps of any other kind are refused.
    turn = tf.Rope(64)
    m = torch.randn((20, 512), device=DEV)
    keep = m.clone()
    p = torch.arange(20, dtype=torch.int32, device=DEV)
    turn(m[:, :128], p, out=m[:, 256:384])
    assert torch.equal(m[:, 256:384], turn(keep[:, :128], p))
    assert torch.equal(m[:, :256], keep[:, :256]) and torch.equal(m[:, 384:], keep[:, 384:])
    for x, out in ((m[:, :128], m[:, 64:192]), (m[:19, :128], m[1:, :128]), (m[:, :128], m.view(40, 256)[:20, :128])):
        with pytest.raises(tf.TfError) as e:
            turn(x, p[:len(x)], out=out)
        assert e.value.rc == -5


def test_captured_and_on_another_stream():
    turn = tf.Rope(128)
    x = torch.randn((33, 256), device=DEV).to(BF16)
    p = torch.zeros(33, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            turn(x, p, out=out)
            p.add_(1)
    side.synchronize()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, turn(x, torch.full_like(p, i)))
    tf.tf_device_status()
