"""tf_sample on the GPU: against the header's arithmetic in torch (every token and
probability the same), and against the definition in 64 bits.  A weight's exponent
is at most 22.2 and rounded twice, its exp is within 2 ulp and it is rounded to a
whole number: running sums are within 22.2 * 2^-23 + 2^-22 + vocab * 2^-32 of the
definition's, relatively, and a token must be one that u and the cuts, moved by
no more than that, give."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import DEV, bf16, kept_tokens, sample_ok

pytestmark = pytest.mark.gpu


def edge(vocab):
    return 22.2 * 2.0 ** -23 + 2.0 ** -22 + vocab * 2.0 ** -32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def logits(rng, rows, vocab, kind):
    if kind == "broad":
        x = rng.standard_normal((rows, vocab)) * 0.5
    elif kind == "sharp":
        x = rng.standard_normal((rows, vocab)) * 2
        for r in range(rows):
            x[r, rng.integers(0, vocab, 30)] += 6 + 3 * rng.standard_normal(30)
    elif kind == "ties":
        x = np.round(rng.standard_normal((rows, vocab)) * 2) / 2
    elif kind == "flat":
        x = np.full((rows, vocab), 1.5)
    elif kind == "masked":
        x = rng.standard_normal((rows, vocab)) * 2
        x[rng.random((rows, vocab)) < 0.9] = -np.inf
        x[:, vocab // 2] = 0.25
    elif kind == "lowest":
        x = rng.standard_normal((rows, vocab)) * 2
        x[rng.random((rows, vocab)) < 0.9] = np.finfo(np.float32).min
        x[:, vocab // 2] = 0.25
    return x.astype(np.float32)


def header(x, u, temperature, top_k, top_p, min_p):
    """The header's arithmetic: whole weights, sums in 64-bit integers."""
    x = x.float()
    x = torch.where(torch.isnan(x), -torch.inf, x)
    vocab = x.shape[1]
    top, best = x.amax(1, keepdim=True), x.argmax(1)
    z = torch.where(x == top, 0.0, (x - top) * (1.0 / temperature)[:, None])
    w = torch.where(x == -torch.inf, 0, (torch.exp(z) * 2.0 ** 31).round().to(torch.int64))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    run = ws.cumsum(1)
    place = torch.arange(vocab, device=DEV)
    k = torch.where(top_k > 0, top_k, vocab).clamp(max=vocab).long()[:, None]
    p = top_p.double()[:, None]
    keep = (place < k) & ((place == 0) | (p >= 1) | ((run - ws).double() < p * run.gather(1, k - 1).double()))
    keep &= ws.double() >= min_p.clamp(max=1.0).double()[:, None] * 2.0 ** 31
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0))
    run = w.cumsum(1)
    all_ = run[:, -1].double()
    token = (run.double() > (u.double() * all_)[:, None]).to(torch.uint8).argmax(1)
    greedy, dead = ~(temperature > 0), top[:, 0] == -torch.inf
    token = torch.where(greedy, best, token)
    prob = torch.where(greedy, 1.0, (w.gather(1, token[:, None])[:, 0].double() / all_).float())
    return torch.where(dead, -1, token).int(), torch.where(dead, 0.0, prob)


def check(x, par, seed, dtype=torch.float32, pad=0, shift=0):
    """par: rows of (temperature, top_k, top_p, min_p)."""
    rng = np.random.default_rng(seed)
    rows, vocab = x.shape
    if dtype == torch.bfloat16:
        x = bf16(x)
    u = rng.random(rows).astype(np.float32).clip(0, 1 - 2.0 ** -24)
    m = torch.full((rows * (vocab + pad) + shift,), 50.0, dtype=dtype, device=DEV)[shift:].view(rows, vocab + pad)
    m[:, :vocab] = torch.from_numpy(x).to(DEV).to(dtype)
    f32 = [torch.tensor([p[i] for p in par], dtype=torch.float32, device=DEV) for i in (0, 2, 3)]
    k = torch.tensor([p[1] for p in par], dtype=torch.int32, device=DEV)
    args = (m[:, :vocab], torch.from_numpy(u).to(DEV), f32[0], k, f32[1], f32[2])
    tokens, probs = tf.sample(*args)
    want, prob = header(*args)
    assert torch.equal(tokens, want) and torch.equal(probs, prob)
    tokens, probs = tokens.cpu().tolist(), probs.cpu().tolist()
    sure = 0
    for r in range(rows):
        one = [float(np.float32(v)) if i != 1 else v for i, v in enumerate(par[r])]
        ok, alone = sample_ok(tokens[r], probs[r], x[r], float(u[r]), *one, edge(vocab))
        assert ok, (r, tokens[r], probs[r], float(u[r]), one)
        sure += alone
    return sure


PARAMS = [(1.0, 0, 1.0, 0.0), (0.7, 1, 1.0, 0.0), (1.0, 7, 1.0, 0.0), (1.3, 50, 0.9, 0.0), (0.9, 0, 0.5, 0.0),
          (1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02), (1.0, 1000, 0.99, 0.001), (0.0, 5, 0.5, 0.1),
          (1.0, 0, 0.0, 0.0), (5.0, 0, 0.3, 0.0), (0.05, 0, 0.999, 0.0), (1.0, 10 ** 9, 2.0, -1.0), (1.0, -3, 1.0, 7.0)]


@pytest.mark.parametrize("kind", ["broad", "sharp", "ties", "flat", "masked", "lowest"])
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 4097, 32003, 70001])
def test_every_parameter(kind, vocab):
    rng = np.random.default_rng(vocab)
    sure = check(logits(rng, len(PARAMS), vocab, kind), PARAMS, 1)
    # Small vocabularies leave no choice, unless a cut lies among equal weights.
    assert vocab > 4097 or kind in ("flat", "ties") or sure >= len(PARAMS) - 2


@pytest.mark.parametrize("kind", ["broad", "sharp", "ties"])
@pytest.mark.parametrize("rows", [1, 3, 20])
def test_language_model_head(kind, rows):
    rng = np.random.default_rng(rows)
    par = [PARAMS[i] for i in rng.integers(0, len(PARAMS), rows)]
    check(logits(rng, rows, 248320, kind), par, 2)


@pytest.mark.parametrize("vocab,rows", [(777, 400), (5000, 200), (300007, 5), (1 << 20, 2)])
def test_many_rows_and_large_vocabularies(vocab, rows):
    rng = np.random.default_rng(rows)
    par = [PARAMS[i] for i in rng.integers(0, len(PARAMS), rows)]
    check(logits(rng, rows, vocab, "sharp"), par, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (0, 3), (13, 1), (64, 8)])
@pytest.mark.parametrize("vocab", [512, 20003, 100001])
def test_types_strides_and_alignment(dtype, pad, shift, vocab):
    rng = np.random.default_rng(pad)
    check(logits(rng, len(PARAMS), vocab, "sharp"), PARAMS, 4, dtype, pad, shift)


def test_ties_go_to_the_lowest_index():
    x = np.zeros((4, 50000), np.float32)
    x[:, [20, 21, 40000, 49999]] = 3
    x[3, 7] = -0.0
    u = torch.tensor([0.0, 0.4, 0.9, 0.99], device=DEV)
    for k, want in ((1, [20] * 4), (2, [20, 20, 21, 21]), (3, [20, 21, 40000, 40000]), (4, [20, 21, 49999, 49999])):
        got, p = tf.sample(torch.from_numpy(x).to(DEV), u, top_k=torch.full((4,), k, dtype=torch.int32, device=DEV))
        assert got.cpu().tolist() == want
        assert torch.allclose(p, torch.full_like(p, 1 / k))
    # The fifth best is the first of the zeros; -0 and 0 are equal.
    got, _ = tf.sample(torch.from_numpy(x).to(DEV), torch.full((4,), 0.0, device=DEV),
                       top_k=torch.full((4,), 5, dtype=torch.int32, device=DEV))
    assert got.cpu().tolist() == [0] * 4
    got, _ = tf.sample(torch.from_numpy(x).to(DEV), u, temperature=torch.zeros(4, device=DEV))
    assert got.cpu().tolist() == [20] * 4


def test_rows_without_tokens_and_odd_values():
    inf, nan = np.inf, np.nan
    x = np.full((6, 9000), -inf, np.float32)
    x[1, 100] = -5                                  # one token
    x[2] = nan                                      # nothing but NaN
    x[3, [3, 8000]] = inf                           # two infinities and others
    x[3, 4] = 100
    x[4, 5:8] = nan
    x[4, 8] = 2
    x[5, :] = np.finfo(np.float32).min              # every token masked alike: each as likely
    u = torch.tensor([0.5, 0.999, 0.5, 0.75, 0.0, 0.50001], device=DEV)
    for par in (dict(), dict(top_p=torch.full((6,), 0.99995, device=DEV)), dict(top_k=torch.full((6,), 8999, dtype=torch.int32, device=DEV)),
                dict(temperature=torch.zeros(6, device=DEV))):
        got, p = tf.sample(torch.from_numpy(x).to(DEV), u, **par)
        got, p = got.cpu().tolist(), p.cpu().tolist()
        greedy = "temperature" in par
        assert got[:3] == [-1, 100, -1] and p[0] == 0 and p[1] == 1 and p[2] == 0
        assert got[3] == (3 if greedy else 8000) and (greedy or p[3] == 0.5)
        assert got[4] == 8 and p[4] == 1
        assert got[5] == 0 if greedy else got[5] in (4499, 4500)
    got, _ = tf.sample(torch.from_numpy(x).to(DEV), torch.full((6,), 1.0, device=DEV))
    assert got.cpu().tolist() == [-1, 100, -1, 8000, 8, 8999]
    hot = torch.full((6,), float("inf"), device=DEV)
    got, _ = tf.sample(torch.from_numpy(logits(np.random.default_rng(1), 6, 9000, "sharp")).to(DEV), u, temperature=hot,
                       top_p=torch.full((6,), 0.999, device=DEV))
    assert all(0 <= t < 9000 for t in got.cpu().tolist())


def test_frequencies_follow_the_probabilities():
    rng = np.random.default_rng(9)
    x = logits(rng, 1, 300, "sharp")
    n = 4096
    rows = torch.from_numpy(np.repeat(x, n, axis=0)).to(DEV)
    u = (torch.arange(n, device=DEV) + 0.5) / n
    tokens, _ = tf.sample(rows, u, top_p=torch.full((n,), 0.9, device=DEV))
    at, w = kept_tokens(x[0], 1.0, 0, float(np.float32(0.9)), 0.0)
    counts = np.bincount(tokens.cpu().numpy(), minlength=300)
    want = np.zeros(300)
    want[at] = w / w.sum() * n
    assert np.all(np.abs(counts - want) <= 1.01)     # u's grid: at most one step at each end


def test_again_and_on_other_streams():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(logits(rng, 7, 248320, "broad")).to(DEV)
    u = torch.rand(7, device=DEV)
    par = dict(top_p=torch.full((7,), 0.9, device=DEV), top_k=torch.full((7,), 5000, dtype=torch.int32, device=DEV))
    first = tf.sample(x, u, **par)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None):
        tokens, probs = torch.empty_like(first[0]), torch.empty_like(first[1])
        torch.cuda.synchronize()
        tf.sample(x, u, tokens=tokens, probs=probs, stream=stream, **par)
        torch.cuda.synchronize()
        assert torch.equal(tokens, first[0]) and torch.equal(probs, first[1])


@pytest.mark.parametrize("vocab", [1000, 32003, 248320])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_temperatures_that_are_not_above_zero(vocab, dtype):
    # NaN and negative ones too: the first largest logit, whatever the other parameters.
    rng = np.random.default_rng(vocab + 1)
    cold = [np.nan, -np.nan, -1.0, -np.inf, -0.0, 0.0]
    par = [(t, k, p, m) for t in cold for k, p, m in ((0, 1.0, 0.0), (50, 0.9, 0.05), (0, 0.3, 0.0))]
    x = logits(rng, len(par), vocab, "broad")
    check(x, par, 6, dtype)
    m = torch.from_numpy(x).to(DEV).to(dtype)
    tokens, probs = tf.sample(m, torch.rand(len(par), device=DEV), temperature=torch.tensor([p[0] for p in par], device=DEV))
    assert torch.equal(tokens.long(), m.float().argmax(1)) and torch.all(probs == 1)


def test_other_parameters_that_are_not_numbers():
    # top-p and min-p of NaN keep everything (they are not below 1, not above 0).
    rng = np.random.default_rng(3)
    m = torch.from_numpy(logits(rng, 4, 5000, "sharp")).to(DEV)
    u, nan = torch.rand(4, device=DEV), torch.full((4,), float("nan"), device=DEV)
    want = tf.sample(m, u)
    for par in (dict(top_p=nan), dict(min_p=nan), dict(top_p=nan, min_p=nan)):
        got = tf.sample(m, u, **par)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
