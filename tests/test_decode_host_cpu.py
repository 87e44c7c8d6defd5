"""Host checks of the kernels' own rules for the cache, attention and sampling (no GPU)."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_numbers_in_device_memory(tmp_path):
    # Row starts whose difference wraps around among them: no row outside the matrices is taken for a sequence's own.
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "seq_rows_test")
    subprocess.check_call([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                           os.path.join(ROOT, "tests", "seq_rows_host_test.cu"), "-o", exe])
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0 and "PASS" in run.stdout, run.stdout


class Ring:
    """Which originals an open ring holds: a call's tokens of its last two pages."""

    def __init__(self, block):
        self.block, self.places, self.tokens, self.calls = block, {}, {}, 0
        self.begun = self.longest = 0

    def may(self, start):
        """The header's rule on where a call may go on."""
        return start % self.block == 0 or start >= max(self.begun, self.longest - self.block)

    def append(self, start, end):
        """Whether the originals of the page that is gone on with were there."""
        b, self.calls = self.block, self.calls + 1
        there = all(self.places.get(p % (2 * b)) == (p, self.tokens[p]) for p in range(start // b * b, start))
        if start % b == 0 and start < self.longest - b:
            self.begun, self.longest = start, start
        for p in range(start, end):
            self.tokens[p] = self.calls
            if p // b >= (end - 1) // b - 1:
                self.places[p % (2 * b)] = (p, self.calls)
        self.longest = max(self.longest, end)
        return there


def test_where_a_sequence_may_be_rewound_to():
    # Wherever the rule allows a call, the ring has what it needs.
    rng = random.Random(1)
    for block in (1, 2, 4, 16):
        for _ in range(300):
            ring, length = Ring(block), 0
            for _ in range(60):
                starts = [p for p in range(length + 1) if ring.may(p)]
                start = rng.choice([length, rng.choice(starts), min(starts, key=lambda p: (p % block == 0, p))])
                if not ring.may(start):
                    start = length
                length = start + rng.choice([1, 1, rng.randint(1, block), rng.randint(1, 4 * block)])
                assert ring.append(start, length), (block, start, length)


def test_rewinding_twice_goes_further_than_the_ring():
    # Each of these calls begins within a page of the length before it; the third finds a draft's token in page 0's place.
    ring = Ring(16)
    assert ring.append(0, 32) and ring.append(32, 33) and ring.append(17, 18)
    assert not ring.may(2)
    assert not ring.append(2, 3)


class Elsewhere:
    """A tensor that says it is on another device; a call that passed it on would show (no library is loaded here)."""

    def __init__(self, t, device):
        self.t, self.device_number = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_number


@pytest.fixture
def tf(monkeypatch):
    import mlx_affine_bit_gb300 as tf

    def called(*a, **k):
        raise AssertionError("the library was called")

    monkeypatch.setattr(tf, "lib", called)
    monkeypatch.setattr(tf, "_get_device", lambda: 0)
    return tf


def test_tensors_on_other_devices_are_refused(tf):
    import torch
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)      # noqa: E731
    at = Elsewhere
    pools = [torch.zeros((4, 2, 16, 64), dtype=torch.int8) for _ in range(2)] + [torch.zeros((4, 2)) for _ in range(2)] + \
        [torch.zeros((2, 2, 32, 64), dtype=torch.bfloat16) for _ in range(2)] + [torch.zeros((2, 2, 2, 32))]
    lens, table, slots, starts = i32(3, 5), torch.zeros((2, 2), dtype=torch.int32), i32(0, 1), i32(0, 1, 2)
    cache = lambda *d: tf.KvCache(*[at(t, n) for t, n in zip(pools, d)])         # noqa: E731
    # A cache and a batch are on one device ...
    for wrong in range(1, 7):
        with pytest.raises(ValueError, match="on"):
            cache(*[-1 if i == wrong else 0 for i in range(7)])
    for d in ((0, -1, 0, 0), (0, 0, 1, 0), (0, 0, 0, -1), (-1, 0, 0, 0)):
        with pytest.raises(ValueError, match="on"):
            tf.KvBatch(at(lens, d[0]), at(table, d[1]), 5, row_start=at(starts, d[2]), rows=2, slots=at(slots, d[3]))
    # ... the same, and the current GPU; so are the rows of each call.
    good, b = cache(*[0] * 7), tf.KvBatch(at(lens, 0), at(table, 0), 5)
    rows = lambda d: at(torch.zeros((2, 128), dtype=torch.bfloat16), d)          # noqa: E731
    for c, batch, where in ((good, b, -1), (good, b, 1), (good, tf.KvBatch(lens, table, 5), 0), (cache(*[-1] * 7), tf.KvBatch(lens, table, 5), -1),
                            (cache(*[1] * 7), tf.KvBatch(at(lens, 1), at(table, 1), 5), 1)):
        home = c.device
        for call in (lambda: c.append(rows(where), rows(home), batch, stream=0), lambda: c.append(rows(home), rows(where), batch, stream=0),
                     lambda: c.read(batch, k_out=rows(where), v_out=rows(home), stream=0),
                     lambda: c.attend(rows(where), batch, out=rows(home), stream=0),
                     lambda: c.attend(rows(home), batch, out=rows(where), stream=0)):
            with pytest.raises(ValueError, match="on|device"):
                call()
    with pytest.raises(AssertionError):          # (and what fits goes on to the library)
        good.append(rows(0), rows(0), b, stream=0)


def test_sampling_on_other_devices_is_refused(tf):
    import torch
    x, u, k = torch.zeros((2, 10)), torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    at = Elsewhere
    for name, t in (("u", u), ("temperature", u), ("top_k", k), ("top_p", u), ("min_p", u), ("tokens", k), ("probs", u)):
        par = dict(u=at(u, 0), tokens=at(k, 0), probs=at(u, 0))
        par[name] = t
        with pytest.raises(ValueError, match=name):
            tf.sample(at(x, 0), stream=0, **par)
    for d in (-1, 1):
        with pytest.raises(ValueError, match="logits"):
            tf.sample(at(x, d), at(u, d), tokens=at(k, d), probs=at(u, d), stream=0)
    with pytest.raises(AssertionError):
        tf.sample(at(x, 0), at(u, 0), tokens=at(k, 0), probs=at(u, 0), stream=0)


def test_generation_refuses_empty_prompts(tf):
    # (The last row of a prompt without rows would be another's.)
    from mlx_affine_bit_gb300.decode import Decoder
    d = Decoder(layers=1, width=256, heads=2, kv_heads=1, dim=64, vocab=64, seqs=2, max_len=32, device="cpu")
    for prompts, n in (([[1], []], 2), ([[], []], 2), ([[1], [2]], 0), ([[1], [2]], -1), ([[1]], 2), ([], 2), ([[1], [2] * 31], 2)):
        with pytest.raises(ValueError):
            d.generate(prompts, n)


def test_reading_with_one_output_given(tf, monkeypatch):
    # The other is made, of the same type, whatever the cache was appended from.
    import torch
    cache = tf.KvCache.empty(4, 2, 64, 16, 2, torch.float32, "cpu")
    b = tf.KvBatch(torch.tensor([3, 5], dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32), 5)
    monkeypatch.setattr(tf, "_on_gpu", lambda *a: None)
    calls = []
    monkeypatch.setattr(tf, "tf_kv_read", lambda *a: calls.append(a))
    for dtype, flags in ((torch.bfloat16, tf.TF_OUT_BF16), (torch.float32, 0)):
        mine = torch.zeros((2, 128), dtype=dtype)
        for k, v in ((mine, None), (None, mine)):
            got = cache.read(b, k_out=k, v_out=v)
            assert got[0 if k is not None else 1] is mine and got[0].dtype == got[1].dtype == dtype
            assert calls[-1][6] == flags
    assert cache.read(b)[0].dtype == torch.float32 and cache.read(b, torch.bfloat16)[1].dtype == torch.bfloat16
    with pytest.raises(TypeError):               # (two types are refused as before)
        cache.read(b, k_out=torch.zeros((2, 128)), v_out=torch.zeros((2, 128), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        cache.read(b, torch.bfloat16, k_out=torch.zeros((2, 128)))
