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
