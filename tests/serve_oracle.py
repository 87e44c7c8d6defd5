"""Plain implementations of include/tfserve.h -- pages, rotary positions, the 4-bit
cache and attention over it -- in Python and 64-bit numpy, and the builders of their
test inputs."""
import math
from fractions import Fraction

import numpy as np
import torch

import mlx_affine_bit_gb300 as tf
from tests.decode_oracle import bf16

DEV = torch.device("cuda:0")
MOST = 2.0 ** 126


# ----------------------------------------------------------------- pages --

class Pages:
    """The state of tf_kv_pages as lists, and its step."""

    def __init__(self, n_seqs, max_pages, block, free):
        self.block, self.max_pages, self.n_blocks = block, max_pages, len(free)
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.kv_len, self.free = [0] * n_seqs, list(free)

    def step(self, change, rows, max_rows, max_len):
        """(row_start, positions, slots, info)"""
        hold = lambda n: -(-n // self.block)                             # noqa: E731
        room = min(max_len, self.max_pages * self.block)
        n = len(self.kv_len)

        def refused(code, few=0):
            return [0] * (n + 1), [-1] * rows, [-1] * rows, [code, few, 0, max(self.kv_len)]

        ends = [a + c for a, c in zip(self.kv_len, change)]
        if any(not 0 <= e <= room or c > max_rows for e, c in zip(ends, change)):
            return refused(2)
        if rows and sum(max(0, c) for c in change) > rows:
            return refused(2)
        back = [p for row, a, e in zip(self.table, self.kv_len, ends) for p in row[hold(e):hold(a)]]
        need = sum(max(0, hold(e) - hold(a)) for a, e in zip(self.kv_len, ends))
        if need > len(self.free) + len(back):
            return refused(1, need - len(self.free) - len(back))
        self.free += back[::-1]
        for row, a, e in zip(self.table, self.kv_len, ends):
            for i in range(hold(e), hold(a)):
                row[i] = -1
        starts, positions, slots = [0], [], []
        for row, a, e in zip(self.table, self.kv_len, ends):
            for i in range(hold(a), hold(e)):
                row[i] = self.free.pop()
            positions += range(a, e)
            slots += [row[p // self.block] * self.block + p % self.block for p in range(a, e)]
            starts.append(starts[-1] + max(0, e - a))
        self.kv_len = ends
        pad = [-1] * (rows - len(positions))
        return starts, positions[:rows] + pad, slots[:rows] + pad, [0, 0, starts[-1], max(ends)]


# ------------------------------------------------------------------ rope --

def rope(x, positions, turns, factor, rot, interleaved, back):
    """x [rows][heads][dim] -> (y, |a| + |b| of each value's pair) in fp64; turns: whole numbers of 2^-64 of a turn."""
    part = np.array([[(p * t % 2 ** 64) / 2.0 ** 64 for t in turns] for p in positions]).reshape(len(positions), 1, len(turns))
    angle = 2 * np.pi * part
    c, s = factor * np.cos(angle), factor * np.sin(angle) * (-1 if back else 1)
    x = x.astype(np.float64)
    y, size = x.copy(), np.zeros(x.shape)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


# ----------------------------------------------------------------- cache --

def below(x):
    """The largest bf16 number not above each x (fp32)."""
    b = np.ascontiguousarray(x, np.float32).view(np.int32)
    cut = b & np.int32(-65536)
    return np.where((b < 0) & (cut != b), cut + np.int32(65536), cut).astype(np.int32).view(np.float32) + np.float32(0)


def above(x):
    """The smallest bf16 number not below each x (fp64, not negative)."""
    y = x.astype(np.float32)
    y = np.where(y.astype(np.float64) < x, np.nextafter(y, np.float32(np.inf)), y)
    return ((y.view(np.uint32).astype(np.uint64) + 65535) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def quantise4(x):
    """[...][dim] fp32 -> codes [...][dim], scales and biases [...][dim / 64] fp32, by the header's definition: in 64 bits,
    and where those might decide otherwise (a tiny value next to a large bias) with fractions."""
    g = x.reshape(*x.shape[:-1], -1, 64).astype(np.float64)
    whole = np.isfinite(g)
    held = np.clip(np.nan_to_num(g, nan=0.0, posinf=MOST, neginf=-MOST), -MOST, MOST)
    some = whole.any(-1)
    lo = np.where(some, np.where(whole, held, np.inf).min(-1), 0.0)
    hi = np.where(some, np.where(whole, held, -np.inf).max(-1), 0.0)
    bias = below(lo.astype(np.float32))
    reach = (hi - bias.astype(np.float64)) / 15.0
    scale = above(reach)
    for at in np.argwhere((above(reach * (1 - 2.0 ** -50)) != above(reach * (1 + 2.0 ** -50))) & (reach > 0)):
        at = tuple(at)
        want = Fraction(float(hi[at])) - Fraction(float(bias[at]))
        near = [v for v in (above(np.array(reach[at] * f)) for f in (1 - 2.0 ** -50, 1 + 2.0 ** -50)) if 15 * Fraction(float(v)) >= want]
        scale[at] = near[0]
    s = scale.astype(np.float64)[..., None]
    with np.errstate(all="ignore"):
        q = np.where(s > 0, (held - bias.astype(np.float64)[..., None]) / s, 0.0)
        code = np.clip(np.rint(q), 0, 15)
        near = np.argwhere((np.abs(q - np.floor(q) - 0.5) < 2.0 ** -40) & (q < 15))
    for at in near:
        at = tuple(at)
        t = Fraction(float(held[at])) - Fraction(float(bias[at[:-1]])) - (int(np.floor(q[at])) + Fraction(1, 2)) * Fraction(float(scale[at[:-1]]))
        low = int(np.floor(q[at]))
        code[at] = low + (t > 0 or (t == 0 and low % 2))
    return code.reshape(x.shape).astype(np.uint8), scale, bias


def values4(code, scale, bias):
    """fp32 values: scale * code + bias rounded once."""
    s, b = (np.repeat(t.astype(np.float64), 64, axis=-1) for t in (scale, bias))
    with np.errstate(all="ignore"):
        return (s * code + b).astype(np.float32)


def attend4(q, k, v, scale, causal, window, f32_q):
    """q [n][heads][dim]; k, v: (codes, scales, biases) of [len][kv_heads] -> (out, bound) [n][heads][dim] in fp64.

    The bound counts the header's roundings, for either kernel, each at its most:
      the output to bf16                                    2^-8 |out|
      p times a scale to fp16, where the bias counts in full   2^-11 p (|v| + |b|), and 2^-25 of what 2^18 stands for, times
                                                            a code of 15: below 2^-39 of the row's largest p (15 s or |b|)
      values to fp16 (tiles)                                2^-11 |v| and 2^-21 of the largest of 16 tokens
      p: its exponent's error, twice (it is in the sum, too)
    and of a score: dim fp32 sums of products of |q| (s c + |b|), fp32 q to fp16 (2^-11), and q below 2^-14 of a 16th of
    its row's largest to 2^-21 of that; keys to fp16 (tiles) like the values; a few roundings of the scaled score."""
    (kc, ks, kb), (vc, vs, vb) = k, v
    length, kvh, dim = kc.shape
    wide = lambda t: np.repeat(t.astype(np.float64), 64, axis=-1)        # noqa: E731
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    g = q.shape[1] // kvh

    def parts(c, s, b):
        x = wide(s) * c + wide(b)
        size = wide(s) * c + np.abs(wide(b))
        most = np.maximum(15 * np.abs(wide(s)), np.abs(wide(b))).max(-1)                    # [len]
        blocks = np.array([most[i // 16 * 16:i // 16 * 16 + 16].max() for i in range(length)])
        return x, size, most, 2 * blocks

    for kv in range(kvh):
        kk, k_size, _, k_unit = parts(kc[:, kv], ks[:, kv], kb[:, kv])
        vv, v_size, v_most, v_unit = parts(vc[:, kv], vs[:, kv], vb[:, kv])
        for h in range(kv * g, kv * g + g):
            qq = q[:, h].astype(np.float64)
            aq = np.abs(qq)
            s = qq @ kk.T * scale
            err = (aq @ k_size.T * (dim * 2.0 ** -23 + (2.0 ** -11 if f32_q else 0)) + aq @ np.abs(kk).T * 2.0 ** -11 +
                   aq.sum(1, keepdims=True) * k_unit[None] * 2.0 ** -20 +
                   aq.max(1, keepdims=True) * k_size.sum(1)[None] * 2.0 ** -21) * abs(scale)
            pos, j = length - len(q) + np.arange(len(q)), np.arange(length)
            see = np.ones(s.shape, bool)
            if causal:
                see = j[None] <= pos[:, None]
                if window:
                    see &= j[None] > pos[:, None] - window
            for i in range(len(q)):
                at = np.nonzero(see[i])[0]
                if at.size == 0:
                    continue
                si = s[i, at]
                p = np.exp(si - si.max())
                p /= p.sum()
                out[i, h] = p @ vv[at]
                ds = err[i, at].max() + np.abs(si).max() * 2.0 ** -21 + 2.0 ** -20
                bound[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + (2.02 * 2.0 ** -11 + 2 * ds) * (p @ (v_size[at] + np.abs(wide(vb)[at, kv]))) + \
                    2.0 ** -20 * (p @ v_unit[at]) + at.size * 2.0 ** -38 * np.max(p * v_most[at]) + 1e-30
    return out, bound


class Sequences4:
    """Sequences in a 4-bit cache with shuffled pages, and their tokens as numpy arrays."""

    def __init__(self, lens, kv_heads, dim, block, dtype=torch.bfloat16, seed=0, spare=2, n_blocks=None):
        self.rng = np.random.default_rng(seed)
        self.h, self.d, self.b, self.dtype, self.lens = kv_heads, dim, block, dtype, lens
        pages = [-(-max(n, 1) // block) for n in lens]
        total = sum(pages) + spare
        self.n_blocks = n_blocks or total
        ids = self.n_blocks - total + self.rng.permutation(total)
        self.table = np.full((len(lens), max(pages)), -1, np.int32)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.cache = tf.Kv4Cache.empty(self.n_blocks, kv_heads, dim, block, DEV)
        self.k = [self.tokens(n) for n in lens]
        self.v = [self.tokens(n) for n in lens]

    def tokens(self, n):
        x = self.rng.standard_normal((n, self.h, self.d)) * np.exp(0.5 * self.rng.standard_normal((n, self.h, 1)))
        x += 0.3 * self.rng.standard_normal((1, self.h, 1))
        return bf16(x) if self.dtype == torch.bfloat16 else x.astype(np.float32)

    def batch(self, lens, rows, seqs=None):
        seqs = list(range(len(lens))) if seqs is None else seqs
        i32 = dict(dtype=torch.int32, device=DEV)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(rows)]).tolist(), **i32)
        return tf.KvBatch(torch.tensor(lens, **i32), torch.from_numpy(self.table[seqs]).to(DEV), max(max(lens), 1), starts,
                          sum(rows), max(rows))

    def slots(self, spans):
        """Slots of the tokens [from, to) of each sequence, one after another."""
        out = [self.table[s, p // self.b].astype(np.int64) * self.b + p % self.b for s, (f, t) in enumerate(spans) for p in range(f, t)]
        return torch.tensor(out, dtype=torch.int64, device=DEV)

    def rows(self, parts, pad=0, shift=0):
        """Rows of several sequences as one device matrix with `pad` extra columns, `shift` elements off alignment."""
        x = np.concatenate(parts).reshape(-1, self.h * self.d)
        m = torch.zeros((x.shape[0] * (x.shape[1] + pad) + shift,), dtype=self.dtype, device=DEV)
        m = m[shift:].view(x.shape[0], x.shape[1] + pad)[:, :x.shape[1]]
        m.copy_(torch.from_numpy(x).to(DEV).to(self.dtype))
        return m

    def append(self, spans, pad=0, shift=0):
        """spans: (from, to) of each sequence's tokens."""
        self.cache.append(self.rows([x[f:t] for x, (f, t) in zip(self.k, spans)], pad, shift),
                          self.rows([x[f:t] for x, (f, t) in zip(self.v, spans)], pad, shift), self.slots(spans))

    def stored(self, s, n):
        """(codes, scales, biases) of keys and of values of the first n tokens of sequence s, from the device."""
        pages = torch.from_numpy(self.table[s, :-(-n // self.b)].astype(np.int64)).to(DEV)
        out = []
        for pool, pair in ((self.cache.k, self.cache.k_affine), (self.cache.v, self.cache.v_affine)):
            line = lambda t: np.moveaxis(t[pages].cpu().numpy(), 1, 2).reshape(-1, self.h, *t.shape[3:])[:n]     # noqa: E731
            c, a = line(pool), line(pair.float())
            out.append((np.stack([c & 15, c >> 4], -1).reshape(n, self.h, self.d), a[..., 0], a[..., 1]))
        return out

    def check(self, s, n):
        """Sequence s holds exactly its first n tokens, quantized."""
        for x, got in zip((self.k[s][:n], self.v[s][:n]), self.stored(s, n)):
            for a, b in zip(got, quantise4(x)):
                assert np.array_equal(a, b)


def filled4(lens, kv_heads, dim, block, seed):
    """A cache with random pages: any codes, scales over some octaves, biases on either side; NaN, infinities and whatever
    else past every sequence's end and in pages of no sequence."""
    q = Sequences4(lens, kv_heads, dim, block, seed=seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    held = torch.zeros(q.n_blocks * block, dtype=torch.bool, device=DEV)
    held[q.slots([(0, n) for n in lens])] = True
    held = held.view(q.n_blocks, 1, block, 1)
    for pool, pair in ((q.cache.k, q.cache.k_affine), (q.cache.v, q.cache.v_affine)):
        pool.copy_(torch.randint(0, 256, pool.shape, generator=gen, device=DEV, dtype=torch.uint8))
        scale = torch.exp(torch.randn(pair.shape[:-1], generator=gen, device=DEV)) * 0.1
        bias = -7.5 * scale * (1 + 0.5 * torch.randn(scale.shape, generator=gen, device=DEV))
        bad = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device=DEV)
        other = bad[torch.randint(0, 4, scale.shape, generator=gen, device=DEV)]
        pair.copy_(torch.stack([torch.where(held, scale, other), torch.where(held, bias, other)], -1))
    return q
