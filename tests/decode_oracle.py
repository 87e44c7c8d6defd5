"""Plain 64-bit implementations of the cache, the attention and the sampling of
include/tfdecode.h, in numpy, and the builders of their test inputs."""
import numpy as np
import torch

import mlx_affine_bit_gb300 as tf

DEV = torch.device("cuda:0")


def bf16(a):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def quantise(x):
    """One page of one head, [tokens][dim] fp32: (scale, codes), the header's fp32 arithmetic."""
    mag = np.abs(x.astype(np.float32))
    amax = np.max(np.where(np.isfinite(mag), mag, 0), initial=0)
    scale = np.float32(amax) * (np.float32(1) / np.float32(127))
    with np.errstate(all="ignore"):
        c = np.rint(x.astype(np.float32) / scale)
    c = np.clip(np.where(np.isnan(c), 0, c), -127, 127)
    return scale, c.astype(np.int8)


def cache_of(tokens, block):
    """[tokens][heads][dim] -> (codes like tokens, scales [pages][heads])."""
    n, h, _ = tokens.shape
    codes = np.zeros(tokens.shape, np.int8)
    scales = np.zeros(((n + block - 1) // block, h), np.float32)
    for p in range(scales.shape[0]):
        for i in range(h):
            scales[p, i], codes[p * block:(p + 1) * block, i] = quantise(tokens[p * block:(p + 1) * block, i])
    return codes, scales


def attend(q, k, v, vs, scale, n, causal, window, f32_q):
    """q [n][heads][dim], k, v [len][kv_heads][dim], the values' scales vs [len][kv_heads] -> (out, bound)
    [n][heads][dim] in fp64.

    The bound follows the header's precision: the result's rounding to bf16 (8 bits: 2^-8 of it at most), the
    rounding of p * vs to 11 bits (2^-11 at most), or below 2^-29 of the row's largest to 2^-40 of that (a code is
    128 at most), and p's own relative error, twice (in the sum that it is divided by
    too), which is that of its exponent: dim products in fp32 sums, fp32 q rounded to 11 bits (2^-11), and a few
    roundings of the scaled score."""
    length, kvh, dim = k.shape
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    g = q.shape[1] // kvh
    for h in range(q.shape[1]):
        kk, vv, qq = k[:, h // g].astype(np.float64), v[:, h // g].astype(np.float64), q[:, h].astype(np.float64)
        s = qq @ kk.T * scale
        mag = np.abs(qq) @ np.abs(kk).T * abs(scale)
        pos = length - n + np.arange(n)
        j = np.arange(length)
        see = np.ones((n, length), bool)
        if causal:
            see = j[None] <= pos[:, None]
            if window:
                see &= j[None] > pos[:, None] - window
        for i in range(n):
            at = np.nonzero(see[i])[0]
            if at.size == 0:
                continue
            si = s[i, at]
            p = np.exp(si - si.max())
            p /= p.sum()
            out[i, h] = p @ vv[at]
            ds = mag[i, at].max() * (dim * 2.0 ** -23 + (2.0 ** -11 if f32_q else 0)) + np.abs(si).max() * 2.0 ** -21 + 2.0 ** -20
            bound[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + (1.01 * 2.0 ** -11 + 2 * ds) * (p @ np.abs(vv[at])) + \
                at.size * 2.0 ** -40 * 128 * np.max(p * vs[at, h // g]) + 1e-30
    return out, bound


def rank(x):
    """Indexes by (logit descending, index ascending); NaN is -inf."""
    x = np.where(np.isnan(x), -np.inf, x)
    return np.lexsort((np.arange(x.size), -x)), x


def weights(x, temperature):
    x = x.astype(np.float64)
    top = x.max()
    with np.errstate(invalid="ignore"):
        z = np.where(x == top, 0.0, (x - top) / temperature)
    return np.where(x == -np.inf, 0.0, np.exp(z))


def kept_tokens(x, temperature, top_k, top_p, min_p):
    """Indexes kept, ascending, and their weights."""
    order, x = rank(x)
    w = weights(x, temperature)[order]
    n = top_k if 0 < top_k < x.size else x.size
    if top_p < 1:
        run = np.cumsum(w[:n])
        n = min(n, int(np.searchsorted(run, top_p * run[-1])) + 1)
    if min_p > 0:
        n = min(n, int((w >= min(min_p, 1.0)).sum()))
    at = np.sort(order[:max(n, 1)])
    return at, weights(x, temperature)[at]


def sample_ok(token, prob, x, u, temperature, top_k, top_p, min_p, edge):
    """Whether a token (and its probability) is one that the definition gives for a u and cuts moved by no more than
    `edge`, the relative error of sums of weights; and whether that leaves one token only."""
    order, xx = rank(x)
    if xx.max() == -np.inf:
        return token == -1 and prob == 0, True
    if not temperature > 0:
        return token == order[0] and prob == 1, True
    # The smallest and the largest set that the cuts may leave.
    wide, ww = kept_tokens(x, temperature, top_k, top_p + edge if top_p < 1 else top_p, min_p * (1 - edge))
    tight, wt = kept_tokens(x, temperature, top_k, top_p - edge if top_p < 1 else top_p, min_p * (1 + edge) if min_p < 1 else min_p)
    if token not in wide:
        return False, False
    slack = edge + (ww.sum() - wt.sum()) / wt.sum()
    run = np.cumsum(ww) / ww.sum()
    i = int(np.searchsorted(wide, token))
    near = (run[i - 1] if i else 0.0) - slack <= u <= run[i] + slack
    share = ww[i] / ww.sum()
    first, last = (int(np.searchsorted(run, v, side="right")) for v in (max(u - slack, 0), min(u + slack, 1 - 1e-15)))
    return near and abs(prob - share) <= (slack + 1e-5) * share + 2.0 ** -31, first == last


class Sequences:
    """Sequences in a paged cache with shuffled pages, and their tokens as numpy arrays."""

    def __init__(self, lens, kv_heads, dim, block, dtype, seed, spare=2, slots=None, n_blocks=None):
        self.rng = np.random.default_rng(seed)
        self.h, self.d, self.b, self.dtype = kv_heads, dim, block, dtype
        pages = [-(-max(n, 1) // block) for n in lens]
        total = sum(pages) + spare
        self.n_blocks = n_blocks or total
        ids = self.n_blocks - total + self.rng.permutation(total)
        self.width = max(pages)
        self.table = np.full((len(lens), self.width), self.n_blocks - 1, np.int32)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.slots = slots
        n_slots = (max(slots) if slots is not None else len(lens) - 1) + 1
        self.cache = tf.KvCache.empty(self.n_blocks, kv_heads, dim, block, n_slots, dtype, DEV)
        self.k = [self.tokens(n) for n in lens]
        self.v = [self.tokens(n) for n in lens]

    def tokens(self, n):
        x = self.rng.standard_normal((n, self.h, self.d)) * np.exp(0.5 * self.rng.standard_normal((n, self.h, 1)))
        return bf16(x) if self.dtype == torch.bfloat16 else x.astype(np.float32)

    def batch(self, lens, rows, seqs=None, uniform=False):
        seqs = list(range(len(lens))) if seqs is None else seqs
        i32 = dict(dtype=torch.int32, device=DEV)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(rows)]).tolist(), **i32)
        slots = None
        if self.slots is not None or seqs != list(range(len(seqs))):
            slots = torch.tensor([self.slots[s] if self.slots is not None else s for s in seqs], **i32)
        return tf.KvBatch(torch.tensor(lens, **i32), torch.from_numpy(self.table[seqs]).to(DEV), max(max(lens), 1),
                          None if uniform else starts, None if uniform else sum(rows), max(rows), slots)

    def rows(self, parts, pad=0, shift=0):
        """Rows of several sequences as one device matrix with `pad` extra columns, `shift` elements off alignment."""
        x = np.concatenate(parts).reshape(-1, self.h * self.d)
        m = torch.zeros((x.shape[0] * (x.shape[1] + pad) + shift,), dtype=self.dtype, device=DEV)
        m = m[shift:].view(x.shape[0], x.shape[1] + pad)
        m[:, :x.shape[1]] = torch.from_numpy(x).to(DEV).to(self.dtype)
        return m[:, :x.shape[1]]

    def append(self, spans, pad=0, shift=0, seqs=None):
        """spans: (from, to) of each sequence's tokens."""
        seqs = list(range(len(spans))) if seqs is None else seqs
        b = self.batch([t for _, t in spans], [t - f for f, t in spans], seqs)
        self.cache.append(self.rows([self.k[s][f:t] for s, (f, t) in zip(seqs, spans)], pad, shift),
                          self.rows([self.v[s][f:t] for s, (f, t) in zip(seqs, spans)], pad, shift), b)

    def stored(self, s, n):
        """(k codes, k scales, v codes, v scales) of the first n tokens of sequence s, from the device."""
        pages = torch.from_numpy(self.table[s, :-(-n // self.b)].astype(np.int64)).to(DEV)
        out = []
        for pool, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            c = pool[pages].cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, self.h, self.d)[:n]
            out += [c, scale[pages].cpu().numpy()]
        return out

    def check(self, s, n):
        """Sequence s holds exactly its first n tokens, quantized."""
        got = self.stored(s, n)
        for x, c, sc in ((self.k[s][:n], got[0], got[1]), (self.v[s][:n], got[2], got[3])):
            want_c, want_s = cache_of(x, self.b)
            assert np.array_equal(sc, want_s)
            assert np.array_equal(c, want_c)

    def value_scales(self, s, n):
        """The value scales [n][heads] of the first n tokens of sequence s."""
        return np.repeat(self.stored(s, n)[3], self.b, axis=0)[:n].astype(np.float64)

    def values(self, s, n):
        """The fp32 values that the first n tokens of sequence s stand for: k, v [n][heads][dim]."""
        kc, ks, vc, vs = self.stored(s, n)
        per = lambda sc: np.repeat(sc, self.b, axis=0)[:n, :, None]       # noqa: E731
        return per(ks) * kc.astype(np.float32), per(vs) * vc.astype(np.float32)
