"""Pages, positions and the 4-bit cache of growing sequences, on torch tensors
(``include/tfserve.h``).

    pages = tf.KvPages.empty(n_seqs=48, n_blocks=4000, max_pages=128)
    cache = tf.Kv4Cache.empty(pages.n_blocks, kv_heads=8, dim=128, block=pages.block)
    turn = tf.Rope(128, base=5e5)
    step = pages.plan(rows=48, max_rows=1, max_len=8192)      # buffers of a step, kept
    ...
    step.step(change)                                         # a token each, say: int32 [48] on the device
    y = tf.qmm(x, W, s, b, bits, G)                           # q | k | v
    qk = turn(y[:, :nq + nk], step.positions)
    cache.append(qk[:, nq:], y[:, nq + nk:], step.slots)
    a = cache.attend(qk[:, :nq], step.batch)

All of it reads what the device holds at the time of the call, so that a step can be one CUDA graph.
"""
from __future__ import annotations

import math

import mlx_affine_bit_gb300 as tf
from mlx_affine_bit_gb300 import _on_gpu, _ptr, _rows, _tensor


class KvPages:
    """The pages of growing sequences (tf_kv_pages).

    table [n_seqs][max_pages] int32 (-1 beyond a sequence's pages), kv_len [n_seqs] int32, free_pages [n_blocks] int32,
    n_free [1] int32: the first n_free of free_pages are those that no sequence holds.  plan() makes steps."""

    def __init__(self, table, kv_len, free_pages, n_free, block=64):
        import torch
        i32 = (torch.int32,)
        if table.dim() != 2:
            raise ValueError("table must be [n_seqs][max_pages]")
        n_seqs, max_pages = table.shape
        _tensor(table, "table", i32, contiguous=False)
        self.device = device = table.get_device()
        if max_pages > 1 and table.stride(1) != 1 or n_seqs > 1 and table.stride(0) < max_pages:
            raise ValueError("table must have contiguous rows that do not overlap")
        _tensor(kv_len, "kv_len", i32, (n_seqs,), device=device)
        _tensor(free_pages, "free_pages", i32, (free_pages.numel(),), device=device)
        _tensor(n_free, "n_free", i32, (1,), device=device)
        self.table, self.kv_len, self.free_pages, self.n_free = table, kv_len, free_pages, n_free
        self.n_seqs, self.max_pages, self.n_blocks, self.block = n_seqs, max_pages, free_pages.numel(), block
        self.c = tf.TfKvPages(_ptr(table), table.stride(0) if n_seqs > 1 else max_pages, _ptr(kv_len), _ptr(free_pages),
                              _ptr(n_free), n_seqs, self.n_blocks, max_pages, block)

    @classmethod
    def empty(cls, n_seqs, n_blocks, max_pages, block=64, device="cuda"):
        """n_seqs sequences without tokens, and all n_blocks pages free (page 0 is taken first)."""
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((n_seqs, max_pages), -1, **i32), torch.zeros(n_seqs, **i32),
                   torch.arange(n_blocks - 1, -1, -1, **i32), torch.full((1,), n_blocks, **i32), block)

    def plan(self, rows, max_rows=1, max_len=None):
        """The buffers of a step of up to `rows` rows (0: a step that only gives tokens back or reserves), of up to
        max_rows of a sequence, to lengths of up to max_len (by default all that the table has room for)."""
        return KvPlan(self, rows, max_rows, max_len)


class KvPlan:
    """One kind of step of a KvPages, and what it leaves on the device: row_start [n_seqs + 1], positions [rows] int32,
    slots [rows] int64, info [4] (include/tfserve.h), and batch, the KvBatch of the step's rows.

    All of it is of the plan's last step, and batch of the pages as they stand then: it reads their lengths and table, with
    this plan's row_start.  After a step of another plan of the same pages it means other tokens; use it before."""

    def __init__(self, pages, rows, max_rows=1, max_len=None):
        import torch
        if rows < 0 or max_rows < 1:
            raise ValueError("rows must not be negative, max_rows at least 1")
        room = pages.max_pages * pages.block
        max_len = room if max_len is None else max_len
        if not 1 <= max_len <= room:
            raise ValueError("max_len must be in [1, max_pages * block]")
        self.pages, self.rows, self.max_rows, self.max_len = pages, rows, max_rows, max_len
        i32 = dict(dtype=torch.int32, device=pages.table.device)
        self.row_start = torch.zeros(pages.n_seqs + 1, **i32)
        self.info = torch.zeros(4, **i32)
        self.positions = self.slots = self.batch = None
        if rows:
            self.positions = torch.full((rows,), -1, **i32)
            self.slots = torch.full((rows,), -1, dtype=torch.int64, device=pages.table.device)
            self.batch = tf.KvBatch(pages.kv_len, pages.table, max_len, self.row_start, rows, min(max_rows, rows), block=pages.block)
            self.slots.block = pages.block       # (of the tensor itself, as Kv4Cache.append looks at it)

    def step(self, change, stream=None):
        """Each sequence gets change[s] tokens (int32 [n_seqs]) or gives -change[s] back; returns self."""
        import torch
        p = self.pages
        if change.dtype != torch.int32 or change.shape != (p.n_seqs,) or not change.is_contiguous() or change.get_device() != p.device:
            _tensor(change, "change", (torch.int32,), (p.n_seqs,), device=p.device)
        _on_gpu(p.device, "the table")
        tf.tf_kv_plan(p.c, change, self.rows, self.max_rows, self.max_len, self.row_start, self.positions, self.slots,
                      self.info, stream)
        return self


class Rope:
    """Rotary positions of heads of `dim` values, the first rot_dim of which turn (tf_rope).

    Pair i turns by base ** (-2 i / rot_dim) a position; pairs are (i, i + rot_dim / 2), or neighbours (2 i, 2 i + 1)
    if interleaved.  scaling, for contexts longer than a model was made for:
        {"type": "linear", "factor"}      positions divided by factor
        {"type": "ntk", "factor"}         a larger base: base * factor ** (rot_dim / (rot_dim - 2))
        {"type": "bands", "factor", "low", "high", "original"}
                                          pairs that make more than `high` turns within the original context stay, those
                                          of less than `low` are divided by factor, in between the two are mixed
        {"type": "yarn", "factor", "original", "fast" (32), "slow" (1), "attention" (0.1 ln(factor) + 1)}
                                          the same by the pairs' numbers, between those of fast and slow turns; cosines
                                          and sines are multiplied by `attention`
    frequencies: radians a position of each pair, instead of base and scaling.

    Calls turn rows of any number of heads; `inverse` turns back (gradients)."""

    def __init__(self, dim, rot_dim=None, base=10000.0, scaling=None, interleaved=False, frequencies=None, factor=1.0,
                 device="cuda"):
        import torch
        rot = dim if rot_dim is None else rot_dim
        if dim < 2 or dim % 2 or dim > 1024 or rot < 2 or rot % 2 or rot > dim:
            raise ValueError("dim must be even, 2 to 1024, and rot_dim even, 2 to dim")
        if frequencies is None:
            if not base > 0:
                raise ValueError("base must be positive")
            frequencies, by = self.scaled(rot, base, scaling)
            factor *= by
        elif scaling is not None:
            raise ValueError("frequencies are given as they are, without scaling")
        if len(frequencies) != rot // 2 or not all(math.isfinite(f) for f in frequencies):
            raise ValueError("rot_dim / 2 finite frequencies are needed")
        self.dim, self.rot_dim, self.interleaved, self.factor = dim, rot, interleaved, factor
        self.frequencies = list(frequencies)
        # In 2^-64 of a turn, as the int64 of the same bits.
        turns = [round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for f in frequencies]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = self.turns.get_device()

    @staticmethod
    def scaled(rot, base, scaling):
        """Radians a position of each pair, and the factor of cosines and sines."""
        f = [base ** (-2 * i / rot) for i in range(rot // 2)]
        if scaling is None:
            return f, 1.0
        kind = scaling["type"]
        factor = float(scaling["factor"])
        if not factor > 0:
            raise ValueError("scaling's factor must be positive")
        if kind == "linear":
            return [x / factor for x in f], 1.0
        if kind == "ntk":
            if rot == 2:
                return f, 1.0
            base = base * factor ** (rot / (rot - 2))
            return [base ** (-2 * i / rot) for i in range(rot // 2)], 1.0
        if kind == "bands":
            low, high, original = (float(scaling[n]) for n in ("low", "high", "original"))
            if not (high > low and original > 0):
                raise ValueError("bands need low < high and a positive original")
            keep = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
            return [x * (k + (1 - k) / factor) for x, k in zip(f, keep)], 1.0
        if kind == "yarn":
            original = float(scaling["original"])
            if not original > 0 or base == 1:
                raise ValueError("yarn needs a positive original, and a base other than 1")

            def pair_of(turns):
                return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

            first = max(math.floor(pair_of(scaling.get("fast", 32.0))), 0)
            last = min(math.ceil(pair_of(scaling.get("slow", 1.0))), rot - 1)
            keep = [1 - min(max((i - first) / max(last - first, 0.001), 0.0), 1.0) for i in range(rot // 2)]
            return ([x * (k + (1 - k) / factor) for x, k in zip(f, keep)],
                    float(scaling.get("attention", 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)))
        raise ValueError("unknown scaling %r" % kind)

    def __call__(self, x, positions, out=None, inverse=False, stream=None):
        """Rows x [rows][heads * dim] (bf16 or fp32, row stride free) turned by positions [rows] int32; rows of a
        negative position are left as they are in `out`.  out: bf16 or fp32, x itself or other memory; a new tensor of
        x's type by default (zeros in rows of no position)."""
        import torch
        types = (torch.bfloat16, torch.float32)
        rows, width = x.shape
        xs = _rows(x, "x", types, rows, width, self.device)
        if out is None:
            out, os_ = torch.zeros((rows, width), dtype=x.dtype, device=x.device), width
        else:
            os_ = _rows(out, "out", types, rows, width, self.device)
        if positions.dtype != torch.int32 or positions.shape != (rows,) or not positions.is_contiguous() or positions.get_device() != self.device:
            _tensor(positions, "positions", (torch.int32,), (rows,), device=self.device)
        if width % self.dim or not width:
            raise ValueError("x's rows must hold heads * dim values")
        _on_gpu(self.device, "x")
        tf.tf_rope(self.turns, self.rot_dim, self.factor, positions, rows, x, xs, out, os_, width // self.dim, self.dim,
                   (tf.TF_IN_F32 if x.dtype == torch.float32 else 0) | (tf.TF_OUT_BF16 if out.dtype == torch.bfloat16 else 0) |
                   (tf.TF_ROPE_PAIRS if self.interleaved else 0) | (tf.TF_ROPE_BACK if inverse else 0), stream)
        return out


class Kv4Cache:
    """A 4-bit paged key/value cache (tf_kv4): a scale and a bias for every 64 values of a token's head.

    k, v [n_blocks][kv_heads][block][dim / 2] uint8 (two codes a byte, the low half first), k_affine, v_affine
    [n_blocks][kv_heads][block][dim / 64][2] bf16."""

    def __init__(self, k, v, k_affine, v_affine):
        import torch
        if k.dim() != 4:
            raise ValueError("k must be [n_blocks][kv_heads][block][dim / 2]")
        n_blocks, heads, block, half = k.shape
        _tensor(k, "k", (torch.uint8,))
        self.device = device = k.get_device()
        _tensor(v, "v", (torch.uint8,), k.shape, device=device)
        for t, name in ((k_affine, "k_affine"), (v_affine, "v_affine")):
            _tensor(t, name, (torch.bfloat16,), (n_blocks, heads, block, half // 32, 2), device=device)
        self.k, self.v, self.k_affine, self.v_affine = k, v, k_affine, v_affine
        self.kv_heads, self.block, self.dim = heads, block, 2 * half
        self.c = tf.TfKv4(_ptr(k), _ptr(v), _ptr(k_affine), _ptr(v_affine), n_blocks, heads, block, self.dim)

    @classmethod
    def empty(cls, n_blocks, kv_heads, dim, block=64, device="cuda"):
        """A new cache of n_blocks pages."""
        import torch
        code = dict(dtype=torch.uint8, device=device)
        pair = dict(dtype=torch.bfloat16, device=device)
        shape, groups = (n_blocks, kv_heads, block, dim // 2), (n_blocks, kv_heads, block, dim // 64, 2)
        return cls(torch.zeros(shape, **code), torch.zeros(shape, **code), torch.zeros(groups, **pair), torch.zeros(groups, **pair))

    _batch = tf.KvCache._batch

    def append(self, k, v, slots, stream=None) -> None:
        """Quantize rows k, v [rows][kv_heads * dim] (bf16 or fp32, row stride free) into slots [rows] int64
        (page * block + place in the page, -1: left out), as KvPlan gives them.  A plan's own slots are refused where its
        pages are of another size than the cache's; other tensors, slices of a plan's among them, are taken at their word."""
        import torch
        if getattr(slots, "block", self.block) != self.block:
            raise ValueError("the slots are of pages of %d tokens, the cache's hold %d" % (slots.block, self.block))
        rows, width = slots.shape[0], self.kv_heads * self.dim
        types = (torch.bfloat16, torch.float32)
        ks = _rows(k, "k", types, rows, width, self.device)
        vs = _rows(v, "v", (k.dtype,), rows, width, self.device)
        if slots.dtype != torch.int64 or slots.shape != (rows,) or not slots.is_contiguous() or slots.get_device() != self.device:
            _tensor(slots, "slots", (torch.int64,), (rows,), device=self.device)
        _on_gpu(self.device, "the cache")
        tf.tf_kv4_append(self.c, slots, rows, k, ks, v, vs, tf.TF_IN_F32 if k.dtype == torch.float32 else 0, stream)

    def read(self, batch, dtype=None, k_out=None, v_out=None, stream=None):
        """The batch's tokens as k, v rows [rows][kv_heads * dim] of dtype (by default the type of the output that is
        given, or bf16).  An output that is not given is made."""
        import torch
        types = (torch.bfloat16, torch.float32)
        given = k_out if k_out is not None else v_out
        dtype = dtype or (torch.bfloat16 if given is None else given.dtype)
        width = self.kv_heads * self.dim
        if dtype not in types:
            raise TypeError("read gives bf16 or fp32")
        k_out = torch.empty((batch.rows, width), dtype=dtype, device=self.k.device) if k_out is None else k_out
        v_out = torch.empty((batch.rows, width), dtype=dtype, device=self.k.device) if v_out is None else v_out
        ks = _rows(k_out, "k_out", (dtype,), batch.rows, width, self.device)
        vs = _rows(v_out, "v_out", (dtype,), batch.rows, width, self.device)
        tf.tf_kv4_read(self.c, self._batch(batch), k_out, ks, v_out, vs, tf.TF_OUT_BF16 if dtype == torch.bfloat16 else 0, stream)
        return k_out, v_out

    def attend(self, q, batch, out=None, scale=None, causal=True, window=0, stream=None, kernel=0):
        """Attention of q [rows][heads * dim] (bf16 or fp32) over the cache; out is bf16, scale 1/sqrt(dim) by default.

        kernel: 0 (by the call's sizes), TF_KV_BY_ROWS or TF_KV_BY_TILES."""
        import torch
        rows, width = q.shape
        qs = _rows(q, "q", (torch.bfloat16, torch.float32), batch.rows, width, self.device)
        if out is None:
            out = torch.empty((rows, width), dtype=torch.bfloat16, device=q.device)
            os_ = width
        else:
            os_ = _rows(out, "out", (torch.bfloat16,), rows, width, self.device)
        if width % self.dim:
            raise ValueError("q's rows must hold heads * dim values")
        tf.tf_kv4_attend(self.c, self._batch(batch), q, qs, width // self.dim, out, os_,
                         self.dim ** -0.5 if scale is None else scale, window,
                         (tf.TF_KV_CAUSAL if causal else 0) | (tf.TF_IN_F32 if q.dtype == torch.float32 else 0) | kernel, stream)
        return out
