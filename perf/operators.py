"""The decode-side operators and the cases they are measured on.

* ``cache``: new tokens' keys and values are quantised into an 8-bit paged cache (one scale per
  block of tokens and head), then the blocks they touched are read back.
* ``attend``: attention of new tokens over that cache, one token a sequence up to whole prompts.
* ``sample``: a token per row of logits, by temperature, top-k, top-p and min-p, from given random
  numbers.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls the framework.
"""
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --

def _cache(name, seqs, new, ragged, before, kv_heads, dim, block, dtype, gap, lens):
    """seqs sequences append up to `new` tokens each (ragged: 1..new) after up to `before` others; rows of
    the source are `gap` elements longer than the keys (a slice of a fused projection's output)."""
    return dict(name=name, op="cache", seqs=seqs, new=new, ragged=ragged, before=before, kv_heads=kv_heads,
                dim=dim, block=block, dtype=dtype, gap=gap, lens=lens)


def _attend(name, seqs, new, ragged, length, heads, kv_heads, dim, block, dtype, causal, window, lens):
    """seqs sequences of up to `length` cached tokens (ragged: from an eighth of that), the last `new` of which ask."""
    return dict(name=name, op="attend", seqs=seqs, new=new, ragged=ragged, length=length, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, causal=causal, window=window, lens=lens)


def _sample(name, rows, vocab, gap, dtype, mixed, masked, temperature, top_k, top_p, min_p):
    """rows of `vocab` logits; mixed: each row its own parameters around the given ones; masked: the share
    of tokens that a grammar forbids (logit -inf)."""
    return dict(name=name, op="sample", rows=rows, vocab=vocab, gap=gap, dtype=dtype, mixed=mixed, masked=masked,
                temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)


def listed():
    return [
        # One decode step of a batch: a token for each of 48 sequences, bf16 keys and values.
        _cache("cache_step", 48, 1, False, 4000, 8, 128, 64, "bf16", 0, 1),
        # Several prompts of different lengths in one call, short blocks, wide heads.
        _cache("cache_ragged", 7, 1000, True, 300, 2, 256, 32, "bf16", 4096, 2),
        # A whole prompt, fp32 rows out of a fused projection.
        _cache("cache_prompt", 1, 4000, False, 0, 8, 128, 64, "fp32", 4096, 3),
        # The smallest call: one sequence, a short conversation, one token; 4096 columns of queries.
        _attend("attend_one", 1, 1, False, 700, 16, 2, 256, 64, "bf16", True, 0, 4),
        # An ordinary decode step: a ragged batch.
        _attend("attend_batch", 48, 1, True, 8000, 32, 8, 128, 64, "bf16", True, 0, 5),
        # One sequence with a long document behind it.
        _attend("attend_long", 1, 1, False, 130977, 32, 8, 128, 128, "bf16", True, 0, 6),
        # Five drafted tokens a sequence are checked at once, fp32 queries.
        _attend("attend_verify", 16, 5, True, 4100, 16, 2, 256, 32, "fp32", True, 0, 7),
        # A whole prompt attends to itself.
        _attend("attend_prompt", 1, 4000, False, 4000, 32, 8, 128, 64, "bf16", True, 0, 8),
        # Prompts that go in by chunks, with a sliding window.
        _attend("attend_chunk", 3, 509, True, 12000, 16, 2, 256, 64, "bf16", True, 4096, 9),
        # The language model head's logits of one sequence (248320 tokens).
        _sample("sample_one", 1, 248320, 0, "fp32", False, 0.0, 0.8, 50, 0.95, 0.0),
        # The same for a batch whose requests ask for different things, some under a grammar.
        _sample("sample_batch", 48, 248320, 0, "fp32", True, 0.5, 1.0, 200, 0.9, 0.02),
        # Many rows of a small, odd vocabulary in bf16, with padded rows.
        _sample("sample_rows", 300, 32003, 61, "bf16", True, 0.0, 0.7, 0, 0.8, 0.05),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "sample"])
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (16, 2, 256), (8, 8, 64), (28, 4, 128), (16, 1, 64), (6, 2, 128)])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    lens = rng.randrange(1 << 30)
    if op == "cache":
        new = rng.choice([1, 1, _log(rng, 2, 4000)])
        seqs = _log(rng, 1, max(1, min(256, 5000 // (new + block))))
        case = _cache("", seqs, new, rng.random() < 0.5, _log(rng, 1, 4000), kv_heads, dim, block, dtype,
                      rng.choice([0, 0, 8, 4096]), lens)
    elif op == "attend":
        new = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 10, 4000)])
        length = _log(rng, max(new, 16), 4000 if new > 600 else 16000 if new > 8 else 130000)
        # No more than the largest listed cases' cache and pairs.
        seqs = 1 if new > 600 else _log(rng, 1, max(1, min(64, 190000 // length, 8000000 // (new * length))))
        window = rng.choice([0, 0, 0, _log(rng, 16, 8000)])
        case = _attend("", seqs, new, rng.random() < 0.5, length, heads, kv_heads, dim, block, dtype,
                       window > 0 or new > 600 or rng.random() < 0.8, window, lens)
    else:
        vocab = _log(rng, 1000, 248320)
        rows = _log(rng, 1, max(1, min(512, 48 * 248320 // vocab)))
        case = _sample("", rows, vocab, rng.choice([0, 0, 5, 64]), rng.choice(["fp32", "bf16"]), rng.random() < 0.5,
                       rng.choice([0.0, 0.0, 0.6]), round(0.3 + rng.random(), 3), rng.choice([0, 1, _log(rng, 2, 1000)]),
                       rng.choice([1.0, round(0.5 + 0.5 * rng.random(), 3)]),
                       rng.choice([0.0, round(0.2 * rng.random(), 3)]))
    del case["name"]
    return case


def _lengths(case):
    """Per sequence: tokens in the cache with the new ones, and new ones."""
    r = random.Random(case["lens"])
    total, new = [], []
    for i in range(case["seqs"]):
        n = r.randint(1, case["new"]) if case["ragged"] else case["new"]
        if case["op"] == "cache":
            b = r.randint(0, case["before"])
            total.append(b + n)
        else:
            lo = max(n, case["length"] // 8)
            total.append(max(n, r.randint(lo, case["length"]) if case["ragged"] and i else case["length"]))
        new.append(n)
    return total, new


# ---------------------------------------------------------------- inputs --

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _starts(counts):
    return [0] + np.cumsum(counts).tolist()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    state = dict(case)
    dt = _TYPES[case["dtype"]]
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        width = vocab + case["gap"]
        logits = randn(rows, width) * 2.0
        # A next-token distribution: a broad body and a few tokens far above it.
        hot = torch.randint(0, vocab, (rows, 40), generator=gen, device=DEV)
        logits.scatter_add_(1, hot, 6.0 + 2.5 * randn(rows, 40))
        if case["masked"]:
            logits[torch.rand((rows, width), generator=gen, device=DEV) < case["masked"]] = -torch.inf
        state["logits"] = logits.to(dt)[:, :vocab]
        mix = torch.rand((4, rows), generator=gen, device=DEV) if case["mixed"] else torch.zeros((4, rows), device=DEV)
        state["temperature"] = case["temperature"] * (1 - 0.5 * mix[0])
        state["top_k"] = (case["top_k"] * (1 - 0.9 * mix[1])).to(torch.int32)
        state["top_p"] = case["top_p"] + (1 - case["top_p"]) * mix[2]
        state["min_p"] = case["min_p"] * (1 - mix[3])
        state["u"] = torch.rand(rows, generator=gen, device=DEV)
        if own:
            import mlx_affine_bit_gb300 as tf
            state["tf"] = tf
        return state

    H, D, T, S = case["kv_heads"], case["dim"], case["block"], case["seqs"]
    total, new = _lengths(case)
    width = -(-max(total) // T)
    need = [-(-n // T) for n in total]
    n_blocks = sum(need) + 3
    pages = torch.randperm(n_blocks, generator=gen, device=DEV)[:sum(need)].to(torch.int32)
    table = torch.zeros((S, width), dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < ints(need)[:, None]] = pages
    rows = sum(new)
    state.update(table=table, kv_len=ints(total), row_start=ints(_starts(new)), rows=rows, max_new=max(new),
                 max_len=max(total))
    if case["op"] == "attend":
        shape = (n_blocks, H, T, D)
        state["k"] = (randn(*shape) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
        state["v"] = (randn(*shape) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
        state["k_scale"] = torch.exp(randn(n_blocks, H) * 0.2) * 0.02
        state["v_scale"] = torch.exp(randn(n_blocks, H) * 0.3) * 0.02
        state["q"] = (randn(rows, case["heads"] * D) * 3.0).to(dt)
        state["open_k"] = state["open_v"] = torch.zeros((S, H, 2 * T, D), dtype=dt, device=DEV)
        state["open_max"] = torch.zeros((S, 2, H, 2 * T), device=DEV)
    else:
        state["k"] = torch.zeros((n_blocks, H, T, D), dtype=torch.int8, device=DEV)
        state["v"] = torch.zeros((n_blocks, H, T, D), dtype=torch.int8, device=DEV)
        state["k_scale"] = torch.zeros((n_blocks, H), device=DEV)
        state["v_scale"] = torch.zeros((n_blocks, H), device=DEV)
        # Keys have channels that stand out; values have not.
        lift = 1.0 + 4.0 * (torch.rand(H * D, generator=gen, device=DEV) < 0.03)
        fused = (randn(rows, 2 * H * D + case["gap"]) * torch.exp(0.3 * randn(rows, 1))).to(dt)
        fused[:, case["gap"]:case["gap"] + H * D] *= lift
        state["new_k"] = fused[:, case["gap"]:case["gap"] + H * D]
        state["new_v"] = fused[:, case["gap"] + H * D:]
        # The blocks that are already begun: their tokens' originals, codes and scales.
        past = state["kv_len"].long() - ints(new)
        state["open_k"] = (randn(S, H, 2 * T, D) * lift.view(1, H, 1, D)).to(dt)
        state["open_v"] = randn(S, H, 2 * T, D).to(dt)
        state["open_max"] = torch.stack([state["open_k"].float().abs().amax(-1), state["open_v"].float().abs().amax(-1)], 1)
        begun = past % T
        at = (past - begun)[:, None] % (2 * T) + torch.arange(T, device=DEV)
        page = table.gather(1, (past // T).clamp(max=width - 1)[:, None])[:, 0].long()
        for ring, pool, scale in ((state["open_k"], state["k"], state["k_scale"]),
                                  (state["open_v"], state["v"], state["v_scale"])):
            x = ring.gather(2, at[:, None, :, None].expand(S, H, T, D)).float()
            x = torch.where((torch.arange(T, device=DEV) < begun[:, None])[:, None, :, None], x, 0.0)
            s = x.abs().amax((2, 3)) / 127.0
            pool[page] = torch.where(s[..., None, None] > 0, (x / s[..., None, None]).round(), 0.0).to(torch.int8)
            scale[page] = s
        # What is read back: the blocks that the new tokens touch.
        back = [n - (n - m) // T * T for n, m in zip(total, new)]
        state.update(back=ints(_starts(back)), back_rows=sum(back), max_back=max(back))
    if own:
        import mlx_affine_bit_gb300 as tf
        state["cache"] = tf.KvCache(state["k"], state["v"], state["k_scale"], state["v_scale"], state["open_k"],
                                    state["open_v"], state["open_max"])
        state["batch"] = tf.KvBatch(state["kv_len"], table, state["max_len"], state["row_start"], rows, max(new))
        if case["op"] == "cache":
            state["reading"] = tf.KvBatch(state["kv_len"], table, state["max_len"], state["back"], sum(back), max(back))
    return state


# ------------------------------------------------------------- plain forms --

def _row_places(starts, rows, kv_len):
    """Of each row: its sequence, its place among that sequence's rows, its position in the sequence."""
    starts = starts.long()
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(starts, r, right=True) - 1
    i = r - starts[seq]
    return seq, i, kv_len.long()[seq] - (starts[seq + 1] - starts[seq]) + i


def _quantise(state, new_rows, pool, scale, ring, peak):
    """Appends one of keys and values: pool, scale, ring and peak (the tokens' magnitudes) are updated."""
    H, D, T, S = state["kv_heads"], state["dim"], state["block"], state["seqs"]
    starts, end = state["row_start"].long(), state["kv_len"].long()
    first = end - (starts[1:] - starts[:-1])
    width = state["table"].shape[1]
    nb = -(-state["max_new"] // T) + 1
    block = (first // T)[:, None] + torch.arange(nb, device=DEV)                      # [S][nb]
    pos = block[..., None] * T + torch.arange(T, device=DEV)                          # [S][nb][T]
    row = (starts[:-1, None, None] + pos - first[:, None, None]).clamp(0, state["rows"] - 1)
    fresh = new_rows.float().view(state["rows"], H, D)[row]                           # [S][nb][T][H][D]
    old = ring.float().permute(0, 2, 1, 3)[torch.arange(S, device=DEV)[:, None, None], pos % (2 * T)]
    x = torch.where((pos < first[:, None, None])[..., None, None], old, fresh)
    x = torch.where((pos < end[:, None, None])[..., None, None], x, 0.0)
    s = x.abs().amax((2, 4)) / 127.0                                                  # [S][nb][H]
    c = torch.where(s[:, :, None, :, None] > 0, (x / s[:, :, None, :, None]).round().clamp(-127, 127), 0.0).to(torch.int8)
    live = block * T < end[:, None]
    page = state["table"].long().gather(1, block.clamp(max=width - 1))[live]
    pool[page] = c.permute(0, 1, 3, 2, 4)[live]
    scale[page] = s[live]
    seq, _, at = _row_places(state["row_start"], state["rows"], state["kv_len"])
    keep = at >= ((end + T - 1) // T * T - 2 * T)[seq]
    values = new_rows.view(state["rows"], H, D)[keep]
    ring[seq[keep], :, at[keep] % (2 * T)] = values
    peak[seq[keep], :, at[keep] % (2 * T)] = values.float().abs().amax(-1)


def _read(state, pool, scale, dt):
    seq, _, at = _row_places(state["back"], state["back_rows"], state["kv_len"])
    page = state["table"].long()[seq, at // state["block"]]
    return (pool[page, :, at % state["block"]].float() * scale[page][..., None]).flatten(1).to(dt)


def _run_cache(state):
    dt = _TYPES[state["dtype"]]
    _quantise(state, state["new_k"], state["k"], state["k_scale"], state["open_k"], state["open_max"][:, 0])
    _quantise(state, state["new_v"], state["v"], state["v_scale"], state["open_v"], state["open_max"][:, 1])
    return _read(state, state["k"], state["k_scale"], dt), _read(state, state["v"], state["v_scale"], dt)


def _run_attend(state):
    S, n, L, T = state["seqs"], state["max_new"], state["max_len"], state["block"]
    Hq, H, D = state["heads"], state["kv_heads"], state["dim"]
    page = state["table"].long()

    def dense(pool, scale):                                                           # [S][H][tokens][D]
        x = pool[page].float() * scale[page][..., None, None]
        return x.transpose(1, 2).reshape(S, H, -1, D)[:, :, :L]

    k = dense(state["k"], state["k_scale"])
    starts, end = state["row_start"].long(), state["kv_len"].long()
    count = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + torch.arange(n, device=DEV)).clamp(max=state["rows"] - 1)
    q = state["q"].float()[row].view(S, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(S, H, -1, D)
    scores = q @ k.transpose(2, 3) * D ** -0.5                                        # [S][H][G n][L]
    del k, q
    key = torch.arange(L, device=DEV)
    seen = (key < end[:, None])[:, None, :].expand(S, n, L)
    if state["causal"]:
        place = (end - count)[:, None] + torch.arange(n, device=DEV)
        seen = seen & (key <= place[..., None])
        if state["window"]:
            seen = seen & (key > place[..., None] - state["window"])
    scores = scores.view(S, H, Hq // H, n, L).masked_fill_(~seen[:, None, None], -torch.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(top == -torch.inf, 0.0, top)))
    del scores
    total = p.sum(-1, keepdim=True)
    out = (p.view(S, H, -1, L) @ dense(state["v"], state["v_scale"])).view(S, H, Hq // H, n, D)
    out = torch.where(total > 0, out / total, 0.0)
    seq, i, _ = _row_places(state["row_start"], state["rows"], state["kv_len"])
    return out.permute(0, 3, 1, 2, 4)[seq, i].reshape(state["rows"], Hq * D).to(torch.bfloat16)


def _run_sample(state):
    x = state["logits"].float()
    vocab = x.shape[1]
    x = torch.where(torch.isnan(x), -torch.inf, x)
    top, best = x.amax(1, keepdim=True), x.argmax(1)
    temperature = state["temperature"]
    greedy = ~(temperature > 0)
    z = torch.where(x == top, 0.0, (x - top) * (1.0 / temperature)[:, None])
    # Weights are whole numbers (31 bits below the largest), so their sums do not depend on the order.
    w = (torch.exp(z) * 2147483648.0).round().to(torch.int64)
    w = torch.where(x == -torch.inf, 0, w)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    run = ws.cumsum(1)
    place = torch.arange(vocab, device=DEV)
    k = torch.where(state["top_k"] > 0, state["top_k"], vocab).clamp(max=vocab).long()
    in_k = run.gather(1, (k - 1)[:, None])
    kept = place < k[:, None]
    p = state["top_p"].double()[:, None]
    kept &= (place == 0) | (p >= 1) | ((run - ws).double() < p * in_k.double())
    kept &= ws.double() >= state["min_p"].clamp(max=1.0).double()[:, None] * 2147483648.0
    w = torch.zeros_like(w).scatter_(1, order, torch.where(kept, ws, 0))
    run = w.cumsum(1)
    whole = run[:, -1]
    hit = run.double() > (state["u"].double() * whole.double())[:, None]
    token = torch.where(greedy, best, hit.to(torch.uint8).argmax(1))
    share = (w.gather(1, token[:, None])[:, 0].double() / whole.double()).float()
    share = torch.where(greedy, 1.0, share)
    dead = top[:, 0] == -torch.inf
    return torch.where(dead, -1, token).to(torch.int32), torch.where(dead, 0.0, share)


def run(state):
    if own:
        if state["op"] == "sample":
            return state["tf"].sample(state["logits"], state["u"], temperature=state["temperature"],
                                      top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
        if state["op"] == "attend":
            return state["cache"].attend(state["q"], state["batch"], causal=state["causal"], window=state["window"])
        state["cache"].append(state["new_k"], state["new_v"], state["batch"])
        k, v = state["cache"].read(state["reading"])
    elif state["op"] == "sample":
        return _run_sample(state)
    elif state["op"] == "attend":
        return _run_attend(state)
    else:
        k, v = _run_cache(state)
    return {"k": k, "v": v, "k_scale": state["k_scale"], "v_scale": state["v_scale"], "open_k": state["open_k"],
            "open_v": state["open_v"], "open_max": state["open_max"]}


# ------------------------------------------------------------ definitions --

def _exact_cache(state):
    """Sequence by sequence and block by block, in 64 bits."""
    H, D, T = state["kv_heads"], state["dim"], state["block"]
    total, new = _lengths(state)
    out = {}
    for name, side in (("k", 0), ("v", 1)):
        ring = state["open_" + name].double().clone()
        peak = state["open_max"][:, side].double().clone()
        scale = state[name + "_scale"].double().clone()
        back, r = [], 0
        for s, (end, n) in enumerate(zip(total, new)):
            first = end - n
            begun = first // T * T
            old = ring[s][:, [p % (2 * T) for p in range(begun, first)]]
            rows = state["new_" + name][r:r + n].double().view(n, H, D).transpose(0, 1)
            x = torch.cat([old, rows], 1)
            for b in range(0, x.shape[1], T):
                part = x[:, b:b + T]
                step = part.abs().flatten(1).max(1).values / 127
                back.append((torch.round(part / step[:, None, None].clamp(min=1e-300)) * step[:, None, None]).transpose(0, 1).flatten(1))
                scale[state["table"][s, (begun + b) // T].long()] = step
            from_ = max(first, ((end + T - 1) // T - 2) * T)
            for p in range(from_, end):
                ring[s][:, p % (2 * T)] = rows[:, p - first]
                peak[s][:, p % (2 * T)] = rows[:, p - first].abs().max(1).values
            r += n
        out[name], out[name + "_scale"], out["open_" + name], out[name + "_max"] = torch.cat(back), scale, ring, peak
    return {"k": out["k"], "v": out["v"], "k_scale": out["k_scale"], "v_scale": out["v_scale"], "open_k": out["open_k"],
            "open_v": out["open_v"], "open_max": torch.stack([out["k_max"], out["v_max"]], 1)}


def _exact_attend(state):
    """Sequence by sequence and head by head, in 64 bits."""
    H, D, G = state["kv_heads"], state["dim"], state["heads"] // state["kv_heads"]
    total, new = _lengths(state)
    result, r = [], 0
    for s, (L, n) in enumerate(zip(total, new)):
        pages = state["table"][s, :-(-L // state["block"])].long()
        heads = []
        for h in range(H):
            k = (state["k"][pages, h].double() * state["k_scale"][pages, h, None, None].double()).flatten(0, 1)[:L]
            v = (state["v"][pages, h].double() * state["v_scale"][pages, h, None, None].double()).flatten(0, 1)[:L]
            for g in range(G):
                column = (h * G + g) * D
                q = state["q"][r:r + n, column:column + D].double()
                score = torch.einsum("id,jd->ij", q, k) / D ** 0.5
                if state["causal"]:
                    i, j = torch.arange(L - n, L, device=DEV)[:, None], torch.arange(L, device=DEV)[None]
                    hidden = j > i
                    if state["window"]:
                        hidden |= i - j >= state["window"]
                    score[hidden] = -torch.inf
                heads.append(torch.softmax(score, 1) @ v)
        result.append(torch.cat(heads, 1))
        r += n
    return torch.cat(result)


def _exact_sample(state):
    """Row by row, in 64 bits and without rounded weights."""
    tokens, shares = [], []
    for row in range(state["rows"]):
        x = state["logits"][row].double().cpu().numpy()
        t, k = float(state["temperature"][row]), int(state["top_k"][row])
        p, m, u = float(state["top_p"][row]), float(state["min_p"][row]), float(state["u"][row])
        order = np.argsort(-x, kind="stable")
        w = np.exp((x[order] - x[order[0]]) / t)
        keep = k if 0 < k < len(w) else len(w)
        if p < 1:
            keep = min(keep, max(1, int(np.searchsorted(np.cumsum(w[:keep]), p * w[:keep].sum())) + 1))
        keep = min(keep, int((w >= m).sum()))
        kept = np.sort(order[:keep])
        weight = np.exp((x[kept] - x[order[0]]) / t)
        at = min(int(np.searchsorted(np.cumsum(weight), u * weight.sum(), side="right")), keep - 1)
        tokens.append(int(kept[at]))
        shares.append(weight[at] / weight.sum())
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(shares, dtype=torch.float64)


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 4e11:
        return None  # 64-bit products of that size take too long
    global own
    mode, own = own, False
    state = prepare(case, seed)
    own = mode
    return {"cache": _exact_cache, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](state)


# ----------------------------------------------------------------- floors --

def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "fp32" else 2
        # Each logit: read, an exponential's worth of arithmetic, a comparison and a sum.
        return {"bytes": case["rows"] * (case["vocab"] * size + 32), "flops": case["rows"] * case["vocab"] * 8}
    total, new = _lengths(case)
    H, D, T = case["kv_heads"], case["dim"], case["block"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "cache":
        back = sum(n - (n - m) // T * T for n, m in zip(total, new))
        blocks = sum(-(-n // T) - (n - m) // T for n, m in zip(total, new))
        kept = sum(min(m, n - (-(-n // T) - 2) * T) for n, m in zip(total, new))
        # Rows in, codes and originals out; codes in, rows out; both of keys and values.
        values = sum(new) * (size + 1) + kept * size + back * (1 + size)
        return {"bytes": 2 * H * (D * values + 4 * kept + 8 * blocks), "flops": 2 * H * D * (4 * sum(new) + back)}
    pairs = seen = 0
    for n, m in zip(total, new):
        if not case["causal"]:
            pairs, seen = pairs + m * n, seen + n
            continue
        w = case["window"] or n
        first = np.arange(n - m, n)
        pairs += int(np.minimum(first + 1, w).sum())
        seen += min(n, m - 1 + w)
    rows = sum(new)
    return {"bytes": 2 * H * seen * (D + 4 / T) + rows * case["heads"] * D * (size + 2) + 4 * sum(-(-n // T) for n in total),
            "flops": 4 * case["heads"] * D * pairs}
