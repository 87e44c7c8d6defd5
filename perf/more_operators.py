"""Operators that serving adds around the products and the 8-bit cache, and the cases they are measured on.

* ``plan``: page tables, row starts, positions and slots of a step, made on the device from how many tokens
  each sequence gets or gives back.
* ``rope``: queries and keys turned by their positions (and gradients turned back): halves or neighbours,
  part of the head, frequencies scaled for long contexts.
* ``cache4``: new tokens' keys and values quantised into a paged cache of 4 bits (a scale and a bias for
  every 64 values of a token's head), then read back.
* ``attend4``: attention of new tokens over that cache, one token a sequence up to whole prompts.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits (angles, and values in
the middle of two codes, in 64); with ``own`` true it calls the framework.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 64              # values that share a scale and a bias


# ------------------------------------------------------------------ cases --

def _plan(name, seqs, new, ragged, held, block, back, pad, lens):
    """seqs sequences of up to `held` tokens get up to `new` each (ragged: 0..new); of a share `back` as many are
    taken away instead; the row buffers have `pad` rows more than the step's."""
    return dict(name=name, op="plan", seqs=seqs, new=new, ragged=ragged, held=held, block=block, back=back, pad=pad,
                lens=lens)


def _rope(name, rows, heads, dim, rot, interleaved, src, dst, gap, base, scaling, far, pad, inverse, lens):
    """rows of `heads` heads, the first `rot` of `dim` values of each turned, `gap` values between the rows (the
    values' columns of a fused projection); positions up to `far`, the last `pad` rows without one."""
    return dict(name=name, op="rope", rows=rows, heads=heads, dim=dim, rot=rot, interleaved=interleaved, src=src,
                dst=dst, gap=gap, base=base, scaling=scaling, far=far, pad=pad, inverse=inverse, lens=lens)


def _cache(name, seqs, new, ragged, before, kv_heads, dim, block, dtype, gap, lens):
    """seqs sequences append up to `new` tokens each (ragged: 1..new) after up to `before` others; rows of
    the source are `gap` elements longer than the keys and values."""
    return dict(name=name, op="cache4", seqs=seqs, new=new, ragged=ragged, before=before, kv_heads=kv_heads,
                dim=dim, block=block, dtype=dtype, gap=gap, lens=lens)


def _attend(name, seqs, new, ragged, length, heads, kv_heads, dim, block, dtype, causal, window, lens):
    """seqs sequences of up to `length` cached tokens (ragged: from an eighth of that), the last `new` of which ask."""
    return dict(name=name, op="attend4", seqs=seqs, new=new, ragged=ragged, length=length, heads=heads,
                kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, causal=causal, window=window, lens=lens)


def listed():
    return [
        # The smallest step: a token for each of 48 sequences is given its place (and taken back, as a rejected draft is).
        _plan("plan_step", 48, 1, False, 4000, 64, 0.0, 16, 1),
        # Prompts of many requests at once, short pages; some requests give tokens back.
        _plan("plan_prompts", 256, 500, True, 8000, 16, 0.1, 40, 2),
        # A decode step's queries and keys out of a fused projection, a quarter of each head turned, far positions.
        _rope("rope_step", 48, 18, 256, 64, False, "fp32", "fp32", 512, 1e7, "bands", 130000, 0, False, 3),
        # A whole prompt's queries and keys, rounded for the attention that follows.
        _rope("rope_prompt", 4000, 40, 128, 128, False, "fp32", "bf16", 1024, 5e5, "yarn", 4000, 7, False, 4),
        # Gradients of queries and keys of a batch of sequences, neighbours turned back.
        _rope("rope_back", 16000, 16, 64, 64, True, "bf16", "bf16", 0, 1e4, "none", 16000, 0, True, 5),
        # One decode step of a batch: a token for each of 48 sequences.
        _cache("cache4_step", 48, 1, False, 4000, 8, 128, 64, "bf16", 0, 6),
        # A whole prompt, fp32 rows out of a fused projection.
        _cache("cache4_prompt", 1, 4000, False, 0, 8, 128, 64, "fp32", 4096, 7),
        # The smallest attention: one sequence, a short conversation, one token, wide heads.
        _attend("attend4_one", 1, 1, False, 700, 16, 2, 256, 64, "bf16", True, 0, 8),
        # An ordinary decode step: a ragged batch.
        _attend("attend4_batch", 48, 1, True, 8000, 32, 8, 128, 64, "bf16", True, 0, 9),
        # One sequence with a long document behind it.
        _attend("attend4_long", 1, 1, False, 130977, 32, 8, 128, 128, "bf16", True, 0, 10),
        # Prompts that go in by chunks, with a sliding window, fp32 queries.
        _attend("attend4_chunk", 3, 509, True, 12000, 16, 2, 256, 64, "fp32", True, 4096, 11),
        # A whole prompt attends to itself.
        _attend("attend4_prompt", 1, 4000, False, 4000, 32, 8, 128, 64, "bf16", True, 0, 12),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["plan", "rope", "cache4", "attend4", "attend4"])
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (16, 2, 256), (8, 8, 64), (28, 4, 128), (16, 1, 64), (6, 2, 128)])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    lens = rng.randrange(1 << 30)
    if op == "plan":
        seqs = _log(rng, 1, 1000)
        new = rng.choice([1, rng.randrange(2, 9), _log(rng, 10, max(20, 120000 // seqs))])
        case = _plan("", seqs, new, rng.random() < 0.7, _log(rng, 1, 8000), block, rng.choice([0.0, 0.0, 0.2]),
                     rng.randrange(50), lens)
    elif op == "rope":
        rows = _log(rng, 1, 800000 // ((heads + kv_heads) * dim // 32))
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        case = _rope("", rows, heads + kv_heads, dim, rot, rng.random() < 0.4, dtype, rng.choice([dtype, "bf16"]),
                     rng.choice([0, kv_heads * dim, 6]), rng.choice([1e4, 5e5, 1e7]),
                     rng.choice(["none", "linear", "ntk", "bands", "yarn"]), _log(rng, 100, 1000000),
                     rng.choice([0, 0, rng.randrange(rows)]), rng.random() < 0.3, lens)
    elif op == "cache4":
        new = rng.choice([1, 1, _log(rng, 2, 4000)])
        seqs = _log(rng, 1, max(1, min(256, 5000 // (new + block))))
        case = _cache("", seqs, new, rng.random() < 0.5, _log(rng, 1, 4000), kv_heads, dim, block, dtype,
                      rng.choice([0, 0, 8, 4096]), lens)
    else:
        new = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 10, 4000)])
        length = _log(rng, max(new, 16), 4000 if new > 600 else 16000 if new > 8 else 130000)
        # No more than the largest listed cases' cache and pairs.
        seqs = 1 if new > 600 else _log(rng, 1, max(1, min(64, 190000 // length, 8000000 // (new * length))))
        window = rng.choice([0, 0, 0, _log(rng, 16, 8000)])
        case = _attend("", seqs, new, rng.random() < 0.5, length, heads, kv_heads, dim, block, dtype,
                       window > 0 or new > 600 or rng.random() < 0.8, window, lens)
    del case["name"]
    return case


def _lengths(case):
    """Per sequence: tokens in the cache with the new ones, and new ones (plan: tokens held before, and their change)."""
    r = random.Random(case["lens"])
    total, new = [], []
    for i in range(case["seqs"]):
        if case["op"] == "plan":
            held = r.randint(0, case["held"])
            n = r.randint(0, case["new"]) if case["ragged"] else case["new"]
            total.append(held)
            new.append(-min(n, held) if r.random() < case["back"] else n)
            continue
        n = r.randint(1, case["new"]) if case["ragged"] else case["new"]
        if case["op"] == "cache4":
            total.append(r.randint(0, case["before"]) + n)
        else:
            lo = max(n, case["length"] // 8)
            total.append(max(n, r.randint(lo, case["length"]) if case["ragged"] and i else case["length"]))
        new.append(n)
    return total, new


# What a model's configuration says of scaled frequencies.
_SCALING = {
    "none": None,
    "linear": dict(type="linear", factor=4.0),
    "ntk": dict(type="ntk", factor=8.0),
    "bands": dict(type="bands", factor=8.0, low=1.0, high=4.0, original=8192),
    "yarn": dict(type="yarn", factor=16.0, original=4096, fast=32.0, slow=1.0),
}


# ---------------------------------------------------------------- inputs --

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _starts(counts):
    return [0] + np.cumsum(counts).tolist()


def _tables(need, width, gen):
    """Pages of sequences that need so many each, in any order, and the other pages."""
    n_blocks = sum(need)
    pages = torch.randperm(n_blocks + n_blocks // 4 + 3, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    held = torch.tensor(need, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < held[:, None]] = pages[:n_blocks]
    return table, pages[n_blocks:], len(pages)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    state = dict(case)
    if own:
        import mlx_affine_bit_gb300 as tf
    if case["op"] == "rope":
        rows, width = case["rows"], case["heads"] * case["dim"]
        state["x"] = (randn(rows, width + case["gap"]) * 2.0).to(_TYPES[case["src"]])[:, :width]
        # Rows of several sequences, each at consecutive positions from anywhere.
        r = random.Random(case["lens"])
        live = rows - case["pad"]
        cuts = sorted(r.randrange(live + 1) for _ in range(min(live, 48)))
        first = torch.randint(0, case["far"], (len(cuts) + 1,), generator=gen, device=DEV)
        at = torch.arange(rows, device=DEV)
        seq = torch.searchsorted(torch.tensor(cuts + [rows + 1], device=DEV), at, right=True)
        position = (first[seq] + at) % case["far"]
        state["position"] = torch.where(at < live, position, -1).to(torch.int32)
        state["out"] = torch.zeros((rows, width), dtype=_TYPES[case["dst"]], device=DEV)
        if own:
            state["turn"] = tf.Rope(case["dim"], case["rot"], base=case["base"], scaling=_SCALING[case["scaling"]],
                                    interleaved=case["interleaved"])
        return state

    T, S = case["block"], case["seqs"]
    total, new = _lengths(case)
    if case["op"] == "plan":
        grown = max(1, max(n + max(m, 0) for n, m in zip(total, new)))
        need = [-(-n // T) for n in total]
        more = sum(max(0, -(-(n + m) // T) - k) for n, m, k in zip(total, new, need))
        width = -(-grown // T) + 2
        table, free, n_blocks = _tables(need, width, gen)
        pool = torch.randperm(n_blocks + more, generator=gen, device=DEV).to(torch.int32)     # every page by another number
        table = torch.where(table < 0, -1, pool[table.clamp(min=0).long()])
        stack = torch.full((n_blocks + more,), -1, dtype=torch.int32, device=DEV)
        stack[:len(free)] = pool[free.long()]
        stack[len(free):len(free) + more] = pool[n_blocks:]
        rows = sum(max(0, m) for m in new) + case["pad"]
        state.update(table=table, kv_len=ints(total), free=stack, n_free=ints([len(free) + more]), change=ints(new),
                     undo=ints([-m for m in new]), rows=rows, max_rows=max(1, max(abs(m) for m in new)), max_len=grown)
        if own:
            pages = tf.KvPages(table, state["kv_len"], stack, state["n_free"], T)
            state["plan"] = pages.plan(rows, state["max_rows"], grown)
            state["take_back"] = pages.plan(0, state["max_rows"], grown)
        return state

    H, D = case["kv_heads"], case["dim"]
    dt = _TYPES[case["dtype"]]
    table, _, n_blocks = _tables([-(-n // T) for n in total], -(-max(total) // T), gen)
    rows = sum(new)
    state.update(table=table, kv_len=ints(total), row_start=ints(_starts(new)), rows=rows, max_new=max(new),
                 max_len=max(total))
    shape, groups = (n_blocks, H, T, D // 2), (n_blocks, H, T, D // GROUP, 2)
    if case["op"] == "attend4":
        for name in ("k", "v"):
            # Codes as rounded normal values have them, a scale and a bias a group.
            code = (randn(n_blocks, H, T, D) * 2.7 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
            state[name] = code[..., 0::2] | (code[..., 1::2] << 4)
            scale = torch.exp(randn(*groups[:-1]) * 0.25) * 0.35
            state[name + "_affine"] = torch.stack([scale, -7.5 * scale * (1 + 0.1 * randn(*groups[:-1]))], -1).to(torch.bfloat16)
        state["q"] = (randn(rows, case["heads"] * D) * 3.0).to(dt)
    else:
        for name in ("k", "v"):
            state[name] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            state[name + "_affine"] = torch.zeros(groups, dtype=torch.bfloat16, device=DEV)
        # Keys have channels that stand out; values have not.
        lift = 1.0 + 4.0 * (torch.rand(H * D, generator=gen, device=DEV) < 0.03)
        fused = (randn(rows, 2 * H * D + case["gap"]) * torch.exp(0.3 * randn(rows, 1))).to(dt)
        fused[:, case["gap"]:case["gap"] + H * D] *= lift
        state["new_k"] = fused[:, case["gap"]:case["gap"] + H * D]
        state["new_v"] = fused[:, case["gap"] + H * D:]
        seq, at = _row_places(state)
        state["slots"] = table.long()[seq, at // T] * T + at % T
    if own:
        state["cache"] = tf.Kv4Cache(state["k"], state["v"], state["k_affine"], state["v_affine"])
        state["batch"] = tf.KvBatch(state["kv_len"], table, state["max_len"], state["row_start"], rows, max(new))
    return state


# ------------------------------------------------------------- plain forms --

def _row_places(state):
    """Of each row: its sequence, its position in the sequence."""
    starts, end = state["row_start"].long(), state["kv_len"].long()
    r = torch.arange(state["rows"], device=DEV)
    seq = torch.searchsorted(starts, r, right=True) - 1
    return seq, end[seq] - starts[seq + 1] + r


def _run_plan(state, change, rows):
    """Pages given back go onto the stack, then pages are taken from it, sequence by sequence."""
    T, width = state["block"], state["table"].shape[1]
    old = state["kv_len"].long()
    end = old + change
    had, has = (old + T - 1) // T, (end + T - 1) // T
    gone, more = (had - has).clamp(min=0), (has - had).clamp(min=0)
    at = torch.arange(width, device=DEV)
    top = state["n_free"].long() + gone.sum()
    leave = (at >= has[:, None]) & (at < had[:, None])
    place = top - 1 - ((gone.cumsum(0) - gone)[:, None] + at - has[:, None])
    n = state["free"].shape[0]
    free = torch.cat([state["free"], state["free"][:1]])
    free[torch.where(leave, place, n)] = state["table"]
    free = free[:n]
    enter = (at >= had[:, None]) & (at < has[:, None])
    place = top - 1 - ((more.cumsum(0) - more)[:, None] + at - had[:, None])
    page = free[place.clamp(0, n - 1)]
    table = torch.where(enter, page, torch.where(leave, -1, state["table"]))
    state["table"].copy_(table)
    state["free"].copy_(free)
    state["kv_len"].copy_(end)
    state["n_free"].copy_(top - more.sum())
    starts = torch.cat([torch.zeros_like(old[:1]), change.long().clamp(min=0).cumsum(0)])
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(starts, r, right=True) - 1
    live = r < starts[-1]
    seq = seq.clamp(max=state["seqs"] - 1)
    position = torch.where(live, old[seq] + r - starts[seq], 0)
    slot = table[seq, position // T].long() * T + position % T
    info = torch.stack([torch.zeros_like(starts[-1]), torch.zeros_like(starts[-1]), starts[-1], end.amax()])
    return (starts.to(torch.int32), torch.where(live, position, -1).to(torch.int32), torch.where(live, slot, -1),
            info.to(torch.int32))


def _frequencies(case):
    """Radians a position of each pair (64 bits), and the factor of cosines and sines."""
    rot, base, s = case["rot"], case["base"], _SCALING[case["scaling"]]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if s is None:
        return base ** (-2 * i / rot), 1.0
    if s["type"] == "ntk":
        return (base * s["factor"] ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    f = base ** (-2 * i / rot)
    if s["type"] == "linear":
        return f / s["factor"], 1.0
    if s["type"] == "bands":
        # Turns within the original context: many are kept, few are stretched, in between both are mixed.
        turns = s["original"] * f / (2 * math.pi)
        keep = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return f * (keep + (1 - keep) / s["factor"]), 1.0

    def pair_of(turns):
        return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(pair_of(s["fast"])), 0), min(math.ceil(pair_of(s["slow"])), rot - 1)
    keep = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (keep + (1 - keep) / s["factor"]), 0.1 * math.log(s["factor"]) + 1.0


def _run_rope(state):
    heads, dim, rot = state["heads"], state["dim"], state["rot"]
    f, factor = _frequencies(state)
    angle = state["position"].double()[:, None] * f
    c = (torch.cos(angle) * factor).float()[:, None]
    s = (torch.sin(angle) * (-factor if state["inverse"] else factor)).float()[:, None]
    x = state["x"].float().view(-1, heads, dim)
    if state["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    y = torch.cat([y, x[..., rot:]], -1).flatten(1).to(state["out"].dtype)
    return torch.where((state["position"] >= 0)[:, None], y, state["out"])


def _bf16_below(x):
    """The largest bf16 number that is not above x (fp32)."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    return torch.where((bits < 0) & (cut != bits), cut + 65536, cut).view(torch.float32) + 0.0


def _bf16_above(x):
    """The smallest bf16 number that is not below x (64 bits, not negative)."""
    y = x.float()
    y = torch.where(y.double() < x, torch.nextafter(y, torch.full_like(y, torch.inf)), y)
    return ((y.view(torch.int32) + 65535) & -65536).view(torch.float32)


def _quantise(state, new, pool, affine):
    H, D, T = state["kv_heads"], state["dim"], state["block"]
    most = 2.0 ** 126
    x = new.float().view(-1, H, D // GROUP, GROUP)
    whole = torch.isfinite(x)
    some = whole.any(-1)
    x = torch.nan_to_num(x, nan=0.0, posinf=most, neginf=-most).clamp(-most, most)
    lo = torch.where(some, torch.where(whole, x, torch.inf).amin(-1), 0.0)
    hi = torch.where(some, torch.where(whole, x, -torch.inf).amax(-1), 0.0)
    bias = _bf16_below(lo)
    scale = _bf16_above((hi.double() - bias.double()) / 15.0)
    wide = scale.double()[..., None]
    code = ((x.double() - bias.double()[..., None]) / torch.where(wide > 0, wide, 1.0)).round().clamp(0, 15)
    code = torch.where(wide > 0, code, 0.0).to(torch.uint8).flatten(2)
    page, at = state["slots"] // T, state["slots"] % T
    pool[page, :, at] = code[..., 0::2] | (code[..., 1::2] << 4)
    affine[page, :, at] = torch.stack([scale, bias], -1).to(torch.bfloat16)


def _values(code, affine):
    """Values of codes [...][dim / 2] with scales and biases [...][dim / 64][2], in 32 bits."""
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2).float()
    c = c.view(*c.shape[:-1], -1, GROUP)
    a = affine.float()
    return (c * a[..., :1] + a[..., 1:]).flatten(-2)


def _run_cache(state):
    _quantise(state, state["new_k"], state["k"], state["k_affine"])
    _quantise(state, state["new_v"], state["v"], state["v_affine"])
    page, at = state["slots"] // state["block"], state["slots"] % state["block"]
    dt = _TYPES[state["dtype"]]
    return (_values(state["k"][page, :, at], state["k_affine"][page, :, at]).flatten(1).to(dt),
            _values(state["v"][page, :, at], state["v_affine"][page, :, at]).flatten(1).to(dt))


def _run_attend(state):
    S, n, L = state["seqs"], state["max_new"], state["max_len"]
    Hq, H, D = state["heads"], state["kv_heads"], state["dim"]
    page = state["table"].long().clamp(min=0)

    def dense(name):                                                                  # [S][H][tokens][D]
        x = _values(state[name][page], state[name + "_affine"][page])
        return x.transpose(1, 2).reshape(S, H, -1, D)[:, :, :L]

    k = dense("k")
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
    out = (p.view(S, H, -1, L) @ dense("v")).view(S, H, Hq // H, n, D)
    out = torch.where(total > 0, out / total, 0.0)
    seq, at = _row_places(state)
    return out.permute(0, 3, 1, 2, 4)[seq, at - (end - count)[seq]].reshape(state["rows"], Hq * D).to(torch.bfloat16)


def run(state):
    if state["op"] == "plan":
        # A round of drafts: their places, and the tokens taken back again.
        if own:
            plan = state["plan"]
            plan.step(state["change"])
            state["take_back"].step(state["undo"])
            starts, position, slot, info = plan.row_start, plan.positions, plan.slots, plan.info
        else:
            starts, position, slot, info = _run_plan(state, state["change"], state["rows"])
            _run_plan(state, state["undo"], 0)
        return {"row_start": starts, "position": position, "slot": slot, "info": info, "table": state["table"],
                "kv_len": state["kv_len"], "free": state["free"], "n_free": state["n_free"]}
    if state["op"] == "rope":
        if own:
            return state["turn"](state["x"], state["position"], out=state["out"], inverse=state["inverse"])
        return _run_rope(state)
    if state["op"] == "attend4":
        if own:
            return state["cache"].attend(state["q"], state["batch"], causal=state["causal"], window=state["window"])
        return _run_attend(state)
    if own:
        state["cache"].append(state["new_k"], state["new_v"], state["slots"])
        k, v = state["cache"].read(state["batch"], dtype=_TYPES[state["dtype"]])
    else:
        k, v = _run_cache(state)
    return {"k": k, "v": v, "k_affine": state["k_affine"], "v_affine": state["v_affine"]}


# ------------------------------------------------------------ definitions --

def _exact_rope(state):
    """Row by row as complex numbers, whose angle is taken modulo a turn first."""
    f, factor = _frequencies(state)
    rot, dim = state["rot"], state["dim"]
    turns = torch.outer(state["position"].double(), f / (2 * math.pi)) % 1.0
    z = torch.polar(torch.full_like(turns, factor), 2 * math.pi * (-turns if state["inverse"] else turns))
    x = state["x"].double().view(-1, state["heads"], dim)
    y = x.clone()
    first = slice(0, rot, 2) if state["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if state["interleaved"] else slice(rot // 2, rot)
    w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z[:, None]
    y[..., first], y[..., second] = w.real, w.imag
    return torch.where((state["position"] >= 0)[:, None], y.flatten(1), 0.0)


def _exact_cache(state):
    """Group by group of 64, in 64 bits, with numbers of 8 significant bits below and above."""
    def eight_bits(x, up):
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -120))) - 7)
        return (torch.ceil(x / step) if up else torch.floor(x / step)) * step

    page, at = state["slots"] // state["block"], state["slots"] % state["block"]
    out = {}
    for name in ("k", "v"):
        x = state["new_" + name].double().view(state["rows"], state["kv_heads"], -1, GROUP)
        bias = eight_bits(x.min(-1).values, False)
        scale = eight_bits((x.max(-1).values - bias) / 15, True)
        code = torch.round((x - bias[..., None]) / scale[..., None].clamp(min=1e-300))
        out[name] = (code * scale[..., None] + bias[..., None]).flatten(1)
        pairs = torch.zeros(state[name + "_affine"].shape, dtype=torch.float64, device=DEV)
        pairs[page, :, at] = torch.stack([scale, bias], -1)
        out[name + "_affine"] = pairs
    return {n: out[n] for n in ("k", "v", "k_affine", "v_affine")}


def _exact_attend(state):
    """Sequence by sequence and head by head, in 64 bits."""
    H, D, G = state["kv_heads"], state["dim"], state["heads"] // state["kv_heads"]
    total, new = _lengths(state)

    def values(name, pages, h, L):
        code, pair = state[name][pages, h].flatten(0, 1)[:L], state[name + "_affine"][pages, h].flatten(0, 1)[:L].double()
        x = torch.empty((L, D), dtype=torch.float64, device=DEV)
        x[:, 0::2], x[:, 1::2] = (code % 16).double(), (code // 16).double()
        return x * pair[..., 0].repeat_interleave(GROUP, 1) + pair[..., 1].repeat_interleave(GROUP, 1)

    result, r = [], 0
    for s, (L, n) in enumerate(zip(total, new)):
        pages = state["table"][s, :-(-L // state["block"])].long()
        heads = []
        for h in range(H):
            k, v = values("k", pages, h, L), values("v", pages, h, L)
            for g in range(G):
                column = (h * G + g) * D
                score = torch.einsum("id,jd->ij", state["q"][r:r + n, column:column + D].double(), k) / D ** 0.5
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


def exact(case, seed):
    if case["op"] == "plan" or (case["op"] == "attend4" and work(case)["flops"] > 4e11):
        return None  # whole numbers; 64-bit products of that size take too long
    global own
    mode, own = own, False
    state = prepare(case, seed)
    own = mode
    return {"rope": _exact_rope, "cache4": _exact_cache, "attend4": _exact_attend}[case["op"]](state)


# ----------------------------------------------------------------- floors --

def work(case):
    if case["op"] == "rope":
        live, size = case["rows"] - case["pad"], {"bf16": 2, "fp32": 4}
        return {"bytes": 4 * case["rows"] + live * case["heads"] * case["dim"] * (size[case["src"]] + size[case["dst"]]),
                "flops": live * case["rot"] * (3 * case["heads"] + 20)}
    total, new = _lengths(case)
    if case["op"] == "plan":
        T = case["block"]
        moved = sum(abs(-(-(n + m) // T) - -(-n // T)) for n, m in zip(total, new))
        rows = sum(max(0, m) for m in new) + case["pad"]
        # Both ways: lengths, changes and row starts, and pages between the stack and the tables; once each row's place.
        return {"bytes": 2 * (16 * case["seqs"] + 12 * moved) + 12 * rows, "flops": 2 * (8 * case["seqs"] + 4 * moved) + 8 * rows}
    H, D, T = case["kv_heads"], case["dim"], case["block"]
    size = 4 if case["dtype"] == "fp32" else 2
    held = D // 2 + D // GROUP * 4                       # bytes of a token's head: codes, scales and biases
    rows = sum(new)
    if case["op"] == "cache4":
        # Rows in and codes out; codes in and rows out; both of keys and values.
        return {"bytes": 2 * rows * H * 2 * (D * size + held) + 8 * rows, "flops": 2 * rows * H * D * 8}
    pairs = seen = 0
    for n, m in zip(total, new):
        if not case["causal"]:
            pairs, seen = pairs + m * n, seen + n
            continue
        w = case["window"] or n
        first = np.arange(n - m, n)
        pairs += int(np.minimum(first + 1, w).sum())
        seen += min(n, m - 1 + w)
    return {"bytes": 2 * H * seen * held + rows * case["heads"] * D * (size + 2) + 4 * sum(-(-n // T) for n in total),
            "flops": 4 * case["heads"] * D * pairs}
