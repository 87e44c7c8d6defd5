"""Pages and places of a step, rotary positions, the 4-bit cache and attention over it, as the serving example runs
them: each against its definition on what the one before it left, drafts that are taken back, and graphs."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from mlx_affine_bit_gb300.decode import ServingDecoder
from tests.serve_oracle import Pages, attend4, quantise4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def decoder(**kw):
    return ServingDecoder(**{**dict(layers=1, width=512, heads=8, kv_heads=2, dim=128, vocab=777, seqs=3, max_len=192, block=64), **kw})


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("heads,kv_heads,dim,block", [(8, 2, 128, 64), (4, 4, 64, 16), (6, 1, 256, 32)])
def test_steps(heads, kv_heads, dim, block):
    d = decoder(heads=heads, kv_heads=kv_heads, dim=dim, block=block)
    pages, cache, nq, nk = d.pages, d.caches[0], heads * dim, kv_heads * dim
    model = Pages(3, pages.max_pages, block, pages.free_pages.tolist())
    gen = torch.Generator().manual_seed(5)
    keys, values = [np.zeros((0, kv_heads, dim))] * 3, [np.zeros((0, kv_heads, dim))] * 3
    # A ragged prompt, single tokens, drafts of which some are taken back while others grow, an ended sequence.
    for change in ([130, 1, 63], [1, 1, 1], [4, 0, 3], [-3, 4, -1], [1, -2, 1], [2, -3, 1]):
        rows = sum(max(0, c) for c in change) + 2
        plan = pages.plan(rows, max(change), d.max_len)
        tokens = torch.randint(0, 777, (rows,), generator=gen).to(DEV)
        plan.step(i32(change))
        start, positions, slots, info = model.step(change, rows, max(change), d.max_len)
        assert plan.row_start.tolist() == start and plan.positions.tolist() == positions and plan.slots.tolist() == slots
        assert plan.info.tolist() == info and pages.table.tolist() == model.table and pages.kv_len.tolist() == model.kv_len
        # What step() does in its layer, once more: the same calls, the same bits.
        y = d.qkv[0](d.embed[tokens])
        turned = d.turn(y[:, :nq + nk], plan.positions, out=y[:, :nq + nk].clone())
        live = start[-1]
        q, k = (t[:live].cpu().numpy().reshape(live, -1, dim) for t in (turned[:, :nq], turned[:, nq:]))
        v = y[:live, nq + nk:].cpu().numpy().reshape(live, -1, dim)
        d.step(tokens, plan)
        out = cache.attend(turned[:, :nq], plan.batch)[:live].float().cpu().numpy().astype(np.float64).reshape(live, heads, dim)
        for s, c in enumerate(change):
            n = model.kv_len[s] - max(0, c)
            keys[s], values[s] = (np.concatenate([x[s][:n], z[start[s]:start[s + 1]]]).astype(np.float32) for x, z in ((keys, k), (values, v)))
            stored = [quantise4(x[s]) for x in (keys, values)]
            places = [model.table[s][p // block] * block + p % block for p in range(model.kv_len[s])]
            for pool, pair, (code, scale, bias) in ((cache.k, cache.k_affine, stored[0]), (cache.v, cache.v_affine, stored[1])):
                got, a = (t.cpu().transpose(1, 2).flatten(0, 1)[places].numpy() for t in (pool, pair.float()))
                assert np.array_equal(np.stack([got & 15, got >> 4], -1).reshape(code.shape), code)
                assert np.array_equal(a[..., 0], scale) and np.array_equal(a[..., 1], bias)
            if c > 0:
                want, bound = attend4(q[start[s]:start[s + 1]], *stored, dim ** -0.5, True, 0, True)
                assert np.all(np.abs(out[start[s]:start[s + 1]] - want) <= bound)
    tf.tf_device_status()


def test_drafts_taken_back_leave_no_trace():
    # Logits of single tokens with rejected drafts between them, and without: the same bits, whatever the pages are.
    gen = torch.Generator().manual_seed(6)
    prompt, after = torch.randint(0, 777, (194,), generator=gen).to(DEV), torch.randint(0, 777, (5, 3), generator=gen).to(DEV)
    drafts = torch.randint(0, 777, (5, 12), generator=gen).to(DEV)
    results = []
    for speculate in (False, True):
        d = decoder(layers=2, block=16)
        first, single, _ = d.begin([130, 1, 63])
        logits = [d.step(prompt, first)]
        many, back = d.pages.plan(12, 4, d.max_len), d.pages.plan(0, 1, d.max_len)
        for i in range(5):
            if speculate:
                d.step(drafts[i], many.step(i32([4, 4, 4])))
                back.step(i32([-4, -4, -4]))
            logits.append(d.step(after[i], single.step(i32([1, 1, 1]))))
        results.append(torch.cat(logits))
    tf.tf_device_status()
    assert torch.equal(*results)


def test_generation_by_graph():
    prompts = [[(31 * s + 7 * i) % 4096 for i in range(n)] for s, n in enumerate((70, 1, 33, 64))]
    results = []
    with torch.cuda.stream(torch.cuda.Stream()):
        d = ServingDecoder(max_len=100)
        for graph in (False, True, True):        # (one decoder: its sequences begin again)
            results.append(d.generate(prompts, 20, graph=graph)[0].cpu())
    assert results[0].shape == (20, 4) and int(results[0].min()) >= 0 and int(results[0].max()) < 4096
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
    assert d.pages.kv_len.tolist() == [89, 20, 52, 83]


def test_refuses_other_sequences():
    with pytest.raises(ValueError):
        decoder(max_len=32).generate([[1], [2] * 31, [3]], 2)
