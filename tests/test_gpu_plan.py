"""tf_kv_plan on the GPU against a plain simulation of stacks and tables: whole
numbers, so everything has to be equal."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from tests.serve_oracle import DEV, Pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(n_seqs, max_pages, block, n_blocks, seed=0, gap=0):
    """The same state on the device (rows of the table `gap` longer) and as lists."""
    free = np.random.default_rng(seed).permutation(n_blocks).astype(np.int32)
    table = torch.full((n_seqs, max_pages + gap), -1, dtype=torch.int32, device=DEV)
    pages = tf.KvPages(table[:, :max_pages], torch.zeros(n_seqs, dtype=torch.int32, device=DEV), torch.from_numpy(free).to(DEV),
                       torch.tensor([n_blocks], dtype=torch.int32, device=DEV), block)
    return pages, Pages(n_seqs, max_pages, block, free.tolist())


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def same(plan, pages, want, plain):
    torch.cuda.synchronize()
    starts, positions, slots, info = want
    assert plan.info.tolist() == info
    assert plan.row_start.tolist() == starts
    if plan.rows:
        assert plan.positions.tolist() == positions and plan.slots.tolist() == slots
    assert pages.kv_len.tolist() == plain.kv_len and pages.table.tolist() == plain.table
    n = pages.n_free.item()
    assert n == len(plain.free) and pages.free_pages[:n].tolist() == plain.free


@pytest.mark.parametrize("n_seqs,block,most", [(1, 16, 40), (5, 64, 200), (48, 32, 3), (257, 16, 30), (1025, 128, 5), (4096, 16, 4),
                                               (3, 16, 3000)])
def test_steps_of_all_kinds(n_seqs, block, most):
    rng = np.random.default_rng(n_seqs)
    max_pages = -(-4 * most // block) + 1
    pages, plain = make(n_seqs, max_pages, block, n_seqs * max_pages * 2 // 3 + 2, n_seqs, gap=3)
    rows = n_seqs * most + 7
    plan = pages.plan(rows, most)
    made = 0
    for _ in range(12):
        change = []
        for n in plain.kv_len:
            kind = rng.choice(["more", "one", "none", "back", "end"], p=[0.4, 0.2, 0.1, 0.2, 0.1])
            c = dict(more=int(rng.integers(0, most + 1)), one=1, none=0, back=-int(rng.integers(0, n + 1)), end=-n)[kind]
            change.append(min(c, max_pages * block - n))
        want = plain.step(change, rows, most, max_pages * block)
        same(plan.step(ints(change)), pages, want, plain)
        made += want[3][0] == 0
    assert made > 0
    tf.tf_device_status()


@pytest.mark.parametrize("n_seqs,block", [(7, 16), (300, 64)])
def test_a_step_and_its_opposite(n_seqs, block):
    # Drafts taken back leave stack, table and lengths as they were, to the order of the stack.
    rng = np.random.default_rng(block)
    pages, _ = make(n_seqs, 20, block, n_seqs * 20, 1)
    pages.plan(n_seqs * 300, 300).step(ints(rng.integers(0, 200, n_seqs).tolist()))
    lens = pages.kv_len.tolist()
    before = [t.clone() for t in (pages.table, pages.kv_len, pages.free_pages[:pages.n_free.item()])]
    change = [int(rng.integers(-n, 60)) for n in lens]
    pages.plan(n_seqs * 60, 60).step(ints(change))
    assert not torch.equal(pages.table, before[0])
    pages.plan(0, 300).step(ints([-c for c in change]))
    torch.cuda.synchronize()
    after = [pages.table, pages.kv_len, pages.free_pages[:pages.n_free.item()]]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    tf.tf_device_status()


def test_too_few_pages_change_nothing():
    pages, plain = make(3, 8, 16, 5)
    plan = pages.plan(200, 100)
    for change in ([30, 1, 0], [40, 40, 40], [0, 100, 0], [-30, 79, 0], [0, 0, 0], [0, -80, 17], [0, 1, 0]):
        want = plain.step(change, 200, 100, 128)
        same(plan.step(ints(change)), pages, want, plain)
    tf.tf_device_status()                                 # (too few pages are no error)


@pytest.mark.parametrize("bad", ["below zero", "above the table", "above max_rows", "more than rows", "length", "n_free", "page held",
                                 "page free", "int32"])
def test_numbers_that_do_not_fit_change_nothing(bad):
    pages, plain = make(4, 8, 16, 40)
    plan = pages.plan(60, 50, 100)
    same(plan.step(ints([20, 0, 33, 5])), pages, plain.step([20, 0, 33, 5], 60, 50, 100), plain)
    change = [1, 2, 3, 4]
    if bad == "below zero":
        change[2] = -34
    elif bad == "above the table":
        change[2] = 68
        plan.max_rows = 200
    elif bad == "above max_rows":
        change[1] = 51
    elif bad == "more than rows":
        change = [31, 30, 0, 0]
    elif bad == "length":
        pages.kv_len[1] = 129
    elif bad == "n_free":
        pages.n_free[0] = 41
    elif bad == "page held":
        change[2] = -33
        pages.table[2, 1] = 40
    elif bad == "page free":
        change[0] = 45
        pages.free_pages[pages.n_free.item() - 2] = -7
    elif bad == "int32":
        change = [2 ** 31 - 1] * 4
        plan.max_rows = 2 ** 31 - 1
    state = [t.clone() for t in (pages.table, pages.kv_len, pages.free_pages, pages.n_free)]
    plan.step(ints(change))
    torch.cuda.synchronize()
    with pytest.raises(tf.TfError) as e:
        tf.tf_device_status()
    assert e.value.rc == -14
    assert plan.info[:3].tolist() == [2, 0, 0] and plan.row_start.tolist() == [0] * 5
    assert torch.all(plan.positions == -1) and torch.all(plan.slots == -1)
    assert all(torch.equal(a, b) for a, b in zip(state, (pages.table, pages.kv_len, pages.free_pages, pages.n_free)))


def test_more_pages_than_a_pass_looks_at():
    # 7000 pages and more move in a step, either way and both; a bad number far down the stack stops all of it.
    rng = np.random.default_rng(9)
    pages, plain = make(60, 260, 16, 16000, 9, gap=1)
    plan = pages.plan(60 * 2000, 2000)
    for low, high in ((1800, 2001), (1900, 2001), (-2000, -1800), (-1500, 2001)):
        change = [max(-n, int(rng.integers(low, high))) for n in plain.kv_len]
        want = plain.step(change, plan.rows, 2000, 260 * 16)
        assert want[3][0] == 0
        same(plan.step(ints(change)), pages, want, plain)
    tf.tf_device_status()
    change = [min(2000, 260 * 16 - n) for n in plain.kv_len]
    taken = sum(-(-(n + c) // 16) - -(-n // 16) for n, c in zip(plain.kv_len, change))
    assert 4500 < taken <= len(plain.free)
    pages.free_pages[pages.n_free.item() - 1 - (taken - 2)] = 16000
    state = [t.clone() for t in (pages.table, pages.kv_len, pages.free_pages, pages.n_free)]
    plan.step(ints(change))
    torch.cuda.synchronize()
    with pytest.raises(tf.TfError):
        tf.tf_device_status()
    assert plan.info[0].item() == 2 and all(torch.equal(a, b) for a, b in zip(state, (pages.table, pages.kv_len, pages.free_pages, pages.n_free)))


def test_slots_past_32_bits_and_outputs_left_out():
    # Page numbers of a pool of 2^26 pages of 128 tokens (none of it is touched); positions or slots alone.
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    free = torch.arange((1 << 26) - 8, 1 << 26, dtype=torch.int32, device=DEV)
    state = dict(table=table, kv_len=ints([0, 0]), free=free, n_free=ints([8]))
    c = tf.TfKvPages(table.data_ptr(), 4, state["kv_len"].data_ptr(), free.data_ptr(), state["n_free"].data_ptr(), 2, 1 << 26, 4, 128)
    starts, info = ints([0] * 3), ints([0] * 4)
    slots = torch.zeros(300, dtype=torch.int64, device=DEV)
    tf.tf_kv_plan(c, ints([130, 5]), 300, 200, 512, starts, None, slots, info)
    torch.cuda.synchronize()
    last = (1 << 26) - 1
    assert slots[:130].tolist() == [last * 128 + i for i in range(128)] + [(last - 1) * 128, (last - 1) * 128 + 1]
    assert slots[130:135].tolist() == [(last - 2) * 128 + i for i in range(5)] and torch.all(slots[135:] == -1)
    positions = ints([9] * 4)
    tf.tf_kv_plan(c, ints([1, 2]), 4, 200, 512, starts, positions, None, info)
    torch.cuda.synchronize()
    assert positions.tolist() == [130, 5, 6, -1] and info.tolist() == [0, 0, 3, 131]
    tf.tf_device_status()


@pytest.mark.parametrize("rows", [64, 6000])
def test_captured_steps_on_another_stream(rows):
    # A graph of a step, replayed with changes that the device holds; both ways of filling the rows.
    pages, plain = make(16, 40, 16, 16 * 40)
    side = torch.cuda.Stream()
    change = ints([0] * 16)
    with torch.cuda.stream(side):
        plan = pages.plan(rows, rows)
        plan.step(change)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.step(change)
    side.synchronize()
    rng = np.random.default_rng(rows)
    for _ in range(6):
        by = [int(rng.integers(-min(n, 3), min(rows // 16, 640 - n) + 1)) for n in plain.kv_len]
        change.copy_(ints(by))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(plan, pages, plain.step(by, rows, rows, 640), plain)
    tf.tf_device_status()


def test_a_refused_step_is_a_batch_of_no_rows():
    # Attention and appends of the step's batch leave everything as it is.
    pages = tf.KvPages.empty(2, 3, 8, 16)
    plan = pages.plan(60, 50)
    cache = tf.Kv4Cache.empty(3, 1, 64, 16)
    plan.step(ints([20, 70]))
    k = torch.randn((60, 64), device=DEV).to(torch.bfloat16)
    cache.append(k, k, plan.slots)
    out = torch.full((60, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cache.attend(k, plan.batch, out=out)
    torch.cuda.synchronize()
    assert plan.info.tolist() == [2, 0, 0, 0]
    assert torch.all(out == 7.0) and torch.all(cache.k == 0) and torch.all(cache.v_affine == 0)
    with pytest.raises(tf.TfError):
        tf.tf_device_status()
