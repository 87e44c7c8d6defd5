"""CPU checks of include/tfserve.h: exported symbols, structs, what the calls refuse on
the host before any CUDA call, and the frequencies of rotary positions."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096        # a 16-byte aligned stand-in address; no call below reaches the device


@pytest.fixture(scope="module")
def tf():
    from mlx_affine_bit_gb300.build import build
    build()
    import mlx_affine_bit_gb300 as tf
    tf.lib()
    return tf


def test_exports_every_declared_symbol(tf):
    hdr = open(os.path.join(ROOT, "include", "tfserve.h")).read()
    declared = set(re.findall(r"^(?:int|const char \*)\s*(tf_\w+)\s*\(", hdr, re.M))
    assert declared == {"tf_kv_plan", "tf_rope", "tf_kv4_append", "tf_kv4_read", "tf_kv4_attend"}
    for so in (tf.SO, tf.SO_DEBUG):
        out = subprocess.check_output(["nm", "-D", "--defined-only", so]).decode()
        assert declared <= set(re.findall(r"\sT\s(tf_\w+)$", out, re.M))
    assert declared <= set(tf.SYMBOLS)


def test_structs_and_flags_match_the_header(tf, tmp_path):
    src = tmp_path / "size.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tfserve.h"\nint main(void){printf("%zu %zu %zu %zu %d %d", '
                   'sizeof(tf_kv_pages), sizeof(tf_kv4), offsetof(tf_kv_pages, block), offsetof(tf_kv4, dim), TF_ROPE_PAIRS, TF_ROPE_BACK);'
                   'return 0;}')
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "size")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "size")]).split()]
    assert got == [ctypes.sizeof(tf.TfKvPages), ctypes.sizeof(tf.TfKv4), tf.TfKvPages.block.offset, tf.TfKv4.dim.offset,
                   tf.TF_ROPE_PAIRS, tf.TF_ROPE_BACK]


def pages(tf, **kw):
    d = dict(table=A, table_stride=8, kv_len=A, free_pages=A, n_free=A, n_seqs=4, n_blocks=10, max_pages=8, block=16)
    d.update(kw)
    return tf.TfKvPages(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(table=None), -5), (dict(kv_len=None), -5), (dict(free_pages=A + 2), -5), (dict(n_free=None), -5), (dict(n_seqs=0), -6),
    (dict(n_seqs=4097), -6), (dict(n_blocks=0), -6), (dict(max_pages=0), -6), (dict(max_pages=65537, table_stride=70000), -6),
    (dict(table_stride=7), -4), (dict(block=48), -6), (dict(block=0), -6)])
def test_pages_refusals(tf, bad, code):
    assert tf.lib().tf_kv_plan(pages(tf, **bad), A, 10, 4, 100, A, A, A, A, None) == code
    assert tf.lib().tf_last_error_string()


def test_plan_refusals(tf):
    L, p = tf.lib(), pages(tf)
    call = lambda change=A, rows=10, most=4, length=100, starts=A, pos=A, slots=A, info=A: L.tf_kv_plan(  # noqa: E731
        p, change, rows, most, length, starts, pos, slots, info, None)
    assert L.tf_kv_plan(None, A, 10, 4, 100, A, A, A, A, None) == -5
    assert call(change=None) == -5 and call(starts=None) == -5 and call(info=None) == -5 and call(slots=A + 4) == -5 and call(pos=A + 1) == -5
    assert call(rows=-1) == -3 and call(most=0) == -3 and call(rows=0) == -3 and call(pos=None, slots=None) == -3
    assert call(length=0) == -6 and call(length=(1 << 20) + 1) == -6


def test_rope_refusals(tf):
    L = tf.lib()
    call = lambda turns=A, rot=64, pos=A, rows=3, x=A, xs=256, out=1 << 20, os_=256, heads=2, dim=128, flags=0: L.tf_rope(  # noqa: E731
        turns, rot, 1.0, pos, rows, x, xs, out, os_, heads, dim, flags, None)
    assert call(turns=None) == -5 and call(turns=A + 4) == -5 and call(pos=None) == -5 and call(x=None) == -5 and call(out=None) == -5
    assert call(x=A + 1) == -5 and call(x=A + 2, flags=4) == -5 and call(out=A + 2) == -5 and call(out=(1 << 20) + 1, flags=1) == -5
    assert call(rows=0) == -3
    for bad in (dict(rot=0), dict(rot=63), dict(rot=130), dict(dim=127), dict(dim=1026), dict(heads=0), dict(heads=65537)):
        assert call(**bad) == -6, bad
    assert call(xs=255) == -4 and call(os_=255) == -4
    assert call(flags=2) == -12 and call(flags=8) == -12
    # Overlaps: the same rows of another type or stride, shifted columns, a row further.
    assert call(out=A) == -5 and call(out=A, flags=5, xs=512) == -5 and call(out=A, flags=4, os_=300) == -5
    assert call(out=A + 128 * 2, flags=1, xs=1024, os_=1024) == -5 and call(out=A + 1024 * 2, flags=1, xs=1024, os_=1024) == -5
    assert call(out=A + 900 * 2, flags=1, xs=1024, os_=1024) == -5        # (runs into the next row)


def kv4(tf, **kw):
    d = dict(k=A, v=A, k_affine=A, v_affine=A, n_blocks=10, kv_heads=2, block=16, dim=64)
    d.update(kw)
    return tf.TfKv4(**d)


def batch(tf, **kw):
    d = dict(n_seqs=2, rows=6, max_rows=4, max_len=40, row_start=A, kv_len=A, table=A, table_stride=3, slots=None)
    d.update(kw)
    return tf.TfKvBatch(**d)


@pytest.mark.parametrize("bad,code", [(dict(k=None), -5), (dict(v=A + 8), -5), (dict(k_affine=None), -5), (dict(v_affine=A + 4), -5),
                                      (dict(block=8), -6), (dict(block=48), -6), (dict(dim=96), -6), (dict(kv_heads=0), -6),
                                      (dict(kv_heads=1025), -6), (dict(n_blocks=0), -6)])
def test_cache_refusals(tf, bad, code):
    L, c, b = tf.lib(), kv4(tf, **bad), batch(tf)
    assert L.tf_kv4_append(c, A, 2, A, 128, A, 128, 0, None) == code
    assert L.tf_kv4_read(c, b, A, 128, A, 128, 0, None) == code
    assert L.tf_kv4_attend(c, b, A, 256, 4, A, 256, 1.0, 0, 8, None) == code
    assert L.tf_last_error_string()


@pytest.mark.parametrize("bad,code", [(dict(kv_len=None), -5), (dict(table=A + 2), -5), (dict(n_seqs=0), -6), (dict(rows=0), -3),
                                      (dict(max_rows=7), -3), (dict(row_start=None), -3), (dict(max_len=0), -6), (dict(table_stride=2), -4)])
def test_batch_refusals(tf, bad, code):
    L, c, b = tf.lib(), kv4(tf), batch(tf, **bad)
    assert L.tf_kv4_read(c, b, A, 128, A, 128, 0, None) == code
    assert L.tf_kv4_attend(c, b, A, 256, 4, A, 256, 1.0, 0, 8, None) == code


def test_call_refusals(tf):
    L, c, b = tf.lib(), kv4(tf), batch(tf)
    append = lambda slots=A, rows=2, k=A, ks=128, v=A, vs=128, flags=0: L.tf_kv4_append(c, slots, rows, k, ks, v, vs, flags, None)  # noqa: E731
    assert append(slots=None) == -5 and append(slots=A + 4) == -5 and append(k=None) == -5 and append(v=A + 1) == -5
    assert append(k=A + 2, flags=4) == -5 and append(rows=0) == -3 and append(ks=127) == -4 and append(vs=0) == -4 and append(flags=1) == -12
    read = lambda k=A, ks=128, v=A, vs=128, flags=0: L.tf_kv4_read(c, b, k, ks, v, vs, flags, None)     # noqa: E731
    assert read(k=None, v=None) == -5 and read(k=A + 2) == -5 and read(v=A + 1, flags=1) == -5
    assert read(ks=127) == -4 and read(vs=127) == -4 and read(flags=4) == -12
    attend = lambda q=A, qs=256, heads=4, out=A, os_=256, window=0, flags=8: L.tf_kv4_attend(  # noqa: E731
        c, b, q, qs, heads, out, os_, 1.0, window, flags, None)
    assert attend(heads=0) == -6 and attend(heads=3) == -6 and attend(window=-1) == -6 and attend(window=5, flags=0) == -6
    assert attend(q=None) == -5 and attend(out=A + 1) == -5 and attend(q=A + 2, flags=12) == -5
    assert attend(qs=255) == -4 and attend(os_=255) == -4 and attend(flags=1) == -12 and attend(flags=8 + 64 + 128) == -12


def test_tensors_of_the_wrong_kind_are_refused(tf):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)      # noqa: E731
    bf = dict(dtype=torch.bfloat16)
    p = tf.KvPages.empty(2, 10, 4, 16, "cpu")
    assert p.table.shape == (2, 4) and p.n_free.item() == 10 and p.free_pages[-1] == 0
    plan = p.plan(8, 4, 60)
    for change, error in ((i32(1, 2, 3), ValueError), (torch.zeros(2), TypeError), (i32(1, 9, 2, 9)[::2], ValueError), (i32(1, 2), ValueError)):
        with pytest.raises(error):
            plan.step(change, stream=0)                      # (the last: not on a GPU)
    for bad in (dict(rows=-1), dict(rows=4, max_rows=0), dict(rows=4, max_len=0), dict(rows=4, max_len=65)):
        with pytest.raises(ValueError):
            p.plan(**bad)
    with pytest.raises(TypeError):
        tf.KvPages(p.table.long(), p.kv_len, p.free_pages, p.n_free, 16)
    with pytest.raises(ValueError):
        tf.KvPages(p.table, i32(1), p.free_pages, p.n_free, 16)
    with pytest.raises(ValueError):
        tf.KvPages(p.table[:1].expand(2, 4), p.kv_len, p.free_pages, p.n_free, 16)

    turn = tf.Rope(64, device="cpu")
    x = torch.zeros((3, 128), **bf)
    for y, at, error in ((x.half(), i32(1, 2, 3), TypeError), (x, i32(1, 2), ValueError), (x, torch.zeros(3), TypeError),
                         (x[:, :100], i32(1, 2, 3), ValueError), (x.t(), i32(*range(128)), ValueError), (x, i32(1, 2, 3), ValueError)):
        with pytest.raises(error):
            turn(y, at, stream=0)                            # (the last: not on a GPU)
    with pytest.raises(ValueError):
        turn(x, i32(1, 2, 3), out=x[:2], stream=0)

    c = tf.Kv4Cache.empty(4, 2, 64, 16, "cpu")
    k, slots = torch.zeros((2, 128), **bf), torch.zeros(2, dtype=torch.int64)
    for args, error in (((k, k.float(), slots), TypeError), ((k[:1], k, slots), ValueError), ((k, k, slots.int()), TypeError),
                        ((k.half(), k.half(), slots), TypeError), ((k, torch.zeros((128, 2), **bf).t(), slots), ValueError),
                        ((k, k, slots), ValueError)):
        with pytest.raises(error):
            c.append(*args, stream=0)                        # (the last: not on a GPU)
    b = tf.KvBatch(i32(3, 5), torch.zeros((2, 2), dtype=torch.int32), 5)
    with pytest.raises(TypeError):
        c.read(b, dtype=torch.float16, stream=0)
    with pytest.raises(TypeError):
        c.read(b, k_out=k, v_out=k.float(), stream=0)
    with pytest.raises(TypeError):
        c.attend(k.half(), b, stream=0)
    with pytest.raises(ValueError):
        c.attend(torch.zeros((2, 100), **bf), b, stream=0)
    with pytest.raises(ValueError):
        tf.Kv4Cache(c.k, c.v, c.k_affine, c.v_affine[:2])
    with pytest.raises(TypeError):
        tf.Kv4Cache(c.k.view(torch.int8), c.v, c.k_affine, c.v_affine)


def test_frequencies(tf):
    # Whole numbers of 2^-64 of a turn, and every kind of scaling against its formula at a few pairs.
    r = tf.Rope(128, 64, base=1e4, device="cpu")
    for i in (0, 1, 31):
        want = 1e4 ** (-2 * i / 64) / (2 * math.pi)
        # (a few roundings of 2^-53, and the whole number's of half of 2^-64)
        assert abs((r.turns[i].item() % 2 ** 64) / 2 ** 64 - want) <= 2.0 ** -52 * want + 2.0 ** -65
    assert r.factor == 1.0 and len(r.frequencies) == 32
    linear = tf.Rope(64, base=1e4, scaling=dict(type="linear", factor=4), device="cpu").frequencies
    assert linear[5] == pytest.approx(1e4 ** (-10 / 64) / 4, rel=1e-14)
    ntk = tf.Rope(64, base=1e4, scaling=dict(type="ntk", factor=8), device="cpu").frequencies
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(1e4 ** (-62 / 64) / 8, rel=1e-12)      # the slowest pair: the whole factor
    bands = dict(type="bands", factor=8, low=1, high=4, original=8192)
    f = tf.Rope(128, base=5e5, scaling=bands, device="cpu").frequencies
    plain = [5e5 ** (-2 * i / 128) for i in range(64)]
    for a, b in zip(f, plain):
        length = 2 * math.pi / b
        if length < 8192 / 4:
            assert a == pytest.approx(b, rel=1e-14)
        elif length > 8192:
            assert a == pytest.approx(b / 8, rel=1e-14)
        else:
            assert b / 8 < a < b
    yarn = tf.Rope(128, base=1e4, scaling=dict(type="yarn", factor=16, original=4096), device="cpu")
    assert yarn.factor == pytest.approx(0.1 * math.log(16) + 1)
    assert yarn.frequencies[0] == 1.0 and yarn.frequencies[-1] == pytest.approx(1e4 ** (-126 / 128) / 16, rel=1e-12)
    given = tf.Rope(8, frequencies=[0.5, -0.25, 7.0, 0.0], factor=2.0, device="cpu")
    assert [t % 2 ** 64 for t in given.turns.tolist()][3] == 0 and given.turns[1] < 0 and given.factor == 2.0
    for bad in (dict(dim=63), dict(dim=64, rot_dim=66), dict(dim=64, rot_dim=3), dict(dim=64, base=0), dict(dim=2048),
                dict(dim=8, frequencies=[1.0]), dict(dim=8, frequencies=[1.0, 1, 1, math.inf]),
                dict(dim=64, scaling=dict(type="linear", factor=0)), dict(dim=64, scaling=dict(type="other", factor=2)),
                dict(dim=64, scaling=dict(type="bands", factor=2, low=4, high=1, original=100)),
                dict(dim=8, frequencies=[1.0] * 4, scaling=dict(type="linear", factor=2))):
        with pytest.raises(ValueError):
            tf.Rope(**bad, device="cpu")


def test_a_plan_goes_with_caches_of_its_pages_only(tf):
    # Pages of 16 tokens in a cache of 32 a page, and the other way round: places and lengths would be taken for others.
    plan = tf.KvPages.empty(2, 10, 8, 16, "cpu").plan(2, 1, 64)
    k = torch.zeros((2, 128), dtype=torch.bfloat16)
    for block in (32, 64):
        other = tf.Kv4Cache.empty(5, 2, 64, block, "cpu")
        eight = tf.KvCache.empty(5, 2, 64, block, 2, device="cpu")
        for call in (lambda: other.append(k, k, plan.slots, stream=0), lambda: other.attend(k, plan.batch, stream=0),
                     lambda: other.read(plan.batch, stream=0), lambda: eight.attend(k, plan.batch, stream=0),
                     lambda: eight.read(plan.batch, stream=0), lambda: eight.append(k, k, plan.batch, stream=0)):
            with pytest.raises(ValueError, match="pages"):
                call()
    # Of the same size, and tensors that say nothing of pages: only that there is no GPU stands against them.
    same = tf.Kv4Cache.empty(5, 2, 64, 16, "cpu")
    for call in (lambda: same.append(k, k, plan.slots, stream=0), lambda: other.append(k, k, plan.slots[:], stream=0),
                 lambda: same.attend(k, plan.batch, stream=0), lambda: same.read(plan.batch, stream=0)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
