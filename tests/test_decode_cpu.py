"""CPU checks of include/tfdecode.h: exported symbols, and what the calls refuse on
the host before any CUDA call."""
import ctypes
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
    hdr = open(os.path.join(ROOT, "include", "tfdecode.h")).read()
    declared = set(re.findall(r"^(?:int|const char \*)\s*(tf_\w+)\s*\(", hdr, re.M))
    assert declared == {"tf_kv_append", "tf_kv_read", "tf_kv_attend", "tf_sample"}
    for so in (tf.SO, tf.SO_DEBUG):
        out = subprocess.check_output(["nm", "-D", "--defined-only", so]).decode()
        assert declared <= set(re.findall(r"\sT\s(tf_\w+)$", out, re.M))
    assert declared <= set(tf.SYMBOLS)


def test_structs_match_the_header(tf, tmp_path):
    src = tmp_path / "size.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tfdecode.h"\nint main(void){printf("%zu %zu %zu %zu", '
                   'sizeof(tf_kv), sizeof(tf_kv_batch), offsetof(tf_kv, f32), offsetof(tf_kv_batch, slots));return 0;}')
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "size")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "size")]).split()]
    assert got == [ctypes.sizeof(tf.TfKv), ctypes.sizeof(tf.TfKvBatch), tf.TfKv.f32.offset, tf.TfKvBatch.slots.offset]


def kv(tf, **kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, open_k=A, open_v=A, open_max=A, n_blocks=10, n_slots=4, kv_heads=2, block=16,
             dim=64, f32=0)
    d.update(kw)
    return tf.TfKv(**d)


def batch(tf, **kw):
    d = dict(n_seqs=2, rows=6, max_rows=4, max_len=40, row_start=A, kv_len=A, table=A, table_stride=3, slots=None)
    d.update(kw)
    return tf.TfKvBatch(**d)


BAD_KV = [(dict(k=None), -5), (dict(v=A + 8), -5), (dict(k_scale=None), -5), (dict(v_scale=A + 2), -5), (dict(block=8), -6),
          (dict(block=48), -6), (dict(dim=96), -6), (dict(kv_heads=0), -6), (dict(kv_heads=1025), -6), (dict(n_blocks=0), -6)]
BAD_BATCH = [(dict(kv_len=None), -5), (dict(table=None), -5), (dict(table=A + 2), -5), (dict(row_start=A + 1), -5),
             (dict(n_seqs=0), -6), (dict(n_seqs=65537), -6), (dict(rows=0), -3), (dict(max_rows=0), -3), (dict(max_rows=7), -3),
             (dict(row_start=None), -3), (dict(max_len=0), -6), (dict(max_len=49), -4), (dict(table_stride=2), -4)]


@pytest.mark.parametrize("bad,code", BAD_KV)
def test_cache_refusals(tf, bad, code):
    L, c, b = tf.lib(), kv(tf, **bad), batch(tf)
    assert L.tf_kv_append(c, b, A, 128, A, 128, None) == code
    assert L.tf_kv_read(c, b, A, 128, A, 128, 0, None) == code
    assert L.tf_kv_attend(c, b, A, 256, 4, A, 256, 1.0, 0, 8, None) == code
    assert L.tf_last_error_string()


@pytest.mark.parametrize("bad,code", BAD_BATCH)
def test_batch_refusals(tf, bad, code):
    L, c, b = tf.lib(), kv(tf), batch(tf, **bad)
    assert L.tf_kv_append(c, b, A, 128, A, 128, None) == code
    assert L.tf_kv_read(c, b, A, 128, A, 128, 0, None) == code
    assert L.tf_kv_attend(c, b, A, 256, 4, A, 256, 1.0, 0, 8, None) == code
    assert L.tf_last_error_string()


def test_append_refusals(tf):
    L, b = tf.lib(), batch(tf)
    for bad, code in ((dict(open_k=None), -5), (dict(open_v=A + 2), -5), (dict(open_max=None), -5), (dict(n_slots=0), -6),
                      (dict(n_slots=1), -6), (dict(f32=2), -12)):
        assert L.tf_kv_append(kv(tf, **bad), b, A, 128, A, 128, None) == code, bad
    c = kv(tf)
    assert L.tf_kv_append(None, b, A, 128, A, 128, None) == -5
    assert L.tf_kv_append(c, None, A, 128, A, 128, None) == -5
    assert L.tf_kv_append(c, b, None, 128, A, 128, None) == -5
    assert L.tf_kv_append(c, b, A + 1, 128, A, 128, None) == -5
    assert L.tf_kv_append(kv(tf, f32=1), b, A + 2, 128, A, 128, None) == -5
    assert L.tf_kv_append(c, b, A, 127, A, 128, None) == -4
    assert L.tf_kv_append(c, b, A, 128, A, 100, None) == -4


def test_read_refusals(tf):
    L, c, b = tf.lib(), kv(tf, open_k=None, open_v=None, open_max=None, n_slots=0), batch(tf)
    assert L.tf_kv_read(c, b, None, 0, None, 0, 0, None) == -5
    assert L.tf_kv_read(c, b, A + 2, 128, None, 0, 0, None) == -5
    assert L.tf_kv_read(c, b, A + 1, 128, None, 0, 1, None) == -5
    assert L.tf_kv_read(c, b, A, 127, None, 0, 0, None) == -4
    assert L.tf_kv_read(c, b, A, 128, A, 127, 0, None) == -4
    assert L.tf_kv_read(c, b, A, 128, A, 128, 2, None) == -12


def test_attend_refusals(tf):
    L, c, b = tf.lib(), kv(tf, open_k=None, open_v=None, open_max=None, n_slots=0), batch(tf)
    call = lambda q=A, qs=256, heads=4, out=A, os_=256, window=0, flags=8: L.tf_kv_attend(c, b, q, qs, heads, out, os_, 1.0, window, flags, None)  # noqa: E731
    assert call(heads=0) == -6 and call(heads=3) == -6
    assert call(heads=4098, qs=1 << 20, os_=1 << 20) == -6
    assert call(window=-1) == -6 and call(window=5, flags=0) == -6
    assert call(q=None) == -5 and call(out=None) == -5 and call(q=A + 1) == -5 and call(q=A + 2, flags=12) == -5 and call(out=A + 1) == -5
    assert call(qs=255) == -4 and call(os_=255) == -4
    assert call(flags=1) == -12 and call(flags=32) == -12


def test_sample_refusals(tf):
    L = tf.lib()
    call = lambda x=A, rows=2, vocab=100, stride=100, u=A, t=None, k=None, p=None, m=None, out=A, pr=None, flags=0: L.tf_sample(  # noqa: E731
        x, rows, vocab, stride, u, t, k, p, m, out, pr, flags, None)
    assert call(rows=0) == -3 and call(rows=(1 << 20) + 1) == -3
    assert call(vocab=0) == -6 and call(vocab=(1 << 20) + 1, stride=1 << 21) == -6
    assert call(stride=99) == -4
    assert call(x=None) == -5 and call(u=None) == -5 and call(out=None) == -5 and call(x=A + 2) == -5 and call(x=A + 1, flags=16) == -5
    for name in ("t", "k", "p", "m", "pr"):
        assert call(**{name: A + 2}) == -5
    assert call(flags=1) == -12


def test_tensors_of_the_wrong_kind_are_refused(tf):
    cache = tf.KvCache.empty(4, 2, 64, 16, 2, torch.bfloat16, "cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)      # noqa: E731
    b = tf.KvBatch(i32(3, 5), torch.zeros((2, 2), dtype=torch.int32), 5)
    k = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cache.append(k.float(), k, b, stream=0)
    with pytest.raises(ValueError):
        cache.append(k[:1], k, b, stream=0)
    with pytest.raises(ValueError):
        cache.append(k, torch.zeros((128, 2), dtype=torch.bfloat16).t(), b, stream=0)
    with pytest.raises(TypeError):
        cache.attend(k.half(), b, stream=0)
    with pytest.raises(ValueError):
        cache.attend(torch.zeros((2, 100), dtype=torch.bfloat16), b, stream=0)
    with pytest.raises(ValueError):
        cache.attend(k, tf.KvBatch(i32(3, 5), torch.zeros((2, 2), dtype=torch.int32), 33), stream=0)
    with pytest.raises(TypeError):
        tf.KvBatch(torch.zeros(2), torch.zeros((2, 2), dtype=torch.int32), 5)
    with pytest.raises(ValueError):
        tf.KvBatch(i32(3, 5), torch.zeros((3, 2), dtype=torch.int32), 5)
    with pytest.raises(ValueError):
        tf.KvBatch(i32(3, 5), torch.zeros((2, 2), dtype=torch.int32), 5, row_start=i32(0, 1, 2))
    with pytest.raises(ValueError):
        tf.KvCache(cache.k, cache.v[:2], cache.k_scale, cache.v_scale)
    with pytest.raises(TypeError):
        tf.sample(torch.zeros((2, 10), dtype=torch.float16), torch.zeros(2), stream=0)
    with pytest.raises(ValueError):
        tf.sample(torch.zeros((2, 10)), torch.zeros(3), stream=0)
    with pytest.raises(TypeError):
        tf.sample(torch.zeros((2, 10)), torch.zeros(2), top_k=torch.zeros(2), stream=0)
