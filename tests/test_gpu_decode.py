"""The generation example on the GPU: a step of a prompt and a step of single tokens
against plain fp64 arithmetic on the cache's own content, and the same tokens with
and without a graph.

The bound goes through the step: the products' (K 2^-24 + 2^-20) sum |x w|, the
attention's as the oracle gives it, and the sums' rounding to bf16 (2^-8 of them)."""
import numpy as np
import pytest
import torch

import mlx_affine_bit_gb300 as tf
from mlx_affine_bit_gb300.decode import Decoder, Matrix
from tests import decode_oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def plain(m: Matrix):
    """The matrix in fp64, [N][K]."""
    w = m.W.cpu().numpy().view(np.uint32)
    per = 32 // m.bits
    codes = np.stack([(w >> np.uint32(m.bits * i)) & np.uint32(2 ** m.bits - 1) for i in range(per)], axis=-1).reshape(w.shape[0], -1)
    s, b = (np.repeat(t.float().cpu().numpy().astype(np.float64), m.group, axis=1) for t in (m.scales, m.biases))
    return codes * s + b


def product(x, w, err):
    """x w^T and the bound of the product whose x is err off."""
    return x @ w.T, err @ np.abs(w).T + (w.shape[1] * 2.0 ** -24 + 2.0 ** -20) * (np.abs(x) @ np.abs(w).T)


def check(d, tokens, lengths, logits):
    """The logits of each sequence's last token against the plain form (one layer)."""
    x = d.embed[tokens]
    q = d.qkv[0](x)[:, :d.heads * d.dim].cpu().numpy().astype(np.float64).reshape(len(lengths), d.heads, d.dim)
    cache, block = d.caches[0], d.caches[0].block
    starts = np.concatenate([[0], np.cumsum(lengths)])
    batch = tf.KvBatch(torch.tensor(lengths, dtype=torch.int32, device=DEV), d.table, d.max_len,
                       row_start=torch.tensor(starts, dtype=torch.int32, device=DEV), rows=int(starts[-1]), max_rows=max(lengths))
    k, v = (t.cpu().numpy().astype(np.float64).reshape(-1, d.kv_heads, d.dim) for t in cache.read(batch))
    a, err = np.zeros((len(lengths), d.heads * d.dim)), np.zeros((len(lengths), d.heads * d.dim))
    for s, n in enumerate(lengths):
        pages = d.table[s].long().cpu()
        vs = np.repeat(cache.v_scale.cpu()[pages].numpy(), block, axis=0)[:n]
        o, e = decode_oracle.attend(q[s:s + 1], k[starts[s]:starts[s + 1]], v[starts[s]:starts[s + 1]], vs, d.dim ** -0.5, 1,
                                    True, 0, True)
        a[s], err[s] = o.reshape(-1), e.reshape(-1)
    y, e = product(a, plain(d.out[0]), err)
    h = x.float().cpu().numpy().astype(np.float64) + y
    y, e = product(h, plain(d.head), e + 2.0 ** -8 * np.abs(h))
    off = np.abs(logits.cpu().numpy() - y)
    assert np.all(off <= e), float((off / e).max())


@pytest.mark.parametrize("heads,kv_heads,dim,block", [(8, 2, 128, 64), (4, 4, 64, 16), (6, 1, 256, 32)])
def test_steps(heads, kv_heads, dim, block):
    lengths = [130, 1, 63]
    d = Decoder(layers=1, width=512, heads=heads, kv_heads=kv_heads, dim=dim, vocab=777, seqs=3, max_len=192, block=block)
    gen = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, 777, (sum(lengths),), generator=gen).to(DEV)
    starts = np.concatenate([[0], np.cumsum(lengths)])
    kv_len = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    prompt = tf.KvBatch(kv_len, d.table, d.max_len, row_start=torch.tensor(starts, dtype=torch.int32, device=DEV),
                        rows=sum(lengths), max_rows=max(lengths))
    last = torch.from_numpy(starts[1:] - 1).to(DEV)
    logits = d.step(tokens, prompt, last)
    check(d, tokens[last], lengths, logits)
    one = tf.KvBatch(kv_len, d.table, d.max_len)
    for _ in range(3):
        kv_len.add_(1)
        lengths = [n + 1 for n in lengths]
        tokens = torch.randint(0, 777, (3,), generator=gen).to(DEV)
        logits = d.step(tokens, one)
        check(d, tokens, lengths, logits)
    tf.tf_device_status()


def test_generation_by_graph():
    prompts = [[(31 * s + 7 * i) % 4096 for i in range(n)] for s, n in enumerate((70, 1, 33, 64))]
    results = []
    with torch.cuda.stream(torch.cuda.Stream()):
        for graph in (False, True, True):
            results.append(Decoder(max_len=100).generate(prompts, 20, graph=graph)[0].cpu())
    assert results[0].shape == (20, 4) and int(results[0].min()) >= 0 and int(results[0].max()) < 4096
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])


def test_refuses_other_sequences():
    d = Decoder(layers=1, width=512, vocab=64, seqs=2, max_len=32)
    with pytest.raises(ValueError):
        d.generate([[1]], 2)
    with pytest.raises(ValueError):
        d.generate([[1], [2] * 31], 2)


def test_generation_on_the_default_stream():
    # With a graph, although that stream cannot be captured; the tokens of a stream of one's own.
    prompts = [[(31 * s + 7 * i) % 4096 for i in range(n)] for s, n in enumerate((20, 1, 33, 64))]
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    got = Decoder(max_len=100).generate(prompts, 12)[0].clone()
    assert torch.equal(got, Decoder(max_len=100).generate(prompts, 12, graph=False)[0])
    with torch.cuda.stream(torch.cuda.Stream()):
        want = Decoder(max_len=100).generate(prompts, 12)[0].cpu()
    assert torch.equal(got.cpu(), want)
