"""Generation with the library's parts together: quantized products, the 8-bit
paged cache, attention over it and the sampling of tokens.

    python -m mlx_affine_bit_gb300.decode [--seqs 8] [--prompt 500] [--tokens 64] [--layers 4]

A small decoder of random weights (attention blocks without positions or norms, and
a language-model head) takes a ragged batch of prompts in one step and then a token
a sequence and step.  A step of a layer is four calls:

    y = x [q | k | v]        tf.qmm, one product for the three (fp32 rows)
    cache.append(k, v)       slices of y as they stand, the cache takes a row stride
    a = cache.attend(q)      bf16 rows, the next product's input
    x = x + a out            tf.qmm

and ends in tf.qmm with the head and tf.sample.  Lengths, page tables and tokens stay
on the device, so that a whole step of single tokens is one CUDA graph.  The script
prints the first tokens and the time of a step, launched call by call and as a graph.
"""
from __future__ import annotations

import argparse
import time
from dataclasses import dataclass

import torch

import mlx_affine_bit_gb300 as tf


@dataclass
class Matrix:
    """A quantized matrix [N][K] as the products take it."""
    W: torch.Tensor
    scales: torch.Tensor
    biases: torch.Tensor
    bits: int
    group: int

    @classmethod
    def random(cls, N, K, bits, group, gen):
        """Codes of all values alike, weights of variance 1 / K around 0."""
        words = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=gen, device=gen.device)
        top = 2 ** bits - 1
        scale = (12 / K) ** 0.5 / top * (0.75 + 0.5 * torch.rand((N, K // group), generator=gen, device=gen.device))
        scale = scale.to(torch.bfloat16)
        return cls(words.to(torch.int32), scale, (scale.float() * (-top / 2)).to(torch.bfloat16), bits, group)

    def __call__(self, x):
        return tf.qmm(x, self.W, self.scales, self.biases, self.bits, self.group)


class Decoder:
    """Layers of attention over `seqs` growing sequences of up to max_len tokens, and a head."""

    def __init__(self, layers=2, width=1024, heads=8, kv_heads=2, dim=128, vocab=4096, bits=4, group=64, seqs=4, max_len=512,
                 block=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.seqs, self.max_len = heads, kv_heads, dim, seqs, max_len
        self.embed = torch.randn((vocab, width), generator=gen, device=device).to(torch.bfloat16)
        self.qkv = [Matrix.random((heads + 2 * kv_heads) * dim, width, bits, group, gen) for _ in range(layers)]
        self.out = [Matrix.random(width, heads * dim, bits, group, gen) for _ in range(layers)]
        self.head = Matrix.random(vocab, width, bits, group, gen)
        pages = (max_len + block - 1) // block
        self.caches = [tf.KvCache.empty(seqs * pages, kv_heads, dim, block, seqs, torch.float32, device) for _ in range(layers)]
        # Pages in any order: here those of the sequences in turn.
        self.table = torch.arange(seqs * pages, dtype=torch.int32, device=device).view(pages, seqs).t().contiguous()

    def step(self, tokens, batch, last=None):
        """Logits [seqs][vocab] after the batch's rows of tokens; last: each sequence's last row (every row if None)."""
        x = self.embed[tokens]
        nq, nk = self.heads * self.dim, self.kv_heads * self.dim
        for qkv, out, cache in zip(self.qkv, self.out, self.caches):
            y = qkv(x)
            cache.append(y[:, nq:nq + nk], y[:, nq + nk:], batch)
            a = cache.attend(y[:, :nq], batch)
            x = (x.float() + out(a)).to(torch.bfloat16)
        return self.head(x if last is None else x[last])

    def generate(self, prompts, n, temperature=0.8, top_k=50, top_p=0.95, seed=1, graph=True):
        """n tokens [n][seqs] after the prompts (lists of tokens, one a sequence), and the last step's seconds.

        graph: single-token steps after the first as one CUDA graph, captured on the current stream (torch's default
        stream cannot be captured: then on one of the call's own)."""
        if len(prompts) != self.seqs or max(map(len, prompts)) + n > self.max_len:
            raise ValueError("the decoder was made for %d sequences of up to %d tokens" % (self.seqs, self.max_len))
        if n < 1 or min(map(len, prompts)) < 1:
            raise ValueError("every prompt, and what is generated, must have a token at least")
        if graph and torch.cuda.current_stream() == torch.cuda.default_stream():
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                result = self.generate(prompts, n, temperature, top_k, top_p, seed, graph)
            torch.cuda.current_stream().wait_stream(side)
            result[0].record_stream(torch.cuda.current_stream())
            return result
        dev, seqs = self.table.device, len(prompts)
        gen = torch.Generator(device=dev).manual_seed(seed)
        u = torch.rand((n, seqs), generator=gen, device=dev)
        row_u = torch.empty(seqs, device=dev)
        how = dict(temperature=torch.full((seqs,), temperature, device=dev), top_p=torch.full((seqs,), top_p, device=dev),
                   top_k=torch.full((seqs,), top_k, dtype=torch.int32, device=dev))
        lengths = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        starts = torch.zeros(seqs + 1, dtype=torch.int32, device=dev)
        starts[1:] = lengths.cumsum(0)
        rows = sum(map(len, prompts))
        logits = self.step(torch.tensor([t for p in prompts for t in p], device=dev),
                           tf.KvBatch(lengths, self.table, self.max_len, row_start=starts, rows=rows, max_rows=max(map(len, prompts))),
                           starts[1:].long() - 1)
        tokens, _ = tf.sample(logits, u[0], **how)
        single = tf.KvBatch(lengths, self.table, self.max_len)

        def advance():
            lengths.add_(1)                      # (read by the device at each call)
            tf.sample(self.step(tokens, single), row_u, tokens=tokens, **how)

        result, g, seconds = [tokens.clone()], None, 0.0
        for i in range(1, n):
            row_u.copy_(u[i])
            torch.cuda.synchronize()
            t = time.perf_counter()
            if g is not None:
                g.replay()
            else:
                advance()
            torch.cuda.synchronize()
            seconds = time.perf_counter() - t
            result.append(tokens.clone())
            if graph and g is None:
                # The first step was launched call by call on this stream, and made the library's workspaces there.
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=torch.cuda.current_stream()):
                    advance()
        tf.tf_device_status()
        return torch.stack(result), seconds


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--prompt", type=int, default=500, help="tokens of the longest prompt")
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--layers", type=int, default=4)
    a = p.parse_args()
    prompts = [[(31 * s + 7 * i) % 4096 for i in range(max(1, a.prompt - 37 * s))] for s in range(a.seqs)]
    with torch.cuda.stream(torch.cuda.Stream()):
        for graph in (False, True):
            d = Decoder(layers=a.layers, seqs=a.seqs, max_len=a.prompt + a.tokens)
            tokens, seconds = d.generate(prompts, a.tokens, graph=graph)
            print("%s: %.0f us a step of %d tokens; sequence 0: %s" %
                  ("one graph a step" if graph else "call by call", seconds * 1e6, a.seqs, tokens[:12, 0].tolist()))


if __name__ == "__main__":
    main()
