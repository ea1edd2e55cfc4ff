"""A decoder's layers on the decode operators: prompts, then one token a sequence and step.

    python -m dense_fp16_gemm_hgemm_amd.decode_step [--batch 16 --prompt 500 --steps 32 --layers 2]

Weights are random.  A step is ``w4_linear`` for the projections, ``kv_append`` for the new
keys and values (with the rotation of keys and queries), ``kv_attend`` over the paged 8-bit
cache, and torch for the norms and the gate; it is captured into a graph once and replayed.
Prompts have more tokens than the 4-bit kernel is made for, so their projections run in
``Hgemm`` on the same weights in binary16.
"""
from __future__ import annotations

import argparse
import time
from typing import NamedTuple

import torch

from . import Hgemm
from .decode import W4, Decode, KvCache, rope_table, w4_quantize, w4_unpack


class Config(NamedTuple):
    hidden: int = 4096
    heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    inner: int = 11008
    layers: int = 2
    page_size: int = 64
    group: int = 128
    window: int = 0
    sinks: int = 0


class Linear(NamedTuple):
    """A projection's weights in 4 bits, and the same numbers in binary16."""
    w4: W4
    full: torch.Tensor

    @classmethod
    def random(cls, n, k, group, gen):
        w = w4_quantize((torch.randn((n, k), device="cuda", generator=gen) * k ** -0.5).half(), group)
        return cls(w, w4_unpack(w).half())


class Layer(NamedTuple):
    qkv: Linear
    out: Linear
    gate_up: Linear
    down: Linear
    cache: KvCache


def _norm(x):
    y = x.float()
    return (y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).half()


class Model:
    """Layers, their caches, and the page table that all of them share."""

    def __init__(self, config: Config, batch: int, max_len: int, seed: int = 0, codes=torch.int8):
        self.config, self.batch = config, batch
        gen = torch.Generator(device="cuda").manual_seed(seed)
        c = config
        self.cols = -(-max_len // c.page_size)
        pages = batch * self.cols
        rows = (c.heads + 2 * c.kv_heads) * c.head_dim
        self.layers = [Layer(Linear.random(rows, c.hidden, c.group, gen),
                             Linear.random(c.hidden, c.heads * c.head_dim, c.group, gen),
                             Linear.random(2 * c.inner, c.hidden, c.group, gen),
                             Linear.random(c.hidden, c.inner, c.group, gen),
                             KvCache.empty(pages, c.kv_heads, c.head_dim, c.page_size, codes))
                       for _ in range(c.layers)]
        # pages are handed out in no order; a server would take them from its free list
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(batch, self.cols).to(torch.int32).cuda()
        self.rope = rope_table(self.cols * c.page_size, c.head_dim)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")  # tokens in the cache
        self.longest = 0  # the most of them, as far as the host knows: replays of a graph are not counted
        self.decode, self.gemm = Decode(), Hgemm()

    def close(self):
        self.decode.close()
        self.gemm.close()

    def _linear(self, x, w: Linear, few):
        if few:
            return self.decode.w4_linear(x, w.w4.qweight, w.w4.scales, w.w4.zeros, n=w.w4.n, group=w.w4.group)
        return self.gemm.run(x, w.full)

    def forward(self, x, cu=None, most=None, max_len=None):
        """x [tokens, hidden]: the next tokens of every sequence, one each, or as `cu` says (`most`
        at most, if given); they join the cache, and the layers' output for them is returned.
        More tokens than the page table has room for are refused."""
        c, d = self.config, self.decode
        few = cu is None
        new = 1 if few else cu[1:] - cu[:-1]
        total = self.lens + new
        longest = self.longest + 1 if few else int(total.max())
        if longest > self.cols * c.page_size:
            raise ValueError(f"the page table has room for {self.cols * c.page_size} tokens a sequence, not for {longest}")
        for layer in self.layers:
            qkv = self._linear(_norm(x), layer.qkv, few).view(x.shape[0], -1, c.head_dim)
            q = d.kv_append(layer.cache, qkv[:, c.heads:c.heads + c.kv_heads], qkv[:, c.heads + c.kv_heads:],
                            self.table, self.lens, cu, most, q=qkv[:, :c.heads], rope=self.rope)
            a = d.kv_attend(q, layer.cache, self.table, total, cu, most, max_len=max_len, window=c.window, sinks=c.sinks)
            x = x + self._linear(a.view(x.shape[0], -1), layer.out, few)
            g = self._linear(_norm(x), layer.gate_up, few)
            g = torch.nn.functional.silu(g[:, :c.inner].float()) * g[:, c.inner:].float()
            x = x + self._linear(g.half(), layer.down, few)
        self.lens.copy_(total)
        self.longest = longest
        return x

    def graph(self, x):
        """forward for one token a sequence as a graph: (graph, its input, its output).  The
        graph reads lengths and pages when it is replayed, and advances the lengths: the caller
        sees to it that they stay within the page table."""
        keep, longest, at, out = self.lens.clone(), self.longest, x.clone(), None
        # the warm-up has no pages: x may be anything, and in the caches a large number would
        # grow the scales of pages that hold tokens already
        table, self.table = self.table, torch.full_like(self.table, -1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(at)
        torch.cuda.current_stream().wait_stream(side)
        self.table, self.longest = table, longest
        self.lens.copy_(keep)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = self.forward(at)
        self.longest = longest
        return g, at, out


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 16), ("prompt", 500), ("steps", 32), ("layers", 2)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    config = Config(layers=a.layers)
    m = Model(config, a.batch, a.prompt + a.steps + 1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens = [max(1, a.prompt * (i + 1) // a.batch) for i in range(a.batch)]
    cu = torch.tensor([0] + lens, dtype=torch.int32, device="cuda").cumsum(0).int()
    x = m.forward(torch.randn((sum(lens), config.hidden), device="cuda", generator=gen).half(), cu, max(lens))
    last = x[cu[1:].long() - 1]
    g, at, out = m.graph(last)
    at.copy_(last)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        g.replay()
        at.copy_(out)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    assert torch.isfinite(out).all()
    print(f"{a.batch} sequences, prompts of {min(lens)} to {max(lens)} tokens, {a.layers} layers: "
          f"{us:.0f} us a step, {a.batch / us * 1e6:.0f} tokens/s")
    m.close()


if __name__ == "__main__":
    main()
