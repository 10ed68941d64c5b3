"""One decoder layer's decode step with 4-bit projections, a 4-bit paged key/value
cache and the activation-sparse FFN:

    h  = x + Wo . attend(cache + append(Wq x', Wk x', Wv x')),   x' = x / rms(x)
    y  = h + FFN(h / rms(h))

for one new token of each of a batch of sequences. Everything but the last
addition runs in libsffn's kernels on one stream, and a
step is captured once in a CUDA graph and replayed, the cache lengths and page
tables being read on the device at every replay.

    python examples/decode_layer.py [--batch 1] [--context 4096] [--steps 32]

prints the time per step and how far the attention half is from a plain fp32
computation on the values the cache holds.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gb300 import sffn, workload as W  # noqa: E402


def random_linear(out_features, in_features, group, max_batch, g):
    """A layer with random codes whose outputs have unit variance for unit-variance inputs."""
    codes = torch.randint(-8, 8, (out_features, in_features), generator=g, device="cuda", dtype=torch.int8)
    scales = (0.75 + 0.5 * torch.rand(out_features, in_features // group, generator=g, device="cuda"))
    scales = (scales / (4.6 * math.sqrt(in_features))).half()
    return sffn.Linear.from_weights(codes, scales, max_batch=max_batch), codes, scales


class DecoderLayer:
    """Weights, cache and buffers of one layer for `batch` sequences of up to `context` positions."""

    def __init__(self, spec: W.LayerSpec, heads: int, kv_heads: int, batch: int, context: int, page: int = 64,
                 group: int = 128, kv_group: int = 128, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.d, self.heads, self.kv_heads, self.dim, self.batch = spec.d, heads, kv_heads, spec.d // heads, batch
        self.qkv, self.w_qkv, self.s_qkv = random_linear((heads + 2 * kv_heads) * self.dim, spec.d, group, batch, g)
        self.proj, self.w_proj, self.s_proj = random_linear(spec.d, heads * self.dim, group, batch, g)
        self.ffn = sffn.Layer.from_weights(W.make_layer(spec, seed=seed, layer=0, device="cuda"), spec.group_size, spec.act,
                                           max_batch=batch)
        self.thres = spec.thres
        pages = -(-context // page)
        self.cache = sffn.KvCache(batch * pages, page, kv_heads, self.dim, min(kv_group, self.dim))
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").view(batch, pages).to(torch.int32)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.tokens = sffn.KvBatch(self.table, self.kv_len)       # one new token per sequence
        self.rope = sffn.Rope.of_base(context, self.dim)
        kw = dict(device="cuda")
        self.x = torch.zeros(batch, spec.d, **kw)
        self.rows = torch.empty(batch, heads + 2 * kv_heads, self.dim, **kw)
        self.q, self.k, self.v = self.rows.split((heads, kv_heads, kv_heads), 1)
        self.att = torch.empty(batch, heads, self.dim, **kw)
        self.h, self.y, self.out, self.xn = (torch.empty(batch, spec.d, **kw) for _ in range(4))
        self.masks = self.ffn.masks(batch)
        self.ws_qkv, self.ws_proj = self.qkv.workspace(batch), self.proj.workspace(batch)
        self.ws_att, self.ws_ffn = self.cache.workspace(self.tokens, heads), self.ffn.workspace(batch)

    def norm(self, x: torch.Tensor) -> torch.Tensor:
        sffn.sffn_norm(x, None, torch.finfo(x.dtype).eps, y=self.xn)
        return self.xn

    def fill(self, n: int, seed: int = 1) -> None:
        """Append n positions of random keys and values to every sequence, as a prompt would have."""
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        k, v = (torch.randn(self.batch * n, self.kv_heads, self.dim, generator=g, device="cuda") for _ in range(2))
        self.kv_len.fill_(n)
        start = torch.arange(self.batch + 1, device="cuda", dtype=torch.int32) * n
        sffn.sffn_kv_append(self.cache.handle, sffn.KvBatch(self.table, self.kv_len, start, self.batch * n), None, k, v)

    def step(self) -> None:
        """One token of every sequence: reads self.x, writes self.out."""
        self.kv_len.add_(1)
        sffn.sffn_linear_forward(self.qkv.handle, self.norm(self.x), self.rows.view(self.batch, -1), None, self.ws_qkv)
        sffn.sffn_kv_append(self.cache.handle, self.tokens, self.q, self.k, self.v, self.q, self.rope)
        sffn.sffn_attend(self.cache.handle, self.tokens, self.q, self.att, None, 1.0 / math.sqrt(self.dim), 0, self.ws_att)
        sffn.sffn_linear_forward(self.proj.handle, self.att.view(self.batch, -1), self.h, self.x, self.ws_proj)
        sffn.sffn_decode_step(self.ffn.handle, self.norm(self.h), self.batch, self.thres, self.masks, self.y, None,
                              self.ws_ffn)
        torch.add(self.h, self.y, out=self.out)

    def check_error(self) -> None:
        for part in (self.qkv, self.proj, self.cache, self.ffn):
            part.check_error()

    def plain_attention_half(self) -> torch.Tensor:
        """h of the step that was just run, in plain fp32 torch, on the cache's own values."""
        def weights(codes, scales):
            return codes.float() * scales.float().repeat_interleave(codes.shape[1] // scales.shape[1], 1)
        x = torch.nn.functional.rms_norm(self.x, self.x.shape[-1:])
        rows = (x @ weights(self.w_qkv, self.s_qkv).T).view(self.batch, -1, self.dim)
        n, half = int(self.kv_len[0]), self.dim // 2
        turn = self.rope.table[n - 1]
        a, b = rows[:, :self.heads, :half], rows[:, :self.heads, half:]
        q = torch.cat((a * turn[:, 0] - b * turn[:, 1], b * turn[:, 0] + a * turn[:, 1]), -1)
        k, v = (torch.empty(self.batch * n, self.kv_heads, self.dim, device="cuda") for _ in range(2))
        start = torch.arange(self.batch + 1, device="cuda", dtype=torch.int32) * n
        sffn.sffn_kv_gather(self.cache.handle, sffn.KvBatch(self.table, self.kv_len, start, self.batch * n), k, v)
        k, v = (t.view(self.batch, n, self.kv_heads, self.dim).repeat_interleave(self.heads // self.kv_heads, 2)
                for t in (k, v))
        p = torch.softmax(torch.einsum("bhd,blhd->bhl", q, k) / math.sqrt(self.dim), -1)
        att = torch.einsum("bhl,blhd->bhd", p, v).reshape(self.batch, -1)
        return self.x + att @ weights(self.w_proj, self.s_proj).T


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--workload", default="llama2_70b_reglu_d8192_f28672_bf16_8l", choices=sorted(W.WORKLOADS))
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    layer = DecoderLayer(W.WORKLOADS[a.workload], a.heads, a.kv_heads, a.batch, a.context)
    layer.fill(max(0, a.context - 2 * a.steps - 4))
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step()
        layer.step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.step()
        for _ in range(a.steps):
            graph.replay()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record(stream)
        for _ in range(a.steps):
            graph.replay()
        end.record(stream)
    stream.synchronize()
    layer.check_error()
    want = layer.plain_attention_half()
    off = float((layer.h - want).norm() / (want - layer.x).norm())
    us = begin.elapsed_time(end) / a.steps * 1e3
    print(f"{a.workload}, {a.heads}/{a.kv_heads} heads, batch {a.batch}, {int(layer.kv_len[0])} cached tokens: "
          f"{us:.1f} us per layer step; attention half off the plain fp32 form by {off:.1e} of its norm")
    return {"us": us, "off": off, "finite": bool(layer.out.isfinite().all())}


if __name__ == "__main__":
    main()
