"""Beam search with a small decoder: 8-bit projections, a 4-bit paged key/value cache that
the beams share, and the activation-sparse FFN.

A step takes one token of every beam of every search through

    codes = q8(norm(h))                     sffn_norm, the last FFN's output added on the way
    q, k, v = Wqkv codes                    sffn_linear8_forward
    att = attend(cache + append(q, k, v))   sffn_kv_append, sffn_attend
    h = h + Wo q8(att)                      sffn_quantize, sffn_linear8_forward
    y = FFN(norm(h))                        sffn_norm, sffn_decode_step

for every layer, then the last norm, the output projection, the choice of the best
continuations (sffn_beam_select) and the reordering of every layer's cache by the beams that
go on (sffn_kv_reorder). It is captured once in a CUDA graph and replayed.

    python examples/beam_search.py [--batch 2] [--beams 4] [--steps 24]

prints the time per step, the best sequence of the first search and its score.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gb300 import sffn, workload as W  # noqa: E402

EPS = 1e-5
START = 1


def random_linear8(out_features, in_features, max_batch, g):
    """A layer with random codes whose outputs have unit variance for unit-variance inputs."""
    codes = (32.0 * torch.randn(out_features, in_features, generator=g, device="cuda")).round().clamp(-127, 127)
    scales = (0.75 + 0.5 * torch.rand(out_features, generator=g, device="cuda")) / (32.0 * math.sqrt(in_features))
    return sffn.Linear8.from_weights(codes.to(torch.int8), scales, max_batch=max_batch)


class Decoder:
    """Weights (the same for the same seed), caches and buffers for `batch` searches of `beams` sequences."""

    def __init__(self, d=1024, layers=2, heads=8, kv_heads=2, vocab=5003, batch=2, beams=4, context=256, page=16,
                 ffn=True, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rows, dim = batch * beams, d // heads
        self.d, self.heads, self.kv_heads, self.dim, self.vocab = d, heads, kv_heads, dim, vocab
        self.batch, self.beams, self.rows = batch, beams, rows
        kw = dict(device="cuda")
        spec = W.LayerSpec(name="beam", d=d, f=2 * d, h=128, group_size=64, act="reglu", wdtype="bf16", p_mean=0.1,
                           zipf_alpha=1.0)
        self.thres = spec.thres
        self.embed = torch.randn(vocab, d, generator=g, **kw)
        weight = lambda: 1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")  # noqa: E731
        self.layers = []
        for i in range(layers):
            layer = dict(norm1=weight(), norm2=weight(), qkv=random_linear8((heads + 2 * kv_heads) * dim, d, rows, g),
                         proj=random_linear8(d, heads * dim, rows, g))
            if ffn:
                layer["ffn"] = sffn.Layer.from_weights(W.make_layer(spec, seed=seed, layer=i, device="cuda"),
                                                       spec.group_size, spec.act, max_batch=rows)
                layer["masks"], layer["ws_ffn"] = layer["ffn"].masks(rows), layer["ffn"].workspace(rows)
            self.layers.append(layer)
        self.norm_out, self.head = weight(), random_linear8(vocab, d, rows, g)
        pages = -(-context // page)
        self.cache = [sffn.KvCache(rows * pages, page, kv_heads, dim, min(64, dim)) for _ in range(layers)]
        self.caches = sffn.KvCaches(self.cache)
        self.own_pages = torch.arange(rows * pages, dtype=torch.int32, **kw).view(rows, pages)
        self.table = self.own_pages.clone()
        self.kv_len = torch.zeros(rows, dtype=torch.int32, **kw)
        self.kv = sffn.KvBatch(self.table, self.kv_len)
        self.rope = sffn.Rope.of_base(context, dim)
        self.search = sffn.Beams(vocab, beams, beams, max_batch=batch)
        self.x, self.h, self.xn, self.y = (torch.zeros(rows, d, **kw) for _ in range(4))
        self.codes, self.scales = torch.empty(rows, d, dtype=torch.int8, **kw), torch.empty(rows, **kw)
        self.qkv = torch.empty(rows, heads + 2 * kv_heads, dim, **kw)
        self.q, self.k, self.v = self.qkv.split((heads, kv_heads, kv_heads), 1)
        self.att = torch.empty(rows, heads, dim, **kw)
        self.logits = torch.empty(rows, vocab, **kw)
        self.scores = torch.empty(batch, beams, **kw)
        self.parents, self.tokens = torch.zeros(2, batch, beams, dtype=torch.int32, **kw)
        self.ws_att = self.cache[0].workspace(self.kv, heads)
        self.ws_search = self.search.workspace(batch)
        self.start()

    def start(self) -> None:
        """Empty caches; every beam at the first token, one of each search alive. Reordering shares pages, so that the
        tables start again from pages of each row's own."""
        self.table.copy_(self.own_pages)
        self.kv_len.zero_()
        self.scores.fill_(-math.inf)
        self.scores[:, 0] = 0.0
        self.tokens.fill_(START)

    def forward(self) -> None:
        """Logits of the next token of every row."""
        self.kv_len.add_(1)
        torch.index_select(self.embed, 0, self.tokens.view(-1), out=self.h)
        added = None
        for layer, cache in zip(self.layers, self.cache):
            sffn.sffn_norm(self.h, layer["norm1"], EPS, added, self.h, None, self.codes, self.scales)
            sffn.sffn_linear8_forward(layer["qkv"].handle, self.codes, self.scales, self.qkv.view(self.rows, -1))
            sffn.sffn_kv_append(cache.handle, self.kv, self.q, self.k, self.v, self.q, self.rope)
            sffn.sffn_attend(cache.handle, self.kv, self.q, self.att, None, self.dim ** -0.5, 0, self.ws_att)
            sffn.sffn_quantize(self.att, self.codes, self.scales)
            sffn.sffn_linear8_forward(layer["proj"].handle, self.codes, self.scales, self.h, self.h)
            if "ffn" in layer:
                sffn.sffn_norm(self.h, layer["norm2"], EPS, y=self.xn)
                sffn.sffn_decode_step(layer["ffn"].handle, self.xn, self.rows, self.thres, layer["masks"], self.y, None,
                                      layer["ws_ffn"])
                added = self.y
        sffn.sffn_norm(self.h, self.norm_out, EPS, added, None, None, self.codes, self.scales)
        sffn.sffn_linear8_forward(self.head.handle, self.codes, self.scales, self.logits)

    def step(self) -> None:
        """One token more for every beam."""
        self.forward()
        sffn.sffn_beam_select(self.search.handle, self.logits, self.scores, self.scores, self.parents, self.tokens,
                              ws=self.ws_search)
        sffn.sffn_kv_reorder(self.caches, self.kv, self.parents, self.beams)

    def check_error(self) -> None:
        for part in (*self.cache, self.search, self.head, *(p for x in self.layers for p in (x["qkv"], x["proj"]))):
            part.check_error()

    def run(self, steps: int, graph: bool = True):
        """(sequences (batch, beams, steps), scores) of a search from the start; with the time of a step in `us`."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        taken = []
        with torch.cuda.stream(stream):
            replay = self.step
            if graph:
                self.step()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured, stream=stream):
                    self.step()
                replay = captured.replay
            self.start()
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record(stream)
            for _ in range(steps):
                replay()
                taken.append((self.parents.clone(), self.tokens.clone()))
            end.record(stream)
        stream.synchronize()
        self.us = begin.elapsed_time(end) / steps * 1e3
        self.check_error()
        at = torch.arange(self.beams, device="cuda").expand(self.batch, -1)
        words = []
        for parents, tokens in reversed(taken):
            words.append(tokens.gather(1, at))
            at = parents.gather(1, at).long()
        return torch.stack(words[::-1], -1), self.scores.clone()

    def score_of(self, tokens) -> float:
        """Log-probability of a sequence fed token by token (for a decoder with one row)."""
        self.start()
        total, last = 0.0, START
        for t in tokens:
            self.tokens.fill_(last)
            self.forward()
            total += float(self.logits[0].double().log_softmax(-1)[t])
            last = t
        self.check_error()
        return total


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args(argv)
    decoder = Decoder(batch=a.batch, beams=a.beams, layers=a.layers)
    sequences, scores = decoder.run(a.steps)
    best = sequences[0, 0].tolist()
    print(f"{a.batch} searches of {a.beams} beams, {a.layers} layers: {decoder.us:.1f} us per step; best of the first: "
          f"{float(scores[0, 0]):.3f}, tokens {best[:8]}{' ...' if len(best) > 8 else ''}")
    return {"us": decoder.us, "sequences": sequences, "scores": scores}


if __name__ == "__main__":
    main()
