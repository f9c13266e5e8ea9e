"""The attention of one decoder layer whose query heads share key and value heads, from hidden states to hidden states, on the
library's calls alone.

    python examples/gqa_layer.py [--heads 16] [--kv 4] [--hidden 1024] [--prompt 300] [--steps 8] [--keep 128]

A prompt runs with its own keys and values, which go into the paged 4-bit cache; the tokens after it read that cache and add up
the weight that every cached token gets.  Half-way the cache is cut to the tokens with the most weight (and the newest ones), on
new pages, and the steps go on.  The last lines say how far the outputs are from the layer computed in 64 bits from the same
quantised weights and the same cached rows, and how long a step takes.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import bit_weight_gemv_fmt1_gb300 as coli  # noqa: E402
from mla_layer import int4_matrix  # noqa: E402

D = 128        # dims of a head, all rotary
GS = 32        # elements per scale of the cache
RECENT = 16    # the newest tokens, which an eviction keeps


class GqaLayer:
    """Weights, rotation table and paged cache of one layer; `n_pages` pages of `page` tokens."""

    def __init__(self, hidden: int, heads: int, kv: int, n_pages: int, page: int = 64, seed: int = 0):
        g = np.random.default_rng(seed)
        self.hidden, self.heads, self.kv, self.page = hidden, heads, kv, page
        self.q, self.q_values = int4_matrix(g, heads * D, hidden)
        self.k, self.k_values = int4_matrix(g, kv * D, hidden)
        self.v, self.v_values = int4_matrix(g, kv * D, hidden)
        self.o, self.o_values = int4_matrix(g, hidden, heads * D)
        freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        angle = torch.arange(n_pages * page, dtype=torch.float64)[:, None] * freq
        self.rot = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.scale = 1.0 / math.sqrt(D)
        codes = lambda: torch.zeros(n_pages, kv, page, D // 2, device="cuda", dtype=torch.uint8)  # noqa: E731
        scales = lambda: torch.zeros(n_pages, kv, page, D // GS, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.cache = coli.GqaCache(codes(), codes(), scales(), scales(), weights=torch.zeros(n_pages, kv, page, device="cuda"))

    def _project(self, x, pos, slot, pages):
        """Rotated queries and keys, and values, of tokens x at positions pos; keys and values go to the cache's places `slot` of the
        sequence on `pages`."""
        T = x.shape[0]
        q, k, v = (torch.empty(T, n, D, device="cuda") for n in (self.heads, self.kv, self.kv))
        coli.matmul_multi([self.q, self.k, self.v], x, [q.view(T, -1), k.view(T, -1), v.view(T, -1)])
        for t in (q, k):
            coli.mla_query(t, pos, self.rot, None, t)                    # in place: all of a head's dims are rotary
        slots = pages[0].long()[slot.long() // self.page] * self.page + slot.long() % self.page
        coli.gqa_append(self.cache, k, v, slots)
        return q, k, v

    def _out(self, mixed):
        y = torch.empty(mixed.shape[0], self.hidden, device="cuda")
        coli.matmul(self.o, mixed.view(mixed.shape[0], -1), y)
        return y

    def prompt(self, x, pages):
        """Attention of a prompt x [T, hidden] whose pages [1, n] are empty yet."""
        T = x.shape[0]
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        q, k, v = self._project(x, pos, pos, pages)
        cu = torch.tensor([0, T], device="cuda", dtype=torch.int32)
        out = torch.empty(T, self.heads, D, device="cuda")
        coli.gqa_prefill(q, k, v, cu, cu, self.scale, out)
        return self._out(out)

    def step(self, x, pos: int, length: int, pages):
        """Attention of one new token x [1, hidden] at position pos of the text, the cache's token `length`."""
        at, slot = (torch.tensor([i], device="cuda", dtype=torch.int32) for i in (pos, length))
        q, _, _ = self._project(x, at, slot, pages)
        out = torch.empty(1, 1, self.heads, D, device="cuda")
        coli.gqa_attend(self.cache, q.view(1, 1, self.heads, D), pages, slot + 1, self.scale, out, weigh=True)
        return self._out(out.view(1, self.heads, D))

    def evict(self, length: int, keep: int, pages, fresh):
        """The sequence cut to `keep` tokens on the pages `fresh`; the tokens that stay, of each head."""
        kept = torch.empty(1, self.kv, keep, device="cuda", dtype=torch.int32)
        lens, new = torch.tensor([length], device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)
        coli.gqa_evict(self.cache, pages, lens, keep, min(RECENT, keep), fresh, kept, new)
        return kept

    def rows(self, length: int, pages):
        """The sequence's keys and values as the cache holds them, [length, kv, D]."""
        k, v = (torch.empty(length, self.kv, D, device="cuda") for _ in "kv")
        return coli.gqa_read(self.cache, pages, torch.tensor([0, length], device="cuda", dtype=torch.int32), k, v)

    def _turn(self, x, pos):
        rot = self.rot.cpu().double()[pos, None]
        c, s = rot[..., :D // 2], rot[..., D // 2:]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    def plain(self, x, pos, k=None, v=None):
        """The layer in 64 bits on the host: x [T, hidden] at positions pos; with k, v [n, kv, D] every token sees those, else its own
        and the earlier ones' keys and values."""
        T = x.shape[0]
        q = self._turn((x @ self.q_values.T).view(T, self.heads, D), pos)
        causal = k is None
        if causal:
            k, v = self._turn((x @ self.k_values.T).view(T, self.kv, D), pos), (x @ self.v_values.T).view(T, self.kv, D)
        k, v = (t.repeat_interleave(self.heads // self.kv, 1) for t in (k, v))
        score = torch.einsum("ihd,jhd->hij", q, k) * self.scale
        if causal:
            score = score.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
        return torch.einsum("hij,jhd->ihd", torch.softmax(score, -1), v).reshape(T, -1) @ self.o_values.T


def run(hidden=1024, heads=16, kv=4, prompt=300, steps=8, keep=128, seed=0):
    """Errors (largest difference over the largest value) of the prompt's and the steps' outputs; whether the eviction kept the
    tokens that the weights say; the layer and its state."""
    total = prompt + steps
    n, m = -(-total // 64), -(-(keep + steps) // 64)
    layer = GqaLayer(hidden, heads, kv, n + m + 2, seed=seed)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(total, hidden, generator=g)
    order = torch.randperm(n + m + 2, generator=g).to(torch.int32).cuda()
    pages, fresh = order[None, :n].contiguous(), order[None, n:n + m].contiguous()
    xd, xh = x.cuda(), x.double()
    err = lambda a, b: float((a.cpu().double() - b).abs().max() / b.abs().max())  # noqa: E731
    e_prompt = err(layer.prompt(xd[:prompt], pages), layer.plain(xh[:prompt], torch.arange(prompt)))
    e_step, length, right = 0.0, prompt, True
    for t in range(prompt, total):
        if t == prompt + steps // 2:
            w = layer.cache.weights[pages[0].long()].transpose(0, 1).flatten(1, 2)[:, :length].cpu()
            kept = layer.evict(length, keep, pages, fresh)[0].cpu()
            stay, old = min(keep, length), max(0, length - min(RECENT, keep))
            for h in range(kv):
                best = sorted(range(old), key=lambda i: (-float(w[h, i]), i))[:stay - (length - old)]
                right = right and kept[h, :stay].tolist() == sorted(best) + list(range(old, length))
            pages, length = fresh, stay
        got = layer.step(xd[t:t + 1], t, length, pages)
        length += 1
        k, v = layer.rows(length, pages)
        e_step = max(e_step, err(got, layer.plain(xh[t:t + 1], torch.tensor([t]), k.cpu().double(), v.cpu().double())))
    coli.sync_check()
    return e_prompt, e_step, right, layer, xd, pages, length


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--keep", type=int, default=128)
    a = ap.parse_args()
    e_prompt, e_step, right, layer, x, pages, length = run(a.hidden, a.heads, a.kv, a.prompt, a.steps, a.keep)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(50):
        layer.step(x[-1:], a.prompt + a.steps - 1, length - 1, pages)
    t1.record()
    torch.cuda.synchronize()
    print(f"{a.heads} heads on {a.kv}, prompt {a.prompt}, {a.steps} steps, {length} tokens kept: error of the prompt {e_prompt:.1e}, of the "
          f"steps {e_step:.1e}; the tokens that stay are {'those' if right else 'NOT those'} of most weight; "
          f"{t0.elapsed_time(t1) * 20:.0f} us a step")


if __name__ == "__main__":
    main()
