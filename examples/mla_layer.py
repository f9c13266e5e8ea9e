"""The attention of one MLA decoder layer, from hidden states to hidden states, on the library's calls alone.

    python examples/mla_layer.py [--heads 16] [--hidden 1024] [--prompt 300] [--steps 8] [--bf16]

A prompt runs in the expanded form (every head's keys and values computed from the cached rows with kv_b), the
tokens after it in the absorbed form over the paged cache (E4M3 rows with a scale each, or bf16 with --bf16).
The last lines say how far both are from the layer computed in 64 bits from the same quantised weights and the
same cached rows, and how long a step takes.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_gemv_fmt1_gb300 as coli  # noqa: E402

L, R, N, V = 512, 64, 128, 128     # latent and rotary dims of a cached row; no-position and value dims of a head
GROUP = 64                         # inputs per int4 scale


def int4_matrix(g: np.random.Generator, rows: int, cols: int):
    """A random int4 matrix (fmt=4) and its values."""
    codes = g.integers(0, 16, (rows, cols), dtype=np.uint8)
    scales = (g.uniform(0.5, 1.5, (rows, cols // GROUP)) / (4.0 * math.sqrt(cols))).astype(np.float32)
    data = codes[:, 0::2] | (codes[:, 1::2] << 4)
    values = (codes.astype(np.float64) - 8.0) * np.repeat(scales.astype(np.float64), GROUP, 1)
    return coli.tensor_upload(4, GROUP, rows, cols, data, scales), torch.from_numpy(values)


class MlaLayer:
    """Weights, rotation table and paged cache of one layer; `n_pages` pages of `page` tokens."""

    def __init__(self, hidden: int, heads: int, n_pages: int, page: int = 64, e4m3: bool = True, seed: int = 0):
        g = np.random.default_rng(seed)
        self.hidden, self.heads, self.page = hidden, heads, page
        self.q, self.q_values = int4_matrix(g, heads * (N + R), hidden)
        self.kv_a, self.kv_a_values = int4_matrix(g, L + R, hidden)
        self.kv_b, self.kv_b_values = int4_matrix(g, heads * (N + V), L)
        self.o, self.o_values = int4_matrix(g, hidden, heads * V)
        self.norm = torch.from_numpy(g.uniform(0.5, 1.5, L).astype(np.float32)).cuda()
        freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
        angle = torch.arange(n_pages * page, dtype=torch.float64)[:, None] * freq
        self.rot = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.scale = 1.0 / math.sqrt(N + R)
        rows = torch.zeros(n_pages, page, L + R, device="cuda", dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        self.cache = coli.MlaCache(rows, L, R, torch.zeros(n_pages, page, device="cuda") if e4m3 else None)

    def _store(self, x, pos, pages):
        """The new tokens' rows into the cache, at positions `pos` of a sequence on `pages`."""
        kv = torch.empty(x.shape[0], L + R, device="cuda")
        coli.matmul(self.kv_a, x, kv)
        slots = pages[0].long()[pos.long() // self.page] * self.page + pos.long() % self.page
        coli.mla_append(self.cache, kv, self.norm, 1e-6, pos, self.rot, slots)

    def prompt(self, x, pages):
        """Attention of a prompt x [T, hidden] whose pages [1, n] are empty yet."""
        T, H = x.shape[0], self.heads
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        self._store(x, pos, pages)
        q = torch.empty(T, H, N + R, device="cuda")
        coli.matmul(self.q, x, q.view(T, -1))
        coli.mla_query(q, pos, self.rot, q[..., :N], q[..., N:])          # in place: each thread writes what it read
        cu = torch.tensor([0, T], device="cuda", dtype=torch.int32)
        rows = torch.empty(T, L + R, device="cuda")
        coli.mla_read(self.cache, pages, cu, rows)
        kv = torch.empty(T, H, N + V, device="cuda")
        coli.matmul(self.kv_b, rows[:, :L].contiguous(), kv.view(T, -1))
        out = torch.empty(T, H, V, device="cuda")
        coli.mla_prefill(q, kv, rows[:, L:], cu, cu, self.scale, out)
        y = torch.empty(T, self.hidden, device="cuda")
        coli.matmul(self.o, out.view(T, -1), y)
        return y

    def step(self, x, pos: int, pages):
        """Attention of one new token x [1, hidden] at position pos."""
        H = self.heads
        at = torch.tensor([pos], device="cuda", dtype=torch.int32)
        self._store(x, at, pages)
        q = torch.empty(1, H, N + R, device="cuda")
        coli.matmul(self.q, x, q.view(1, -1))
        nope, rope = torch.empty(1, H, N, device="cuda"), torch.empty(1, H, R, device="cuda")
        coli.mla_query(q, at, self.rot, nope, rope)
        latent, mixed = torch.empty(1, 1, H, L, device="cuda"), torch.empty(1, 1, H, L, device="cuda")
        coli.matmul_rows_t(self.kv_b, 0, N + V, N, H, nope, latent, S=1)
        coli.mla_attend(self.cache, latent, rope.view(1, 1, H, R), pages, at + 1, self.scale, mixed)
        out = torch.empty(1, H, V, device="cuda")
        coli.matmul_rows(self.kv_b, N, N + V, V, H, mixed, out, S=1)
        y = torch.empty(1, self.hidden, device="cuda")
        coli.matmul(self.o, out.view(1, -1), y)
        return y

    def plain(self, x, rows):
        """The layer in 64 bits on the host: x [T, hidden], the cached rows [T, L + R] as they stand."""
        T, H = x.shape[0], self.heads
        q = (x @ self.q_values.T).view(T, H, N + R)
        rot = self.rot.cpu().double()[:T, None]
        c, s = rot[..., :R // 2], rot[..., R // 2:]
        a, b = q[..., N:N + R // 2], q[..., N + R // 2:]
        q = torch.cat([q[..., :N], a * c - b * s, a * s + b * c], -1)
        kv = (rows[:, :L] @ self.kv_b_values.T).view(T, H, N + V)
        k = torch.cat([kv[..., :N], rows[:, None, L:].expand(T, H, R)], -1)
        score = torch.einsum("ihd,jhd->hij", q, k) * self.scale
        score = score.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
        out = torch.einsum("hij,jhd->ihd", torch.softmax(score, -1), kv[..., N:])
        return out.reshape(T, -1) @ self.o_values.T


def run(hidden=1024, heads=16, prompt=300, steps=8, e4m3=True, seed=0):
    """Errors (largest difference over the largest value) of the prompt's and the steps' outputs; the layer and its state."""
    total = prompt + steps
    n = -(-total // 64)
    layer = MlaLayer(hidden, heads, n + 2, e4m3=e4m3, seed=seed)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(total, hidden, generator=g)
    pages = torch.randperm(n + 2, generator=g)[None, :n].to(torch.int32).cuda()
    xd = x.cuda()
    got = [layer.prompt(xd[:prompt], pages)]
    for t in range(prompt, total):
        got.append(layer.step(xd[t:t + 1], t, pages))
    rows = torch.empty(total, L + R, device="cuda")
    coli.mla_read(layer.cache, pages, torch.tensor([0, total], dtype=torch.int32, device="cuda"), rows)
    coli.sync_check()
    want = layer.plain(x.double(), rows.cpu().double())
    err = lambda a, b: float((a.cpu().double() - b).abs().max() / b.abs().max())  # noqa: E731
    return err(got[0], want[:prompt]), err(torch.cat(got[1:]), want[prompt:]), layer, xd, pages


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--bf16", action="store_true", help="a bf16 cache instead of E4M3")
    a = ap.parse_args()
    e_prompt, e_step, layer, x, pages = run(a.hidden, a.heads, a.prompt, a.steps, not a.bf16)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(50):
        layer.step(x[-1:], a.prompt + a.steps - 1, pages)
    t1.record()
    torch.cuda.synchronize()
    print(f"{a.heads} heads, prompt {a.prompt}, {'bf16' if a.bf16 else 'e4m3'} cache: error of the prompt {e_prompt:.1e}, "
          f"of {a.steps} steps {e_step:.1e}; {t0.elapsed_time(t1) * 20:.0f} us a step")


if __name__ == "__main__":
    main()
