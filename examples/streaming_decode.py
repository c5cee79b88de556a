"""A small decoder that streams through a bounded KV cache.

Random weights, no tokenizer: it shows how the library's calls fit together in a decode loop.
Every layer appends the new tokens' keys and values (normed and rotated on the way) and attends
over its slices; when the slices have grown `slack` rows beyond the budget, one eviction step
cuts every slice of every layer back to it. With ``--image`` attention reads the 8-bit image of
the full blocks, which is brought up to date once per step and rebuilt behind an eviction.

    python examples/streaming_decode.py --prompt 4096 --tokens 256 --budget 1024 --slack 128
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from streaming_kv_cache_step_gb300 import nexus  # noqa: E402


class StreamingDecoder:
    """`layers` blocks of attention and a gated feed-forward, bf16, one GPU."""

    def __init__(self, layers=2, seqs=2, kv_heads=2, group=4, head_dim=128, budget=1024, slack=128,
                 chunk=512, window=16, theta=500000.0, image=False, seed=0, device="cuda"):
        self.L, self.S, self.H, self.G, self.d = layers, seqs, kv_heads, group, head_dim
        self.budget, self.slack, self.chunk, self.window = budget, slack, chunk, window
        dev = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)
        width = kv_heads * group * head_dim
        heads = kv_heads * (group + 2) * head_dim

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=dev).div(shape[0] ** 0.5).bfloat16()

        self.qkv = [weight(width, heads) for _ in range(layers)]
        self.out = [weight(width, width) for _ in range(layers)]
        self.up = [weight(width, 2 * width) for _ in range(layers)]
        self.down = [weight(width, width) for _ in range(layers)]
        self.q_norm = [1 + 0.1 * weight(head_dim) for _ in range(layers)]
        self.k_norm = [1 + 0.1 * weight(head_dim) for _ in range(layers)]
        self.rotary = nexus.Rotary([theta ** (-2.0 * i / head_dim) for i in range(head_dim // 2)],
                                   device=dev)
        # rows: the budget, the slack, and the chunk that may arrive before the next eviction
        self.capacity = budget + slack + chunk
        shape = (layers, seqs, kv_heads, self.capacity)
        self.cache = nexus.Cache(
            k=torch.empty(*shape, head_dim, dtype=torch.bfloat16, device=dev),
            v=torch.empty(*shape, head_dim, dtype=torch.bfloat16, device=dev),
            pos=torch.empty(shape, dtype=torch.int32, device=dev),
            lens=torch.zeros(shape[:3], dtype=torch.int32, device=dev), layers=layers, seqs=seqs,
            kv_heads=kv_heads, group=group, head_dim=head_dim, capacity=self.capacity)
        self.image = nexus.new_image(self.cache) if image else None
        self.status = nexus.new_status(dev)
        self.attend_ws = nexus.alloc_attend_workspace(self.cache, tokens=seqs * chunk,
                                                      max_tokens=chunk)
        self.params = nexus.Params(
            budget=torch.full((seqs,), budget, dtype=torch.int32, device=dev), budget_max=budget,
            window=window, walk_len=min(3, window), n_sink=min(32, budget // 4),
            n_recent=min(32, budget // 4), seed=0x243F6A8885A308D3)
        self.evict_ws = nexus.alloc_workspace(self.cache, self.params)
        # the last `window` queries of every layer, newest last: what an eviction scores with
        self.queries = torch.zeros(layers, seqs, kv_heads * group, window, head_dim,
                                   dtype=torch.bfloat16, device=dev)
        self.held = 0              # rows of every slice, known on the host
        self.position = 0          # of the next token
        self.evictions = 0

    def forward(self, x):
        """x [seqs, n, width], the next n <= chunk tokens of every sequence; returns the same
        shape. Evicts first if the tokens would take the slices beyond budget + slack + chunk."""
        S, n, width = x.shape
        if n > self.chunk:
            raise ValueError(f"at most {self.chunk} tokens at once")
        if self.held + n > self.capacity or self.held > self.budget + self.slack:
            self.evict()
        H, G, d = self.H, self.G, self.d
        x = x.reshape(S * n, width)
        pos = torch.arange(self.position, self.position + n, dtype=torch.int32, device=x.device)
        pos = pos.repeat(S)
        q = torch.empty(S * n, H * G, d, dtype=torch.bfloat16, device=x.device)
        y = torch.empty_like(q)
        for l in range(self.L):
            p = (_rms(x) @ self.qkv[l]).view(S * n, H * (G + 2), d)
            nexus.append(self.cache, l, p[:, :H * G], p[:, H * G:-H], p[:, -H:], pos, q,
                         self.status, max_tokens=n, rotary=self.rotary, q_norm=self.q_norm[l],
                         k_norm=self.k_norm[l])
            nexus.attend(self.cache, l, q, y, self.attend_ws, self.status, max_tokens=n,
                         image=self.image)
            self._keep_queries(l, q.view(S, n, H * G, d))
            x = x + y.view(S * n, width) @ self.out[l]
            a, b = (_rms(x) @ self.up[l]).chunk(2, dim=-1)
            x = x + (torch.nn.functional.silu(a) * b) @ self.down[l]
        self.held += n
        self.position += n
        if self.image is not None:     # the blocks that became full in this step
            nexus.quantize(self.cache, self.image, self.status)
        return x.view(S, n, width)

    def _keep_queries(self, l, q):
        w, n = self.window, q.shape[1]
        new = q[:, max(0, n - w):].transpose(1, 2)
        if n >= w:
            self.queries[l] = new
        else:
            self.queries[l] = torch.cat([self.queries[l, :, :, n:], new], dim=2)

    def evict(self):
        """One eviction step over all layers; returns the kept slots per slice."""
        keep = torch.empty(self.cache.n_slices, self.capacity, dtype=torch.int32,
                           device=self.cache.k.device)
        self.params.step = self.evictions
        nexus.evict_step(self.cache, self.queries, self.params, keep, self.evict_ws, self.status)
        self.held = min(self.held, self.budget)
        self.evictions += 1
        if self.image is not None:     # the rows moved: the image starts over
            self.image.rows.zero_()
            nexus.quantize(self.cache, self.image, self.status)
        return keep

    def check(self):
        """Raises if any call since the last check found something wrong on the device."""
        got = int(self.status.item())
        self.status.zero_()
        if got:
            raise RuntimeError(f"device status {got}")


def _rms(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--budget", type=int, default=1024)
    ap.add_argument("--slack", type=int, default=128)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--image", action="store_true")
    a = ap.parse_args()
    m = StreamingDecoder(layers=a.layers, seqs=a.seqs, kv_heads=8, budget=a.budget, slack=a.slack,
                         chunk=a.chunk, image=a.image)
    width = m.H * m.G * m.d
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in range(0, a.prompt, a.chunk):
        n = min(a.chunk, a.prompt - at)
        x = m.forward(torch.randn(a.seqs, n, width, generator=g, device="cuda").bfloat16())
    m.check()
    x = x[:, -1:]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens):
        x = m.forward(_rms(x))
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    m.check()
    print(f"{a.tokens} tokens of {a.seqs} sequences in {1e3 * t:.1f} ms "
          f"({1e6 * t / a.tokens / a.layers:.0f} us per layer and step), {m.evictions} evictions, "
          f"{m.held} rows of {m.position} positions held")


if __name__ == "__main__":
    main()
