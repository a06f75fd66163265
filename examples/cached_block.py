"""A transformer block over the paged 4-bit cache, from the library's operators alone.

    python examples/cached_block.py [--width 1024] [--prompt 500] [--tokens 16]

Each block norms, modulates and quantizes (block_norm to INT8 codes), projects (masked_qgemm at
the step's weight bits), appends keys and values (kv_append, rotated), attends (kv_attention),
projects out, joins the residual stream and norms again (block_norm with its gate) and runs the
MLP (gelu_quant_act folds the GELU into the down projection's quantizer).  A prompt goes through
as one chunk, then tokens follow one at a time; the same tokens in one chunk show how far the two
ways differ.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import timestep_adaptive_bit_amd as T  # noqa: E402

DEV = "cuda:0"
HAD = 32


class Block:
    """Weights, modulation and cache of one block for up to `max_len` tokens of one sequence."""

    def __init__(self, ctx, width=1024, q_heads=16, kv_heads=4, head_dim=64, hidden=4096, max_len=1024,
                 page=16, k_bits=0, seed=0):
        self.ctx, self.width, self.hq, self.hk, self.D, self.k_bits = ctx, width, q_heads, kv_heads, head_dim, k_bits
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
        w = lambda n, k: ctx.quantize_weights((r(n, k) / math.sqrt(k)).bfloat16().to(DEV), HAD)   # noqa: E731
        self.qkv = w((q_heads + 2 * kv_heads) * head_dim, width)
        self.out = w(width, q_heads * head_dim)
        self.up, self.down = w(hidden, width), w(width, hidden)
        # gate, scale, shift of the attention and of the MLP: rows of one conditioning output
        self.mod = (0.2 * r(1, 6, width)).bfloat16().to(DEV)
        self.norm = (1 + 0.1 * r(4, width)).bfloat16().to(DEV)
        pages = (max_len + page - 1) // page
        self.cache = T.KVCache.empty(pages, page, kv_heads, head_dim, had_block=HAD, device=DEV)
        self.table = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)[None]
        self.page, self.max_len = page, max_len
        angle = torch.arange(max_len)[:, None] / 10000.0 ** (torch.arange(head_dim // 2) / (head_dim // 2))
        self.rope = T.Rope(angle.cos().to(DEV), angle.sin().to(DEV))
        self.used = 0

    def _linear(self, codes, scales, w):
        return self.ctx.masked_qgemm(codes, scales, w["w_q"], w["w_scale"], self.k_bits)[0]

    def forward(self, x):
        """x bf16 [n][width], the sequence's next n tokens: their new residual stream."""
        ctx, n, first = self.ctx, x.shape[0], self.used
        if first + n > self.max_len:
            raise ValueError(f"{first} + {n} tokens do not fit {self.max_len}")
        m, nw = self.mod, self.norm
        pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
        at = pos.long()
        slots = self.table[0].long()[at // self.page] * self.page + at % self.page
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        lens = torch.tensor([first + n], dtype=torch.int32, device=DEV)

        _, h, hs = ctx.block_norm(x, pre=T.NORM_LAYER, pre_weight=nw[0], scale=m[:, 1], shift=m[:, 2],
                                  fmt=T.FMT_INT8, had_block=HAD, want_x=False)
        qkv = self._linear(h, hs, self.qkv)
        heads = qkv.unflatten(1, (self.hq + 2 * self.hk, self.D))
        q, k, v = heads.split([self.hq, self.hk, self.hk], dim=1)      # slices: no copies
        ctx.kv_append(self.cache, k, v, slots, rope=self.rope, positions=pos)
        self.used = first + n
        a = ctx.kv_attention(self.cache, q, cu, self.table, lens, n, self.used, causal=True,
                             rope=self.rope, positions=pos)
        y = self._linear(*ctx.hadamard_quant_act(a.flatten(1), HAD), self.out)
        x, h, hs = ctx.block_norm(x, y, post=T.NORM_RMS, post_weight=nw[1], gate=m[:, 0],
                                  pre=T.NORM_LAYER, pre_weight=nw[2], scale=m[:, 4], shift=m[:, 5],
                                  fmt=T.FMT_INT8, had_block=HAD)
        y = self._linear(*ctx.gelu_quant_act(self._linear(h, hs, self.up), HAD), self.down)
        x, _, _ = ctx.block_norm(x, y, post=T.NORM_RMS, post_weight=nw[3], gate=m[:, 3], want_h=False)
        return x


def run(width=1024, q_heads=16, kv_heads=4, head_dim=64, hidden=4096, prompt=500, tokens=16, blocks=2):
    """The stream after `blocks` blocks of prompt + tokens: in one chunk, and with the tokens one
    at a time; and the milliseconds a single token took."""
    with torch.no_grad():
        ctx = T.Context()
        n = prompt + tokens
        g = torch.Generator().manual_seed(1)
        x = torch.randn(n, width, generator=g).bfloat16().to(DEV)

        def make():
            return [Block(ctx, width, q_heads, kv_heads, head_dim, hidden, n, seed=i) for i in range(blocks)]

        def through(stack, rows):
            for b in stack:
                rows = b.forward(rows)
            return rows

        whole = through(make(), x)
        stack = make()
        parts = [through(stack, x[:prompt])]
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(prompt, n):
            parts.append(through(stack, x[i:i + 1]))
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t) * 1e3 / max(tokens, 1)
        step = torch.cat(parts)
        ctx.close()
        return whole, step, ms


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--tokens", type=int, default=16)
    a = p.parse_args()
    whole, step, ms = run(width=a.width, hidden=4 * a.width, prompt=a.prompt, tokens=a.tokens)
    d = (whole.double() - step.double()).norm() / whole.double().norm()
    print(f"{a.prompt} + {a.tokens} tokens: one chunk and token by token differ by {d:.2e}; {ms:.2f} ms a token")
