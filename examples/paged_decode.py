"""Serving with an MXFP8 key/value cache: prompts enter in chunks beside requests that decode.

One attention layer with MXFP8 projections (mx_quantize, mx_gemm), rotary positions, a
paged cache (mx_kv_append) and attention over it (mx_paged_attention).  Every request's
tokens are fed in steps of a mixed batch: a chunk while it has more than one token left,
then one token a step.  The layer's outputs over all steps are compared with the same
layer computed at once in float32 from the same quantized weights.

    python examples/paged_decode.py [--requests 6] [--dim 128] [--steps-of 48]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_block_scaled_quantize_amd as mxa  # noqa: E402


class Layer:
    """Fused q, k, v projection and output projection, weights in MXFP8."""

    def __init__(self, width, heads, kv_heads, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.dim = width, heads, kv_heads, dim
        self.w = {}
        for name, rows, cols in (("qkv", (heads + 2 * kv_heads) * dim, width), ("out", width, heads * dim)):
            w = torch.randn((rows, cols), device="cuda", generator=g) * cols ** -0.5
            self.w[name] = mxa.mx_quantize(w.bfloat16())

    def project(self, name, x):
        return mxa.mx_gemm(*mxa.mx_quantize(x), *self.w[name])

    def step(self, x, state, slots, pos, page_table, cu, lens, max_q, max_kv):
        """x [tokens][width] bfloat16: the new tokens of all requests in a row."""
        qkv = self.project("qkv", x).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = mxa.mx_kv_append(k, v, state["cache"], slots, pos, state["rope"], q=q)
        o = mxa.mx_paged_attention(q, state["cache"], page_table, cu, lens, max_q=max_q, max_kv=max_kv)
        return self.project("out", o.flatten(1))

    def reference(self, x, rope):
        """One request's tokens at once, float32 but for the quantized weights and activations."""
        def matmul(name, x):
            w = mxa.mx_dequantize(*self.w[name], *self.shape(name))
            a = mxa.mx_dequantize(*mxa.mx_quantize(x.bfloat16()), *x.shape)
            return a @ w.T
        n = x.shape[0]
        q, k, v = matmul("qkv", x).view(n, -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], 1)
        c, s = rope[:n, None, :, 0], rope[:n, None, :, 1]
        half = self.dim // 2
        turn = lambda t: torch.cat([t[..., :half] * c - t[..., half:] * s, t[..., half:] * c + t[..., :half] * s], -1)  # noqa: E731
        q, k = turn(q), turn(k)
        group = self.heads // self.kv_heads
        k, v = (t.repeat_interleave(group, 1).transpose(0, 1).contiguous() for t in (k, v))
        a = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * self.dim ** -0.5
        a = a.masked_fill(torch.ones((n, n), dtype=torch.bool, device=a.device).triu(1), -float("inf"))
        return matmul("out", torch.matmul(a.softmax(-1), v).transpose(0, 1).flatten(1))

    def shape(self, name):
        inner = (self.heads + 2 * self.kv_heads) * self.dim
        return (inner, self.width) if name == "qkv" else (self.width, self.heads * self.dim)


def serve(requests=6, width=512, heads=8, kv_heads=2, dim=128, page=16, chunk=48, seed=0):
    """Feeds requests of uneven lengths; returns the largest relative error of a request's outputs."""
    g = torch.Generator().manual_seed(seed)
    layer = Layer(width, heads, kv_heads, dim, seed)
    lengths = [int(n) for n in torch.randint(chunk // 2, 5 * chunk, (requests,), generator=g)]
    x = [torch.randn((n, width), generator=g).bfloat16().cuda() for n in lengths]
    need = [-(-n // page) for n in lengths]
    free = torch.randperm(sum(need), generator=g).int()
    table = torch.zeros((requests, max(need)), dtype=torch.int32)
    for r, n in enumerate(need):
        table[r, :n], free = free[:n], free[n:]
    on_gpu = table.cuda()
    state = {"cache": mxa.new_kv_cache(sum(need), kv_heads, page, dim), "rope": mxa.mx_rope_table(max(lengths), dim)}
    done, outputs, steps = [0] * requests, [[] for _ in x], 0
    while any(d < n for d, n in zip(done, lengths)):
        # whole chunks of the prompt, then its last tokens one by one as if they had just been sampled
        new = [0 if d == n else chunk if n - d > chunk else 1 for d, n in zip(done, lengths)]
        slots, pos = [], []
        for r, m in enumerate(new):
            for p in range(done[r], done[r] + m):
                slots.append(int(table[r, p // page]) * page + p % page)
                pos.append(p)
        lens = [d + m for d, m in zip(done, new)]
        cu = torch.tensor([0] + new).cumsum(0).int().cuda()
        y = layer.step(torch.cat([t[d:d + m] for t, d, m in zip(x, done, new)]), state, torch.tensor(slots).cuda(),
                       torch.tensor(pos, dtype=torch.int32).cuda(), on_gpu, cu,
                       torch.tensor(lens, dtype=torch.int32).cuda(), max(new), max(lens))
        for r, part in enumerate(y.split(new)):
            outputs[r].append(part)
        done, steps = lens, steps + 1
    worst = 0.0
    for r, t in enumerate(x):
        want = layer.reference(t.float(), state["rope"])
        worst = max(worst, float((torch.cat(outputs[r]).float() - want).norm() / want.norm()))
    return worst, steps, sum(lengths)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--steps-of", type=int, default=48)
    a = ap.parse_args()
    worst, steps, tokens = serve(a.requests, dim=a.dim, chunk=a.steps_of)
    print(f"{tokens} tokens of {a.requests} requests in {steps} steps, relative error against float32 attention {worst:.4f}")


if __name__ == "__main__":
    main()
