"""Beam search over an MXFP8 key/value cache whose pages the beams share.

A small transformer of random weights (rotary attention over the paged cache, residual, tied output
projection) generates with several beams for each request.  Between two steps nothing leaves the GPU:
mx_beam_select chooses the next beams and reorders their tokens, mx_kv_fork gives them their parents' pages,
pages and slots for their next token and copies of partly filled pages in every layer, mx_kv_append and
mx_paged_attention take its table, lengths and slots as they are.  Now and then the pool is compacted; at
the end all pages are given back.  ``replay`` feeds the sequences found one by one, each in pages of its own,
and returns their log-probabilities: what the search's scores have to be.

    python examples/beam_search.py [--requests 3] [--beams 4] [--steps 24]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_block_scaled_quantize_amd as mxa  # noqa: E402


class Model:
    def __init__(self, vocab=500, layers=2, heads=4, kv_heads=2, dim=64, longest=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.heads, self.kv_heads, self.dim, self.width = vocab, heads, kv_heads, dim, heads * dim
        normal = lambda *n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
        self.embedding = normal(vocab, self.width)
        self.qkv = [normal(self.width, (heads + 2 * kv_heads) * dim) * self.width ** -0.5 for _ in range(layers)]
        self.rope = mxa.mx_rope_table(longest, dim)

    def new_caches(self, pages, page):
        return [mxa.new_kv_cache(pages, self.kv_heads, page, self.dim) for _ in self.qkv]

    def step(self, caches, tokens, pos, cu, fork, max_q, max_kv):
        """New tokens of all sequences in a row, at positions pos; logits behind each sequence's last one."""
        x = self.embedding[tokens.long()]
        for w, cache in zip(self.qkv, caches):
            # row by row the same whatever the other rows are
            qkv = (x[:, :, None] * w).sum(1).bfloat16().unflatten(1, (-1, self.dim))
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
            q = mxa.mx_kv_append(k, v, cache, fork.slots, pos, self.rope, q=q)
            o = mxa.mx_paged_attention(q, cache, fork.page_table, cu, fork.lens, max_q=max_q, max_kv=max_kv)
            x = x + o.flatten(1).float()
        last = x[(cu[1:] - 1).long()]
        return (last[:, :, None] * self.embedding.T).sum(1) * (4.0 * self.width ** -0.5 / len(self.qkv))


def feed_prompts(model, prompts, caches, refs, cols, longest):
    """A sequence for each prompt, and the logits behind it."""
    n = [len(p) for p in prompts]
    cu = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
    none = torch.zeros((0, cols), dtype=torch.int32, device="cuda")
    new = torch.full((len(n),), -1, dtype=torch.int32, device="cuda")
    fork = mxa.mx_kv_fork(caches, refs, none, none[:, 0].contiguous(), cu, parents=new, tokens=sum(n))
    tokens = torch.tensor(sum(prompts, []), dtype=torch.int32, device="cuda")
    pos = torch.tensor([i for m in n for i in range(m)], dtype=torch.int32, device="cuda")
    return fork, model.step(caches, tokens, pos, cu, fork, max(n), longest)


def search(model, prompts, beams, steps, page=16, eos=-1, compact_every=5):
    """Returns the best beams' tokens [requests][beams][steps], lengths, scores and finished flags, and how many pages
    were in use at most.  The pool has as many pages as beams that share nothing behind their prompts can need."""
    requests, longest = len(prompts), max(map(len, prompts)) + steps
    cols = -(-longest // page)
    pages = sum(-(-len(p) // page) + beams * (-(-steps // page) + 2) for p in prompts)
    caches, most = model.new_caches(pages, page), 0
    fork, logits = feed_prompts(model, prompts, caches, mxa.new_page_refs(pages), cols, longest)
    step = mxa.mx_beam_select(logits.unflatten(0, (requests, 1)), torch.zeros((requests, 1), device="cuda"), beams, eos=eos,
                              history=torch.zeros((requests, 1, steps), dtype=torch.int32, device="cuda"),
                              lens=torch.zeros((requests, 1), dtype=torch.int32, device="cuda"))
    one = torch.arange(requests * beams + 1, dtype=torch.int32, device="cuda")
    for t in range(1, steps):
        fork = mxa.mx_kv_fork(caches, fork.refs, fork.page_table, fork.lens, one, parents=step.parents,
                              tokens=requests * beams)
        logits = model.step(caches, step.tokens.flatten(), fork.lens - 1, one, fork, 1, longest)
        if t % compact_every == 0:
            refs, table, used = mxa.mx_kv_compact(caches, fork.refs, fork.page_table, fork.lens)
            fork = fork._replace(refs=refs, page_table=table)
            most = max(most, int(used))
        step = mxa.mx_beam_select(logits.unflatten(0, (requests, beams)), step.scores, finished=step.finished, eos=eos,
                                  history=step.history, lens=step.lens)
    refs, _ = mxa.mx_kv_free(fork.refs, fork.page_table, fork.lens, page)
    assert int(refs.abs().sum()) == 0, "pages are left"
    return step, most


def replay(model, prompts, history, lens, page=16):
    """Log-probability of each sequence of history [requests][beams][steps], fed alone in pages of its own."""
    requests, beams, steps = history.shape
    longest = max(map(len, prompts)) + steps
    cols = -(-longest // page)
    pages = requests * beams * cols
    caches = model.new_caches(pages, page)
    fork, logits = feed_prompts(model, [p for p in prompts for _ in range(beams)], caches, mxa.new_page_refs(pages), cols,
                                longest)
    one = torch.arange(requests * beams + 1, dtype=torch.int32, device="cuda")
    total = torch.zeros(requests * beams, dtype=torch.float64, device="cuda")
    for t in range(steps):
        token = history.flatten(0, 1)[:, t]
        p = logits.double().log_softmax(-1).gather(1, token.long()[:, None])[:, 0]
        total += torch.where(t < lens.flatten(), p, 0.0)
        if t + 1 < steps:
            fork = mxa.mx_kv_fork(caches, fork.refs, fork.page_table, fork.lens, one, tokens=requests * beams)
            logits = model.step(caches, token, fork.lens - 1, one, fork, 1, longest)
    return total.unflatten(0, (requests, beams))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (int(n),), generator=g).tolist()
               for n in torch.randint(1, 60, (a.requests,), generator=g)]
    step, most = search(model, prompts, a.beams, a.steps)
    off = (replay(model, prompts, step.history, step.lens) - step.scores).abs().max()
    print(f"{a.requests} requests of {a.beams} beams, {a.steps} steps, at most {most} pages in use; best scores "
          f"{[round(x, 3) for x in step.scores[:, 0].tolist()]}, off by at most {float(off):.1e} when fed alone")


if __name__ == "__main__":
    main()
