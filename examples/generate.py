"""A small decoder with random 4-bit weights, run the way a serving loop runs one: prompts of different lengths go
through in one call, then each step feeds every sequence its last token, from a HIP graph if asked.

Per layer: one fused q/k/v projection (mxq_linear), rotary positions on views of it (mxq_rope, in place), the new
keys and values into the 8-bit paged cache (mxq_kv_append), attention over it (mxq_attention), the output projection
and a gated MLP; then lm_head and the next token's draw (mxq_sample).  With norms of each head's queries and keys, the
norms, the rotation and the append are one call (mxq_rope_append); the cache may be held in 4 bits (KvCache4).

    python examples/generate.py [--steps 32] [--graph] [--norms] [--bits 4]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import dequant_matmul_qmv_amd as mxq  # noqa: E402

DEV = "cuda:0"


class Linear:
    """y = x W^T with random 4-bit codes, groups of 64, zero on average."""

    def __init__(self, n, k, gen):
        self.w = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=gen, dtype=torch.int64).to(torch.int32).to(DEV)
        scale = (0.5 + torch.rand(n, k // 64, generator=gen)) * 0.2 / k ** 0.5
        self.scales, self.biases = scale.half().to(DEV), (-7.5 * scale).half().to(DEV)

    def __call__(self, x):
        return mxq.mxq_linear(x, self.w, self.scales, self.biases, bits=4, group_size=64)


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Decoder:
    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, ffn=1024, vocab=4099, pages=64, block=16, seed=0,
                 norms=False, bits=8):
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.ffn, self.block = heads, kv_heads, dim, ffn, block
        self.embed = torch.randn(vocab, hidden, generator=gen).half().to(DEV)
        self.layers = [(Linear((heads + 2 * kv_heads) * dim, hidden, gen), Linear(hidden, heads * dim, gen),
                        Linear(2 * ffn, hidden, gen), Linear(hidden, ffn, gen)) for _ in range(layers)]
        self.head = Linear(vocab, hidden, gen)
        self.inv_freq = (500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).float().to(DEV)
        self.norms = None
        if norms:
            self.norms = [[(1 + 0.2 * torch.randn(dim, generator=gen)).half().to(DEV) for _ in range(2)] for _ in range(layers)]
        kind = mxq.KvCache if bits == 8 else mxq.KvCache4
        self.caches = [kind.empty(pages, kv_heads, block, dim, DEV) for _ in range(layers)]

    def __call__(self, ids, positions, table, lens, starts=None):
        """Logits of each sequence's last token.  `lens` counts the new tokens; `starts` as in mxq_kv_append."""
        x, n = self.embed[ids], ids.shape[0]
        q_end, k_end = self.heads * self.dim, (self.heads + self.kv_heads) * self.dim
        for i, ((qkv_proj, o_proj, up, down), cache) in enumerate(zip(self.layers, self.caches)):
            qkv = qkv_proj(norm(x))
            q = qkv[:, :q_end].view(n, self.heads, self.dim)
            k = qkv[:, q_end:k_end].view(n, self.kv_heads, self.dim)
            v = qkv[:, k_end:].view(n, self.kv_heads, self.dim)
            if self.norms:
                mxq.mxq_rope_append(cache, q, k, v, self.inv_freq, table, lens, starts, *self.norms[i], q, positions=positions)
            else:
                mxq.mxq_rope(q, k, self.inv_freq, positions, q, k)
                mxq.mxq_kv_append(cache, k, v, table, lens, starts)
            y = mxq.mxq_attention(q, cache, table, lens, starts)
            x = x + o_proj(y.view(n, q_end))
            g = up(norm(x))
            x = x + down(torch.nn.functional.silu(g[:, :self.ffn]) * g[:, self.ffn:])
        if starts is not None:
            x = x[starts[1:].long() - 1]
        return self.head(norm(x))


def generate(model, prompts, steps, graph=False, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, seed=0):
    """`steps` tokens for each prompt (lists of token ids): an int32 tensor [prompts, steps]."""
    n, lengths = len(prompts), [len(p) for p in prompts]
    pages = -(-(max(lengths) + steps) // model.block)
    if n * pages > model.caches[0].blocks:
        raise ValueError(f"{n} sequences of {pages} pages do not fit a cache of {model.caches[0].blocks}")
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.arange(n * pages, dtype=torch.int32, device=DEV).view(n, pages)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    starts = torch.tensor([sum(lengths[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
    ids = torch.tensor([t for p in prompts for t in p], device=DEV)
    positions = torch.cat([torch.arange(m, dtype=torch.int32, device=DEV) for m in lengths])
    draws = torch.rand(steps, n, generator=gen, device=DEV)
    settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    out = torch.empty(steps, n, dtype=torch.int32, device=DEV)
    token, _ = mxq.mxq_sample(model(ids, positions, table, lens, starts), draws[0], **settings)
    out[0] = token
    # the step's own inputs, which the graph reads at their place
    at, u = lens.clone(), draws[0].clone()

    def step():
        lens.copy_(at + 1)
        logits = model(token.long(), at, table, lens)
        mxq.mxq_sample(logits, u, token, probs, **settings)
        at.copy_(lens)

    probs = torch.empty(n, device=DEV)
    replay = None
    for i in range(1, steps):
        u.copy_(draws[i])
        if i < 3 or not graph:  # the first steps run eagerly: they also load what the capture needs
            step()
        else:
            if replay is None:
                replay = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(replay):
                    step()
            replay.replay()
        out[i] = token
    return out.T.contiguous()


def main():
    args = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    args.add_argument("--steps", type=int, default=32)
    args.add_argument("--graph", action="store_true")
    args.add_argument("--norms", action="store_true")
    args.add_argument("--bits", type=int, choices=(4, 8), default=8)
    args = args.parse_args()
    prompts = [[1, 5, 9, 200, 31], list(range(100, 140)), [7]]
    for tokens in generate(Decoder(pages=256, norms=args.norms, bits=args.bits), prompts, args.steps, args.graph).tolist():
        print(tokens)


if __name__ == "__main__":
    main()
