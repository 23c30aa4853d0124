"""A decode loop on the library's operators: one attention layer and a head.

    python examples/decode_loop.py [--steps 32] [--cache mxfp8]

Prompts of ragged lengths are written into a paged key-value cache; every step
then takes the last token of each sequence through NVFP4 projections
(gemm_nvfp4_act), appends its key and value, attends to the cache while the
attention's weights accumulate, and reports the chosen token's log
probability, the entropy and the alternatives.  When a sequence outgrows its
budget, the tokens with the least accumulated weight are evicted into fresh
pages and the old pages are freed.  Weights are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_03_amd as fp4  # noqa: E402

FORMATS = {"bf16": fp4.KV_BF16, "mxfp8": fp4.KV_MXFP8, "mxfp4": fp4.KV_MXFP4}


class Layer:
    """One attention layer with an output head, its weights in NVFP4."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            return fp4.quantize(w, fp4.NVFP4)

        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.vocab = hidden, q_heads, kv_heads, head_dim, vocab
        self.embed = torch.randn(vocab, hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        self.head = weight(vocab, hidden)

    def project(self, x):
        """q, k, v of rows x, as views of one product (rows x heads x head_dim)."""
        heads = self.q_heads + 2 * self.kv_heads
        # (The fused decode product takes up to 32 rows; a prompt takes the tiled one.)
        if fp4.fp4_gemm_nvfp4_act_supported(x.shape[0], heads * self.head_dim, self.hidden, fp4.BF16):
            y = fp4.gemm_nvfp4_act(x, self.qkv)
        else:
            y = fp4.gemm(fp4.quantize(x, fp4.NVFP4), self.qkv)
        y = y.view(x.shape[0], heads, self.head_dim)
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)


class Sequences:
    """The cache of a batch: a pool of pages, who holds which, and the accumulated weights."""

    def __init__(self, layer, batch, tokens, page_size, fmt):
        self.width = -(-tokens // page_size)
        self.cache = fp4.KVCache.empty(2 * batch * self.width, page_size, layer.kv_heads, layer.head_dim, fmt)
        self.free = list(range(2 * batch * self.width))
        self.table = self.pages(batch)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros(batch, layer.kv_heads, self.width * page_size, device="cuda")
        self.ids = torch.arange(batch, dtype=torch.int32, device="cuda")

    def pages(self, batch):
        n = batch * self.width
        got, self.free = self.free[:n], self.free[n:]
        return torch.tensor(got, dtype=torch.int32, device="cuda").view(batch, self.width)

    def evict(self, budget, recent):
        """Every sequence down to `budget` tokens, in fresh pages."""
        table = self.pages(self.table.shape[0])
        self.lens, self.weights, kept = fp4.kv_evict(self.cache, self.table, self.lens, self.weights, budget, recent,
                                                     table)
        self.free += self.table.flatten().tolist()
        self.table = table
        return kept


def run(steps=32, batch=4, prompt=200, budget=96, recent=16, cache="mxfp8", hidden=512, q_heads=8, kv_heads=2,
        head_dim=64, vocab=2048, page_size=16, top_k=5, seed=0):
    layer = Layer(hidden, q_heads, kv_heads, head_dim, vocab, seed)
    g = torch.Generator().manual_seed(seed)
    lens = [1 + int(torch.randint(0, prompt, (1,), generator=g)) for _ in range(batch)]
    seqs = Sequences(layer, batch, max(prompt, budget) + steps + 1, page_size, FORMATS[cache])

    # The prompts, all rows at once: row i is token pos[i] of sequence seq[i].
    seq = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(lens)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    tokens = torch.randint(0, vocab, (len(seq),), generator=g).cuda()
    _, k, v = layer.project(layer.embed[tokens])
    fp4.kv_append(seqs.cache, k, v, seqs.table, seq, pos)
    seqs.lens += torch.tensor(lens, dtype=torch.int32, device="cuda")

    token = tokens[torch.tensor(lens).cumsum(0).cuda() - 1]
    ws = fp4.attention_workspace(seqs.cache, batch, q_heads, seqs.table.shape[1] * page_size, weights=True)
    lp_ws = fp4.logprobs_workspace(batch, vocab, top_k)
    longest, history = max(lens), []
    for _ in range(steps):
        x = layer.embed[token]
        q, k, v = layer.project(x)
        fp4.kv_append(seqs.cache, k, v, seqs.table, seqs.ids, seqs.lens)
        seqs.lens += 1
        longest += 1
        a = fp4.decode_attention(q, seqs.cache, seqs.table, seqs.lens, weights=seqs.weights, weights_out=seqs.weights,
                                 ws=ws)
        y = x + fp4.gemm_nvfp4_act(a.view(batch, -1), layer.out)
        logits = fp4.gemm_nvfp4_act(y, layer.head, out_dtype=torch.float32)
        best = fp4.logprobs(logits, token.to(torch.int32).view(-1, 1), top_k=top_k, ws=lp_ws)
        token = best.top_index[:, 0].long()
        history.append({"token": token, "logp": best.top_logp[:, 0], "entropy": best.entropy, "logits": logits,
                        "alternatives": best.top_index, "lens": seqs.lens.clone()})
        if longest >= budget + recent:
            seqs.evict(budget, recent)
            longest = budget
    return history


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--cache", choices=sorted(FORMATS), default="mxfp8")
    a = p.parse_args()
    for i, h in enumerate(run(steps=a.steps, cache=a.cache)):
        print("step %d  lens %s  tokens %s  logp %s  entropy %s" % (
            i, h["lens"].tolist(), h["token"].tolist(), ["%.2f" % v for v in h["logp"].tolist()],
            ["%.2f" % v for v in h["entropy"].tolist()]))


if __name__ == "__main__":
    main()
