"""A speculative decode loop of a mixture-of-experts layer on the library's operators.

    python examples/moe_decode.py [--steps 16] [--drafts 3]

Every step takes the last token of each sequence and a few drafted ones through
NVFP4 projections, norms the queries and keys of each head and turns them to
their positions, appends keys and values to a paged cache, attends to it (a row
of the batch for each drafted token), routes the rows to their experts, runs
the MXFP4 experts on the rows in expert order and joins what they give, and
verifies the drafts against the head's logits.  What was drafted wrongly stays
in the cache behind the sequence's end and is overwritten by the next step.
Weights are random; the draft model is a table of the tokens' successors.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_03_amd as fp4  # noqa: E402


class Layer:
    """Attention with query and key norms, a mixture of experts, and an output head."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, experts, top_k, inner, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k, fmt=fp4.NVFP4):
            return fp4.quantize(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5, fmt)

        def expert_weights(n, k):
            q = [weight(n, k, fp4.MXFP4) for _ in range(experts)]
            return torch.stack([w.codes for w in q]), torch.stack([w.scales for w in q])

        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.vocab = hidden, q_heads, kv_heads, head_dim, vocab
        self.experts, self.top_k, self.inner = experts, top_k, inner
        self.embed = torch.randn(vocab, hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.q_norm = 1.0 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")
        self.k_norm = 1.0 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")
        pairs = head_dim // 2
        self.rope = fp4.Rope(torch.pow(10000.0, -torch.arange(pairs, device="cuda") / pairs).float())
        self.out = weight(hidden, q_heads * head_dim)
        self.router = weight(experts, hidden)
        self.up, self.down = expert_weights(inner, hidden), expert_weights(hidden, inner)
        self.head = weight(vocab, hidden)
        # The draft model: logits of the token after each.
        self.successor = torch.randn(vocab, vocab, generator=g, device="cuda").to(torch.bfloat16)

    def mixture(self, x):
        """The experts' outputs for rows x, weighted by the router."""
        logits = fp4.gemm(fp4.quantize(x, fp4.NVFP4), self.router, out_dtype=torch.float32)
        ids, w = fp4.moe_route(logits, self.top_k)
        off, rows, pos = fp4.moe_sort(ids, self.experts)
        up = fp4.gemm_grouped(fp4.quantize(x, fp4.MXFP4), rows, off, *self.up, self.inner, self.hidden, fp4.MXFP4)
        h = torch.relu_(up)
        own = torch.arange(h.shape[0], dtype=torch.int32, device="cuda")  # (rows are in expert order already)
        y = fp4.gemm_grouped(fp4.quantize(h, fp4.MXFP4), own, off, *self.down, self.hidden, self.inner, fp4.MXFP4)
        return fp4.moe_combine(y, pos, w)

    def forward(self, tokens, seq, pos, cache, table):
        """Logits of rows of tokens: row i is token pos[i] of sequence seq[i]."""
        x = self.embed[tokens]
        heads = self.q_heads + 2 * self.kv_heads
        y = fp4.gemm(fp4.quantize(x, fp4.NVFP4), self.qkv, out_dtype=torch.bfloat16).view(-1, heads, self.head_dim)
        q, k, v = y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        q, k = fp4.qk_norm_rope(q, k, self.rope, pos, self.q_norm, self.k_norm, q_out=q, k_out=k)
        fp4.kv_append(cache, k, v, table, seq, pos)
        rows = q.contiguous()
        a = fp4.decode_attention(rows, cache, table[seq.long()], pos + 1)
        x = x + fp4.gemm(fp4.quantize(a.view(len(a), -1), fp4.NVFP4), self.out, out_dtype=torch.bfloat16)
        x = x + self.mixture(x)
        return fp4.gemm(fp4.quantize(x, fp4.NVFP4), self.head, out_dtype=torch.float32)


def run(steps=16, batch=4, drafts=3, prompt=40, hidden=512, q_heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2,
        inner=256, vocab=1024, page_size=16, seed=0):
    layer = Layer(hidden, q_heads, kv_heads, head_dim, experts, top_k, inner, vocab, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-(prompt + steps * (drafts + 1) + drafts + 1) // page_size)
    cache = fp4.KVCache.empty(batch * width, page_size, kv_heads, head_dim, fp4.KV_MXFP8)
    table = torch.randperm(batch * width, generator=g, device="cuda").to(torch.int32).view(batch, width)
    # Requests at temperatures of their own, the first one greedy.
    temperature = torch.arange(batch, device="cuda") * 0.4

    # The prompts; the last token of each is the first to be decoded.
    tokens = torch.randint(0, vocab, (batch, prompt), generator=g, device="cuda")
    seq = torch.arange(batch, dtype=torch.int32, device="cuda")
    at = torch.arange(prompt - 1, dtype=torch.int32, device="cuda")
    layer.forward(tokens[:, :-1].reshape(-1), seq.repeat_interleave(prompt - 1), at.repeat(batch), cache, table)
    last = tokens[:, -1]
    lens = torch.full((batch,), prompt - 1, dtype=torch.int32, device="cuda")   # tokens in the cache

    step_seq = seq.repeat_interleave(drafts + 1)
    ahead = torch.arange(drafts + 1, dtype=torch.int32, device="cuda")
    ws, history = fp4.verify_workspace(batch, drafts, vocab), []
    for _ in range(steps):
        # Drafts drawn one after the other from the draft model, at each request's temperature.
        drafted, draft_logits, token = [], [], last
        for _ in range(drafts):
            y = layer.successor[token]
            noise = torch.empty(batch, vocab, device="cuda").exponential_(generator=g)
            token = (y.float() - temperature[:, None] * torch.log(noise)).argmax(1)
            draft_logits.append(y.float())
            drafted.append(token.to(torch.int32))
        rows = torch.stack([last.to(torch.int32)] + drafted, 1)
        pos = (lens[:, None] + ahead).reshape(-1)
        logits = layer.forward(rows.long().reshape(-1), step_seq, pos, cache, table).view(batch, drafts + 1, vocab)
        u = torch.rand(batch, drafts + 1, generator=g, device="cuda")
        # (Without drafts a step draws one token from the target's distribution.)
        drafted, draft_logits = rows[:, 1:].contiguous(), torch.stack(draft_logits, 1) if drafts else None
        if drafts:   # (the two models are unrelated: some of the draft's logits make some of its tokens welcome)
            logits[:, :drafts] += 1.5 * draft_logits
        out, kept, chance = fp4.verify_drafts(logits, draft_logits, drafted, u, temperature, ws=ws)
        last = out.gather(1, kept.long()[:, None])[:, 0].long()
        lens = lens + kept + 1
        history.append({"out": out, "kept": kept, "chance": chance, "target": logits, "draft": draft_logits,
                        "tokens": drafted, "u": u, "temperature": temperature, "lens": lens})
    return history


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--drafts", type=int, default=3)
    a = p.parse_args()
    for i, h in enumerate(run(steps=a.steps, drafts=a.drafts)):
        print("step %d  kept %s  emitted %s  lens %s" % (i, h["kept"].tolist(), h["out"].tolist(), h["lens"].tolist()))


if __name__ == "__main__":
    main()
