"""The decode-step operators at sizes of real use: plain forms, the library's calls, and what each has to move.

kv_append, decode_attention, kv_evict, logprobs and logprobs_backward of
block_scaled_fp4_03_amd, each beside its plain form: elementary torch
operations in FP32 (own = False) computing the same outputs from the same
inputs.  exact() computes them again from the definitions in FP64.
"""
import math

import torch

own = False

PAGE = 64          # tokens of a cache page, unless a case says otherwise


def listed():
    return [
        # One new token of each of 64 sequences into a BF16 cache: the write of every decode step.
        {"name": "append_decode_bf16", "op": "append", "rows": 64, "seqs": 64, "hkv": 8, "d": 128, "fmt": "bf16",
         "start": 97, "page": 64},
        # A batch of prompts (16384 tokens in 8 sequences) quantised into an MXFP8 cache.
        {"name": "append_prompt_mxfp8", "op": "append", "rows": 16384, "seqs": 8, "hkv": 8, "d": 128, "fmt": "mxfp8",
         "start": 5, "page": 64},
        # One sequence shortly after its prompt began: the smallest call, where latency counts.
        {"name": "attn_single_bf16", "op": "attn", "b": 1, "hq": 32, "hkv": 8, "d": 128, "len": 129, "ragged": False,
         "fmt": "bf16", "weights": False, "page": 64},
        # A serving batch of ragged lengths (one of them empty), with the weights accumulated for eviction.
        {"name": "attn_ragged_weights", "op": "attn", "b": 48, "hq": 64, "hkv": 8, "d": 64, "len": 4099,
         "ragged": True, "fmt": "bf16", "weights": True, "page": 32},
        # Few very long sequences: the length has to be split over the chip.
        {"name": "attn_long_mxfp8", "op": "attn", "b": 4, "hq": 64, "hkv": 8, "d": 128, "len": 131071,
         "ragged": False, "fmt": "mxfp8", "weights": False, "page": 64},
        # A large batch over a 4-bit cache: the most decoding work per byte.
        {"name": "attn_batch_mxfp4", "op": "attn", "b": 32, "hq": 32, "hkv": 8, "d": 128, "len": 16384,
         "ragged": True, "fmt": "mxfp4", "weights": False, "page": 64},
        # Two sequences a little over their budget: the periodic eviction while decoding.
        {"name": "evict_decode_bf16", "op": "evict", "b": 2, "hkv": 8, "d": 128, "len": 1100, "budget": 1024,
         "recent": 128, "fmt": "bf16", "page": 64},
        # Long prompts cut to an eighth right after they were read.
        {"name": "evict_prompt_mxfp8", "op": "evict", "b": 16, "hkv": 8, "d": 128, "len": 32768, "budget": 4096,
         "recent": 512, "fmt": "mxfp8", "page": 64},
        # What a serving step reports for one token: its log probability, the entropy and 20 alternatives.
        {"name": "logprobs_step_f32", "op": "logprobs", "n": 1, "v": 131072, "m": 1, "k": 20, "dtype": "f32"},
        # Scoring a batch of texts, a vocabulary of odd size (rows start at every alignment).
        {"name": "logprobs_score_bf16", "op": "logprobs", "n": 4096, "v": 100003, "m": 1, "k": 8, "dtype": "bf16"},
        # The gradient for a small step in FP32, several tokens a row.
        {"name": "logprobs_grad_f32", "op": "grad", "n": 256, "v": 32768, "m": 4, "dtype": "f32"},
        # The gradient of a training batch.
        {"name": "logprobs_grad_bf16", "op": "grad", "n": 4096, "v": 100003, "m": 1, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "evict", "logprobs", "grad"])
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    fmt, page = rng.choice(["bf16", "mxfp8", "mxfp4"]), rng.choice([16, 32, 64, 128])
    if op == "append":
        fmt = rng.choice(["bf16", "mxfp8"])
        seqs = _log_int(rng, 1, 64)
        return {"op": op, "rows": seqs * _log_int(rng, 1, max(1, 16384 * 1024 // (seqs * hkv * d * 2))), "seqs": seqs,
                "hkv": hkv, "d": d, "fmt": fmt, "start": _log_int(rng, 1, 200), "page": page}
    if op == "attn":
        b = _log_int(rng, 1, 64)
        # Cache values (K and V) up to half of the largest listed case's.
        most = min(131072, (1 << 28) // (b * hkv * d))
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        return {"op": op, "b": b, "hq": hkv * group, "hkv": hkv, "d": d, "len": _log_int(rng, 1, most),
                "ragged": rng.random() < 0.6, "fmt": fmt, "weights": rng.random() < 0.3, "page": page}
    if op == "evict":
        fmt = rng.choice(["bf16", "mxfp8"])
        b = _log_int(rng, 1, 16)
        length = _log_int(rng, 64, min(32768, (1 << 27) // (b * hkv * d)))
        budget = max(1, int(length * rng.uniform(0.05, 1.0)))
        return {"op": op, "b": b, "hkv": hkv, "d": d, "len": length, "budget": budget,
                "recent": int(budget * rng.uniform(0.0, 0.5)), "fmt": fmt, "page": page}
    v = _log_int(rng, 2000, 200000)
    n = _log_int(rng, 1, min(8192, (1 << 28) // v))
    dtype = rng.choice(["f32", "bf16"])
    if op == "logprobs":
        return {"op": op, "n": n, "v": v, "m": rng.choice([1, 1, 2, 5]), "k": rng.choice([0, 1, 5, 8, 20]),
                "dtype": dtype}
    return {"op": op, "n": n, "v": v, "m": rng.choice([1, 1, 2, 5]), "dtype": dtype}


# ---- inputs ------------------------------------------------------------------
def _lens(case):
    """Lengths of the batch: all `len`, or ragged from none to `len` (the longest first, an empty one last)."""
    b, most = case["b"], case["len"]
    if not case.get("ragged"):
        return [most] * b
    got = [1 + int((most - 1) * ((i * 0.6180339887 + 1.0) % 1.0)) for i in range(b)]
    got[0] = most
    if b > 2:
        got[-1] = 0
    return got


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _tables(g, b, width, first=0):
    """A page table with the pages of every sequence scattered over the pool."""
    return (first + torch.randperm(b * width, generator=g, device="cuda")).to(torch.int32).view(b, width)


def _pool(g, fmt, pages, hkv, page, d):
    """Cache rows as a serving process finds them: values of about unit size (codes and scales for the MX formats)."""
    if fmt == "bf16":
        return _randn(g, pages, hkv, page, d).to(torch.bfloat16), None
    codes = torch.randint(0, 256, (pages, hkv, page, d if fmt == "mxfp8" else d // 2), generator=g, device="cuda",
                          dtype=torch.int16).to(torch.uint8)
    if fmt == "mxfp8":
        # E4M3 bytes of exponent fields 9..14 (values to 240; no NaN pattern), the block scale 2^-7 or 2^-6.
        codes = (codes & 0x87) | ((9 + ((codes >> 3) & 15).to(torch.int16) * 6 // 16).to(torch.uint8) << 3)
        low = 120
    else:
        low = 125
    scales = torch.randint(low, low + 2, (pages, hkv, page, d // 32), generator=g, device="cuda",
                           dtype=torch.int16).to(torch.uint8)
    return codes, scales


def _handle(k, ks, v, vs):
    """The library's handle on the pools, which a serving process makes once (the plain form needs none)."""
    if not own:
        return None
    import block_scaled_fp4_03_amd as fp4
    return fp4.KVCache(k, v, ks, vs)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    if op == "append":
        n, seqs, page = case["rows"], case["seqs"], case["page"]
        each = -(-n // seqs)
        width = -(-(case["start"] + each) // page)
        s["k"], s["ks"] = _pool(g, case["fmt"], seqs * width, case["hkv"], page, case["d"])
        s["v"], s["vs"] = _pool(g, case["fmt"], seqs * width, case["hkv"], page, case["d"])
        s["table"] = _tables(g, seqs, width)
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        s["seq"], s["pos"] = torch.div(i, each, rounding_mode="floor").to(torch.int32), i % each + case["start"]
        # The new keys and values are columns of one fused projection's output, as they come from it.
        qkv = _randn(g, n, 3, case["hkv"], case["d"]).to(torch.bfloat16)
        s["new_k"], s["new_v"] = qkv[:, 1], qkv[:, 2]
        s["cache"] = _handle(s["k"], s["ks"], s["v"], s["vs"])
    elif op == "attn":
        b, page = case["b"], case["page"]
        lens = _lens(case)
        width = -(-max(lens) // page)
        s["k"], s["ks"] = _pool(g, case["fmt"], b * width, case["hkv"], page, case["d"])
        s["v"], s["vs"] = _pool(g, case["fmt"], b * width, case["hkv"], page, case["d"])
        s["table"] = _tables(g, b, width)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _randn(g, b, case["hq"], case["d"]).to(torch.bfloat16)
        s["win"] = s["wout"] = None
        if case["weights"]:
            s["win"] = torch.rand(b, case["hkv"], width * page, generator=g, device="cuda")
            s["wout"] = torch.zeros_like(s["win"])
        s["cache"] = _handle(s["k"], s["ks"], s["v"], s["vs"])
        if own:   # the workspace of the split, kept by the program from step to step
            import block_scaled_fp4_03_amd as fp4
            s["ws"] = fp4.attention_workspace(s["cache"], b, case["hq"], width * page, weights=case["weights"])
    elif op == "evict":
        b, page = case["b"], case["page"]
        width, width2 = -(-case["len"] // page), -(-min(case["len"], case["budget"]) // page)
        pages = b * (width + width2)
        s["k"], s["ks"] = _pool(g, case["fmt"], pages, case["hkv"], page, case["d"])
        s["v"], s["vs"] = _pool(g, case["fmt"], pages, case["hkv"], page, case["d"])
        s["table"], s["table2"] = _tables(g, b, width), _tables(g, b, width2, b * width)
        s["lens"] = torch.full((b,), case["len"], dtype=torch.int32, device="cuda")
        # Accumulated weights: a few tokens hold most of them.
        s["w"] = torch.exp(2.0 * _randn(g, b, case["hkv"], width * page))
        s["cache"] = _handle(s["k"], s["ks"], s["v"], s["vs"])
        if own:
            import block_scaled_fp4_03_amd as fp4
            s["ws"] = fp4.evict_workspace(s["cache"], b, width * page, case["budget"])
    else:
        n, v, m = case["n"], case["v"], case["m"]
        s["x"] = (3.0 * _randn(g, n, v)).to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        s["tokens"] = torch.randint(0, v, (n, m), generator=g, device="cuda", dtype=torch.int32)
        if op == "grad":
            s["g"], s["gh"] = _randn(g, n, m), 0.01 * _randn(g, n)
            y = s["x"].float()
            s["lse"] = torch.logsumexp(y, 1)
            p = torch.exp(y - s["lse"][:, None])
            s["ent"] = s["lse"] - (p * y).sum(1)
            del y, p
        elif own:
            import block_scaled_fp4_03_amd as fp4
            s["ws"] = fp4.logprobs_workspace(n, v, case["k"])
    return s


# ---- the operators -----------------------------------------------------------
def _values(codes, scales, fmt):
    """Cache rows as FP32 values."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "mxfp8":
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        grid = torch.cat([grid, -grid])
        byte = torch.arange(256, device=codes.device)
        x = torch.stack([grid[byte & 15], grid[byte >> 4]], 1)[codes.int()].flatten(-2)
    e = torch.exp2(scales.float() - 127.0)
    return (x.unflatten(-1, (-1, 32)) * e[..., None]).flatten(-2)


def _rows(pool, table):
    """Pool rows of every token of the table: [b, hkv, tokens, row]."""
    if pool is None:
        return None
    return pool[table.int()].permute(0, 2, 1, 3, 4).flatten(2, 3)


def _quantise(x, fmt):
    """MXFP8 codes and scales of rows of 32-value blocks: the smallest e with amax <= 448 * 2^e."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    blocks = x.float().unflatten(-1, (-1, 32))
    bits = blocks.abs().amax(-1).view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
    y = (blocks * torch.exp2(127.0 - byte.float())[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), byte.to(torch.uint8)


def _shown(t, fmt):
    """A pool as an output: 8-bit codes as E4M3 values."""
    return t.view(torch.float8_e4m3fn) if fmt == "mxfp8" else t


def _pools_out(s):
    c = s["case"]
    return {"k": _shown(s["k"], c["fmt"]), "v": _shown(s["v"], c["fmt"]), "ks": s["ks"], "vs": s["vs"]}


def _run_append(s):
    c = s["case"]
    if own:
        import block_scaled_fp4_03_amd as fp4
        fp4.kv_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["seq"], s["pos"])
        return _pools_out(s)
    page, slot = s["table"][s["seq"].long(), (s["pos"] // c["page"]).long()].long(), (s["pos"] % c["page"]).long()
    k, ks = _quantise(s["new_k"], c["fmt"])
    v, vs = _quantise(s["new_v"], c["fmt"])
    s["k"][page, :, slot], s["v"][page, :, slot] = k, v
    if ks is not None:
        s["ks"][page, :, slot], s["vs"][page, :, slot] = ks, vs
    return _pools_out(s)


def _run_attn(s):
    c = s["case"]
    if own:
        import block_scaled_fp4_03_amd as fp4
        out = fp4.decode_attention(s["q"], s["cache"], s["table"], s["lens"], weights=s["win"],
                                   weights_out=s["wout"], ws=s["ws"])
        return {"out": out, "weights": s["wout"]}
    b, hkv, d = c["b"], c["hkv"], c["d"]
    k = _values(_rows(s["k"], s["table"]), _rows(s["ks"], s["table"]), c["fmt"])
    valid = (torch.arange(k.shape[2], device=k.device)[None] < s["lens"][:, None])[:, None, None]
    score = torch.matmul(s["q"].float().view(b, hkv, -1, d), k.transpose(2, 3)) / math.sqrt(d)
    del k
    score = torch.where(valid, score, -math.inf)
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total == 0.0, 1.0, total)
    v = _values(_rows(s["v"], s["table"]), _rows(s["vs"], s["table"]), c["fmt"])
    out = torch.matmul(p, torch.where(valid.transpose(2, 3), v, 0.0)).view(b, c["hq"], d).to(torch.bfloat16)
    if not c["weights"]:
        return {"out": out, "weights": None}
    return {"out": out, "weights": torch.where(valid[:, 0], s["win"] + p.sum(2), 0.0)}


def _run_evict(s):
    c = s["case"]
    if own:
        import block_scaled_fp4_03_amd as fp4
        lens, w, kept = fp4.kv_evict(s["cache"], s["table"], s["lens"], s["w"], c["budget"], c["recent"], s["table2"],
                                     ws=s["ws"])
        return {**_pools_out(s), "lens": lens, "w": w, "kept": kept}
    b, page, length = c["b"], c["page"], c["len"]
    keep = min(length, c["budget"])
    index = torch.arange(length, device=s["w"].device)
    w = s["w"][:, :, :length]
    if keep < length:
        # Weights are not negative, so their bits order them; the lower index wins a tie.
        key = torch.where(index >= length - min(c["recent"], keep), 0x7FFFFFFF, w.view(torch.int32)).long()
        kept = torch.topk((key << 32) | (length - 1 - index), keep, 2).indices.sort(2).values
    else:
        kept = index.expand(b, c["hkv"], length)
    to = torch.arange(keep, device=kept.device)
    head = torch.arange(c["hkv"], device=kept.device)[None, :, None]
    seq = torch.arange(b, device=kept.device)[:, None, None]
    src = s["table"][seq, torch.div(kept, page, rounding_mode="floor")].long()
    dst = s["table2"][:, None, torch.div(to, page, rounding_mode="floor")].long().expand_as(src)
    slot = (to % page).expand_as(src)
    s["k"][dst, head, slot] = s["k"][src, head, kept % page]
    s["v"][dst, head, slot] = s["v"][src, head, kept % page]
    if s["ks"] is not None:
        s["ks"][dst, head, slot] = s["ks"][src, head, kept % page]
        s["vs"][dst, head, slot] = s["vs"][src, head, kept % page]
    cap = s["table2"].shape[1] * page
    out_w = torch.zeros(b, c["hkv"], cap, device=w.device)
    out_w[:, :, :keep] = torch.gather(w, 2, kept)
    out_kept = torch.full((b, c["hkv"], c["budget"]), -1, dtype=torch.int32, device=w.device)
    out_kept[:, :, :keep] = kept.to(torch.int32)
    return {**_pools_out(s), "lens": s["lens"].clamp(max=c["budget"]), "w": out_w, "kept": out_kept}


def _run_logprobs(s):
    c = s["case"]
    if own:
        import block_scaled_fp4_03_amd as fp4
        r = fp4.logprobs(s["x"], s["tokens"], top_k=c["k"], ws=s["ws"])
        return {"logp": r.logp, "entropy": r.entropy, "lse": r.lse, "top": r.top_logp, "index": r.top_index}
    y = s["x"].float()
    top = y.amax(1, keepdim=True)
    e = torch.exp(y - top)
    total = e.sum(1)
    lse = top[:, 0] + torch.log(total)
    entropy = torch.log(total) - (e * (y - top)).sum(1) / total
    logp = torch.gather(y, 1, s["tokens"].long()) - lse[:, None]
    if not c["k"]:
        return {"logp": logp, "entropy": entropy, "lse": lse, "top": None, "index": None}
    # An integer key of each value (-0 as +0), and the lower index wins a tie.
    bits = (y + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
    index = torch.topk(key | (c["v"] - 1 - torch.arange(c["v"], device=y.device)), c["k"], 1).indices
    return {"logp": logp, "entropy": entropy, "lse": lse, "top": torch.gather(y, 1, index) - lse[:, None],
            "index": index.to(torch.int32)}


def _run_grad(s):
    c = s["case"]
    if own:
        import block_scaled_fp4_03_amd as fp4
        return fp4.logprobs_backward(s["x"], s["tokens"], s["lse"], s["g"], s["ent"], s["gh"])
    logp = s["x"].float() - s["lse"][:, None]
    p = torch.exp(logp)
    d = -p * (s["g"].sum(1, keepdim=True) + s["gh"][:, None] * (logp + s["ent"][:, None]))
    d.scatter_add_(1, s["tokens"].long(), s["g"])
    return d.to(s["x"].dtype)


def run(state):
    return {"append": _run_append, "attn": _run_attn, "evict": _run_evict, "logprobs": _run_logprobs,
            "grad": _run_grad}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------
def _row_bytes(case):
    return {"bf16": 2 * case["d"], "mxfp8": case["d"] + case["d"] // 32,
            "mxfp4": case["d"] // 2 + case["d"] // 32}[case["fmt"]]


def work(case):
    op = case["op"]
    if op == "append":
        rows = 2 * case["rows"] * case["hkv"]
        return {"bytes": rows * (2 * case["d"] + _row_bytes(case)) + 8 * case["rows"], "flops": 2 * rows * case["d"]}
    if op == "attn":
        tokens, small = sum(_lens(case)), 4 * case["b"] * case["hq"] * case["d"]
        weights = 8 * tokens * case["hkv"] if case["weights"] else 0
        return {"bytes": 2 * tokens * case["hkv"] * _row_bytes(case) + small + weights + 4 * -(-tokens // case["page"]),
                "flops": 4 * tokens * case["hq"] * case["d"]}
    if op == "evict":
        keep, heads = min(case["len"], case["budget"]), case["b"] * case["hkv"]
        return {"bytes": heads * (4 * case["len"] + keep * (2 * 2 * _row_bytes(case) + 8)), "flops": heads * case["len"]}
    size, elem = case["n"] * case["v"], 4 if case["dtype"] == "f32" else 2
    if op == "logprobs":
        return {"bytes": size * elem + case["n"] * (8 * case["m"] + 8 * case["k"] + 8), "flops": 6 * size}
    return {"bytes": 2 * size * elem + case["n"] * (8 * case["m"] + 12), "flops": 6 * size}


# ---- the definitions in FP64 ---------------------------------------------------
def _exact_value(codes, scales, fmt):
    """FP64 values of cache rows, from the formats' definitions."""
    if fmt == "bf16":
        return codes.double()
    if fmt == "mxfp8":
        e, m = (codes >> 3).int() & 15, (codes & 7).double()
        mag = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
        x = torch.where(codes >= 128, -mag, mag)
    else:
        code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        e, m = (code.int() >> 1) & 3, (code & 1).double()
        mag = torch.where(e == 0, m * 0.5, (1.0 + m / 2.0) * torch.exp2((e - 1).double()))
        x = torch.where(code >= 8, -mag, mag)
    return x * torch.exp2(scales.double() - 127.0).repeat_interleave(32, -1)


def _exact_attn(s):
    c = s["case"]
    group, page = c["hq"] // c["hkv"], c["page"]
    out = torch.zeros(c["b"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    weights = torch.zeros(s["win"].shape, dtype=torch.float64, device="cuda") if c["weights"] else None
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(c["hkv"]):
            def rows(pool):
                return None if pool is None else pool[pages, h].reshape(len(pages) * page, -1)[:n]
            k = _exact_value(rows(s["k"]), rows(s["ks"]), c["fmt"])
            v = _exact_value(rows(s["v"]), rows(s["vs"]), c["fmt"])
            z = k @ s["q"][b, h * group:(h + 1) * group].double().T / c["d"] ** 0.5
            p = torch.softmax(z, 0)
            out[b, h * group:(h + 1) * group] = p.T @ v
            if weights is not None:
                weights[b, h, :n] = s["win"][b, h, :n].double() + p.sum(1)
    return {"out": out, "weights": weights}


def _exact_rows(s):
    """FP64 of logits rows, a few at a time."""
    c = s["case"]
    step = max(1, (1 << 25) // c["v"])
    for at in range(0, c["n"], step):
        yield slice(at, at + step), s["x"][at:at + step].double()


def _exact_logprobs(s):
    c, got = s["case"], []
    for at, y in _exact_rows(s):
        lp = torch.log_softmax(y, 1)
        row = [torch.gather(lp, 1, s["tokens"][at].long()), -(torch.exp(lp) * lp).sum(1), torch.logsumexp(y, 1)]
        if c["k"]:
            row.append(torch.topk(lp, c["k"], 1).values)
        got.append(row)
    got = [torch.cat(col) for col in zip(*got)]
    return {"logp": got[0], "entropy": got[1], "lse": got[2], "top": got[3] if c["k"] else None, "index": None}


def _exact_grad(s):
    got = []
    for at, y in _exact_rows(s):
        lp = torch.log_softmax(y, 1)
        p = torch.exp(lp)
        h = -(p * lp).sum(1, keepdim=True)
        g = s["g"][at].double()
        hot = torch.zeros_like(p).scatter_add_(1, s["tokens"][at].long(), g)
        # The output's precision is enough to keep of each element, and half the memory.
        got.append((hot - p * g.sum(1, keepdim=True) - s["gh"][at].double()[:, None] * p * (lp + h)))
    return torch.cat(got)


def _exact_append(s):
    c = s["case"]
    got = {"ks": None, "vs": None}
    seq, pos = s["seq"].tolist(), s["pos"].tolist()
    table = s["table"].tolist()
    page = torch.tensor([table[b][t // c["page"]] for b, t in zip(seq, pos)], device="cuda")
    slot = torch.tensor([t % c["page"] for t in pos], device="cuda")
    for name, scales, new in (("k", "ks", "new_k"), ("v", "vs", "new_v")):
        x = s[new].double()
        if c["fmt"] == "mxfp8":
            x = x.reshape(*x.shape[:-1], -1, 32)
            unit = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448.0)))
            y = x / unit
            step = torch.exp2(torch.floor(torch.log2(y.abs())).clamp(min=-6.0) - 3.0)
            x = (torch.round(y / step) * step).flatten(-2)
            # The pool's 8-bit elements stand for E4M3 values; their block scales are outputs of their own.
            pool = _exact_value(s[name], torch.full_like(s[scales], 127), "mxfp8")
        else:
            pool = s[name].double()
        pool[page, :, slot] = x
        got[name] = pool
    return got


def exact(case, seed):
    if case["op"] == "evict":
        # Copies: the outputs have no other value than the plain form's.
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "logprobs": _exact_logprobs,
            "grad": _exact_grad}[case["op"]](s)
