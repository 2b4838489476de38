"""Measured cases of the operators around the decode step: attention over whole prompts, the append to a
cache held in 4 bits and the attention that reads it, and the log probabilities of given tokens.

A case is a dict of plain values; prepare() makes its inputs from a seed, run() makes one pass: in
the operators' plain form (elementary torch operations), or through the package when `own` is set."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
DEV = "cuda"
BLOCK = 32  # elements of a head that share a power of two in the 4-bit cache
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases


def _prompt(name, seqs, lo, hi, q_heads, kv_heads, head_dim, dtype, lse):
    return {"name": name, "op": "prompt", "seqs": seqs, "lo": lo, "hi": hi, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "lse": lse}


def _append(name, tokens, q_heads, kv_heads, head_dim, rot_dim, pairs, src, dst, gains, far, page):
    return {"name": name, "op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "pairs": pairs, "src": src, "dst": dst, "gains": gains, "far": far,
            "page": page}


def _attn(name, seqs, q_lo, q_hi, q_heads, kv_heads, head_dim, dtype, page, lo, hi):
    return {"name": name, "op": "attention", "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype, "page": page, "lo": lo, "hi": hi}


def _logprobs(name, tokens, vocab, dtype, top, scale):
    return {"name": name, "op": "logprobs", "tokens": tokens, "vocab": vocab, "dtype": dtype, "top": top, "scale": scale}


def listed():
    return [
        # a few short questions: the smallest prompt call
        _prompt("prompt-short", 4, 3, 60, 20, 5, 128, "bf16", False),
        # a batch of requests of all lengths, packed, heads of an odd size
        _prompt("prompt-ragged", 24, 1, 1500, 12, 4, 80, "f16", True),
        # one ordinary prompt
        _prompt("prompt-one", 1, 2048, 2048, 20, 5, 128, "bf16", False),
        # a long document
        _prompt("prompt-long", 1, 16384, 16384, 32, 8, 128, "bf16", False),
        # a decode step of 64 sequences: queries out, keys and values into their pages
        _append("append4-step", 64, 20, 5, 128, 128, "halves", "f32", "bf16", True, 8192, 16),
        # a prompt's tokens into the cache, its queries, and what its own attention reads
        _append("append4-prompt", 8192, 32, 8, 128, 128, "halves", "bf16", "bf16", True, 65536, 64),
        # one sequence of some hundred tokens
        _attn("attn4-one-sequence", 1, 1, 1, 20, 5, 128, "bf16", 16, 700, 700),
        # drafted tokens of a batch, ragged everywhere, small heads
        _attn("attn4-drafts", 24, 1, 5, 32, 8, 64, "f16", 32, 5, 4000),
        # few sequences with long histories: one stream over the cache
        _attn("attn4-long", 8, 1, 1, 32, 8, 128, "bf16", 64, 50000, 65536),
        # one answer token, alternatives shown
        _logprobs("logprobs-one", 1, 128256, "f32", 5, 1.0),
        # a decode step of 64 sequences, sampled at a temperature
        _logprobs("logprobs-batch", 64, 128256, "f32", 20, 1.25),
        # the scores of a prompt's own tokens
        _logprobs("logprobs-prompt", 2048, 128256, "bf16", 1, 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append", "attention", "attention", "logprobs"))
    kv_heads = rng.randint(1, 8)
    group = rng.randint(1, 8)
    page = rng.choice((16, 32, 64, 128))
    if op == "prompt":
        head_dim = rng.choice((64, 72, 80, 96, 128, 128, 256))
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 16384 // seqs))
        lo = rng.randint(1, hi)
        # no more multiply-adds than the largest listed case
        while seqs * hi * hi * group * kv_heads * head_dim > 16384 * 16384 * 32 * 128:
            lo, hi = max(1, lo // 2), max(1, hi // 2)
        case = _prompt("", seqs, lo, hi, group * kv_heads, kv_heads, head_dim, rng.choice(("bf16", "bf16", "f16")),
                       rng.random() < 0.4)
    elif op == "append":
        head_dim = rng.choice((32, 64, 96, 128, 128, 256))
        most = 8192 * 48 * 128 // ((2 + group) * kv_heads * head_dim)
        rot_dim = 2 * rng.randint(1, head_dim // 2) if rng.random() < 0.3 else head_dim
        tokens = _log_int(rng, 1, min(most, 8192))
        src, dst = rng.choice((("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f16")))
        case = _append("", tokens, group * kv_heads if rng.random() < 0.6 else 0, kv_heads, head_dim, rot_dim,
                       rng.choice(("halves", "adjacent")), src, dst, rng.random() < 0.6,
                       _log_int(rng, tokens + 1, 65536 + tokens), page)
    elif op == "attention":
        head_dim = rng.choice((32, 64, 64, 96, 128, 128, 160, 256))
        seqs = _log_int(rng, 1, 64)
        q_hi = rng.choice((1, 1, 1, rng.randint(2, 8)))
        hi = _log_int(rng, q_hi, max(q_hi, min(65536, 8 * 57344 * 8 * 128 // (seqs * kv_heads * head_dim))))
        case = _attn("", seqs, rng.randint(1, q_hi), q_hi, group * kv_heads, kv_heads, head_dim,
                     rng.choice(("bf16", "f16")), page, rng.randint(q_hi, hi), hi)
    else:
        vocab, dtype = _log_int(rng, 1000, 128256), rng.choice(("f32", "f32", "bf16", "f16"))
        tokens = _log_int(rng, 1, min(4096, 2048 * 128256 * 2 // (vocab * SIZE[dtype])))
        case = _logprobs("", tokens, vocab, dtype, rng.choice((0, 1, 5, 20, rng.randint(1, 32))),
                         rng.choice((1.0, 1.0, 1.25, 0.7)))
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n whole numbers of [lo, hi], scattered, the same for every seed (the work depends on them)."""
    return [lo + (i * 2654435761 + 40503) % 1000003 % (hi - lo + 1) for i in range(n)]


def _starts(counts):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    return starts


# ------------------------------------------------------------------------------ the 4-bit format


def _powers(dtype):
    return torch.tensor([2.0 ** (i - 127) for i in range(1, 254)], dtype=dtype, device=DEV)


def _to_codes(x):
    """x [..., head_dim] of float32 or float64 -> the bytes of its elements, low half first, and those of its blocks'
    powers of two (2^(byte - 127)): the smallest that leaves no element above 7 of it, 2^-125 at least."""
    b = x.unflatten(-1, (-1, BLOCK))
    mant, exponent = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(mant == 0, -125, (exponent - 3 + (mant > 0.875)).clamp(-125, 125))
    a = b.abs() * _powers(x.dtype)[126 - e]
    code = sum(c.to(torch.uint8) for c in (a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0))
    code = (code + 8 * (b < 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e[..., 0] + 127).to(torch.uint8)


def _from_codes(codes, scales, dtype):
    """The values that bytes of codes and scales stand for."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=DEV)
    x = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * _powers(dtype)[scales.int() - 1][..., None]).flatten(-2)


# ------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"prompt": _prepare_prompt, "append": _prepare_append, "attention": _prepare_attn,
            "logprobs": _prepare_logprobs}[case["op"]](case, gen)


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


def _prepare_prompt(case, gen):
    Hq, Hk, D, dtype = case["q_heads"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    starts = _starts(_spread(case["seqs"], case["lo"], case["hi"]))
    T = starts[-1]
    # queries and keys as the norm leaves them, values still inside the rows of a fused projection
    rows = _randn(gen, T, 3 * Hk * D, dtype=dtype)
    s = {"case": case, "q": _randn(gen, T, Hq, D, dtype=dtype, scale=1.5), "k": _randn(gen, T, Hk, D, dtype=dtype),
         "v": rows.view(T, 3 * Hk, D)[:, 2 * Hk:], "out": torch.empty(T, Hq, D, dtype=dtype, device=DEV),
         "lse": torch.empty(T, Hq, device=DEV) if case["lse"] else None,
         "starts": torch.tensor(starts, dtype=torch.int32, device=DEV)}
    if own:
        import bit_plane_weight_amd as bpw
        s["plan"] = bpw.PromptAttnPlan(s["q"], s["k"], s["v"], s["out"], s["starts"], lse=s["lse"])
    return s


def _prepare_append(case, gen):
    T, Hq, Hk, D, R, P = (case[x] for x in ("tokens", "q_heads", "kv_heads", "head_dim", "rot_dim", "page"))
    src, dst = DTYPES[case["src"]], DTYPES[case["dst"]]
    heads = _randn(gen, T, (Hq + 2 * Hk) * D, dtype=src, scale=1.5).view(T, Hq + 2 * Hk, D)
    first = int(torch.randint(0, case["far"] - T + 1, (1,), generator=gen, device=DEV))
    pages = T // P + 8
    order = torch.randperm(pages, generator=gen, device=DEV)
    start = int(torch.randint(0, 7 * P, (1,), generator=gen, device=DEV))
    if T <= 256:  # a decode step: one token each, scattered over the pages
        slots = torch.randperm(pages * P, generator=gen, device=DEV)[:T].contiguous()
    else:  # one sequence: consecutive offsets over its pages
        at = torch.arange(start, start + T, device=DEV)
        slots = order[at // P] * P + at % P
    s = {"case": case, "q": heads[:, :Hq] if Hq else None, "k": heads[:, Hq:Hq + Hk], "v": heads[:, Hq + Hk:],
         "slots": slots, "positions": torch.arange(first, first + T, dtype=torch.int32, device=DEV),
         "inv_freq": 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R),
         "q_gain": 1 + _randn(gen, D, scale=0.1) if case["gains"] and Hq else None,
         "k_gain": 1 + _randn(gen, D, scale=0.1) if case["gains"] else None,
         "q_out": torch.empty(T, Hq, D, dtype=dst, device=DEV) if Hq else None}
    for x in "kv":
        s[x + "_codes"] = torch.zeros(pages, Hk, P, D // 2, dtype=torch.uint8, device=DEV)
        s[x + "_scales"] = torch.full((pages, Hk, P, D // BLOCK), 127, dtype=torch.uint8, device=DEV)
        s[x + "_values"] = torch.empty(T, Hk, D, dtype=dst, device=DEV)
    if own:
        import bit_plane_weight_amd as bpw
        kv = bpw.PagedKv4(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["plan"] = bpw.Kv4AppendPlan(kv, s["k"], s["v"], slots, positions=s["positions"], inv_freq=s["inv_freq"],
                                      k_gain=s["k_gain"], q=s["q"], q_out=s["q_out"], q_gain=s["q_gain"], eps=EPS,
                                      interleaved=case["pairs"] == "adjacent", k_values=s["k_values"],
                                      v_values=s["v_values"])
    return s


def _attn_lengths(case):
    n_q = _spread(case["seqs"], case["q_lo"], case["q_hi"])
    lens = [max(a, n) for a, n in zip(_spread(case["seqs"], case["lo"], case["hi"]), n_q)]
    return n_q, lens


def _prepare_attn(case, gen):
    B, Hq, Hk, D, P = (case[x] for x in ("seqs", "q_heads", "kv_heads", "head_dim", "page"))
    dtype = DTYPES[case["dtype"]]
    n_q, lens = _attn_lengths(case)
    T = sum(n_q)
    per_seq = [-(-n // P) for n in lens]
    pages = sum(per_seq) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    # each sequence's row of the table: its own pages, then pages that are not read
    at = torch.tensor(per_seq, device=DEV)
    first = torch.cumsum(at, 0) - at
    col = torch.arange(max(per_seq), device=DEV)
    table = order[torch.where(col[None] < at[:, None], first[:, None] + col[None], 0)].contiguous()
    s = {"case": case, "max_q": max(n_q), "q": _randn(gen, T, Hq, D, dtype=dtype, scale=1.5),
         "out": torch.empty(T, Hq, D, dtype=dtype, device=DEV), "lse": torch.empty(T, Hq, device=DEV), "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "q_starts": torch.tensor(_starts(n_q), dtype=torch.int32, device=DEV)}
    for x in "kv":
        s[x + "_codes"] = torch.empty(pages, Hk, P, D // 2, dtype=torch.uint8, device=DEV)
        s[x + "_scales"] = torch.empty(pages, Hk, P, D // BLOCK, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 25) // (Hk * P * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            s[x + "_codes"][p:p + n], s[x + "_scales"][p:p + n] = _to_codes(_randn(gen, n, Hk, P, D))
    if own:
        import bit_plane_weight_amd as bpw
        kv = bpw.PagedKv4(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        ws = torch.empty(bpw.bpw_kv4_attn_workspace_bytes(kv, s["q"], B, s["max_q"], table.shape[1]), dtype=torch.uint8,
                         device=DEV)
        s["plan"] = bpw.Kv4AttnPlan(kv, s["q"], s["out"], table, s["lens"], s["q_starts"], s["max_q"], ws, lse=s["lse"])
    return s


def _prepare_logprobs(case, gen):
    T, V, K, dtype = case["tokens"], case["vocab"], case["top"], DTYPES[case["dtype"]]
    logits = torch.empty(T, V, dtype=dtype, device=DEV)
    for t in range(0, T, 256):
        logits[t:t + 256] = _randn(gen, min(256, T - t), V, scale=2.5)
    # a few likely tokens a row, the given one often among them
    likely = torch.randint(0, V, (T, 4), generator=gen, device=DEV)
    logits.scatter_add_(1, likely, (8 + 4 * torch.rand(T, 4, generator=gen, device=DEV)).to(dtype))
    other = torch.randint(0, V, (T,), generator=gen, device=DEV)
    tokens = torch.where(torch.rand(T, generator=gen, device=DEV) < 0.7, likely[:, 0], other).to(torch.int32)
    s = {"case": case, "logits": logits, "tokens": tokens, "logprobs": torch.empty(T, device=DEV),
         "entropy": torch.empty(T, device=DEV),
         "top_tokens": torch.empty(T, K, dtype=torch.int32, device=DEV) if K else None,
         "top_logprobs": torch.empty(T, K, device=DEV) if K else None}
    if own:
        import bit_plane_weight_amd as bpw
        ws = torch.empty(bpw.bpw_token_logprobs_workspace_bytes(T, V, K), dtype=torch.uint8, device=DEV)
        s["plan"] = bpw.TokenLogprobsPlan(logits, tokens, s["logprobs"], ws, entropy=s["entropy"],
                                          top_tokens=s["top_tokens"], top_logprobs=s["top_logprobs"], scale=case["scale"])
    return s


# ------------------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        s["plan"].run()
    else:
        {"prompt": _plain_prompt, "append": _plain_append, "attention": _plain_attn, "logprobs": _plain_logprobs}[op](s)
    names = {"prompt": ("out", "lse"), "append": ("k_values", "v_values", "q_out"), "attention": ("out", "lse"),
             "logprobs": ("logprobs", "entropy", "top_tokens", "top_logprobs")}[op]
    return {n: s[n] for n in names if s[n] is not None}


def _plain_prompt(s):
    c = s["case"]
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    starts = _starts(_spread(c["seqs"], c["lo"], c["hi"]))
    for a, b in zip(starts, starts[1:]):
        n = b - a
        later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        for h in range(Hk):
            group = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            q = s["q"][a:b, group].float().transpose(0, 1)
            k, v = s["k"][a:b, h].float(), s["v"][a:b, h].float()
            score = torch.matmul(q, k.t()).mul_(1.0 / math.sqrt(D)).masked_fill_(later, -math.inf)
            top = score.amax(-1, keepdim=True)
            w = score.sub_(top).exp_()
            total = w.sum(-1, keepdim=True)
            s["out"][a:b, group] = (torch.matmul(w, v) / total).transpose(0, 1).to(s["out"].dtype)
            if s["lse"] is not None:
                s["lse"][a:b, group] = (top + torch.log(total))[..., 0].t()


def _plain_norm_rotate(x, gain, s):
    """In 64 bits: a key's element may lie next to the border of two codes."""
    x = x.double()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.double()
    angle = (s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    cos, sin, R = angle.cos(), angle.sin(), 2 * s["inv_freq"].numel()
    if s["case"]["pairs"] == "adjacent":
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_append(s):
    P = s["case"]["page"]
    page, at = s["slots"] // P, s["slots"] % P
    for x, rows in (("k", _plain_norm_rotate(s["k"], s["k_gain"], s)), ("v", s["v"].float())):
        codes, scales = _to_codes(rows)
        s[x + "_codes"][page, :, at], s[x + "_scales"][page, :, at] = codes, scales
        s[x + "_values"].copy_(_from_codes(codes, scales, torch.float32))
    if s["q"] is not None:
        s["q_out"].copy_(_plain_norm_rotate(s["q"], s["q_gain"], s))


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hk, D, M = c["seqs"], c["q_heads"], c["kv_heads"], c["head_dim"], s["max_q"]
    G, T, starts = Hq // Hk, s["q"].shape[0], s["q_starts"].long()
    # tokens as rows [sequence, j], the rows past a sequence's own repeated from others and not used
    j = torch.arange(M, device=DEV)
    row = (starts[:-1, None] + j[None]).clamp(max=T - 1)
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(starts, token, right=True) - 1
    place = seq * M + token - starts[seq]
    q = s["q"].float().view(T, Hk, G, D)[row].permute(0, 2, 1, 3, 4).reshape(B, Hk, M * G, D)
    L = s["table"].shape[1] * c["page"]
    keys, values = (_from_codes(*(s[f"{x}_{y}"][s["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, -1)
                                  for y in ("codes", "scales")), torch.float32) for x in "kv")
    # token j of n sees the first len - (n - 1 - j)
    n_q = starts[1:] - starts[:-1]
    sees = s["lens"].long()[:, None] - (n_q[:, None] - 1 - j[None])
    hidden = torch.arange(L, device=DEV) >= sees[..., None]  # [B, M, L]
    score = torch.matmul(q, keys.transpose(-1, -2)).view(B, Hk, M, G, L) / math.sqrt(D)
    score = score.masked_fill(hidden[:, None, :, None], -math.inf).view(B, Hk, M * G, L)
    top = score.amax(-1)
    base = torch.where(torch.isinf(top), 0.0, top)
    w = torch.exp(score - base[..., None])
    total = w.sum(-1)
    out = torch.matmul(w, values) / total[..., None]
    lse = base + torch.log(total)
    out = out.view(B, Hk, M, G, D).transpose(1, 2).reshape(B * M, Hq, D)
    lse = lse.view(B, Hk, M, G).transpose(1, 2).reshape(B * M, Hq)
    s["out"].copy_(out[place])
    s["lse"].copy_(lse[place])


def _plain_logprobs(s):
    K, V, rows = s["case"]["top"], s["case"]["vocab"], 256
    order = torch.arange(V - 1, -1, -1, device=DEV)
    for t in range(0, s["case"]["tokens"], rows):
        x = s["logits"][t:t + rows].float()
        y = x * s["case"]["scale"]
        y = y - y.amax(-1, keepdim=True)
        e = torch.exp(y)
        total = e.sum(-1)
        lse = torch.log(total)
        s["logprobs"][t:t + rows] = y.gather(-1, s["tokens"][t:t + rows, None].long())[:, 0] - lse
        s["entropy"][t:t + rows] = lse - (e * y).sum(-1) / total
        if K:  # ties go to the lowest index: whole numbers that rise with the logit, then fall with the index
            bits = (x + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * V + order
            at = key.topk(K, -1).indices
            s["top_tokens"][t:t + rows] = at.int()
            s["top_logprobs"][t:t + rows] = y.gather(-1, at) - lse[:, None]


# ------------------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "append": _exact_append, "attention": _exact_attn,
            "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_prompt(case, s):
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    bounds = s["starts"].tolist()
    for a, b in zip(bounds, bounds[1:]):
        for hq in range(Hq):
            h = hq // (Hq // Hk)
            k, v = s["k"][a:b, h].to(torch.float64), s["v"][a:b, h].to(torch.float64)
            for i in range(a, b, 4096):  # some rows at a time, against the positions up to the last of them
                e = min(b, i + 4096)
                score = s["q"][i:e, hq].to(torch.float64) @ k[:e - a].T / math.sqrt(D)
                at = torch.arange(e - a, device=DEV)
                score[at[None] > torch.arange(i - a, e - a, device=DEV)[:, None]] = -math.inf
                lse[i:e, hq] = torch.logsumexp(score, -1)
                out[i:e, hq] = torch.softmax(score, -1) @ v[:e - a]
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_heads(case, x, gain, s):
    x = x.to(torch.float64)
    if gain is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.to(torch.float64)
    R = case["rot_dim"]
    inv = s["inv_freq"]
    turn = torch.polar(torch.ones_like(inv)[None], s["positions"].to(torch.float64)[:, None] * inv[None])[:, None]
    y = x.clone()
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["pairs"] == "adjacent" else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_nearest(x):
    """The value of the 4-bit format nearest to each element, of two as near the one with the even code."""
    b = x.unflatten(-1, (-1, BLOCK))
    most = b.abs().amax(-1, keepdim=True)
    unit = torch.full_like(most, 2.0 ** -125)
    for e in range(-124, 126):
        unit = torch.where(most > 7 * unit, unit * 2, unit)
    near, best = torch.zeros_like(b), torch.full_like(b, math.inf)
    for value in E2M1[0::2] + E2M1[1::2]:  # even codes first
        off = (b.abs() - value * unit).abs()
        near = torch.where(off < best, value * unit, near)
        best = torch.minimum(off, best)
    return torch.where(b < 0, -near, near).flatten(-2)


def _exact_append(case, s):
    got = {"k_values": _exact_nearest(_exact_heads(case, s["k"], s["k_gain"], s)),
           "v_values": _exact_nearest(s["v"].to(torch.float64))}
    if s["q"] is not None:
        got["q_out"] = _exact_heads(case, s["q"], s["q_gain"], s)
    return got


def _exact_rows(s, x, b, n):
    """Positions 0 .. n-1 of sequence b of the cache's keys or values [kv_heads, n, head_dim]."""
    ids = s["table"][b].long()
    codes, scales = (s[f"{x}_{y}"][ids].transpose(0, 1).flatten(1, 2)[:, :n].to(torch.int64) for y in ("codes", "scales"))
    half = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
    size, exponent = half % 2, half % 8 // 2  # E2M1: a bit of mantissa, two of exponent, the sign
    value = torch.where(exponent == 0, size * 0.5, (1 + size * 0.5) * 2.0 ** (exponent - 1).double())
    value = torch.where(half >= 8, -value, value)
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), scales.double() - 127)
    return value * unit.repeat_interleave(BLOCK, -1)


def _exact_attn(case, s):
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    n_q, lens = _attn_lengths(case)
    out, lse, t = [], [], 0
    for b, (n, length) in enumerate(zip(n_q, lens)):
        k, v = (_exact_rows(s, x, b, length) for x in "kv")
        q = s["q"][t:t + n].to(torch.float64).view(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)  # [Hk, G, n, D]
        score = (q.reshape(Hk, -1, D) @ k.transpose(1, 2) / math.sqrt(D)).view(Hk, Hq // Hk, n, -1)
        score[..., torch.arange(length, device=DEV)[None] > length - n + torch.arange(n, device=DEV)[:, None]] = -math.inf
        lse.append(torch.logsumexp(score, -1).permute(2, 0, 1).reshape(n, Hq))
        w = torch.softmax(score, -1).view(Hk, -1, length)
        out.append((w @ v).view(Hk, Hq // Hk, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D))
        t += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_logprobs(case, s):
    K, parts = case["top"], {"logprobs": [], "entropy": [], "top_tokens": [], "top_logprobs": []}
    for t in range(0, case["tokens"], 128):
        x = s["logits"][t:t + 128].to(torch.float64)
        logp = torch.log_softmax(x * case["scale"], -1)
        parts["logprobs"].append(logp.gather(-1, s["tokens"][t:t + 128, None].long())[:, 0])
        parts["entropy"].append(-(logp.exp() * logp).sum(-1))
        if K:
            at = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :K]
            parts["top_tokens"].append(at.int())
            parts["top_logprobs"].append(logp.gather(-1, at))
    return {n: torch.cat(x) for n, x in parts.items() if x}


# ------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "prompt":
        counts = _spread(case["seqs"], case["lo"], case["hi"])
        Hq, Hk, D, T = case["q_heads"], case["kv_heads"], case["head_dim"], sum(counts)
        return {"bytes": 2 * T * (Hq + Hk) * D * SIZE[case["dtype"]] + (T * Hq * 4 if case["lse"] else 0),
                "flops": 4 * Hq * D * sum(n * (n + 1) // 2 for n in counts)}
    if case["op"] == "append":
        T, Hq, Hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        moved = T * (Hq + 2 * Hk) * D * (SIZE[case["src"]] + SIZE[case["dst"]])
        return {"bytes": moved + T * 2 * Hk * (D // 2 + D // BLOCK) + T * 12, "flops": 8 * T * (Hq + 2 * Hk) * D}
    if case["op"] == "attention":
        n_q, lens = _attn_lengths(case)
        Hq, Hk, D, T = case["q_heads"], case["kv_heads"], case["head_dim"], sum(n_q)
        seen = sum(n * length - n * (n - 1) // 2 for n, length in zip(n_q, lens))
        return {"bytes": 2 * T * Hq * D * SIZE[case["dtype"]] + T * Hq * 4 + 2 * sum(lens) * Hk * (D // 2 + D // BLOCK),
                "flops": 4 * seen * Hq * D}
    n = case["tokens"] * case["vocab"]
    return {"bytes": n * SIZE[case["dtype"]] + case["tokens"] * (12 + 8 * case["top"]), "flops": 5 * n}
