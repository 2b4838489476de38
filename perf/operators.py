"""Measured cases of the decode-step operators: the norm and rotation of query and key heads, the
append to a paged cache, attention over a shared prefix and per-sequence suffixes, and the
verification of drafted tokens.

A case is a dict of plain values; prepare() makes its inputs from a seed, run() makes one pass: in
the operators' plain form (elementary torch operations), or through the package when `own` is set."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------ cases


def _rope(name, tokens, q_heads, kv_heads, head_dim, rot_dim, pairs, src, dst, gains, far):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "pairs": pairs, "src": src, "dst": dst, "gains": gains, "far": far}


def _append(name, tokens, q_heads, kv_heads, head_dim, rot_dim, pairs, src, dst, gains, far, page):
    return {**_rope(name, tokens, q_heads, kv_heads, head_dim, rot_dim, pairs, src, dst, gains, far), "op": "kv_append",
            "page": page}


def _attn(name, seqs, q_lo, q_hi, q_heads, kv_heads, head_dim, dtype, page, prefix, lo, hi):
    return {"name": name, "op": "attention", "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype, "page": page, "prefix": prefix, "lo": lo, "hi": hi}


def _verify(name, seqs, drafts, ragged, vocab, with_draft, dtype):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "ragged": ragged, "vocab": vocab,
            "with_draft": with_draft, "dtype": dtype}


def listed():
    return [
        # one token's query and key heads as the float32 GEMV leaves them, rounded for the attention
        _rope("rope-one-token", 1, 20, 5, 128, 128, "halves", "f32", "bf16", True, 4096),
        # a ragged batch of a model with small heads, a part of each rotated, adjacent pairs
        _rope("rope-part-of-head", 777, 12, 4, 80, 32, "adjacent", "f16", "f16", True, 8192),
        # the heads of a long prompt, positions far out
        _rope("rope-prompt", 16384, 32, 8, 128, 128, "halves", "bf16", "bf16", True, 131072),
        # a decode step of 64 sequences: queries out, keys and values into their pages
        _append("append-step", 64, 20, 5, 128, 128, "halves", "f32", "bf16", True, 8192, 16),
        # a chunk of a prompt into the cache, no queries and no norms
        _append("append-prompt", 8192, 0, 8, 128, 128, "halves", "bf16", "bf16", False, 65536, 64),
        # one sequence of some hundred tokens, nothing shared: the smallest attention call
        _attn("attn-one-sequence", 1, 1, 1, 20, 5, 128, "bf16", 16, 0, 700, 700),
        # a decode step of 16 sequences under one system prompt
        _attn("attn-step", 16, 1, 1, 20, 5, 128, "bf16", 16, 2048, 1, 512),
        # drafted tokens of 8 sequences, the prefix ending inside a page, ragged everywhere
        _attn("attn-drafts", 8, 1, 5, 32, 8, 64, "f16", 32, 1000, 5, 1500),
        # few sequences with long histories of their own: one stream over the cache
        _attn("attn-long-suffix", 4, 1, 1, 32, 8, 128, "bf16", 64, 0, 50000, 65536),
        # many sequences with drafted tokens over one long document: matrix-core work
        _attn("attn-long-prefix", 64, 4, 4, 32, 8, 128, "bf16", 64, 32768, 16, 1024),
        # four drafted tokens of one sequence
        _verify("verify-one-sequence", 1, 4, False, 128256, True, "f32"),
        # a batch with up to eight drafted tokens each
        _verify("verify-batch", 64, 8, True, 128256, True, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "kv_append", "attention", "attention", "verify"))
    kv_heads = rng.randint(1, 8)
    group = rng.randint(1, 8)
    head_dim = rng.choice((64, 80, 96, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    if op in ("norm_rope", "kv_append"):
        most = 16384 * 40 * 128 // ((2 + group) * kv_heads * head_dim)
        rot_dim = 2 * rng.randint(1, head_dim // 2) if rng.random() < 0.4 else head_dim
        tokens = _log_int(rng, 1, min(most, 16384))
        src, dst = rng.choice((("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f16")))
        c = (tokens, group * kv_heads, kv_heads, head_dim, rot_dim, rng.choice(("halves", "adjacent")), src, dst,
             rng.random() < 0.6, _log_int(rng, tokens + 1, 131072 + tokens))
        case = _rope("", *c) if op == "norm_rope" else _append("", *c, page)
        if op == "kv_append" and rng.random() < 0.4:
            case["q_heads"] = 0
    elif op == "attention":
        seqs = _log_int(rng, 1, 64)
        q_hi = rng.choice((1, 1, 1, rng.randint(2, 8)))
        prefix = 0 if rng.random() < 0.3 else _log_int(rng, 16, 32768)
        bytes_per = kv_heads * head_dim * 4
        hi = _log_int(rng, q_hi, max(q_hi, min(65536, (1 << 30) // (seqs * bytes_per))))
        lo = rng.randint(q_hi, hi)
        # no more multiply-adds than the largest listed case
        most = 64 * 4 * 32 * 128 * 32768
        while seqs * q_hi * group * kv_heads * head_dim * prefix > most:
            prefix //= 2
        case = _attn("", seqs, rng.randint(1, q_hi), q_hi, group * kv_heads, kv_heads, head_dim,
                     rng.choice(("bf16", "f16")), page, prefix, lo, hi)
    else:
        case = _verify("", _log_int(rng, 1, 64), rng.randint(1, 8), rng.random() < 0.5, _log_int(rng, 1000, 128256),
                       rng.random() < 0.8, rng.choice(("f32", "f32", "bf16")))
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n whole numbers of [lo, hi], scattered, the same for every seed (the work depends on them)."""
    return [lo + (i * 2654435761 + 40503) % 1000003 % (hi - lo + 1) for i in range(n)]


# ------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"norm_rope": _prepare_rope, "kv_append": _prepare_rope, "attention": _prepare_attn,
            "verify": _prepare_verify}[case["op"]](case, gen)


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


def _prepare_rope(case, gen):
    T, Hq, Hk, D, R = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["rot_dim"]
    src, dst = DTYPES[case["src"]], DTYPES[case["dst"]]
    # one projection's rows hold queries, keys and values side by side, as a fused product leaves them
    rows = _randn(gen, T, (Hq + 2 * Hk) * D, dtype=src, scale=1.5)
    heads = rows.view(T, Hq + 2 * Hk, D)
    first = int(torch.randint(0, case["far"] - T + 1, (1,), generator=gen, device=DEV))
    s = {"case": case, "q": heads[:, :Hq] if Hq else None, "k": heads[:, Hq:Hq + Hk], "v": heads[:, Hq + Hk:],
         "positions": torch.arange(first, first + T, dtype=torch.int32, device=DEV),
         "inv_freq": 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R),
         "q_gain": 1 + _randn(gen, D, scale=0.1) if case["gains"] and Hq else None,
         "k_gain": 1 + _randn(gen, D, scale=0.1) if case["gains"] else None,
         "q_out": torch.empty(T, Hq, D, dtype=dst, device=DEV) if Hq else None}
    if case["op"] == "norm_rope":
        s["k_out"] = torch.empty(T, Hk, D, dtype=dst, device=DEV)
        if own:
            import bit_plane_weight_amd as bpw
            s["plan"] = bpw.QkNormRopePlan(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["inv_freq"],
                                           q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS,
                                           interleaved=case["pairs"] == "adjacent")
    else:
        P = case["page"]
        pages = T // P + 8
        s["k_pages"] = _randn(gen, pages, Hk, P, D, dtype=dst)
        s["v_pages"] = _randn(gen, pages, Hk, P, D, dtype=dst)
        order = torch.randperm(pages, generator=gen, device=DEV)
        start = int(torch.randint(0, 7 * P, (1,), generator=gen, device=DEV))
        if T <= 256:  # a decode step: one token each, scattered over the pages
            s["slots"] = torch.randperm(pages * P, generator=gen, device=DEV)[:T].contiguous()
        else:  # a chunk of one sequence: consecutive offsets over its pages
            at = torch.arange(start, start + T, device=DEV)
            s["slots"] = order[at // P] * P + at % P
        if own:
            import bit_plane_weight_amd as bpw
            s["plan"] = bpw.KvAppendPlan(bpw.PagedKv(s["k_pages"], s["v_pages"]), s["k"], s["v"], s["slots"],
                                         positions=s["positions"], inv_freq=s["inv_freq"], k_gain=s["k_gain"],
                                         q=s["q"], q_out=s["q_out"], q_gain=s["q_gain"], eps=EPS,
                                         interleaved=case["pairs"] == "adjacent")
    return s


def _attn_lengths(case):
    n_q = _spread(case["seqs"], case["q_lo"], case["q_hi"])
    lens = [max(a, n) for a, n in zip(_spread(case["seqs"], case["lo"], case["hi"]), n_q)]
    return n_q, lens


def _prepare_attn(case, gen):
    B, Hq, Hk, D, P = case["seqs"], case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    n_q, lens = _attn_lengths(case)
    T = sum(n_q)
    starts = [0]
    for n in n_q:
        starts.append(starts[-1] + n)
    prefix_pages = -(-case["prefix"] // P)
    per_seq = [-(-n // P) for n in lens]
    pages = prefix_pages + sum(per_seq) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    # each sequence's row of the table: its own pages, then pages that are not read
    width = max(per_seq)
    at = torch.tensor(per_seq, device=DEV)
    first = prefix_pages + torch.cumsum(at, 0) - at
    col = torch.arange(width, device=DEV)
    table = order[torch.where(col[None] < at[:, None], first[:, None] + col[None], 0)].contiguous()
    s = {"case": case, "max_q": max(n_q),
         "q": _randn(gen, T, Hq, D, dtype=dtype, scale=1.5), "out": torch.empty(T, Hq, D, dtype=dtype, device=DEV),
         "lse": torch.empty(T, Hq, dtype=torch.float32, device=DEV),
         "k_pages": _randn(gen, pages, Hk, P, D, dtype=dtype), "v_pages": _randn(gen, pages, Hk, P, D, dtype=dtype),
         "prefix_pages": order[:prefix_pages].contiguous(), "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "q_starts": torch.tensor(starts, dtype=torch.int32, device=DEV)}
    if own:
        import bit_plane_weight_amd as bpw
        kv = bpw.PagedKv(s["k_pages"], s["v_pages"])
        ws = torch.empty(bpw.bpw_attn_shared_prefix_workspace_bytes(kv, s["q"], case["prefix"], B, s["max_q"]),
                         dtype=torch.uint8, device=DEV)
        s["plan"] = bpw.SharedPrefixAttnPlan(kv, s["q"], s["out"], s["prefix_pages"], case["prefix"], table, s["lens"],
                                             s["q_starts"], s["max_q"], ws, lse=s["lse"])
    return s


def _prepare_verify(case, gen):
    B, K, V = case["seqs"], case["drafts"], case["vocab"]
    dtype = DTYPES[case["dtype"]]
    logits = _randn(gen, B, K + 1, V, scale=3.0)
    s = {"case": case, "target": torch.softmax(logits, -1).to(dtype),
         "n_draft": torch.tensor(_spread(B, 0, K) if case["ragged"] else [K] * B, dtype=torch.int32, device=DEV)}
    guess = torch.softmax(logits[:, :K] + _randn(gen, B, K, V, scale=0.4), -1).to(dtype)
    del logits
    s["tokens"] = torch.multinomial(guess.float().view(B * K, V), 1, generator=gen).view(B, K).to(torch.int32)
    s["draft"] = guess if case["with_draft"] else None
    s["accept_u"] = torch.rand(B, K, generator=gen, device=DEV)
    s["sample_u"] = torch.rand(B, generator=gen, device=DEV)
    s["out_tokens"] = torch.empty(B, K + 1, dtype=torch.int32, device=DEV)
    s["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
    if own:
        import bit_plane_weight_amd as bpw
        ws = torch.empty(bpw.bpw_verify_draft_workspace_bytes(B, V), dtype=torch.uint8, device=DEV)
        s["plan"] = bpw.DraftVerifyPlan(s["target"], s["draft"], s["tokens"], s["accept_u"], s["sample_u"],
                                        s["out_tokens"], s["accepted"], ws, n_draft=s["n_draft"])
    return s


# ------------------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        s["plan"].run()
    else:
        {"norm_rope": _plain_rope, "kv_append": _plain_append, "attention": _plain_attn, "verify": _plain_verify}[op](s)
    if op == "norm_rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "kv_append":
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], **({} if s["q"] is None else {"q": s["q_out"]})}
    if op == "attention":
        return {"out": s["out"], "lse": s["lse"]}
    return {"tokens": s["out_tokens"], "accepted": s["accepted"]}


def _plain_norm_rotate(x, gain, cos, sin, adjacent):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    R = 2 * cos.shape[-1]
    c, n = cos[:, None], sin[:, None]
    if adjacent:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_angles(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    return angle.cos().float(), angle.sin().float()


def _plain_rope(s):
    cos, sin = _plain_angles(s)
    adjacent = s["case"]["pairs"] == "adjacent"
    s["q_out"].copy_(_plain_norm_rotate(s["q"], s["q_gain"], cos, sin, adjacent))
    s["k_out"].copy_(_plain_norm_rotate(s["k"], s["k_gain"], cos, sin, adjacent))


def _plain_append(s):
    cos, sin = _plain_angles(s)
    adjacent, P, dst = s["case"]["pairs"] == "adjacent", s["case"]["page"], s["k_pages"].dtype
    page, at = s["slots"] // P, s["slots"] % P
    s["k_pages"][page, :, at] = _plain_norm_rotate(s["k"], s["k_gain"], cos, sin, adjacent).to(dst)
    s["v_pages"][page, :, at] = s["v"].to(dst)
    if s["q"] is not None:
        s["q_out"].copy_(_plain_norm_rotate(s["q"], s["q_gain"], cos, sin, adjacent))


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hk, D, P, Lp, M = c["seqs"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], c["prefix"], s["max_q"]
    G, T, starts = Hq // Hk, s["q"].shape[0], s["q_starts"].long()
    scale = 1.0 / math.sqrt(D)
    # tokens as rows [sequence, j], the rows past a sequence's own repeated from others and not used
    j = torch.arange(M, device=DEV)
    row = (starts[:-1, None] + j[None]).clamp(max=T - 1)
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(starts, token, right=True) - 1
    place = seq * M + token - starts[seq]
    q = s["q"].float().view(T, Hk, G, D)[row].permute(0, 2, 1, 3, 4)  # [B, Hk, M, G, D]
    # scores against each sequence's own keys; token j of n sees the first len - (n - 1 - j)
    L = s["table"].shape[1] * P
    keys, values = (x[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D).float()
                    for x in (s["k_pages"], s["v_pages"]))
    n_q = starts[1:] - starts[:-1]
    sees = s["lens"].long()[:, None] - (n_q[:, None] - 1 - j[None])
    hidden = torch.arange(L, device=DEV) >= sees[..., None]  # [B, M, L]
    own_s = torch.matmul(q.reshape(B, Hk, M * G, D), keys.transpose(-1, -2)).view(B, Hk, M, G, L) * scale
    own_s = own_s.masked_fill(hidden[:, None, :, None], -math.inf).view(B, Hk, M * G, L)
    top = own_s.amax(-1)
    if Lp:
        pk, pv = (x[s["prefix_pages"].long()].permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :Lp].float()
                  for x in (s["k_pages"], s["v_pages"]))
        qp = q.permute(1, 0, 2, 3, 4).reshape(Hk, B * M * G, D)
        pre_s = torch.matmul(qp, pk.transpose(-1, -2)) * scale  # [Hk, B*M*G, Lp]
        top = torch.maximum(top, pre_s.amax(-1).view(Hk, B, M * G).transpose(0, 1))
    base = torch.where(torch.isinf(top), 0.0, top)
    own_p = torch.exp(own_s - base[..., None])
    total, out = own_p.sum(-1), torch.matmul(own_p, values)
    if Lp:
        pre_p = torch.exp(pre_s - base.transpose(0, 1).reshape(Hk, B * M * G, 1))
        total = total + pre_p.sum(-1).view(Hk, B, M * G).transpose(0, 1)
        out = out + torch.matmul(pre_p, pv).view(Hk, B, M * G, D).transpose(0, 1)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = base + torch.log(total)
    out = out.view(B, Hk, M, G, D).transpose(1, 2).reshape(B * M, Hq, D)
    lse = lse.view(B, Hk, M, G).transpose(1, 2).reshape(B * M, Hq)
    s["out"].copy_(out[place])
    s["lse"].copy_(lse[place])


def _plain_verify(s):
    B, K, V = s["case"]["seqs"], s["case"]["drafts"], s["case"]["vocab"]
    tok, step = s["tokens"].long(), torch.arange(K, device=DEV)
    p = s["target"][:, :K].gather(-1, tok[..., None])[..., 0].double()
    q = 1.0 if s["draft"] is None else s["draft"].gather(-1, tok[..., None])[..., 0].double()
    ok = (s["accept_u"].double() * q < p) & (step < s["n_draft"][:, None])
    n = ok.long().cumprod(-1).sum(-1)
    seq = torch.arange(B, device=DEV)
    mass = s["target"][seq, n].double()
    at = n.clamp(max=K - 1)
    if s["draft"] is None:
        rest = mass.scatter(-1, tok[seq, at][:, None], 0.0)
    else:
        rest = (mass - s["draft"][seq, at].double()).clamp(min=0.0)
    rejected = (n < s["n_draft"])[:, None] & (rest.sum(-1, keepdim=True) > 0)
    mass = torch.where(rejected, rest, mass)
    cum = mass.cumsum(-1)
    last = torch.where(mass > 0, torch.arange(V, device=DEV), -1).amax(-1)
    pick = torch.minimum((cum <= s["sample_u"].double()[:, None] * cum[:, -1:]).sum(-1), last)
    step = torch.arange(K + 1, device=DEV)
    drafts = torch.cat((tok, tok[:, -1:]), -1)
    out = torch.where(step < n[:, None], drafts, torch.where(step == n[:, None], pick[:, None], -1))
    s["out_tokens"].copy_(out)
    s["accepted"].copy_(n)


# ------------------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_rope, "kv_append": _exact_append, "attention": _exact_attn,
            "verify": _exact_verify}[case["op"]](case, s)


def _exact_heads(case, x, gain, positions, inv_freq):
    x = x.to(torch.float64)
    if gain is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.to(torch.float64)
    R = case["rot_dim"]
    turn = torch.polar(torch.ones_like(inv_freq)[None], positions.to(torch.float64)[:, None] * inv_freq[None])[:, None]
    y = x.clone()
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["pairs"] == "adjacent" else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rope(case, s):
    return {n: _exact_heads(case, s[n], s[n + "_gain"], s["positions"], s["inv_freq"]) for n in ("q", "k")}


def _exact_append(case, s):
    P = case["page"]
    k, v = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
    page, at = torch.div(s["slots"], P, rounding_mode="floor"), torch.remainder(s["slots"], P)
    k[page, :, at] = _exact_heads(case, s["k"], s["k_gain"], s["positions"], s["inv_freq"])
    v[page, :, at] = s["v"].to(torch.float64)
    got = {"k_pages": k, "v_pages": v}
    if s["q"] is not None:
        got["q"] = _exact_heads(case, s["q"], s["q_gain"], s["positions"], s["inv_freq"])
    return got


def _exact_attn(case, s):
    Hq, Hk, D, P = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    n_q, lens = _attn_lengths(case)

    def rows(pages, ids, n):
        return pages[ids.long()].transpose(0, 1).reshape(Hk, -1, D)[:, :n].to(torch.float64)

    shared = [rows(s[x], s["prefix_pages"], case["prefix"]) for x in ("k_pages", "v_pages")]
    out, lse, t = [], [], 0
    for b, (n, length) in enumerate(zip(n_q, lens)):
        k, v = (torch.cat((shared[i], rows(s[x], s["table"][b], length)), 1)
                for i, x in enumerate(("k_pages", "v_pages")))
        q = s["q"][t:t + n].to(torch.float64).view(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)  # [Hk, G, n, D]
        score = q.reshape(Hk, -1, D) @ k.transpose(1, 2) / math.sqrt(D)
        score = score.view(Hk, Hq // Hk, n, -1)
        far = torch.arange(k.shape[1], device=DEV)[None] > case["prefix"] + length - n + torch.arange(n, device=DEV)[:, None]
        score[..., far] = -math.inf
        lse.append(torch.logsumexp(score, -1).permute(2, 0, 1).reshape(n, Hq))
        w = torch.softmax(score, -1).view(Hk, -1, k.shape[1])
        out.append((w @ v).view(Hk, Hq // Hk, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D))
        t += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_verify(case, s):
    K, V = case["drafts"], case["vocab"]
    tokens, accepted = torch.full((case["seqs"], K + 1), -1), torch.zeros(case["seqs"], dtype=torch.int64)
    for b in range(case["seqs"]):
        n, most = 0, int(s["n_draft"][b])
        while n < most:
            x = int(s["tokens"][b, n])
            q = 1.0 if s["draft"] is None else float(s["draft"][b, n, x])
            if not float(s["accept_u"][b, n]) * q < float(s["target"][b, n, x]):
                break
            tokens[b, n] = x
            n += 1
        mass = s["target"][b, n].double().cpu()
        if n < most:
            guess = torch.zeros(V, dtype=torch.float64)
            if s["draft"] is None:
                guess[int(s["tokens"][b, n])] = 1.0
            else:
                guess = s["draft"][b, n].double().cpu()
            rest = torch.maximum(mass - guess, torch.zeros(1, dtype=torch.float64))
            mass = rest if float(rest.sum()) > 0 else mass
        cum = torch.cumsum(mass, 0)
        above = torch.nonzero(cum > float(s["sample_u"][b]) * float(cum[-1]))
        tokens[b, n] = int(above[0]) if len(above) else int(torch.nonzero(mass > 0)[-1])
        accepted[b] = n
    return {"tokens": tokens.int(), "accepted": accepted.int()}


# ------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] in ("norm_rope", "kv_append"):
        heads = case["q_heads"] + (1 if case["op"] == "norm_rope" else 2) * case["kv_heads"]
        n = case["tokens"] * heads * case["head_dim"]
        return {"bytes": n * (SIZE[case["src"]] + SIZE[case["dst"]]) + case["tokens"] * 12, "flops": 8 * n}
    if case["op"] == "attention":
        n_q, lens = _attn_lengths(case)
        Hq, Hk, D, T = case["q_heads"], case["kv_heads"], case["head_dim"], sum(n_q)
        size = SIZE[case["dtype"]]
        seen = T * case["prefix"] + sum(n * length - n * (n - 1) // 2 for n, length in zip(n_q, lens))
        return {"bytes": 2 * T * Hq * D * size + T * Hq * 4 + 2 * (case["prefix"] + sum(lens)) * Hk * D * size,
                "flops": 4 * seen * Hq * D}
    # the one row of the target that each sequence draws its last token from, and the draft's beside it
    rows = case["seqs"] * (2 if case["with_draft"] else 1)
    return {"bytes": rows * case["vocab"] * SIZE[case["dtype"]] + case["seqs"] * (case["drafts"] * 20 + 12),
            "flops": 2 * rows * case["vocab"]}
