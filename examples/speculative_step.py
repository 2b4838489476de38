"""One attention block and the verification of a speculative decode step, from ternary projections to accepted tokens.

Several sequences share a prefix (a system prompt, a document) and have drafted some tokens each. For all drafted
tokens at once: the q, k and v projections (grouped ternary small batch), norm + rotation + append to the paged cache
in one launch, attention over the shared prefix and each sequence's own pages, the output projection, a small dense
head, and the verification of the drafts against its probabilities. Weights and inputs are random; with --check the
block is compared with a float64 reference on the CPU.

    python examples/speculative_step.py --sequences 8 --drafts 3 --prefix 2048 --check
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_plane_weight_amd as bpw  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, VOCAB = 2560, 20, 5, 128, 16, 4096


def ternary(rng, rows, cols, dev):
    """A random ternary matrix on the GPU, and its dequantised copy for the reference."""
    w = rng.integers(-1, 2, (rows, cols)).astype(np.int8)
    scale = float(np.float32(1.0 / math.sqrt(cols)))
    host = bpw.bpw_load(bpw.bpw_pack_i8(w), rows, cols, scale)
    return bpw.bpw_upload(host, torch.empty(host.nbytes, dtype=torch.uint8, device=dev)), w.astype(np.float64) * scale


class Projections:
    """Matrices that read the same int8 activations [tokens, cols], in one launch (bpw.SmallBatchPlan)."""

    def __init__(self, mats, tokens, scales, dev):
        cols = mats[0].cols
        self.x = torch.zeros(tokens, (cols + 63) // 64 * 64, dtype=torch.int8, device=dev)
        self.out = [torch.empty(tokens, m.rows, device=dev) for m in mats]
        sums = [torch.empty(tokens, m.rows, dtype=torch.int32, device=dev) for m in mats]
        jobs = [bpw.sb_job(m, self.x, scales, s, o) for m, s, o in zip(mats, sums, self.out)]
        ws = torch.empty(bpw.bpw_gemm_small_batch_workspace_bytes(jobs, tokens), dtype=torch.uint8, device=dev)
        self.plan = bpw.SmallBatchPlan(jobs, tokens, ws)


def codes(x):
    """Absmax int8 codes of each row, and their scales."""
    scale = x.abs().amax(-1, keepdim=True).clamp(min=1e-12) / 127
    return torch.round(x / scale).to(torch.int8), scale


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--prefix", type=int, default=2048)
    ap.add_argument("--suffix", type=int, default=300, help="most positions of a sequence's own before this step")
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    B, K = a.sequences, a.drafts
    N = K + 1  # the last accepted token and the drafts: one query token each
    T = B * N
    if T > 64:
        ap.error("sequences * (drafts + 1) is the small batch: 64 tokens at most")
    dev = torch.device("cuda:0")
    rng, gen = np.random.default_rng(a.seed), torch.Generator(device=dev).manual_seed(a.seed)

    # projections: one launch for q, k, v; one for the output projection (activation scales applied after it)
    mats, dense = zip(*(ternary(rng, r, HIDDEN, dev) for r in (Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, HIDDEN)))
    x_scale = np.full(T, 0.02, np.float32)
    qkv = Projections(mats[:3], T, x_scale, dev)
    out_proj = Projections(mats[3:], T, np.ones(T, np.float32), dev)
    head_w = (torch.randn(VOCAB, HIDDEN, generator=gen, device=dev) / 64).to(torch.bfloat16)

    # the paged cache: prefix pages shared, then each sequence's own
    lens = [int(n) for n in rng.integers(0, a.suffix + 1, B)]
    prefix_pages = -(-a.prefix // PAGE)
    own_pages = -(-(a.suffix + N) // PAGE)
    pages = prefix_pages + B * own_pages
    cache = [torch.randn(pages, KV_HEADS, PAGE, HEAD_DIM, generator=gen, device=dev).to(torch.bfloat16) for _ in range(2)]
    kv = bpw.PagedKv(*cache)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    prefix, table = order[:prefix_pages].contiguous(), order[prefix_pages:].view(B, own_pages).contiguous()
    place = torch.tensor([[n + j for j in range(N)] for n in lens], device=dev)  # own positions of the new tokens
    slots = (torch.gather(table, 1, place // PAGE) * PAGE + place % PAGE).flatten().long()
    positions = (a.prefix + place).flatten().to(torch.int32)
    len_after = torch.tensor([n + N for n in lens], dtype=torch.int32, device=dev)
    starts = torch.arange(0, T + 1, N, dtype=torch.int32, device=dev)
    inv_freq = 500000.0 ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64, device=dev) / HEAD_DIM)
    q_gain, k_gain = (1 + 0.1 * torch.randn(HEAD_DIM, generator=gen, device=dev) for _ in range(2))

    q = torch.empty(T, Q_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=dev)
    attended = torch.empty_like(q)
    as_heads = lambda t: t.unflatten(-1, (-1, HEAD_DIM))  # noqa: E731
    append = bpw.KvAppendPlan(kv, as_heads(qkv.out[1]), as_heads(qkv.out[2]), slots, positions, inv_freq, k_gain=k_gain,
                              q=as_heads(qkv.out[0]), q_out=q, q_gain=q_gain)
    ws = torch.empty(bpw.bpw_attn_shared_prefix_workspace_bytes(kv, q, a.prefix, B, N, own_pages), dtype=torch.uint8, device=dev)
    attention = bpw.SharedPrefixAttnPlan(kv, q, attended, prefix, a.prefix, table, len_after, starts, N, ws)

    # the step: what the framework runs is launches only, so a graph can hold them
    qkv.x.copy_(torch.randint(-127, 128, qkv.x.shape, generator=gen, device=dev, dtype=torch.int8))
    qkv.plan.run()
    append.run()
    attention.run()
    c, scale = codes(attended.flatten(1).float())
    out_proj.x.copy_(c)
    out_proj.plan.run()
    hidden = out_proj.out[0] * scale
    logits = torch.empty(T, VOCAB, device=dev)
    normed = (hidden / hidden.square().mean(-1, keepdim=True).sqrt()).to(torch.bfloat16)
    for t in range(T):
        bpw.bpw_dense_head_gemv(head_w, normed[t], logits[t])

    # drafts from a model that is nearly this one, and the verdict on them
    target = torch.softmax(4 * logits, -1).view(B, N, VOCAB)
    guess = torch.softmax(4 * logits + 0.3 * torch.randn(logits.shape, generator=gen, device=dev), -1).view(B, N, VOCAB)[:, :K].contiguous()
    drafted = torch.multinomial(guess.view(B * K, VOCAB), 1, generator=gen).view(B, K).to(torch.int32)
    tokens, accepted = torch.empty(B, N, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    u, r = torch.rand(B, K, generator=gen, device=dev), torch.rand(B, generator=gen, device=dev)
    vws = torch.empty(bpw.bpw_verify_draft_workspace_bytes(B, VOCAB), dtype=torch.uint8, device=dev)
    bpw.bpw_verify_draft(target, guess, drafted, u, r, tokens, accepted, vws)
    torch.cuda.synchronize()
    print(f"{B} sequences, {K} drafts each, prefix {a.prefix}: accepted {accepted.tolist()}")
    print("tokens of the first sequence:", tokens[0].tolist())
    if a.check:
        check(a, qkv.x, x_scale, dense, kv, prefix, table, len_after, starts, positions, inv_freq, q_gain, k_gain, slots, q,
              attended, target, guess, drafted, u, r, tokens, accepted)
        print("check: ok")
    return accepted


def check(a, x, x_scale, dense, kv, prefix, table, len_after, starts, positions, inv_freq, q_gain, k_gain, slots, q, attended,
          target, guess, drafted, u, r, tokens, accepted):
    """The block against float64: queries, appended keys and attention within a bfloat16 step of what their rounded
    inputs give, the verdict equal."""
    from oracle import decode_ops
    f64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    heads = [(f64(x)[:, :HIDDEN] * x_scale[:, None]) @ w.T for w in dense[:3]]
    heads = [h.reshape(h.shape[0], -1, HEAD_DIM) for h in heads]
    step = 2.0 ** -7
    for got, want, gain in ((f64(q), heads[0], q_gain),
                            (f64(kv.k_pages)[(slots // PAGE).cpu(), :, (slots % PAGE).cpu()], heads[1], k_gain)):
        want, mag = decode_ops.norm_rope(want, f64(gain), positions.tolist(), inv_freq.tolist(), 1e-6, False)
        assert np.all(np.abs(got - want) <= step * np.abs(want) + 1e-4 * mag), "queries or keys"
    out, _, mag = decode_ops.attention(f64(q), f64(kv.k_pages), f64(kv.v_pages), prefix.tolist(), a.prefix, table.cpu().numpy(),
                                       len_after.tolist(), starts.tolist(), a.drafts + 1, HEAD_DIM ** -0.5)
    assert np.all(np.abs(f64(attended) - out) <= step * (np.abs(out) + mag)), "attention"
    toks, n = decode_ops.verify(f64(target), f64(guess), drafted.cpu().numpy(), None, u.cpu().numpy(), r.cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), toks) and np.array_equal(accepted.cpu().numpy(), n), "verdict"


if __name__ == "__main__":
    main()
