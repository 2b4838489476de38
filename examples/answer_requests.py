"""Requests from prompt to scored answers over a cache held in 4 bits: append, prompt attention, decode steps, log probabilities.

Several prompts of different lengths arrive packed one after another. One launch norms and rotates their heads, writes
keys and values to the 4-bit pages and hands out the values that the codes stand for, which the attention over the
prompts reads, so that a token sees the same numbers there as the decode steps will. The prompt's own tokens are
scored. Then every request takes decode steps: append, attention over its pages, the head, and the log probability,
entropy and alternatives of the token it answers with (append, attention and scores in one graph). Weights are random; with
--check all of it is compared with float64 references on the CPU.

    python examples/answer_requests.py --requests 4 --longest 200 --answer 6 --check
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_plane_weight_amd as bpw  # noqa: E402

Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, VOCAB, TOP, HEAT = 20, 5, 128, 16, 4096, 4, 1.25
I32, BF16, U8 = torch.int32, torch.bfloat16, torch.uint8


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--longest", type=int, default=200, help="most tokens of a prompt")
    ap.add_argument("--answer", type=int, default=6, help="decode steps")
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    B, dev = a.requests, torch.device("cuda:0")
    rng, gen = np.random.default_rng(a.seed), torch.Generator(device=dev).manual_seed(a.seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731

    # a token's heads stand in one row: what a fused projection of its embedding would give
    table_of_rows = randn(VOCAB, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM).to(BF16)
    head_w = (randn(VOCAB, Q_HEADS * HEAD_DIM) / 32).to(BF16)
    q_gain, k_gain = (1 + 0.1 * randn(HEAD_DIM) for _ in range(2))
    inv_freq = 500000.0 ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64, device=dev) / HEAD_DIM)

    lens = [int(n) for n in rng.integers(1, a.longest + 1, B)]
    starts = np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1])
    prompt = torch.tensor(rng.integers(0, VOCAB, T), device=dev)

    # pages in a scattered order, enough for prompts and answers
    per_request = -(-(max(lens) + a.answer) // PAGE)
    pages = B * per_request
    codes = [torch.zeros(pages, KV_HEADS, PAGE, HEAD_DIM // 2, dtype=U8, device=dev) for _ in range(2)]
    powers = [torch.full((pages, KV_HEADS, PAGE, HEAD_DIM // 32), 127, dtype=U8, device=dev) for _ in range(2)]
    kv = bpw.PagedKv4(*codes, *powers)
    table = torch.randperm(pages, generator=gen, device=dev).to(I32).view(B, per_request).contiguous()

    def slots_of(request, place):
        return (table[request, place // PAGE] * PAGE + place % PAGE).long()

    def heads(rows):
        return rows.view(-1, Q_HEADS + 2 * KV_HEADS, HEAD_DIM).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)

    def logits_of(attended, out):
        for t in range(out.shape[0]):
            bpw.bpw_dense_head_gemv(head_w, attended[t].flatten(), out[t])

    # ---- the prompts
    request = torch.tensor(np.repeat(np.arange(B), lens), device=dev)
    place = torch.tensor(np.concatenate([np.arange(n) for n in lens]), device=dev)
    slots, positions = slots_of(request, place), place.to(I32)
    q, k, v = heads(table_of_rows[prompt])
    q_out, attended = (torch.empty(T, Q_HEADS, HEAD_DIM, dtype=BF16, device=dev) for _ in range(2))
    k_seen, v_seen = (torch.empty(T, KV_HEADS, HEAD_DIM, dtype=BF16, device=dev) for _ in range(2))
    bpw.bpw_kv4_append(kv, k, v, slots, positions, inv_freq, k_gain=k_gain, q=q, q_out=q_out, q_gain=q_gain, k_values=k_seen,
                       v_values=v_seen)
    bpw.bpw_prompt_attn(q_out, k_seen, v_seen, attended, torch.tensor(starts, dtype=I32, device=dev))
    logits = torch.empty(T, VOCAB, device=dev)
    logits_of(attended, logits)
    following = torch.roll(prompt, -1).to(I32)  # (of a request's last token: another request's first, not used)
    scores, answer = torch.empty(T, device=dev), torch.empty(T, 1, dtype=I32, device=dev)
    ws = torch.empty(bpw.bpw_token_logprobs_workspace_bytes(T, VOCAB, 1), dtype=U8, device=dev)
    bpw.bpw_token_logprobs(logits, following, scores, ws, top_tokens=answer, top_logprobs=torch.empty(T, 1, device=dev))
    torch.cuda.synchronize()
    own = [float(scores[starts[i]:starts[i + 1] - 1].sum()) for i in range(B)]
    print(f"{B} prompts of {lens} tokens, log probabilities {[round(x, 1) for x in own]}")
    f64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    if a.check:
        from oracle import decode_ops, request_ops
        where = ((slots // PAGE).cpu(), slice(None), (slots % PAGE).cpu())
        for seen, x, y in ((k_seen, codes[0], powers[0]), (v_seen, codes[1], powers[1])):
            held = request_ops.from_codes(request_ops.unpacked(x.cpu().numpy()), y.cpu().numpy())[where]
            assert np.array_equal(f64(seen), held), "values handed out and held"
        turned, mag = decode_ops.norm_rope(f64(k), f64(k_gain), positions.tolist(), inv_freq.tolist(), 1e-6, False)
        want, power, near = request_ops.to_codes(turned)
        got = request_ops.unpacked(codes[0].cpu().numpy())[where]
        assert np.all((got == want) | (near < 1e-9)), "codes of keys"
        assert np.array_equal(powers[0].cpu().numpy()[where], power), "powers of keys"
        out, _, mag = request_ops.prompt(f64(q_out), f64(k_seen), f64(v_seen), starts, HEAD_DIM ** -0.5)
        assert np.all(np.abs(f64(attended) - out) <= 2.0 ** -7 * (np.abs(out) + mag)), "attention of the prompts"
        lp = request_ops.logprobs(f64(logits), following.cpu().numpy(), 1, 1.0)
        assert np.all(np.abs(f64(scores) - lp[0]) <= 1e-5 * (1 + np.abs(lp[0]))), "scores of the prompts"
        assert np.array_equal(answer.cpu().numpy(), lp[2]), "most likely tokens"

    # ---- the answers: buffers that a graph can read
    token = answer[torch.tensor(starts[1:] - 1, device=dev), 0].clone()
    rows = torch.zeros(B, table_of_rows.shape[1], dtype=BF16, device=dev)
    q1, k1, v1 = heads(rows)
    slot1, len1 = torch.zeros(B, dtype=torch.int64, device=dev), torch.zeros(B, dtype=I32, device=dev)
    pos1, one_each = torch.zeros(B, dtype=I32, device=dev), torch.arange(B + 1, dtype=I32, device=dev)
    q1_out, attended1 = (torch.empty(B, Q_HEADS, HEAD_DIM, dtype=BF16, device=dev) for _ in range(2))
    logits1 = torch.empty(B, VOCAB, device=dev)
    logprob, entropy = torch.empty(B, device=dev), torch.empty(B, device=dev)
    top, top_lp = torch.empty(B, TOP, dtype=I32, device=dev), torch.empty(B, TOP, device=dev)
    append = bpw.Kv4AppendPlan(kv, k1, v1, slot1, pos1, inv_freq, k_gain=k_gain, q=q1, q_out=q1_out, q_gain=q_gain)
    ws4 = torch.empty(bpw.bpw_kv4_attn_workspace_bytes(kv, q1_out, B, 1, per_request), dtype=U8, device=dev)
    attend = bpw.Kv4AttnPlan(kv, q1_out, attended1, table, len1, one_each, 1, ws4)
    wsl = torch.empty(bpw.bpw_token_logprobs_workspace_bytes(B, VOCAB, TOP), dtype=U8, device=dev)
    likely = torch.empty(B, dtype=I32, device=dev)  # the token that the last logits made most likely
    score = bpw.TokenLogprobsPlan(logits1, likely, logprob, wsl, entropy=entropy, top_tokens=top, top_logprobs=top_lp, scale=HEAT)

    def step():
        append.run()
        attend.run()
        logits_of(attended1, logits1)
        likely.copy_(logits1.argmax(-1))
        score.run()

    graph = None
    total = torch.zeros(B, device=dev)
    for i in range(a.answer):
        at = torch.tensor([n + i for n in lens], device=dev)
        rows.copy_(table_of_rows[token.long()])
        slot1.copy_(slots_of(torch.arange(B, device=dev), at))
        pos1.copy_(at)
        len1.copy_(at + 1)
        if i == 1:  # (the first step has run everything once)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        total += logprob
        token = top[:, 0].clone()
        torch.cuda.synchronize()
        print(f"step {i}: tokens {token.tolist()}, log probabilities {[round(x, 2) for x in logprob.tolist()]}")
        if a.check:
            held = [request_ops.from_codes(request_ops.unpacked(x.cpu().numpy()), y.cpu().numpy()) for x, y in zip(codes, powers)]
            out, _, mag = decode_ops.attention(f64(q1_out), *held, [], 0, table.cpu().numpy(), len1.tolist(), one_each.tolist(), 1, HEAD_DIM ** -0.5)
            assert np.all(np.abs(f64(attended1) - out) <= 2.0 ** -7 * np.abs(out) + 1e-4 * mag), "attention of a step"
            lp = request_ops.logprobs(f64(logits1), token.cpu().numpy(), TOP, HEAT)
            assert np.array_equal(top.cpu().numpy(), lp[2]), "alternatives"
            for got, want in ((logprob, lp[0]), (entropy, lp[1]), (top_lp, lp[3])):
                assert np.all(np.abs(f64(got) - want) <= 1e-5 * (1 + np.abs(want))), "scores of a step"
    if a.check:
        print("check: ok")
    return total


if __name__ == "__main__":
    main()
