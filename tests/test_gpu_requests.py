"""Prompt attention, the 4-bit paged cache and token log probabilities on the GPU against the float64 oracle (oracle/request_ops.py,
oracle/decode_ops.py).

Tolerances. A rounding to type t is off by at most eps(t) / 2 of the value; float32 errors are counted by operation where each
bound is formed. Integers and 4-bit codes are equal."""
import importlib.util
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_plane_weight_amd as bpw  # noqa: E402
from conftest import ROOT  # noqa: E402
from oracle import decode_ops, request_ops  # noqa: E402
from test_gpu_decode import BF16, F16, F32, U, attn_tol, dev, f64, half_step, heads_tol, smallest, within  # noqa: E402, F401

pytestmark = pytest.mark.gpu
I32, U8 = torch.int32, torch.uint8


def same_bits(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32), b.view(torch.int16 if b.element_size() == 2 else torch.int32))


# ------------------------------------------------------------------------------ whole prompts


class Prompt:
    """A packed batch: `before` tokens of no sequence, the sequences, `behind` tokens of none. Outputs begin at 77."""

    def __init__(self, dev, counts, Hq, Hk, D, dt=BF16, seed=0, layout="tokens", before=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        T = before + sum(counts) + behind
        q = (torch.randn(T, Hq, D, generator=g) * 1.5).to(dt)
        k, v = (torch.randn(T, Hk, D, generator=g).to(dt) for _ in range(2))
        self.q = q.to(dev)
        if layout == "fused":  # the heads of one projection's rows, with something between them
            rows = torch.full((T, 2 * Hk + 1, D), float("nan"), dtype=dt, device=dev)
            rows[:, :Hk], rows[:, Hk + 1:] = k.to(dev), v.to(dev)
            self.k, self.v = rows[:, :Hk], rows[:, Hk + 1:]
        elif layout == "heads":
            self.q, self.k, self.v = (x.transpose(0, 1).contiguous().to(dev).transpose(0, 1) for x in (q, k, v))
        else:
            self.k, self.v = k.to(dev), v.to(dev)
        self.out = torch.full((T, Hq, D), 77.0, dtype=dt, device=dev)
        self.lse = torch.full((T, Hq), 77.0, device=dev)
        self.starts = torch.tensor(np.concatenate([[before], before + np.cumsum(counts)]), dtype=I32, device=dev)
        self.scale, self.dt = None, dt

    def run(self):
        self.out.fill_(77.0), self.lse.fill_(77.0)
        bpw.bpw_prompt_attn(self.q, self.k, self.v, self.out, self.starts, scale=self.scale, lse=self.lse)
        torch.cuda.synchronize()

    def check(self, what=""):
        D, scale, starts = self.q.shape[-1], self.scale or self.q.shape[-1] ** -0.5, self.starts.tolist()
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        out, lse, mag = request_ops.prompt(q, k, v, starts, scale)
        gone = np.ones(len(lse), bool)  # tokens of no sequence: left as they were
        for a, b in zip(starts, starts[1:]):
            gone[max(a, 0):max(b, 0)] = False
        out[gone], mag[gone], lse[gone] = 77.0, 0.0, 77.0
        L = max(b - a for a, b in zip(starts, starts[1:]))
        tol, tol_lse = attn_tol(out, mag, q, k[np.isfinite(k).all(-1)], v[np.isfinite(v)], D, L, scale, self.dt)
        within(self.out, out, tol, f"{what} out")
        within(self.lse, lse, tol_lse + 4 * U * np.abs(lse), f"{what} lse")


@pytest.mark.parametrize("counts,Hq,Hk,D,dt", [
    ([1], 1, 1, 8, BF16),
    ([1, 1, 2], 4, 2, 64, F16),
    ([5], 20, 5, 128, BF16),
    ([31, 33, 1, 64, 0, 65], 4, 4, 128, BF16),
    ([128, 0, 0, 129, 127], 3, 1, 64, F16),
    ([300, 7], 6, 2, 80, BF16),
    ([257], 14, 2, 96, F16),        # groups that tiles cut
    ([40, 41, 42], 40, 1, 128, BF16),
    ([200], 130, 1, 64, BF16),      # a group beyond one tile
    ([190, 3], 4, 2, 256, F16),
    ([150], 5, 5, 192, BF16),
    ([130, 70], 3, 3, 24, F16),
    ([3 + i % 40 for i in range(150)], 2, 1, 64, BF16),   # more sequences than one round of probes
    ([700], 8, 2, 128, F16),
])
@pytest.mark.parametrize("layout", ["tokens", "fused", "heads"])
def test_prompt(dev, counts, Hq, Hk, D, dt, layout):
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=sum(counts) + D, layout=layout, before=3 if layout == "fused" else 0, behind=2 if layout != "tokens" else 0)
    p.run()
    p.check()


def test_prompt_long_against_blocks(dev):
    """Thousands of positions: the tiles' turns many times over, against float64 products on the GPU."""
    counts, Hq, Hk, D = [5000, 1, 3001], 4, 1, 128
    p = Prompt(dev, counts, Hq, Hk, D, BF16, seed=5)
    p.run()
    a = 0
    for n in counts:
        q, k, v = (x[a:a + n].double().transpose(0, 1) for x in (p.q, p.k, p.v))
        s = q @ k.transpose(1, 2) * D ** -0.5
        s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=dev).triu(1), -math.inf)
        w = torch.softmax(s, -1)
        out, mag, lse = (x.transpose(0, 1).contiguous().cpu().numpy() for x in (w @ v, w @ v.abs(), torch.logsumexp(s, -1)))
        tol, tol_lse = attn_tol(out, mag, f64(p.q[a:a + n]), f64(p.k[a:a + n]), f64(p.v[a:a + n]), D, n, D ** -0.5, BF16)
        within(p.out[a:a + n], out, tol, f"out {n}")
        within(p.lse[a:a + n], lse, tol_lse + 4 * U * np.abs(lse), f"lse {n}")
        a += n


@pytest.mark.parametrize("counts,Hq,Hk,D,dt", [
    ([900, 300, 120], 16, 2, 128, F16),
    ([63, 1, 800, 0, 470], 16, 16, 96, BF16),
    ([700, 333, 1, 290], 16, 4, 256, BF16),
    ([450, 860], 16, 8, 200, F16),
    ([64] * 33, 32, 8, 64, BF16),
    ([1500, 600], 32, 4, 64, F16),
])
def test_prompt_many_rows(dev, counts, Hq, Hk, D, dt):
    """Rows enough for workgroups of 128 of them and the pipeline: as it is, with scores that rise, with values and keys of NaN
    and infinity that some rows of a tile see."""
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=D, layout="fused", before=2, behind=1)
    p.run()
    p.check("as it is")
    longest = 2 + sum(counts[:counts.index(max(counts))])
    p.k[longest:longest + max(counts)] *= torch.linspace(0.1, 4, max(counts), device=dev).to(dt)[:, None, None]
    p.run()
    p.check("rising")
    for at, n, what in ((max(counts) // 2, float("inf"), p.v), (max(counts) - 2, float("nan"), p.v), (max(counts) - 9, float("nan"), p.k)):
        what[longest + at, 0] = n
    p.run()
    p.check("not finite")


def test_prompt_many_sequences(dev):
    """More sequences than two rounds of probes tell apart, most of one token or none."""
    counts = [i % 7 % 3 for i in range(5000)]
    p = Prompt(dev, counts, 2, 2, 8, F16, seed=2)
    p.run()
    p.check()


def test_prompt_starts_out_of_range(dev):
    """Starts are cut to the tokens that there are; an empty call of sequences writes nothing."""
    p = Prompt(dev, [40, 50], 4, 2, 64, F16, seed=3)
    p.starts.copy_(torch.tensor([-5, 40, 10 ** 9], dtype=I32))
    p.run()
    p.starts.copy_(torch.tensor([0, 40, 90], dtype=I32))
    p.check("cut")
    for at in (0, 90, -7, 2 ** 31 - 1):
        p.starts.fill_(at)
        p.run()
        assert (p.out == 77).all() and (p.lse == 77).all()


@pytest.mark.parametrize("D,dt", [(128, BF16), (64, F16), (256, BF16), (80, F16)])
def test_prompt_wide_and_flat_scores(dev, D, dt):
    """Scores that rise along the positions, so that the shift is raised many times; all weights nearly alike."""
    p = Prompt(dev, [200, 90], 4, 2, D, dt, seed=D)
    p.k *= torch.linspace(0.1, 6, p.k.shape[0], device=dev).to(dt)[:, None, None]
    for p.scale in (2.0, 1e-30):
        p.run()
        p.check(str(p.scale))


@pytest.mark.parametrize("Hq,Hk,D,dt", [(4, 4, 128, BF16), (6, 2, 64, F16), (5, 1, 80, BF16), (2, 1, 256, F16)])
def test_prompt_what_is_not_seen_does_not_reach(dev, Hq, Hk, D, dt):
    """NaN and infinities in later tokens' keys and values, in another sequence's, and in tokens of none."""
    p = Prompt(dev, [100, 70], Hq, Hk, D, dt, seed=7, before=4, behind=4)
    p.run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    for x in (p.k, p.v):
        x[:4], x[-4:] = float("nan"), float("inf")
    p.run()
    assert same_bits(p.out, clean) and same_bits(p.lse, clean_lse)
    for at, n, what in ((4 + 61, float("nan"), p.v), (4 + 90, float("inf"), p.v), (4 + 99, -float("inf"), p.v), (4 + 33, float("nan"), p.k)):
        what[at, 0] = n
    p.run()
    assert same_bits(p.out[104:], clean[104:])  # the other sequence
    assert same_bits(p.lse[:4 + 33], clean_lse[:4 + 33])
    first = slice(0, Hq // Hk)  # heads that read the key/value head 0
    assert torch.isfinite(p.out[4:4 + 33].float()).all() and torch.isnan(p.out[4 + 33:4 + 100, first].float()).all()
    p.k[4 + 33, 0] = 0.5
    p.run()
    p.check()  # before 61 all finite, then NaN; the oracle looks at each token's own positions
    assert torch.isfinite(p.out[4:4 + 61].float()).all() and torch.isnan(p.out[4 + 61:4 + 100, first].float()).all()


def test_prompt_nan_query_and_infinite_value(dev):
    p = Prompt(dev, [70, 40], 4, 2, 64, BF16, seed=11)
    p.q[10, 1], p.v[30, 1, 5] = float("nan"), float("inf")
    p.run()
    p.check()
    assert torch.isnan(p.out[10, 1].float()).all() and torch.isnan(p.lse[10, 1]) and torch.isinf(p.out[30:70, 2:, 5].float()).all()


@pytest.mark.parametrize("Hq,Hk,D,counts", [(4, 2, 64, [200, 90]), (4, 1, 128, [300]), (2, 2, 256, [260]), (6, 2, 80, [150, 70]),
                                            (32, 4, 64, [1500, 600]), (16, 2, 128, [900, 300]), (16, 4, 256, [700])])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_prompt_infinite_values_of_small_weight(dev, Hq, Hk, D, counts, dt):
    """An infinite value makes the outputs that see it infinite, also where its weight, 2^-32 to 2^-100 of the largest, is none in
    float16: beside the positions that all rows of a tile see, and on the diagonal."""
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=D)
    p.scale = 1.0
    p.q.zero_(), p.k.zero_()
    p.q[..., 0] = 1.0
    n = counts[0]
    p.k[:n, :, 0] = torch.randn(n, 1, device=dev).to(dt)
    p.k[3, :, 0], p.k[n // 2, :, 0], p.k[n - 40, :, 0] = 30.0, -10.0, 45.0  # a weight of 2^-58 (to 2^-80) at n / 2
    p.v[5, 0, 1], p.v[n // 2, -1, 2], p.v[n // 2, -1, 3], p.v[n - 30, 0, 4] = math.inf, -math.inf, math.inf, -math.inf
    p.run()
    p.check()
    assert torch.isinf(p.out[5:n, :Hq // Hk, 1]).all() and torch.isinf(p.out[n // 2:n, -1, 2:4]).all()
    p.v[n // 2 + 1, -1, 2] = math.inf  # and one of the other sign
    p.run()
    p.check("both signs")
    assert torch.isnan(p.out[n // 2 + 1:n, -1, 2]).all() and torch.isinf(p.out[n // 2:n, -1, 3]).all()


@pytest.mark.parametrize("counts,Hq,Hk,D,dt", [([120, 90], 4, 2, 64, BF16), ([700, 333], 16, 4, 128, F16), ([400], 12, 4, 256, BF16)])
def test_prompt_scores_of_minus_infinity(dev, counts, Hq, Hk, D, dt):
    """Tokens that see nothing but scores of -inf have lse -inf and out NaN (0 / 0); for later ones those positions have no weight."""
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=83)
    n = 70
    p.q.abs_()
    kept = p.k[:n].clone()
    p.k[:n, :, 0] = -math.inf
    p.run()
    assert torch.isnan(p.out[:n]).all() and (p.lse[:n] == -math.inf).all()
    q, k, v = f64(p.q[n:counts[0]]), f64(p.k[n:counts[0]]), f64(p.v[n:counts[0]])
    out, lse, mag = request_ops.prompt(q, k, v, [0, counts[0] - n], D ** -0.5)
    tol, tol_lse = attn_tol(out, mag, q, k, v, D, counts[0], D ** -0.5, dt)
    within(p.out[n:counts[0]], out, tol, "out")
    within(p.lse[n:counts[0]], lse, tol_lse + 4 * U * np.abs(lse), "lse")
    p.k[:n] = kept
    p.run()
    p.check("finite again")


def test_prompt_float16_weights_far_below_the_largest(dev):
    """One position of 32 has all but 2^-25 of the weight and values of zero: the output is what the others add. A step of
    float16's subnormals is 2^-30 of the largest weight, half of one the error."""
    n = 128
    p = Prompt(dev, [n], 2, 1, 64, F16, seed=13)
    p.scale = 1.0
    p.q.zero_(), p.k.zero_()
    p.q[..., 0] = 1.0
    p.v.copy_(p.v.abs() + 500.0)
    p.k[::32, :, 0], p.v[::32] = 17.5, 0.0
    p.run()
    out, lse, mag = request_ops.prompt(f64(p.q), f64(p.k), f64(p.v), [0, n], 1.0)
    assert (out[31:] > 1e-4).all()
    _, tol_lse = attn_tol(out, mag, f64(p.q), f64(p.k), f64(p.v), 64, n, 1.0, F16)
    tol = mag * (2 * tol_lse[..., None] + half_step(F16)) + 32 * 2.0 ** -31 * f64(p.v).max() + half_step(F16) * out + smallest(F16)
    within(p.out, out, tol, "out")
    within(p.lse, lse, tol_lse + 4 * U * np.abs(lse), "lse")


def test_prompt_strides_past_32_bits(dev):
    T, Hk, D, far = 300, 2, 64, 2 ** 23
    p = Prompt(dev, [T - 7, 7], 4, Hk, D, F16, seed=17)
    for name in ("k", "v"):
        wide = torch.empty((T - 1) * far + Hk * D, dtype=F16, device=dev).as_strided((T, Hk, D), (far, D, 1))
        wide.copy_(getattr(p, name))
        setattr(p, name, wide)
    p.run()
    p.check()


def test_prompt_same_bits_on_another_stream_and_in_a_graph(dev):
    """The same bits each time; starts and inputs change between a graph's replays."""
    p = Prompt(dev, [90, 150, 31], 8, 2, 128, BF16, seed=19)
    plan = bpw.PromptAttnPlan(p.q, p.k, p.v, p.out, p.starts, lse=p.lse)
    plan.run()
    first, lse = p.out.clone(), p.lse.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        p.out.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        plan.run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert same_bits(p.out, first) and same_bits(p.lse, lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.run()
    for starts in ([0, 90, 240, 271], [0, 1, 2, 271], [30, 30, 100, 200]):
        p.starts.copy_(torch.tensor(starts, dtype=I32))
        p.v.normal_()
        p.out.fill_(77.0), p.lse.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check(str(starts))
        got = p.out.clone()
        p.run()
        assert same_bits(p.out, got)


@pytest.mark.parametrize("counts,Hq,Hk,D,dt", [
    ([1, 1, 2], 4, 2, 64, F16),
    ([31, 33, 1, 64, 0, 65], 4, 4, 128, BF16),
    ([300, 7], 6, 2, 80, BF16),
    ([190, 3], 4, 2, 256, F16),
    ([150], 5, 5, 192, BF16),
    ([900, 300, 120], 16, 2, 128, F16),   # from here on rows enough for the pipeline
    ([63, 1, 800, 0, 470], 16, 16, 96, BF16),
    ([700, 333, 1, 290], 16, 4, 256, BF16),
    ([450, 860], 16, 8, 200, F16),
    ([700, 600], 16, 4, 160, BF16),
    ([1500, 600], 32, 4, 64, F16),
])
def test_prompt_without_lse(dev, counts, Hq, Hk, D, dt):
    """A kernel of its own, which forms no unrounded sums: the same outputs, bit for bit where they are numbers (no sum that lse
    alone takes enters them), as they are, with scores that rise, with what is not finite."""
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=D + 1, layout="fused", before=2, behind=1)
    n = max(counts)
    longest = 2 + sum(counts[:counts.index(n)])

    def both(what):
        p.run()
        p.check(what)
        out = torch.full_like(p.out, 77.0)
        bpw.bpw_prompt_attn(p.q, p.k, p.v, out, p.starts, scale=p.scale)
        torch.cuda.synchronize()
        assert np.array_equal(f64(out), f64(p.out), equal_nan=True), what

    both("as it is")
    p.k[longest:longest + n] *= torch.linspace(0.1, 4, n, device=dev).to(dt)[:, None, None]
    both("rising")
    for at, x, what in ((n // 2, float("inf"), p.v), (n - 2, float("nan"), p.v), (n - 9, float("nan"), p.k)):
        what[longest + max(at, 0), 0] = x
    both("not finite")


# ------------------------------------------------------------------------------ a cache held in 4 bits


def kv4_cache(dev, pages, Hk, P, D, layout="hnd", seed=0):
    """k_codes, v_codes, k_scales, v_scales of random bytes (powers 2^-3 .. 2^3)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in (D // 2, D // 2, D // 32, D // 32):
        x = torch.randint(0, 256, (pages, P, Hk, n), generator=g, dtype=U8) if n == D // 2 else torch.randint(124, 131, (pages, P, Hk, n), generator=g, dtype=U8)
        out.append(x.to(dev).transpose(1, 2) if layout == "nhd" else x.transpose(1, 2).contiguous().to(dev))
    if layout == "together":  # a row's codes and powers side by side, in a row of a multiple of 16 bytes
        for i in (0, 1):
            width = D // 2 + -(-D // 32 // 16) * 16
            rows = torch.zeros(pages, Hk, P, width, dtype=U8, device=dev)
            rows[..., :D // 2], rows[..., D // 2:D // 2 + D // 32] = out[i], out[2 + i]
            out[i], out[2 + i] = rows[..., :D // 2], rows[..., D // 2:D // 2 + D // 32]
    return out


def held(codes, scales):
    """What a cache stands for, float64 on the CPU [pages, heads, page, dim]."""
    return request_ops.from_codes(request_ops.unpacked(codes.cpu().numpy()), scales.cpu().numpy())


def run_append(dev, T, Hq, Hk, D, R, P, adjacent, src, dst, gains, layout, seed=0, rows=None):
    g = torch.Generator().manual_seed(seed)
    pages = T // P + 4
    cache = kv4_cache(dev, pages, Hk, P, D, layout, seed)
    if rows is None:
        rows = (torch.randn(T, Hq + 2 * Hk, D, generator=g) * 2).to(src)
        rows *= torch.exp2(torch.randint(-6, 7, (T, Hq + 2 * Hk, D // 32), generator=g).float()).repeat_interleave(32, -1).to(src)
    if layout == "odd":  # rows begin one element off
        buf = torch.zeros(rows.numel() + 1, dtype=src, device=dev)
        buf[1:] = rows.flatten().to(dev)
        rows = buf[1:].view(rows.shape)
    rows = rows.to(dev)
    q, k, v = rows[:, :Hq] if Hq else None, rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    slots = torch.randperm(pages * P, generator=g)[:T]
    for i, bad in enumerate((-1, pages * P, -(1 << 60), 1 << 60)):  # padding tokens
        if T > 4 + i:
            slots[4 + i] = bad
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=I32)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)) if R else None
    qg, kg = (1 + torch.randn(D, generator=g) * 0.2 if gains else None for _ in range(2))
    before = [c.clone() for c in cache]
    qo = torch.full((T, Hq, D), float("nan"), dtype=dst, device=dev) if Hq else None
    kv, vv = (torch.full((T, Hk, D), 77.0, dtype=dst, device=dev) for _ in range(2))
    to = lambda x: None if x is None else x.to(dev)  # noqa: E731
    bpw.bpw_kv4_append(bpw.PagedKv4(*cache), k, v, slots.to(dev), to(pos), to(freq), to(kg), q, qo, to(qg), 1e-5, adjacent, kv, vv)
    torch.cuda.synchronize()
    freqs = [] if freq is None else freq.tolist()
    norm = lambda x, w: decode_ops.norm_rope(f64(x), None if w is None else f64(w), pos.tolist(), freqs, 1e-5, adjacent)  # noqa: E731
    left = torch.ones(pages, P, dtype=torch.bool)
    for i, (want, values) in enumerate(((norm(k, kg)[0], kv), (f64(v), vv))):
        codes, power, near = request_ops.to_codes(want)
        computed = near if gains else near[..., :R]  # (the rest is taken as it is)
        assert i == 1 or computed.size == 0 or computed.min() > 1e-8  # no key so near a border that float64 could take either side
        mean = request_ops.from_codes(codes, power)
        assert np.array_equal(f64(values), torch.tensor(mean).to(dst).double().numpy(), equal_nan=True), "values"
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * P:
                left[s // P, s % P] = False
                assert np.array_equal(request_ops.unpacked(cache[i][s // P, :, s % P].cpu().numpy()), codes[t]), f"codes of token {t}"
                assert np.array_equal(cache[2 + i][s // P, :, s % P].cpu().numpy(), power[t]), f"powers of token {t}"
    for c, b in zip(cache, before):
        assert torch.equal(c.transpose(1, 2)[left.to(dev)], b.transpose(1, 2)[left.to(dev)])
    if Hq:
        wq, mq = norm(q, qg)
        within(qo, wq, heads_tol(wq, mq, dst), "queries")


@pytest.mark.parametrize("T,Hq,Hk,D,R,P,adjacent,src,dst,gains,layout", [
    (1, 20, 5, 128, 128, 16, False, F32, BF16, True, "hnd"),
    (1, 0, 1, 32, 32, 16, True, F32, F16, True, "hnd"),
    (64, 4, 2, 64, 64, 32, True, BF16, BF16, True, "nhd"),
    (19, 0, 3, 96, 40, 16, False, F32, F16, False, "hnd"),
    (40, 3, 1, 128, 66, 64, False, F16, F16, True, "together"),
    (9, 6, 2, 160, 160, 64, False, BF16, F16, True, "nhd"),
    (9, 2, 2, 256, 256, 128, False, F32, BF16, True, "odd"),
    (7, 2, 2, 256, 62, 1024, True, BF16, BF16, False, "together"),
    (11, 1, 7, 224, 0, 16, False, F16, BF16, True, "odd"),
])
def test_append4(dev, T, Hq, Hk, D, R, P, adjacent, src, dst, gains, layout):
    run_append(dev, T, Hq, Hk, D, R, P, adjacent, src, dst, gains, layout, seed=T * 31 + D)


@pytest.mark.parametrize("T,Hq,Hk,D,R,P,adjacent,src,dst,gains,layout", [
    (2049, 3, 2, 64, 64, 64, False, BF16, BF16, True, "hnd"),
    (2200, 0, 1, 128, 64, 16, True, F32, F16, True, "nhd"),
    (2048, 5, 1, 96, 96, 32, False, F16, F16, False, "odd"),
    (2050, 2, 1, 256, 256, 64, False, F32, BF16, True, "hnd"),
    (2051, 9, 1, 32, 18, 16, False, BF16, F16, True, "together"),
])
def test_append4_of_a_prompt(dev, T, Hq, Hk, D, R, P, adjacent, src, dst, gains, layout):
    """Tokens enough for a workgroup to take two of them, the last one alone."""
    run_append(dev, T, Hq, Hk, D, R, P, adjacent, src, dst, gains, layout, seed=T)


@pytest.mark.parametrize("src", [F32, BF16, F16])
def test_append4_borders_and_extremes(dev, src):
    """Every border of two codes and its neighbours at several powers, blocks of zeros, of the smallest and largest numbers, with
    an infinity or NaN."""
    T, Hk, D = 12, 1, 64
    info = torch.finfo(src)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], dtype=torch.float64)
    rows = torch.zeros(T, 2 * Hk, D, dtype=torch.float64)
    for t, e in enumerate((0, -3, 5, 9)):
        b = borders * 2.0 ** e
        near = torch.cat([b, b * (1 + info.eps), b * (1 - info.eps), -b])
        rows[t, :, :32] = near
        rows[t, :, 32:] = torch.where(near.abs() > 6.9 * 2.0 ** e, 0.0, near)  # the largest 5
    rows[5, :, 3], rows[5, :, 40] = info.max, -info.max
    rows[6, :, 3], rows[6, :, 40] = info.tiny, info.tiny * info.eps
    rows[7, :, 3], rows[7, :, 40] = math.inf, math.nan
    rows[8, :, 3], rows[8, :, 40] = -math.inf, 1.0
    rows[9] = -0.0
    rows[10] = 7.0
    rows[11, :, ::2] = -7.0 * (1 + info.eps)
    run_append_values(dev, rows.to(src), Hk, D)


def run_append_values(dev, rows, Hk, D):
    T = rows.shape[0]
    cache = kv4_cache(dev, 1, Hk, 16, D)
    k, v = rows[:, :Hk].to(dev), rows[:, Hk:].to(dev)
    kv = torch.empty(T, Hk, D, dtype=BF16, device=dev)
    vv = torch.empty_like(kv)
    bpw.bpw_kv4_append(bpw.PagedKv4(*cache), k, v, torch.arange(T, device=dev), k_values=kv, v_values=vv)
    torch.cuda.synchronize()
    for i, (x, got) in enumerate(((k, kv), (v, vv))):
        codes, power, _ = request_ops.to_codes(f64(x))
        mean = request_ops.from_codes(codes, power)
        assert np.array_equal(cache[2 + i][0, :, :T].transpose(0, 1).cpu().numpy(), power)
        assert np.array_equal(request_ops.unpacked(cache[i][0, :, :T].transpose(0, 1).cpu().numpy()), codes)
        assert np.array_equal(f64(got), mean, equal_nan=True)  # bfloat16 holds them all
    k16, v16 = torch.empty(T, Hk, D, dtype=F16, device=dev), torch.empty(T, Hk, D, dtype=F16, device=dev)
    bpw.bpw_kv4_append(bpw.PagedKv4(*cache), k, v, torch.arange(T, device=dev), v_values=v16)
    bpw.bpw_kv4_append(bpw.PagedKv4(*cache), k, v, torch.arange(T, device=dev), k_values=k16)
    torch.cuda.synchronize()
    assert np.array_equal(f64(v16), torch.tensor(request_ops.from_codes(*request_ops.to_codes(f64(v))[:2])).to(F16).double().numpy(), equal_nan=True)
    assert np.array_equal(f64(k16), f64(v16), equal_nan=True) == np.array_equal(f64(k), f64(v), equal_nan=True)


def attn4_tol(want, mag, q, k, v, D, L, scale, dst):
    """As attn_tol, with weights of two bfloat16 numbers (half a step of the second: 2^-18 of the weight) and exact operands. The
    exponential gives 0 below float32's smallest normal number, 2^-126 of a largest weight that is at least 1: each position may
    lose as much of its value, and its part once more where the parts are joined."""
    ds = (D + 4) * 4 * U * scale * np.linalg.norm(q, axis=-1)[..., None] * (np.max(np.linalg.norm(k, axis=-1)) if k.size else 0)
    chain = 2 * (L / 16 + 64) * U
    rel = 2 * (ds + 2.0 ** -21) + 2 * chain + 2.0 ** -17
    lost = 2 * L * 2.0 ** -126 * (np.max(np.abs(v)) if v.size else 0)
    return rel * mag + lost + half_step(dst) * np.abs(want) * (1 + 64 * U) + smallest(dst), ds[..., 0] + 2.0 ** -21 + chain


class Attn4:
    """One attention call: pages in a scattered order, what no sequence reads with powers of 255 (NaN)."""

    def __init__(self, dev, n_q, lens, Hq, Hk, D, P, dt=BF16, seed=0, layout="hnd", max_pages=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.n_q, self.lens, self.dt = n_q, lens, dt
        B, T = len(n_q), sum(n_q)
        need = [max(0, -(-x // P)) for x in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g)
        width = max(need + [1]) if max_pages is None else max_pages
        table = torch.full((B, width), -7, dtype=I32)
        fill, at = torch.zeros(pages, P, dtype=torch.bool), 0
        for b, n in enumerate(need):
            n = min(n, width)
            table[b, :n] = order[at:at + n].int()
            for i in range(min(lens[b], width * P)):
                fill[table[b, i // P], i % P] = True
            at += n
        self.cache = kv4_cache(dev, pages, Hk, P, D, layout, seed)
        for c in self.cache[2:]:
            c.copy_(torch.where(fill.to(dev)[:, None, :, None], c, 255))
        self.q = (torch.randn(T, Hq, D, generator=g) * 0.3).to(dt).to(dev)
        self.table, self.len_t = table.to(dev), torch.tensor(lens, dtype=I32, device=dev)
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(n_q)]), dtype=I32, device=dev)
        self.out = torch.full((T, Hq, D), 77.0, dtype=dt, device=dev)
        self.lse = torch.full((T, Hq), 77.0, device=dev)
        self.max_q, self.scale = max(max(n_q), 1), None

    def plan(self):
        kv = bpw.PagedKv4(*self.cache)
        n = bpw.bpw_kv4_attn_workspace_bytes(kv, self.q, len(self.n_q), self.max_q, self.table.shape[1])
        ws = torch.full((n,), 255, dtype=U8, device=self.q.device)  # NaN wherever a stale part would be read
        return bpw.Kv4AttnPlan(kv, self.q, self.out, self.table, self.len_t, self.starts, self.max_q, ws, scale=self.scale, lse=self.lse)

    def run(self, what=""):
        self.out.fill_(77.0), self.lse.fill_(77.0)
        self.plan().run()
        torch.cuda.synchronize()
        self.check(what)

    def check(self, what=""):
        q, k, v = f64(self.q), held(self.cache[0], self.cache[2]), held(self.cache[1], self.cache[3])
        D, scale = q.shape[-1], self.scale or q.shape[-1] ** -0.5
        seen = [(self.starts[b].item(), self.starts[b + 1].item()) for b in range(len(self.n_q))]
        out, lse, mag = decode_ops.attention(q, k, v, [], 0, self.table.cpu().numpy(), self.len_t.tolist(), self.starts.tolist(), self.max_q, scale)
        gone = np.ones(len(lse), bool)
        for a, b in seen:
            a, b = min(max(a, 0), len(lse)), min(max(b, 0), len(lse))
            gone[a:min(b, a + self.max_q)] = False
        out[gone], mag[gone], lse[gone] = 77.0, 0.0, 77.0
        L = max(list(self.len_t.tolist()) + [0])
        tol, tol_lse = attn4_tol(out, mag, q, k[np.isfinite(k).all(-1)], v[np.isfinite(v)], D, min(L, k.shape[0] * k.shape[2]), scale,
                                 self.dt)
        within(self.out, out, tol, f"{what} out")
        within(self.lse, lse, tol_lse + 4 * U * np.where(np.isinf(lse), 0, np.abs(lse)), f"{what} lse")


@pytest.mark.parametrize("n_q,lens,Hq,Hk,D,P,dt", [
    ([1], [1], 1, 1, 32, 16, BF16),
    ([1], [700], 20, 5, 128, 16, BF16),
    ([1], [0], 4, 2, 64, 16, F16),                      # nothing to see: zeros
    ([1, 1], [0, 5], 4, 2, 64, 16, F16),
    ([1] * 16, [1 + 31 * i for i in range(16)], 20, 5, 128, 16, BF16),
    ([2, 0, 5, 1, 3], [33, 40, 5, 1, 900], 8, 2, 64, 32, F16),   # an idle sequence
    ([4, 3], [2, 1], 6, 2, 96, 16, BF16),               # fewer positions than query tokens
    ([1, 1, 1], [129, 128, 127], 7, 1, 96, 16, F16),
    ([9, 2], [300, 17], 40, 8, 128, 64, BF16),          # several tiles of rows
    ([3], [260], 40, 1, 128, 128, F16),                 # a group beyond one tile
    ([1, 2], [140, 1000], 4, 4, 256, 16, BF16),
    ([6, 6, 6], [140, 100, 33], 16, 2, 256, 32, F16),
    ([5, 1], [64, 1070], 6, 3, 192, 1024, BF16),
    ([1, 7], [31, 32], 3, 3, 32, 16, F16),
    ([1, 2], [2500, 40], 6, 2, 160, 16, F16),
    ([2] * 40, [3 + 17 * i for i in range(40)], 8, 2, 64, 16, BF16),
])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "together"])
def test_attention4(dev, n_q, lens, Hq, Hk, D, P, dt, layout):
    Attn4(dev, n_q, lens, Hq, Hk, D, P, dt, seed=len(lens) * 7 + D, layout=layout).run()


# Calls of the one-launch kernel and of the two launches, joined by a workgroup or by a wave to a row.
# (n_q, lens, Hq, Hk, D, P, max_pages)
ATTENTION4_PATHS = {
    "short": ([1, 2, 1], [40, 1, 77], 4, 2, 64, 16, 8),
    "short 128": ([5, 0, 1], [40, 1, 300], 12, 2, 128, 16, 20),
    "short 256": ([3, 1], [40, 77], 4, 2, 256, 32, 4),
    "split": ([1, 2, 1], [900, 1, 77], 4, 2, 64, 16, 400),
    "split 128": ([3, 1], [900, 2100], 14, 2, 128, 16, 200),
    "split 256": ([1, 2, 1], [300, 1, 777], 4, 2, 256, 16, 100),
    "split rows": ([3] * 30, [40 + i for i in range(30)], 12, 2, 96, 64, 40),
}


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("path", ATTENTION4_PATHS)
def test_attention4_paths(dev, path, dt):
    """Every path: as it is, with wide and nearly equal scores, with pages missing, with powers of NaN in what a query sees."""
    n_q, lens, Hq, Hk, D, P, pages = ATTENTION4_PATHS[path]
    a = Attn4(dev, n_q, lens, Hq, Hk, D, P, dt, seed=59, max_pages=pages)
    a.run("as it is")
    for a.scale in (2.0, 1e-30):
        a.run(f"scale {a.scale}")
    a.scale = None
    table = a.table.clone()
    a.table[0, 0], a.table[-1, 1] = -1, 2 ** 31 - 1
    a.run("missing pages")
    a.table.fill_(a.cache[0].shape[0])
    a.run("no page")
    a.table.copy_(table)
    a.q[0, 1] = float("nan")
    a.run("a query of NaN")
    a.q[0, 1] = 0.25
    a.cache[2][a.table[0, 1].long(), 0, 3, 0] = 255  # a block of a key that sequence 0 sees (position P + 3)
    a.run("a key of NaN")
    a.cache[2][a.table[0, 1].long(), 0, 3, 0] = 127
    a.cache[3][a.table[0, 1].long(), 0, 3, -1] = 255
    a.run("a value of NaN")
    a.len_t[0] = P + 3
    a.run("and it is not seen")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("layout", ["nhd", "together", "odd"])
@pytest.mark.parametrize("path", ATTENTION4_PATHS)
def test_attention4_paths_of_any_strides(dev, path, layout, dt):
    """Rows of powers apart from one another, or one after another from an odd address: read byte by byte."""
    n_q, lens, Hq, Hk, D, P, pages = ATTENTION4_PATHS[path]
    a = Attn4(dev, n_q, lens, Hq, Hk, D, P, dt, seed=61, max_pages=pages, layout="hnd" if layout == "odd" else layout)
    if layout == "odd":
        for i in (2, 3):
            buf = torch.zeros(a.cache[i].numel() + 1, dtype=U8, device=dev)
            buf[1:] = a.cache[i].flatten()
            a.cache[i] = buf[1:].view(a.cache[i].shape)
    a.run("as it is")
    a.table[0, 0] = -1
    a.run("a page is missing")
    a.table[0, 0] = a.table[0, 1].item()
    a.cache[3][a.table[0, 1].long(), 0, 3, -1] = 255
    a.run("a value of NaN")


@pytest.mark.parametrize("Hq,Hk,D,n,dt", [(3, 1, 64, 5, BF16), (8, 2, 128, 3, F16), (12, 2, 96, 7, BF16), (4, 4, 256, 9, F16)])
def test_attention4_values_of_nan_in_later_drafts(dev, Hq, Hk, D, n, dt):
    """The drafts lie across the end of a 32-position step; those before the NaN are as without it."""
    a = Attn4(dev, [n, 2], [32 + n // 2, 40], Hq, Hk, D, 16, dt, seed=D + n)
    L = a.lens[0]
    a.plan().run()
    clean = a.out.clone()
    a.cache[3][a.table[0, (L - 1) // 16].long(), :, (L - 1) % 16, 0] = 255
    a.run("with NaN")
    keep = n - 1
    assert same_bits(a.out[:keep], clean[:keep]) and same_bits(a.out[n:], clean[n:])
    assert torch.isnan(a.out[n - 1, :, :32].float()).all() and torch.isfinite(a.out[n - 1, :, 32:].float()).all()


def test_attention4_long_splits(dev):
    a = Attn4(dev, [1, 2, 1], [9000, 1, 14000], 16, 8, 64, 64, F16, seed=5)
    a.run()


def test_attention4_many_sequences(dev):
    """Sequence counts past one thread's four and past a wave's 256; most idle or one position long; the most of all."""
    n_q, lens = [i % 3 % 2 for i in range(700)], [(i * 7) % 41 if i % 5 else 0 for i in range(700)]
    Attn4(dev, n_q, lens, 2, 1, 64, 16, F16, seed=3, max_pages=70).run()
    Attn4(dev, [1] * 1024, [1 + i % 3 for i in range(1024)], 2, 1, 256, 16, BF16, seed=31, max_pages=20).run()


def test_attention4_more_workgroups_than_one_launch_over_an_empty_table(dev):
    """A table without columns: nothing to see. A workgroup to each of its (sequence, head, tile) items would be a grid of more
    than 2^32 threads, of which only the first would run."""
    B, T, H, D = 1024, 144, 1024, 32
    kv = bpw.PagedKv4(*kv4_cache(dev, 2, H, 16, D))
    q = torch.randn(T, H, D, device=dev).to(BF16)
    out, lse = torch.full_like(q, 77.0), torch.full((T, H), 77.0, device=dev)
    table, lens = torch.empty(B, 0, dtype=I32, device=dev), torch.full((B,), 5, dtype=I32, device=dev)
    starts = torch.zeros(B + 1, dtype=I32, device=dev)
    starts[-1] = T  # the last sequence has the tokens
    ws = torch.empty(bpw.bpw_kv4_attn_workspace_bytes(kv, q, B, T, 0), dtype=U8, device=dev)
    bpw.bpw_kv4_attn(kv, q, out, table, lens, starts, T, ws, lse=lse)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -math.inf).all()


def test_attention4_runtime_values_out_of_range(dev):
    """Lengths past the table cut, query tokens past the starts or max_q left out."""
    a = Attn4(dev, [1, 1, 3, 2], [100, 64, 40, 208], 4, 2, 64, 16, BF16, seed=9)
    a.len_t[3], a.len_t[2] = 2 ** 31 - 1, -5
    a.run("lengths")
    a.max_q = 2
    a.run("max_q")
    a.starts[-1], a.starts[1] = 100, -3
    a.run("starts")


def test_attention4_offsets_past_32_bits(dev):
    P, Hk, D, far = 16, 2, 64, 2 ** 32 + 8192
    a = Attn4(dev, [1], [40], 4, Hk, D, P, BF16, seed=17)
    n = a.cache[0].shape[0]
    for i, c in enumerate(a.cache):
        stride = far // (n - 1) // 16 * 16 + 16
        buf = torch.empty(stride * (n - 1) + c[0].numel(), dtype=U8, device=dev)
        view = buf.as_strided(c.shape, (stride, c[0, 0].numel(), c.shape[3], 1))
        view.copy_(c)
        a.cache[i] = view
    a.run()
    k, v = torch.randn(1, Hk, D, device=dev), torch.randn(1, Hk, D, device=dev)
    bpw.bpw_kv4_append(bpw.PagedKv4(*a.cache), k, v, torch.tensor([(n - 1) * P + 3], device=dev))
    torch.cuda.synchronize()
    for i, x in ((0, k), (1, v)):
        assert np.array_equal(held(a.cache[i][n - 1:], a.cache[2 + i][n - 1:])[0, :, 3], request_ops.from_codes(*request_ops.to_codes(f64(x[0]))[:2]))


def test_step4_in_a_graph(dev):
    """Append and attention captured once; rows, slots and lengths change between the replays; the same bits on another stream."""
    a = Attn4(dev, [1, 1, 2], [30, 90, 64], 8, 2, 64, 16, BF16, seed=23, spare=6, max_pages=100)
    T, Hk, D, P = 4, 2, 64, 16
    spare = sorted(set(range(a.cache[0].shape[0])) - set(a.table[a.table >= 0].tolist()))
    for b, n in enumerate(a.lens):
        for c in range(-(-n // P), -(-n // P) + 2):
            a.table[b, c] = spare.pop()
    rows = torch.randn(T, 8 + 2 * Hk, D, device=dev)
    slots, pos = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=I32, device=dev)
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    append = bpw.Kv4AppendPlan(bpw.PagedKv4(*a.cache), rows[:, 8:8 + Hk], rows[:, 8 + Hk:], slots, pos, freq, q=rows[:, :8], q_out=a.q)
    attn = a.plan()

    def place():
        """The new tokens are each sequence's last positions."""
        a.len_t += torch.tensor([1, 1, 2], dtype=I32, device=dev)
        lens, tab = a.len_t.tolist(), a.table.tolist()
        own = [(0, lens[0] - 1), (1, lens[1] - 1), (2, lens[2] - 2), (2, lens[2] - 1)]
        slots.copy_(torch.tensor([tab[b][p // P] * P + p % P for b, p in own]))
        pos.copy_(torch.tensor([p for _, p in own], dtype=I32))

    place()
    append.run(), attn.run()
    torch.cuda.synchronize()
    a.check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append.run(), attn.run()
    side = torch.cuda.Stream()
    for i in range(3):
        rows.normal_()
        place()
        graph.replay()
        torch.cuda.synchronize()
        a.check(f"replay {i}")
        got, lse = a.out.clone(), a.lse.clone()
        side.wait_stream(torch.cuda.current_stream())
        append.run(side), attn.run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert same_bits(a.out, got) and same_bits(a.lse, lse)


def two_launches(plan):
    """Runs the plan and says whether it took the split and its join, which alone write the workspace."""
    ws = plan._keep[1]
    ws.fill_(255)
    plan.run()
    torch.cuda.synchronize()
    return bool((ws != 255).any())


def run_split(a, what=""):
    """A call that has to take the two launches."""
    a.out.fill_(77.0), a.lse.fill_(77.0)
    assert two_launches(a.plan()), f"{what}: one launch"
    a.check(what)


def test_attention4_paths_are_those_they_are_named_for(dev):
    for name, (n_q, lens, Hq, Hk, D, P, pages) in ATTENTION4_PATHS.items():
        a = Attn4(dev, n_q, lens, Hq, Hk, D, P, BF16, seed=59, max_pages=pages)
        assert two_launches(a.plan()) == name.startswith("split"), name


@pytest.mark.parametrize("B,n,Hq,Hk,D,positions,two", [
    (1, 1, 32, 8, 64, 1280, False), (1, 1, 32, 8, 64, 1536, True), (4, 1, 32, 8, 64, 1536, False), (4, 1, 32, 8, 64, 2560, True),
    (64, 1, 32, 8, 64, 4096, False), (64, 1, 32, 8, 64, 4160, True), (1, 1, 20, 5, 128, 1280, False), (1, 1, 20, 5, 128, 1344, True),
    (64, 1, 32, 8, 128, 512, False), (128, 1, 32, 8, 128, 512, True), (8, 64, 32, 8, 128, 512, False), (2, 1000, 32, 8, 128, 1024, True),
    (256, 1, 16, 4, 256, 256, False), (512, 1, 16, 4, 256, 256, True), (512, 1, 32, 8, 64, 256, False), (1024, 1, 32, 8, 64, 256, True),
])
def test_attention4_takes_the_launches_that_its_sizes_call_for(dev, B, n, Hq, Hk, D, positions, two):
    """On both sides of every bound of the rule, by the table's columns; few positions of them are in use."""
    a = Attn4(dev, [min(n, 3)] * B, [3 + i % 40 for i in range(B)], 1, 1, D, 64, BF16, seed=67, max_pages=positions // 64)
    a.cache = [c.expand(-1, Hk, -1, -1).contiguous() for c in a.cache]
    T = max(n, min(n, 3) * B)
    a.q = (torch.randn(T, Hq, D, device=dev) * 0.3).to(BF16)
    a.out, a.lse, a.max_q = torch.full_like(a.q, 77.0), torch.full((T, Hq), 77.0, device=dev), n
    assert two_launches(a.plan()) == two
    a.check()


def test_attention4_split_over_many_sequences(dev):
    """Sequence counts past one thread's four and past a wave's 256, most idle or short; the most of all."""
    n_q, lens = [i % 3 % 2 for i in range(700)], [(i * 7) % 41 if i % 5 else 0 for i in range(700)]
    run_split(Attn4(dev, n_q, lens, 2, 1, 64, 16, F16, seed=3, max_pages=1000))
    n_q, lens = [1 + i % 2 for i in range(300)], [(i * 37) % 611 for i in range(300)]
    run_split(Attn4(dev, n_q, lens, 8, 2, 128, 32, BF16, seed=7, max_pages=400))
    run_split(Attn4(dev, [1] * 1024, [1 + i % 3 for i in range(1024)], 2, 1, 256, 16, BF16, seed=31, max_pages=300))
    run_split(Attn4(dev, [1] * 1024, [i % 70 for i in range(1024)], 2, 1, 32, 16, F16, seed=37, max_pages=1000, layout="nhd"))


@pytest.mark.parametrize("D,P,pages,dt", [(64, 16, 1000, BF16), (128, 16, 500, F16), (256, 32, 150, BF16)])
def test_attention4_split_runtime_values_out_of_range(dev, D, P, pages, dt):
    """Lengths past the table cut, query tokens past the starts or max_q left out."""
    a = Attn4(dev, [1, 1, 3, 2], [100, 64, 40, 208], 4, 2, D, P, dt, seed=9, max_pages=pages)
    a.len_t[3], a.len_t[2] = 2 ** 31 - 1, -5
    run_split(a, "lengths")
    a.max_q = 2
    run_split(a, "max_q")
    a.starts[-1], a.starts[1] = 100, -3
    run_split(a, "starts")


@pytest.mark.parametrize("D,Hq,dt", [(64, 8, BF16), (128, 10, F16), (256, 4, BF16)])
def test_attention4_split_in_a_graph_and_on_another_stream(dev, D, Hq, dt):
    """Split and join captured once; queries, pages and lengths change between replays; the same bits on another stream."""
    lens = [300, 2000, 65, 1, 900]
    a = Attn4(dev, [1, 2, 1, 1, 3], lens, Hq, 2, D, 16, dt, seed=23, max_pages=1000)
    plan = a.plan()
    assert two_launches(plan)
    a.check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    side = torch.cuda.Stream()
    for i, order in enumerate(([0, 1, 2, 3, 4], [4, 0, 3, 1, 2], [1, 4, 0, 2, 3])):
        a.q.normal_(std=0.3)
        a.table.copy_(a.table[order].clone())
        a.len_t.copy_(torch.tensor(lens, dtype=I32, device=dev)[order].clone())
        lens = [lens[x] for x in order]
        a.out.fill_(77.0), a.lse.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        a.check(f"replay {i}")
        got, lse = a.out.clone(), a.lse.clone()
        a.out.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        plan.run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert same_bits(a.out, got) and same_bits(a.lse, lse)


# ------------------------------------------------------------------------------ strides of outputs, counts past one launch, no pages


def outputs_of(dev, T, H, D, dt, layout):
    """An output of 77 inside a larger buffer of 77, and that buffer."""
    shape, order = {"wide rows": ((T, H + 3, D + 16), (0, 1, 2)), "heads first": ((H + 1, T + 2, D), (1, 0, 2))}[layout]
    buf = torch.full(shape, 77.0, dtype=dt, device=dev)
    return buf.permute(order)[:T, 1:H + 1, :D] if layout == "wide rows" else buf.permute(order)[1:T + 1, :H], buf


def rest_is_left(view, buf):
    kept = view.clone()
    view.fill_(77.0)
    assert (buf == 77).all()
    return kept


@pytest.mark.parametrize("layout", ["wide rows", "heads first"])
@pytest.mark.parametrize("counts,Hq,Hk,D,dt", [([40, 3], 6, 2, 80, F16), ([900, 300, 120], 16, 2, 128, BF16), ([150], 4, 4, 256, BF16)])
def test_prompt_into_outputs_of_any_strides(dev, counts, Hq, Hk, D, dt, layout):
    p = Prompt(dev, counts, Hq, Hk, D, dt, seed=71)
    p.run()
    out, buf = outputs_of(dev, sum(counts), Hq, D, dt, layout)
    bpw.bpw_prompt_attn(p.q, p.k, p.v, out, p.starts, lse=p.lse)
    torch.cuda.synchronize()
    assert same_bits(rest_is_left(out, buf), p.out)


@pytest.mark.parametrize("layout", ["wide rows", "heads first"])
@pytest.mark.parametrize("T,D,dt", [(33, 64, BF16), (33, 96, F16), (2049, 128, BF16)])
def test_append4_into_outputs_of_any_strides(dev, T, D, dt, layout):
    Hq, Hk = 5, 2
    rows = torch.randn(T, Hq + 2 * Hk, D, device=dev)
    pos, freq = torch.arange(T, dtype=I32, device=dev), 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    cache = [kv4_cache(dev, T // 16 + 1, Hk, 16, D) for _ in range(2)]
    want = [torch.empty(T, h, D, dtype=dt, device=dev) for h in (Hq, Hk, Hk)]
    got = [outputs_of(dev, T, h, D, dt, layout) for h in (Hq, Hk, Hk)]
    for c, (qo, kv, vv) in zip(cache, (want, [x for x, _ in got])):
        bpw.bpw_kv4_append(bpw.PagedKv4(*c), rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:], torch.arange(T, device=dev), pos, freq, q=rows[:, :Hq], q_out=qo,
                           k_values=kv, v_values=vv)
    torch.cuda.synchronize()
    for (view, buf), x in zip(got, want):
        assert same_bits(rest_is_left(view, buf), x)
    assert all(torch.equal(a, b) for a, b in zip(*cache))


@pytest.mark.parametrize("layout", ["wide rows", "heads first"])
@pytest.mark.parametrize("path", ATTENTION4_PATHS)
def test_attention4_into_outputs_of_any_strides(dev, path, layout):
    n_q, lens, Hq, Hk, D, P, pages = ATTENTION4_PATHS[path]
    a = Attn4(dev, n_q, lens, Hq, Hk, D, P, BF16, seed=73, max_pages=pages)
    a.run()
    want = a.out
    a.out, buf = outputs_of(dev, sum(n_q), Hq, D, BF16, layout)
    a.plan().run()
    torch.cuda.synchronize()
    assert same_bits(rest_is_left(a.out, buf), want)


@pytest.mark.parametrize("path", ATTENTION4_PATHS)
def test_attention4_over_a_cache_without_pages(dev, path):
    """Every entry of the table is out of range: zeros."""
    n_q, lens, Hq, Hk, D, P, pages = ATTENTION4_PATHS[path]
    a = Attn4(dev, n_q, lens, Hq, Hk, D, P, F16, seed=79, max_pages=pages)
    a.cache = [c[:0].contiguous() for c in a.cache]
    a.plan().run()
    torch.cuda.synchronize()
    assert (a.out == 0).all() and (a.lse == -math.inf).all()


def test_append4_to_a_cache_without_pages(dev):
    """No slot is inside it; the values are handed out all the same."""
    T, Hk, D = 9, 2, 64
    k, v = torch.randn(T, Hk, D, device=dev), torch.randn(T, Hk, D, device=dev)
    out = [torch.empty(T, Hk, D, dtype=BF16, device=dev) for _ in range(2)]
    kv = bpw.PagedKv4(*(torch.empty(0, Hk, 16, n, dtype=U8, device=dev) for n in (D // 2, D // 2, D // 32, D // 32)))
    bpw.bpw_kv4_append(kv, k, v, torch.arange(T, device=dev), k_values=out[0], v_values=out[1])
    torch.cuda.synchronize()
    for x, got in zip((k, v), out):
        assert np.array_equal(f64(got), request_ops.from_codes(*request_ops.to_codes(f64(x))[:2]))


def test_prompt_of_the_most_sequences(dev):
    """2^20 sequences of one token: more workgroups than one launch takes, and each output is its own value."""
    T, H, D = 1 << 20, 8, 8
    q, k, v = (torch.randn(T, H, D, device=dev).to(BF16) for _ in range(3))
    out, lse = torch.full_like(q, 77.0), torch.full((T, H), 77.0, device=dev)
    bpw.bpw_prompt_attn(q, k, v, out, torch.arange(T + 1, dtype=I32, device=dev), scale=0.5, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out, v)
    s = (q.double() * k.double()).sum(-1) * 0.5
    assert ((lse.double() - s).abs() <= (D + 8) * 2 * U * 0.5 * (q.double() * k.double()).abs().sum(-1) + 4 * U * s.abs() + 2.0 ** -22).all()


def test_append4_of_more_tokens_than_one_launch(dev):
    """2^23 workgroups' tokens and some more, rows that repeat; the last ones alone have slots."""
    T, D, n = (1 << 23) + 5, 32, 64
    rows = torch.randn(n, 1, D, device=dev).to(BF16)
    k = rows.repeat(T // n + 1, 1, 1)[:T]
    slots = torch.full((T,), -1, dtype=torch.int64, device=dev)
    slots[-16:] = torch.arange(16, device=dev)
    cache, small = kv4_cache(dev, 1, 1, 16, D), kv4_cache(dev, 1, 1, 16, D)
    out = torch.full_like(k, 77.0)
    bpw.bpw_kv4_append(bpw.PagedKv4(*cache), k, k, slots, k_values=out)
    want = torch.empty_like(rows)
    bpw.bpw_kv4_append(bpw.PagedKv4(*small), rows, rows, torch.full((n,), -1, dtype=torch.int64, device=dev), k_values=want)
    bpw.bpw_kv4_append(bpw.PagedKv4(*small), k[-16:].contiguous(), k[-16:].contiguous(), torch.arange(16, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(out[:T // n * n].view(-1, n, 1, D), want.expand(T // n, n, 1, D)) and torch.equal(out[T // n * n:], want[:T % n])
    assert all(torch.equal(a, b) for a, b in zip(cache, small))


def test_logprobs_of_more_rows_than_one_launch(dev):
    T, V = (1 << 22) + 7, 3
    x = torch.randn(T, V, device=dev)
    tokens = torch.randint(0, V, (T,), device=dev).int()
    lp, ent, top, top_lp = torch.empty(T, device=dev), torch.empty(T, device=dev), torch.empty(T, 1, dtype=I32, device=dev), torch.empty(T, 1, device=dev)
    bpw.bpw_token_logprobs(x, tokens, lp, None, ent, top, top_lp)
    torch.cuda.synchronize()
    want = torch.log_softmax(x.double(), -1)
    assert torch.equal(top[:, 0].long(), want.argmax(-1))
    # at most three weights: two additions, the exponentials, log and result in half steps of values up to some twenty
    for got, y in ((lp, want.gather(1, tokens[:, None].long())[:, 0]), (ent, -(want.exp() * want).sum(-1)), (top_lp[:, 0], want.amax(-1))):
        assert ((got.double() - y).abs() <= 2.0 ** -20 * (1 + y.abs())).all()


# ------------------------------------------------------------------------------ log probabilities


def logprobs_tol(x, scale):
    """For each row: of log sum exp, and of a log probability at scaled distance d from the largest logit (to be added per entry).
    Weights: a difference, a product by a factor of two roundings (4 U |d|), the exponential 2^-21; the sum: a chain of at most
    8 additions a round of 2048 entries, 64 more across lanes, waves and parts; E|d| and E d^2 under the row's own
    probabilities. A shift raised at the end: 2^-20."""
    with np.errstate(invalid="ignore", over="ignore"):
        d = scale * (x - x.max(-1, keepdims=True))
        p = np.exp(d) / np.exp(d).sum(-1, keepdims=True)
        e1, e2 = np.where(p > 0, p * -d, 0).sum(-1), np.where(p > 0, p * d * d, 0).sum(-1)
        log_l = np.log(np.exp(d).sum(-1))
    chain = U * (8 * (x.shape[1] / 2048 + 2) + 64) + 2.0 ** -20
    lse = chain + 4 * U * e1 + 2 * U * np.abs(log_l)
    return lse, lse + e1 * (2 * chain + 8 * U * e1) + 4 * U * e2 + 4 * U * (np.abs(log_l) + e1)


def run_logprobs(dev, x, tokens, n_top, scale=1.0, ws=None):
    T, V = x.shape
    lp, ent = torch.full((T,), 77.0, device=dev), torch.full((T,), 77.0, device=dev)
    top, top_lp = (torch.full((T, n_top), 77, dtype=t, device=dev) for t in (I32, F32)) if n_top else (None, None)
    n = bpw.bpw_token_logprobs_workspace_bytes(T, V, n_top)
    ws = torch.full((n,), 255, dtype=U8, device=dev)
    xd = x.to(dev)
    bpw.bpw_token_logprobs(xd, tokens.to(dev), lp, ws, ent, top, top_lp, scale)
    torch.cuda.synchronize()
    x64 = f64(x)
    want = list(request_ops.logprobs(x64, tokens.tolist(), n_top, scale))
    for i in (0, 3):  # what float32 does not reach is infinite
        want[i] = np.where(want[i] < -np.finfo(np.float32).max, -np.inf, want[i])
    tol_lse, tol_ent = logprobs_tol(x64, np.float64(np.float32(scale)))
    tol_lse, tol_ent = np.nan_to_num(tol_lse, nan=0, posinf=0), np.nan_to_num(tol_ent, nan=0, posinf=0)
    entry = lambda y, tol: tol + 4 * U * np.where(np.isfinite(y), np.abs(y) + 30, 0)  # noqa: E731
    within(lp, want[0], entry(want[0], tol_lse), "logprobs")
    within(ent, want[1], tol_ent, "entropy")
    if n_top:
        assert np.array_equal(top.cpu().numpy(), want[2])
        within(top_lp, want[3], entry(want[3], tol_lse[:, None]), "top")
    return lp, ent, top, top_lp


@pytest.mark.parametrize("T,V,K,dt,scale", [
    (1, 1, 1, F32, 1.0), (1, 1, 0, BF16, 1.0), (3, 7, 32, F32, 1.0), (5, 63, 5, F16, 0.5), (2, 512, 3, BF16, 1.0), (2, 2047, 20, F32, 2.0),
    (4, 2049, 1, BF16, 1.25), (7, 5001, 32, F32, 1.0), (1, 128256, 5, F32, 1.0), (3, 128257, 20, BF16, 0.7), (2, 300001, 8, F16, 1.0),
    (1100, 4100, 3, F32, 1.0), (1030, 2100, 0, F16, 1.0), (300, 9000, 20, BF16, 1.0),
])
def test_logprobs(dev, T, V, K, dt, scale):
    g = torch.Generator().manual_seed(T + V)
    x = (torch.randn(T, V, generator=g) * 3).to(dt)
    run_logprobs(dev, x, torch.randint(0, V, (T,), generator=g).int(), K, scale)


def test_logprobs_ties_and_orders(dev):
    """Equal logits, zeros of both signs, entries that rise (every one is better than all before) and fall."""
    V = 20000
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(8, V)
    x[0] = torch.randint(0, 3, (V,), generator=g).float()
    x[1] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    x[2], x[3] = torch.arange(V) / 1000.0, -torch.arange(V) / 1000.0
    x[4] = torch.randint(-2, 2, (V,), generator=g).float() * 1e-42  # subnormal
    x[5, 9999] = 50.0
    x[6] = torch.randn(V, generator=g).bfloat16().float()
    x[7, -1], x[7, 0] = 3.0, 3.0
    tokens = torch.tensor([5, 0, V - 1, 0, 7, 9999, 1, V - 1]).int()
    for K in (1, 7, 32):
        run_logprobs(dev, x, tokens, K)
        run_logprobs(dev, x.repeat(200, 1), tokens.repeat(200), K)  # one launch


@pytest.mark.parametrize("many", [1, 150])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_logprobs_masks_and_extremes(dev, dt, many):
    """Vocabularies masked by -inf and by the type's lowest value, rows of nothing, of one entry, of the lowest value alone, with NaN
    or +inf; differences that overflow; tokens outside the vocabulary."""
    V, low = 9000, torch.finfo(dt).min
    g = torch.Generator().manual_seed(5)
    x = torch.randn(10, V, generator=g).to(dt)
    x[0, torch.rand(V, generator=g) < 0.99] = -math.inf
    x[1, torch.rand(V, generator=g) < 0.99] = low
    x[2] = -math.inf
    x[3], x[3, 4321] = -math.inf, 2.0
    x[4] = low
    x[5, 77] = math.nan
    x[6, 8888], x[6, 5] = math.inf, math.nan
    x[7], x[7, 123] = low, torch.finfo(dt).max
    x[8], x[8, 8999] = -math.inf, low
    tokens = torch.tensor([3, 3, 3, 4321, 17, 5, 8888, 5, 8999, V]).int()
    for K in (0, 1, 20):
        run_logprobs(dev, x.repeat(many, 1), tokens.repeat(many), K)
    tokens.copy_(torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31, -1, -1, -1, 123, 0, -1]))
    run_logprobs(dev, x.repeat(many, 1), tokens.repeat(many), 2)
    if dt == F32:
        run_logprobs(dev, x[:5].repeat(many, 1), tokens[:5].repeat(many), 3, 1e-20)
        run_logprobs(dev, x[:4].repeat(many, 1), tokens[:4].repeat(many), 3, 1e3)


def test_logprobs_nearly_certain(dev):
    """One entry has all but 1e-6 of the mass: its log probability and the entropy keep their digits, to float32's steps at 1."""
    x = torch.full((2, 30000), -30.0)
    x[:, 20000] = 0.0
    x[1, 7] = -14.0
    lp, ent, *_ = run_logprobs(dev, x, torch.tensor([20000, 20000]).int(), 2)
    want = request_ops.logprobs(f64(x), [20000, 20000], 0, 1.0)
    assert np.all(np.abs(f64(lp) - want[0]) <= 4 * U) and np.all(np.abs(f64(ent) - want[1]) <= 4 * U + 1e-3 * want[1])


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("gap", [2.0, 8.0, 10.5, 11.0])
def test_logprobs_nearly_certain_after_a_smaller_maximum(dev, dt, gap):
    """A lane meets an entry `gap` below the row's largest long before that one, and nothing else. l is the sum of 1 and one weight,
    off by half a step at 1 (all other additions add zero); the weight, and with it t, by the scale's roundings (3 U of the gap),
    the exponential and the quotient (4 U each): less than 2^-18 of it."""
    V, T = 12000, 1030  # one part a row, the two in the first and the second group of a lane's rounds
    x = torch.full((1, V), -math.inf)
    x[0, 40], x[0, 8192 + 40] = -gap, 0.0
    x = x.to(dt)
    lp, ent = torch.empty(T, device=dev), torch.empty(T, device=dev)
    bpw.bpw_token_logprobs(x.to(dev).expand(T, V), torch.full((T,), 8192 + 40, dtype=I32, device=dev), lp, None, entropy=ent)
    torch.cuda.synchronize()
    want = request_ops.logprobs(f64(x), [8192 + 40], 0, 1.0)
    assert np.all(np.abs(f64(lp) - want[0]) <= U + 2.0 ** -18 * abs(want[0]))
    assert np.all(np.abs(f64(ent) - want[1]) <= U + 2.0 ** -18 * want[1])


@pytest.mark.parametrize("V", [262144, 1 << 20])
@pytest.mark.parametrize("weight", [0.55, 0.61, 0.7, 0.9])
def test_logprobs_of_flat_rows(dev, V, weight):
    """Entries nearly all alike, four above them: roundings of one chain of a lane's sums would all go the same way. l is a chain of 32
    entries, of its groups, of 6 additions over lanes and 4 over waves; a weight is off by a product of two roundings' factor
    (2 U of |d|) and 2^-22; log l by a step of it; the results by half a step."""
    T, low = 1024, math.log(weight)  # (1024 rows: one part a row)
    x = torch.full((1, V), low)
    x[0, :1024:256] = 0.0  # (one to each of the waves that share a row: their shifts are alike)
    lp, ent = torch.empty(T, device=dev), torch.empty(T, device=dev)
    bpw.bpw_token_logprobs(x.to(dev).expand(T, V), torch.full((T,), V - 1, dtype=I32, device=dev), lp, None, entropy=ent)
    torch.cuda.synchronize()
    want = request_ops.logprobs(f64(x), [V - 1], 0, 1.0)
    chain = U * (32 + V / 8192 + 10) + 2 * U * abs(low) + 2.0 ** -22
    tol = chain + 3 * U * abs(want[0][0])
    assert np.all(np.abs(f64(lp) - want[0]) <= tol), (f64(lp)[0] - want[0][0], tol)
    # t / l: both chains, of at most |low| (a mean of the distances), its quotient's and its product's roundings among them
    assert np.all(np.abs(f64(ent) - want[1]) <= tol + abs(low) * (2 * chain + 4 * U)), (f64(ent)[0] - want[1][0], tol)


@pytest.mark.parametrize("offset", [1e4, -3e4, 1e6, 1e9, -1e20, 1e29])
def test_logprobs_far_from_zero(dev, offset):
    """Logits that share a large offset: only their differences count."""
    g = torch.Generator().manual_seed(17)
    x = torch.randn(3, 20001, generator=g) * 3 + offset
    for T in (1, 400):
        run_logprobs(dev, x.repeat(T, 1), torch.tensor([5, 17, 20000]).int().repeat(T), 4, 1.25)


def test_logprobs_rows_of_any_alignment_in_a_graph(dev):
    """Rows inside wider ones, at addresses no vector is aligned to; captured once, contents changed between replays; no tokens."""
    T, V, K = 5, 5003, 6
    wide = torch.randn(T, V + 13, device=dev).to(BF16)
    view = wide[:, 3:V + 3]
    tokens = torch.randint(0, V, (T,), device=dev).int()
    lp, ent, top, top_lp = torch.empty(T, device=dev), torch.empty(T, device=dev), torch.empty(T, K, dtype=I32, device=dev), torch.empty(T, K, device=dev)
    ws = torch.empty(bpw.bpw_token_logprobs_workspace_bytes(T, V, K), dtype=U8, device=dev)
    plan = bpw.TokenLogprobsPlan(view, tokens, lp, ws, ent, top, top_lp)
    plan.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for _ in range(3):
        wide.normal_(), tokens.random_(0, V)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (lp, ent, top, top_lp)]
        want = run_logprobs(dev, view.cpu(), tokens.cpu(), K)
        assert torch.equal(got[2], want[2]) and all(torch.allclose(a, b, rtol=0, atol=1e-5) for a, b in zip(got[:2], want[:2]))
        plan.run()
        assert all(same_bits(a, b) for a, b in zip(got, (lp, ent, top, top_lp)))
    bpw.bpw_token_logprobs(view, None, None, ws, entropy=ent)
    torch.cuda.synchronize()
    assert torch.allclose(ent, want[1], rtol=0, atol=1e-5)


def test_answer_requests_example(dev):
    """The operators together, from packed prompts to scored answers, the steps in a graph."""
    import importlib.util
    import os
    from conftest import ROOT
    spec = importlib.util.spec_from_file_location("answer_requests", os.path.join(ROOT, "examples", "answer_requests.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.main(["--requests", "5", "--longest", "150", "--answer", "4", "--check"])
