"""The decode-step operators on the GPU against the float64 oracle (oracle/decode_ops.py): head norms with
rotation, the paged append, attention over a shared prefix, draft verification.

Tolerances. A rounding to type t is off by at most eps(t) / 2 of the value; float32 errors are counted by
operation where each bound is formed. Integers are equal."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_plane_weight_amd as bpw  # noqa: E402
from oracle import decode_ops  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24  # half a step of float32


def half_step(t):
    return torch.finfo(t).eps / 2


def smallest(t):
    """Half a step of the type's subnormals."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU (they fail rather than skip)"
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    bpw.bpw_device_check()
    return d


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN where none should be, or none where one should"
    bad = np.abs(got - want) > tol
    bad &= ~np.isnan(want) & ~(got == want)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.max(np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0)):.3g} times the bound")


# ------------------------------------------------------------------------------ heads


def heads_tol(want, mag, dst):
    """float32: the sum of squares is a chain of at most 24 roundings (halved by the root), five more make the
    factor and apply it; sine and cosine are off by pi + 3 half steps (the reduced turn, the function);
    the pair's products and their sum add three."""
    return 32 * U * mag + half_step(dst) * np.abs(want) * (1 + 64 * U) + smallest(dst)


def run_rope(dev, T, Hq, Hk, D, R, adjacent, src, dst, gains, layout="fused", seed=0, positions=None):
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn(T, (Hq + Hk) * D + 8, generator=g) * 2).to(src)
    if layout == "odd":  # rows begin one element off
        buf = torch.zeros(T, (Hq + Hk) * D + 9, dtype=src)
        buf[:, 1:] = rows
        rows_d = buf.to(dev)[:, 1:]
    else:
        rows_d = rows.to(dev)
    heads = rows_d[:, :(Hq + Hk) * D].unflatten(1, (Hq + Hk, D))
    q, k = heads[:, :Hq], heads[:, Hq:]
    if positions is None:
        positions = torch.randint(0, 16_000_000, (T,), generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)) if R else None
    qg = 1 + torch.randn(D, generator=g) * 0.2 if gains else None
    kg = 1 + torch.randn(D, generator=g) * 0.2 if gains else None
    if layout == "in place":
        qo, ko = q, k
    else:
        qo = torch.full((T, Hq, D), float("nan"), dtype=dst, device=dev)
        ko = torch.full((T, Hk, D), float("nan"), dtype=dst, device=dev)
    to = lambda x: None if x is None else x.to(dev)  # noqa: E731
    want = [decode_ops.norm_rope(f64(x), None if w is None else f64(w), positions.tolist(), [] if freq is None else freq.tolist(),
                                 1e-5, adjacent) for x, w in ((q, qg), (k, kg))]
    bpw.bpw_qk_norm_rope(q if Hq else None, k if Hk else None, qo if Hq else None, ko if Hk else None, to(positions),
                         to(freq), to(qg), to(kg), eps=1e-5, interleaved=adjacent)
    torch.cuda.synchronize()
    for got, (y, mag), n, name in ((qo, want[0], Hq, "q"), (ko, want[1], Hk, "k")):
        if n:
            within(got, y, heads_tol(y, mag, dst), f"{name} {T}x{n}x{D} rot {R}")


@pytest.mark.parametrize("T,Hq,Hk,D,R,adjacent,src,dst,gains", [
    (1, 20, 5, 128, 128, False, F32, BF16, True),
    (1, 1, 1, 2, 2, True, F32, F32, True),
    (3, 4, 2, 64, 64, True, BF16, BF16, True),
    (5, 3, 1, 80, 32, False, F16, F16, True),
    (5, 3, 1, 80, 80, False, F16, F32, True),
    (7, 5, 5, 96, 96, True, BF16, F32, False),
    (2, 2, 2, 10, 6, False, F32, F16, True),
    (4, 1, 0, 256, 64, False, F32, BF16, True),
    (4, 0, 3, 256, 256, True, F16, BF16, False),
    (2, 2, 1, 1024, 1024, False, F32, F32, True),
    (2, 2, 1, 1022, 510, False, BF16, F16, True),
    (3, 2, 1, 128, 0, False, F32, BF16, True),    # no rotation
    (33, 40, 8, 128, 128, False, BF16, BF16, True),  # more heads than one sweep
    (5, 3, 1, 80, 40, False, BF16, BF16, True),   # pairs that are not whole chunks
    (5, 3, 1, 80, 54, True, F32, F16, True),
    (9, 17, 3, 128, 66, False, F16, F32, True),
    (3, 2, 2, 8, 6, False, BF16, BF16, True),
    (3, 2, 2, 8, 2, True, F32, BF16, False),
    (2, 5, 1, 512, 510, False, BF16, F16, True),
    (2, 5, 1, 504, 130, True, BF16, BF16, True),
    (2053, 2, 1, 72, 34, False, BF16, BF16, True),
    (2051, 3, 1, 64, 64, False, BF16, BF16, True),   # several tokens a workgroup, the last one short
])
def test_norm_rope(dev, T, Hq, Hk, D, R, adjacent, src, dst, gains):
    run_rope(dev, T, Hq, Hk, D, R, adjacent, src, dst, gains)


@pytest.mark.parametrize("layout", ["odd", "in place"])
@pytest.mark.parametrize("D,R,adjacent", [(128, 128, False), (128, 64, True), (36, 20, False), (88, 50, False), (88, 50, True)])
def test_norm_rope_layouts(dev, layout, D, R, adjacent):
    run_rope(dev, 9, 4, 2, D, R, adjacent, BF16, BF16, True, layout)


def test_norm_rope_more_tokens_than_one_launch(dev):
    """A workgroup to a token and more tokens than a launch has workgroups: those about the border and the last are right, and
    every token is written. All tokens read one row; their positions differ."""
    T, H, far = 2 ** 24 + 3, 256, 1 << 20
    q = torch.randn(1, H, 2, device=dev).expand(T, H, 2)
    out = torch.full((T, H, 2), float("nan"), dtype=BF16, device=dev)
    pos = (torch.arange(T, device=dev) % far).int()
    freq = torch.tensor([0.7], dtype=torch.float64, device=dev)
    bpw.bpw_qk_norm_rope(q, None, out, None, pos, freq, q_gain=torch.ones(2, device=dev))
    torch.cuda.synchronize()
    assert all(not torch.isnan(x).any() for x in out.split(1 << 19))
    at = [0, 1, 2 ** 22 - 1, 2 ** 22, 2 ** 24, T - 1]
    want, mag = decode_ops.norm_rope(f64(q[at]), np.ones(2), pos[at].tolist(), freq.tolist(), 1e-6, False)
    within(out[at], want, heads_tol(want, mag, BF16), "tokens")


def test_norm_rope_zero_head_and_far_position(dev):
    """A head of zeros stays zero under eps; the farthest position's angle keeps its digits."""
    q = torch.zeros(1, 2, 64, device=dev)
    out = torch.full_like(q, float("nan"))
    pos = torch.tensor([2 ** 30], dtype=torch.int32, device=dev)
    freq = torch.tensor([2 * math.pi * k / 32 for k in range(32)], dtype=torch.float64, device=dev)
    bpw.bpw_qk_norm_rope(q, None, out, None, pos, freq, q_gain=torch.ones(64, device=dev))
    assert torch.equal(out, q)
    # position 2^30 at frequency 2 pi k / 32 is a whole number of turns: nothing changes, but for the float64
    # product's own rounding: half a step of an angle below 2^33 (2^-21), and 1 / (2 pi) as much again
    q = torch.randn(1, 2, 64, device=dev)
    bpw.bpw_qk_norm_rope(q, None, out, None, pos, freq)
    torch.cuda.synchronize()
    assert (out - q).abs().max().item() <= 2 * q.abs().max().item() * (2.0 ** -19 + 8 * U)


@pytest.mark.parametrize("T,Hq,Hk,D,R,P,src,dst,layout", [
    (1, 20, 5, 128, 128, 16, F32, BF16, "hnd"),
    (64, 4, 2, 64, 64, 32, BF16, BF16, "nhd"),
    (19, 0, 3, 80, 40, 16, F32, F16, "hnd"),
    (300, 0, 1, 128, 128, 1024, F16, F16, "nhd"),
    (9, 6, 2, 36, 36, 64, BF16, F16, "hnd"),
    (5, 2, 2, 256, 256, 128, F32, BF16, "odd"),
])
def test_append(dev, T, Hq, Hk, D, R, P, src, dst, layout):
    g = torch.Generator().manual_seed(T * 31 + D)
    pages = T // P + 4
    if layout == "nhd":
        caches = [torch.randn(pages, P, Hk, D, generator=g).to(dst).to(dev).transpose(1, 2) for _ in range(2)]
    elif layout == "odd":
        caches = [torch.randn(pages * Hk * P * D + 1, generator=g).to(dst).to(dev)[1:].view(pages, Hk, P, D) for _ in range(2)]
    else:  # keys and values of a page side by side
        both = torch.randn(pages, 2, Hk, P, D, generator=g).to(dst).to(dev)
        caches = [both[:, 0], both[:, 1]]
    rows = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(src).to(dev)
    q, k, v = rows[:, :Hq] if Hq else None, rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    slots = torch.randperm(pages * P, generator=g)[:T]
    for i, bad in enumerate((-1, pages * P, -(1 << 60), 1 << 60)):  # padding tokens
        if T > 4 + i:
            slots[4 + i] = bad
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    qg, kg = (1 + torch.randn(D, generator=g) * 0.2 for _ in range(2))
    before = [c.clone() for c in caches]
    qo = torch.full((T, Hq, D), float("nan"), dtype=dst, device=dev) if Hq else None
    bpw.bpw_kv_append(bpw.PagedKv(*caches), k, v, slots.to(dev), pos.to(dev), freq.to(dev), kg.to(dev), q, qo, qg.to(dev))
    torch.cuda.synchronize()
    wk, mk = decode_ops.norm_rope(f64(k), f64(kg), pos.tolist(), freq.tolist(), 1e-6, False)
    tol = heads_tol(wk, mk, dst)
    written = torch.zeros(pages, P, dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * P:
            written[s // P, s % P] = True
            within(caches[0][s // P, :, s % P], wk[t], tol[t], f"key of token {t}")
            assert torch.equal(caches[1][s // P, :, s % P], v[t].to(dst)), f"value of token {t}"
    left = ~written.to(dev)
    for c, b in zip(caches, before):
        assert torch.equal(c.transpose(1, 2)[left].view(torch.int16), b.transpose(1, 2)[left].view(torch.int16))
    if Hq:
        wq, mq = decode_ops.norm_rope(f64(q), f64(qg), pos.tolist(), freq.tolist(), 1e-6, False)
        within(qo, wq, heads_tol(wq, mq, dst), "queries")


# ------------------------------------------------------------------------------ attention


def attn_tol(want, mag, q, k_all, v_all, D, L, scale, dst):
    """Scores: D products accumulated in float32 (two half steps each, in any order), bounded by the norms;
    the exponential and its argument 2^-21; sums and products over L positions: a chain of at most L / 16 + 64
    roundings in each of l and o. The weights are rounded to dst (half a step, or half a step of its
    subnormals where they are smallest: the largest weight is at least 1 in the kernel's scale), and so is the output."""
    ds = (D + 4) * 2 * U * scale * np.linalg.norm(q, axis=-1)[..., None] * (np.max(np.linalg.norm(k_all, axis=-1)) if k_all.size else 0)
    rel = 2 * (ds + 2.0 ** -21) + 2 * (L / 16 + 64) * U * 2 + half_step(dst)
    vmax = np.max(np.abs(v_all)) if v_all.size else 0
    return rel * mag + L * smallest(dst) * vmax + half_step(dst) * np.abs(want) * (1 + 64 * U) + smallest(dst), ds[..., 0] + 2.0 ** -21 + 2 * (L / 16 + 64) * U


class Attn:
    """One attention call's inputs: pages in a scattered order, what no sequence reads filled with NaN."""

    def __init__(self, dev, n_q, lens, Hq, Hk, D, P, prefix, dt=BF16, seed=0, layout="hnd", spare=2, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.n_q, self.lens, self.prefix, self.P, self.dt = n_q, lens, prefix, P, dt
        B, T = len(n_q), sum(n_q)
        need = [max(0, -(-x // P)) for x in lens]
        pp = -(-prefix // P)
        pages = pp + sum(need) + spare
        order = torch.randperm(pages, generator=g)
        width = max(need + [1]) if max_pages is None else max_pages
        table = torch.full((B, width), -7, dtype=torch.int32)
        at = pp
        fill = torch.zeros(pages, P, dtype=torch.bool)
        for b, n in enumerate(need):
            n = min(n, width)
            table[b, :n] = order[at:at + n].int()
            for i in range(min(lens[b], width * P)):
                fill[table[b, i // P], i % P] = True
            at += n
        prefix_pages = order[:pp].int()
        for i in range(prefix):
            fill[prefix_pages[i // P], i % P] = True
        k, v = (torch.randn(pages, P, Hk, D, generator=g).to(dt) for _ in range(2))
        k[~fill], v[~fill] = float("nan"), float("nan")
        if layout == "nhd":
            self.k, self.v = k.to(dev).transpose(1, 2), v.to(dev).transpose(1, 2)
        else:
            self.k, self.v = (x.transpose(1, 2).contiguous().to(dev) for x in (k, v))
        self.q = (torch.randn(T, Hq, D, generator=g) * 1.5).to(dt).to(dev)
        self.table, self.prefix_pages = table.to(dev), prefix_pages.to(dev) if prefix else None
        self.len_t = torch.tensor(lens, dtype=torch.int32, device=dev)
        starts = np.concatenate([[0], np.cumsum(n_q)])
        self.starts = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.out = torch.full((T, Hq, D), 77.0, dtype=dt, device=dev)
        self.lse = torch.full((T, Hq), 77.0, device=dev)
        self.max_q = max(max(n_q), 1)
        self.scale = None

    def plan(self):
        kv = bpw.PagedKv(self.k, self.v)
        n = bpw.bpw_attn_shared_prefix_workspace_bytes(kv, self.q, self.prefix, len(self.n_q), self.max_q, self.table.shape[1])
        ws = torch.full((n,), 255, dtype=torch.uint8, device=self.q.device)  # NaN wherever a stale part would be read
        return bpw.SharedPrefixAttnPlan(kv, self.q, self.out, self.prefix_pages, self.prefix, self.table, self.len_t,
                                        self.starts, self.max_q, ws, scale=self.scale, lse=self.lse)

    def reference(self):
        return decode_ops.attention(f64(self.q), f64(self.k), f64(self.v), [] if not self.prefix else self.prefix_pages.tolist(),
                                    self.prefix, self.table.cpu().numpy(), self.len_t.tolist(), self.starts.tolist(),
                                    self.max_q, self.scale or self.q.shape[-1] ** -0.5)

    def check(self, what=""):
        out, lse, mag = self.reference()
        gone = np.isnan(lse)  # tokens of no sequence: left as they were
        out[gone], mag[gone], lse[gone] = 77.0, 0.0, 77.0
        D, L = self.q.shape[-1], self.prefix + max(list(self.len_t.tolist()) + [0])
        k, v = f64(self.k), f64(self.v)
        k, v = k[~np.isnan(k).any(-1)], v[~np.isnan(v)]
        tol, tol_lse = attn_tol(out, mag, f64(self.q), k, v, D, L, self.scale or D ** -0.5, self.dt)
        within(self.out, out, tol, f"{what} out")
        within(self.lse, lse, tol_lse + 4 * U * np.where(np.isinf(lse), 0, np.abs(lse)), f"{what} lse")


@pytest.mark.parametrize("n_q,lens,Hq,Hk,D,P,prefix,dt", [
    ([1], [1], 1, 1, 8, 16, 0, BF16),
    ([1], [700], 20, 5, 128, 16, 0, BF16),
    ([1], [0], 4, 2, 64, 16, 0, F16),                      # nothing to see: zeros
    ([1, 1], [0, 5], 4, 2, 64, 16, 16, F16),               # only the prefix
    ([1] * 16, [1 + 31 * i for i in range(16)], 20, 5, 128, 16, 517, BF16),
    ([2, 0, 5, 1, 3], [33, 40, 5, 1, 900], 8, 2, 64, 32, 100, F16),   # an idle sequence
    ([4, 3], [2, 1], 6, 2, 80, 16, 0, BF16),               # fewer positions than query tokens
    ([4, 3], [2, 0], 6, 2, 80, 16, 37, BF16),
    ([1, 1, 1], [129, 128, 127], 7, 1, 96, 16, 1, F16),
    ([9, 2], [300, 17], 24, 8, 128, 64, 65, BF16),         # two tiles of rows in a suffix, four in the prefix
    ([3], [260], 40, 1, 128, 128, 129, BF16),              # a group beyond one tile
    ([1, 2], [140, 100], 4, 4, 256, 16, 200, BF16),
    ([6, 6, 6], [140, 100, 33], 16, 2, 256, 32, 300, F16),
    ([5, 1], [64, 70], 6, 3, 192, 1024, 90, BF16),
    ([1, 7], [31, 32], 3, 3, 24, 16, 48, F16),
    ([2] * 40, [3 + 7 * i for i in range(40)], 8, 2, 64, 16, 1400, BF16),
    # prefix rows of 33 .. 64 and beyond: through LDS, with every padding of the head and ragged last tiles of rows
    ([1] * 17, [5] * 17, 8, 2, 128, 16, 333, F16),
    ([3] * 13, [40 + i for i in range(13)], 12, 2, 128, 64, 65, BF16),
    ([4] * 10, [16] * 10, 4, 1, 80, 32, 128, F16),
    ([1] * 45, [1] * 45, 6, 2, 48, 16, 63, BF16),
    ([2] * 10, [70] * 10, 6, 2, 256, 16, 190, BF16),
    ([5] * 9, [70] * 9, 12, 2, 200, 128, 131, F16),
])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_attention(dev, n_q, lens, Hq, Hk, D, P, prefix, dt, layout):
    a = Attn(dev, n_q, lens, Hq, Hk, D, P, prefix, dt, seed=len(lens) * 7 + D, layout=layout)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


@pytest.mark.parametrize("n_q,lens,Hq,Hk,D,P,prefix,pages", [
    # either side of the one-launch kernel's bound on table and prefix, the contents the same
    ([1], [512], 20, 5, 128, 16, 0, 32),
    ([1], [512], 20, 5, 128, 16, 0, 33),
    ([3, 0, 2], [250, 9, 0], 24, 2, 128, 16, 100, 16),
    ([2, 1], [300, 1024], 6, 3, 64, 64, 0, 16),
    ([5, 9], [77, 128], 40, 2, 256, 16, 30, 8),
    ([1, 1], [0, 16], 4, 2, 40, 16, 1, 1),
])
def test_attention_short(dev, n_q, lens, Hq, Hk, D, P, prefix, pages):
    a = Attn(dev, n_q, lens, Hq, Hk, D, P, prefix, F16, seed=sum(lens), max_pages=pages)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_attention_many_sequences(dev):
    """Sequence counts past one thread's four and past a wave's 256; most idle or one position long."""
    n_q = [i % 3 % 2 for i in range(700)]
    lens = [(i * 7) % 41 if i % 5 else 0 for i in range(700)]
    a = Attn(dev, n_q, lens, 2, 1, 64, 16, 20, F16, seed=3)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_attention_long_splits(dev):
    """More units than workgroups in both segments: runs that hold several items and items cut in the middle."""
    a = Attn(dev, [1, 2, 1], [9000, 1, 14000], 16, 8, 64, 64, 7001, F16, seed=5)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_attention_most_parts_of_a_row(dev):
    """A wide prefix in the most pieces beside one suffix that every wave takes a part of: 2112 parts to a row."""
    a = Attn(dev, [1, 1], [122880, 0], 16, 1, 128, 16, 16384, BF16, seed=41)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_attention_runtime_values_out_of_range(dev):
    """Pages that do not exist are hidden, lengths past the table cut, query tokens past the starts or max_q left out."""
    a = Attn(dev, [1, 1, 3, 2], [100, 64, 40, 208], 4, 2, 64, 16, 50, BF16, seed=9)
    a.table[0, 1], a.table[0, 3], a.table[1, 0], a.prefix_pages[1] = -1, 10 ** 9, -2 ** 31, 5000
    a.table[1, 1:] = -1  # nothing left of it
    a.len_t[3] = 2 ** 31 - 1
    a.len_t[2] = -5
    a.plan().run()
    torch.cuda.synchronize()
    a.check("bad pages")
    a.max_q = 2  # the third sequence's last token is left out
    a.out.fill_(77.0), a.lse.fill_(77.0)
    a.plan().run()
    torch.cuda.synchronize()
    a.check("max_q")
    a.starts[-1] = 100
    a.starts[1] = -3
    a.out.fill_(77.0), a.lse.fill_(77.0)
    a.plan().run()
    torch.cuda.synchronize()
    a.check("starts")


@pytest.mark.parametrize("n,D", [(9, 64), (40, 128), (9, 256)])
def test_attention_wide_prefix_with_missing_pages(dev, n, D):
    """The same for a prefix that many rows share: the first, a middle and the last page do not exist."""
    a = Attn(dev, [1] * n, [3] * n, 16, 2, D, 16, 165, F16, seed=n)
    a.prefix_pages[0], a.prefix_pages[4], a.prefix_pages[5], a.prefix_pages[10] = -1, 2 ** 31 - 1, -2 ** 31, a.k.shape[0]
    a.plan().run()
    torch.cuda.synchronize()
    a.check()
    a.prefix_pages.fill_(-1)
    a.len_t.zero_()
    a.plan().run()
    torch.cuda.synchronize()
    a.check("nothing")


def test_attention_wide_peaked_and_wide_scores(dev):
    a = Attn(dev, [2] * 20, [9] * 20, 8, 2, 128, 16, 517, BF16, seed=29)
    a.k *= torch.linspace(0.1, 6, a.k.shape[0], device=dev).to(BF16)[:, None, None, None]
    for a.scale in (2.0, 1e-30):
        a.plan().run()
        torch.cuda.synchronize()
        a.check(str(a.scale))


def test_attention_peaked_and_wide_scores(dev):
    """Scores far above and below one another, and rising along the positions, so that the running maximum
    is raised many times; and a scale that makes all weights equal."""
    a = Attn(dev, [1, 2], [300, 177], 4, 2, 128, 16, 90, BF16, seed=11)
    ramp = torch.linspace(0.1, 6, a.k.shape[0], device=dev).to(BF16)
    a.k *= ramp[:, None, None, None]
    a.scale = 2.0
    a.plan().run()
    torch.cuda.synchronize()
    a.check("wide")
    a.scale = 1e-30
    a.plan().run()
    torch.cuda.synchronize()
    a.check("flat")


def test_attention_nan_and_infinity_where_seen(dev):
    """A NaN key that a query sees makes its output NaN, and no other sequence's."""
    a = Attn(dev, [1, 1], [50, 60], 4, 2, 64, 16, 0, BF16, seed=13)
    a.k[a.table[0, 2].long(), 0, 3] = float("nan")  # head 0, position 35 of sequence 0
    a.plan().run()
    torch.cuda.synchronize()
    got = a.out.float()
    assert torch.isnan(got[0, :2]).all() and not torch.isnan(got[0, 2:]).any() and not torch.isnan(got[1]).any()


# Calls by the path they take: one launch; two, joined by a workgroup or by a wave to a row; a prefix of 64 and of 128 rows
# through LDS. (n_q, lens, Hq, Hk, D, P, prefix, max_pages)
ATTENTION_PATHS = {
    "short": ([1, 2, 1], [40, 1, 77], 4, 2, 64, 16, 20, 8),
    "narrow": ([1, 2, 1], [900, 1, 77], 4, 2, 64, 16, 20, 64),
    "narrow 256": ([1, 2, 1], [300, 1, 77], 4, 2, 256, 16, 40, 64),
    "narrow rows": ([3] * 30, [40 + i for i in range(30)], 12, 2, 128, 64, 65, 8),
    "wide 64": ([1] * 12, [40] * 11 + [1], 8, 2, 128, 16, 3333, 4),
    "wide 128": ([3] * 13, [40 + i for i in range(12)] + [3], 12, 2, 128, 64, 3333, 1),
    "wide 128, padded": ([3] * 13, [40 + i for i in range(12)] + [3], 12, 2, 80, 32, 3333, 2),
    "wide 64, small": ([1] * 30, [40] * 29 + [1], 4, 2, 48, 16, 9000, 4),
    "wide 64, large": ([2] * 10, [70] * 9 + [2], 6, 2, 256, 16, 3333, 5),
    "wide 128, large": ([5] * 9, [70] * 8 + [5], 12, 2, 200, 128, 3333, 1),
}


def check_with_nan(a, what):
    """As Attn.check, where every token belongs to a sequence: NaN has to be where the reference has it, in out and lse."""
    out, lse, mag = a.reference()
    D, L = a.q.shape[-1], a.prefix + max(a.lens)
    q, k, v = f64(a.q), f64(a.k), f64(a.v)
    tol, tol_lse = attn_tol(out, mag, q, k[np.isfinite(k).all(-1)], v[np.isfinite(v)], D, L, a.scale or D ** -0.5, a.dt)
    within(a.out, out, tol, f"{what} out")
    within(a.lse, lse, tol_lse + 4 * U * np.abs(lse), f"{what} lse")


@pytest.mark.parametrize("layout,dt", [("hnd", BF16), ("nhd", F16)])
@pytest.mark.parametrize("path", ATTENTION_PATHS)
def test_attention_paths(dev, path, layout, dt):
    """Every path: as it is, with scores that rise along the pages and with nearly equal weights, and with pages missing: the first,
    some in the middle and the last of the prefix, one of a sequence's, all of them."""
    n_q, lens, Hq, Hk, D, P, prefix, pages = ATTENTION_PATHS[path]
    a = Attn(dev, n_q, lens, Hq, Hk, D, P, prefix, dt, seed=59, layout=layout, max_pages=pages)

    def run(what):
        a.out.fill_(77.0), a.lse.fill_(77.0)
        a.plan().run()
        torch.cuda.synchronize()
        a.check(what)

    run("as it is")
    flat_k = a.k.clone()
    a.k *= torch.linspace(0.1, 6, a.k.shape[0], device=dev).to(dt)[:, None, None, None]
    for a.scale in (2.0, 1e-30):
        run(f"scale {a.scale}")
    a.k, a.scale = flat_k, None
    last = a.prefix_pages.numel() - 1
    for i, bad in ((0, -1), (last // 2, 2 ** 31 - 1), (last // 2 + 1, -2 ** 31), (last, a.k.shape[0])):
        a.prefix_pages[min(i, last)] = bad
    a.table[0, 0] = -1
    run("missing pages")
    a.prefix_pages.fill_(-1)
    run("no prefix page")
    a.table.fill_(a.k.shape[0])
    run("no page")


@pytest.mark.parametrize("path", ATTENTION_PATHS)
def test_attention_nan_scores_are_not_nothing_seen(dev, path):
    """Rows whose scores are all NaN in a part of their positions, or in all: a query of NaN, the one key a sequence has of its
    own, all keys of a sequence or of the prefix, a wave's step of them. out and lse are NaN, and no other row's."""
    n_q, lens, Hq, Hk, D, P, prefix, pages = ATTENTION_PATHS[path]
    a = Attn(dev, n_q, lens, Hq, Hk, D, P, prefix, BF16, seed=43, max_pages=pages)
    clean_q, clean_k = a.q.clone(), a.k.clone()

    def row(b, pos):  # a position of sequence b (None: of the prefix), of key/value head 0
        page = (a.prefix_pages if b is None else a.table[b])[pos // P].long()
        return page, 0, pos % P

    def run(what):
        a.plan().run()
        torch.cuda.synchronize()
        assert np.isnan(f64(a.lse)).any()
        check_with_nan(a, what)
        a.q.copy_(clean_q), a.k.copy_(clean_k)

    a.q[0, 1] = float("nan")
    run("query")
    one = int(np.argmin(lens))
    for pos in range(lens[one]):
        a.k[row(one, pos)] = float("nan")
    run("the sequence of the fewest positions")
    for pos in range(lens[0]):
        a.k[row(0, pos)] = float("nan")
    run("a sequence")
    for pos in range(prefix):
        a.k[row(None, pos)] = float("nan")
    run("the prefix")
    for pos in range(min(32, prefix)):
        a.k[row(None, pos)] = float("nan")
    run("a step of the prefix")


@pytest.mark.parametrize("path", ATTENTION_PATHS)
def test_attention_float16_weights_far_below_the_largest(dev, path):
    """One position of 32 has all but 2^-25 of the weight and values of zero: the output is what the others add. Weights are
    rounded to float16 from 2^6 at the largest, so a step of its subnormals is 2^-30 of it, and half of one the error."""
    n_q, lens, Hq, Hk, D, P, prefix, pages = ATTENTION_PATHS[path]
    a = Attn(dev, n_q, lens, Hq, Hk, D, P, prefix, F16, seed=53, max_pages=pages)
    a.scale = 1.0
    a.q.zero_()
    a.q[..., 0] = 1.0
    a.k.copy_(torch.where(torch.isnan(a.k), a.k, 0.0))
    a.v.copy_(a.v.abs() + 500.0)
    for pages_of, n in [(a.prefix_pages, prefix)] + [(a.table[b], n) for b, n in enumerate(lens)]:
        for pos in range(0, n, 32):
            a.k[pages_of[pos // P].long(), :, pos % P, 0] = 17.5  # exp(-17.5) = 2^-25.2
            a.v[pages_of[pos // P].long(), :, pos % P] = 0.0
    a.plan().run()
    torch.cuda.synchronize()
    out, lse, mag = a.reference()
    assert (out > 1e-4).all()
    k, v = f64(a.k), f64(a.v)
    v = v[np.isfinite(v)]
    _, tol_lse = attn_tol(out, mag, f64(a.q), k[np.isfinite(k).all(-1)], v, D, prefix + max(lens), 1.0, F16)
    # float32 errors as of lse, twice; the weights above and at the subnormals (32 to one of 2^6); the output
    tol = mag * (2 * tol_lse[..., None] + half_step(F16)) + 32 * 2.0 ** -31 * v.max() + half_step(F16) * out + smallest(F16)
    within(a.out, out, tol, "out")
    within(a.lse, lse, tol_lse + 4 * U * np.abs(lse), "lse")


@pytest.mark.parametrize("Hq,Hk,D,n,dt", [(3, 1, 64, 5, BF16), (8, 2, 128, 3, F16), (12, 2, 80, 7, BF16), (4, 4, 256, 9, F16)])
def test_attention_values_that_are_not_finite_in_later_drafts(dev, Hq, Hk, D, n, dt):
    """NaN and infinities in the values of drafts: the tokens before them are as without, the others show them.
    The drafts lie across the end of a 32-position step."""
    a = Attn(dev, [n, 2], [32 + n // 2, 40], Hq, Hk, D, 16, 21, dt, seed=D + n)
    L = a.lens[0]
    a.plan().run()
    clean = a.out.clone()
    row = lambda pos: (a.table[0, pos // 16].long(), slice(None), pos % 16)  # noqa: E731
    a.v[row(L - 1)] = float("nan")
    a.v[row(L - 2)] = float("inf")
    a.plan().run()
    torch.cuda.synchronize()
    got = a.out.float()
    assert torch.equal(a.out[n:].view(torch.int16), clean[n:].view(torch.int16))  # the other sequence
    keep = n - 2  # tokens that see neither
    assert torch.isfinite(got[:keep]).all() and not torch.isfinite(got[n - 2]).any() and torch.isnan(got[n - 1]).all()
    a.out = a.out[:keep]
    a.lse, a.q = a.lse[:keep], a.q[:keep]  # the reference of those alone: drafts they do not see cut off
    a.n_q, a.lens = [keep], [L - 2]
    a.table, a.len_t = a.table[:1], torch.tensor([L - 2], dtype=torch.int32, device=dev)
    a.starts = torch.tensor([0, keep], dtype=torch.int32, device=dev)
    a.v[row(L - 1)] = float("nan")
    a.v[row(L - 2)] = float("nan")
    a.check()


def test_attention_offsets_past_32_bits(dev):
    """Pages further apart than 2^31 elements."""
    P, Hk, D, far = 16, 2, 64, 2 ** 31 + 4096
    a = Attn(dev, [1], [40], 4, Hk, D, P, 20, BF16, seed=17)
    n = a.k.shape[0]
    views = []
    for src in (a.k, a.v):
        stride = far // (n - 1) // 8 * 8 + 8
        buf = torch.empty(stride * (n - 1) + Hk * P * D, dtype=BF16, device=dev)
        view = buf.as_strided((n, Hk, P, D), (stride, P * D, D, 1))
        view.copy_(src)
        views.append(view)
    assert views[0].stride(0) * (n - 1) * 2 > 2 ** 32
    a.k, a.v = views
    slots = torch.tensor([(n - 1) * P + 3], device=dev)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()
    k, v = torch.randn(1, Hk, D, device=dev), torch.randn(1, Hk, D, device=dev)
    bpw.bpw_kv_append(bpw.PagedKv(a.k, a.v), k, v, slots)
    torch.cuda.synchronize()
    assert torch.equal(a.k[n - 1, :, 3], k[0].to(BF16)) and torch.equal(a.v[n - 1, :, 3], v[0].to(BF16))


def test_attention_same_bits_each_time_and_on_another_stream(dev):
    a = Attn(dev, [1, 3, 2], [500, 320, 77], 8, 2, 128, 16, 700, BF16, seed=19)
    plan = a.plan()
    plan.run()
    first, lse = a.out.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.out.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        plan.run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a.out.view(torch.int16), first.view(torch.int16)) and torch.equal(a.lse, lse)


def test_step_in_a_graph(dev):
    """Append and attention captured once; positions, slots, lengths and tables change between the replays."""
    a = Attn(dev, [1, 1, 2], [30, 90, 64], 8, 2, 64, 16, 40, BF16, seed=23, spare=6, max_pages=8)
    T, Hk, D, P = 4, 2, 64, 16
    spare = sorted(set(range(a.k.shape[0])) - set(a.table[a.table >= 0].tolist()) - set(a.prefix_pages.tolist()))
    for b, n in enumerate(a.lens):
        for c in range(-(-n // P), -(-n // P) + 2):
            a.table[b, c] = spare.pop()
    rows = torch.randn(T, 8 + 2 * Hk, D, device=dev)
    slots, pos = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    append = bpw.KvAppendPlan(bpw.PagedKv(a.k, a.v), rows[:, 8:8 + Hk], rows[:, 8 + Hk:], slots, pos, freq, q=rows[:, :8], q_out=a.q)
    attn = a.plan()
    a.len_t += torch.tensor([1, 1, 2], dtype=torch.int32, device=dev)

    def place():
        """The new tokens are each sequence's last positions."""
        lens, tab = a.len_t.tolist(), a.table.tolist()
        own = [(0, lens[0] - 1), (1, lens[1] - 1), (2, lens[2] - 2), (2, lens[2] - 1)]
        slots.copy_(torch.tensor([tab[b][p // P] * P + p % P for b, p in own]))
        pos.copy_(torch.tensor([a.prefix + p for _, p in own], dtype=torch.int32))

    place()
    append.run(), attn.run()
    torch.cuda.synchronize()
    a.check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append.run(), attn.run()
    for i in range(3):
        rows.normal_()
        a.len_t += torch.tensor([1, 1, 2], dtype=torch.int32, device=dev)
        place()
        graph.replay()
        torch.cuda.synchronize()
        a.check(f"replay {i}")
        got = a.out.clone()
        append.run(), attn.run()
        assert torch.equal(got.view(torch.int16), a.out.view(torch.int16))


@pytest.mark.parametrize("n", [3, 60])
def test_attention_without_own_positions(dev, n):
    """A page table of no columns: the prefix is all there is."""
    a = Attn(dev, [1] * n, [0] * n, 8, 4, 64, 32, 75, F16, seed=37, max_pages=0)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_attention_most_sequences(dev):
    """The most sequences a call takes, with the largest tables in LDS beside the largest tiles."""
    n = 1024
    a = Attn(dev, [1] * n, [1 + i % 3 for i in range(n)], 2, 1, 256, 16, 130, BF16, seed=31)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


@pytest.mark.parametrize("tokens,lens,Hq,Hk,prefix,pages", [
    (2049, 0, 32, 2, 600, 0),     # the join: 2^26 query rows, idle sequences' among them
    (4097, 9, 32, 32, 5, 1),      # few positions, 2^23 tiles
])
def test_attention_more_rows_than_one_launch(dev, tokens, lens, Hq, Hk, prefix, pages):
    """The last of the most sequences holds all tokens, so that its rows lie past the first launch's."""
    n = 1024
    a = Attn(dev, [0] * (n - 1) + [tokens], [0] * (n - 1) + [lens], Hq, Hk, 8, 16, prefix, F16, seed=47, max_pages=pages)
    a.plan().run()
    torch.cuda.synchronize()
    a.check()


def test_speculative_step_example(dev):
    """The operators together, from ternary projections to accepted tokens."""
    import importlib.util
    import os
    from conftest import ROOT
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.main(["--sequences", "4", "--drafts", "3", "--prefix", "200", "--suffix", "40", "--check"])


# ------------------------------------------------------------------------------ draft verification


def run_verify(dev, target, draft, tokens, u, r, n_draft=None):
    B, K1, V = target.shape
    out = torch.full((B, K1), 99, dtype=torch.int32, device=dev)
    acc = torch.full((B,), 99, dtype=torch.int32, device=dev)
    ws = torch.full((bpw.bpw_verify_draft_workspace_bytes(B, V),), 255, dtype=torch.uint8, device=dev)
    to = lambda x: None if x is None else x.to(dev)  # noqa: E731
    bpw.bpw_verify_draft(to(target), to(draft), to(tokens), to(u), to(r), out, acc, ws, to(n_draft))
    torch.cuda.synchronize()
    want, n = decode_ops.verify(f64(target), None if draft is None else f64(draft), tokens.numpy(),
                                None if n_draft is None else n_draft.numpy(), u.numpy(), r.numpy())
    assert np.array_equal(acc.cpu().numpy(), n)
    assert np.array_equal(out.cpu().numpy(), want)


def verify_case(B, K, V, dt, seed, noise=0.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=g) * 2
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits[:, :K] + torch.randn(B, K, V, generator=g) * noise, -1).to(dt)
    tokens = torch.multinomial(draft.float().reshape(B * K, V), 1, generator=g).view(B, K).int()
    return target, draft, tokens, torch.rand(B, K, generator=g), torch.rand(B, generator=g)


@pytest.mark.parametrize("B,K,V,dt", [(1, 1, 1, F32), (3, 2, 7, F32), (5, 4, 255, BF16), (4, 8, 4096, F32), (7, 3, 4097, F16),
                                      (2, 64, 300, F32), (9, 5, 32001, F32), (2, 4, 128256, BF16)])
@pytest.mark.parametrize("certain", [False, True])
def test_verify(dev, B, K, V, dt, certain):
    target, draft, tokens, u, r = verify_case(B, K, V, dt, B * 100 + K)
    if certain:  # certain drafts are accepted by the target's probability alone
        tokens = target[:, :K].float().argmax(-1).int()
        draft = None
    run_verify(dev, target, draft, tokens, u, r)
    n = torch.tensor([(i * 3) % (K + 3) - 1 for i in range(B)], dtype=torch.int32)  # below 0 and past K too
    run_verify(dev, target, draft, tokens, u, r, n)
    run_verify(dev, target, draft, tokens, u * 0, r)       # everything with mass is accepted
    run_verify(dev, target, draft, tokens, u * 0 + 2, r)   # next to nothing is


@pytest.mark.parametrize("V", [5000, 9000])
def test_verify_borders(dev, V):
    """Rows with zeros, NaN, infinities and negatives; r at 0 and at 1; a draft equal to the target; rows of no
    mass; drafted tokens outside the vocabulary; the mass in one entry, first and last."""
    K = 2
    g = torch.Generator().manual_seed(3)
    base = torch.zeros(8, K + 1, V)
    base[:, :, 4000:4100] = torch.rand(8, K + 1, 100, generator=g)
    base[1, :, 0] = 5.0
    base[2, :, V - 1] = 5.0
    base[3, :, 4050] = float("nan")
    base[3, :, 4051] = -3.0
    base[3, :, 4052] = float("inf")
    base[4] = 0.0
    draft = base[:, :K].clone()
    draft[0] *= 0.5
    draft[5] = 0.0
    tokens = torch.full((8, K), 4020, dtype=torch.int32)
    tokens[6, 0], tokens[7, 1] = -1, V
    for r in (0.0, 0.25, 1.0 - 2.0 ** -24, 1.0):
        for u in (0.0, 0.9999, 1.0):
            run_verify(dev, base, draft, tokens, torch.full((8, K), u), torch.full((8,), r))
            run_verify(dev, base, None, tokens, torch.full((8, K), u), torch.full((8,), r))


@pytest.mark.parametrize("V", [262145, 300001, 600000])
def test_verify_more_than_a_wave_of_chunks(dev, V):
    """Vocabularies of more than 64 chunks of 4096, the border in each 64 of them; mass only past the first 64; a draft that
    takes all of it."""
    target, draft, tokens, u, r = verify_case(5, 2, V, F32, V)
    target[2, :, :262144] = 0.0
    draft[3] = target[3, :2]
    for x in (r, r * 0, r * 0 + 0.999, r * 0 + (1.0 - 2.0 ** -24), r * 0 + 1.0):
        run_verify(dev, target, draft, tokens, u, x)
    run_verify(dev, target, None, tokens, u, r)


def test_verify_border_within_a_rounding_of_a_chunk(dev):
    """Masses 1, 2^-53 and 2^-53 in the chunks 0, 2 and 3, halves in 10 and 70, r = 1/2: the border 1 + 2^-53 is passed in chunk 3,
    by less than float64 tells from chunk 2's end, and not 60 chunks later."""
    V, at = 71 * 4096, {0: 1.0, 2: 2.0 ** -53, 3: 2.0 ** -53, 10: 0.5, 70: 0.5}
    target = torch.zeros(1, 2, V, device=dev)
    for chunk, mass in at.items():
        target[:, 1, chunk * 4096 + 7] = mass
    target[0, 0, 5] = 1.0
    out, acc = torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.empty(bpw.bpw_verify_draft_workspace_bytes(1, V), dtype=torch.uint8, device=dev)
    bpw.bpw_verify_draft(target, None, torch.full((1, 1), 5, dtype=torch.int32, device=dev), torch.zeros(1, 1, device=dev),
                         torch.full((1,), 0.5, device=dev), out, acc, ws)
    torch.cuda.synchronize()
    assert acc.tolist() == [1] and out.tolist() == [[5, 3 * 4096 + 7]]


def test_verify_strided_rows(dev):
    """Rows inside wider ones, steps out of order in memory, at an address no vector is aligned to."""
    target, draft, tokens, u, r = verify_case(3, 2, 5001, F32, 77)
    wide = torch.zeros(3, 3, 5008, device=dev)
    wide[:, :, 3:5004] = target.to(dev)
    view = wide[:, :, 3:5004]
    turned = draft.to(dev).transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(3, 3, dtype=torch.int32, device=dev)
    acc = torch.empty(3, dtype=torch.int32, device=dev)
    ws = torch.empty(bpw.bpw_verify_draft_workspace_bytes(3, 5001), dtype=torch.uint8, device=dev)
    plan = bpw.DraftVerifyPlan(view, turned, tokens.to(dev), u.to(dev), r.to(dev), out, acc, ws)
    graph = torch.cuda.CUDAGraph()
    plan.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.run()
    want, n = decode_ops.verify(f64(target), f64(draft), tokens.numpy(), None, u.numpy(), r.numpy())
    for _ in range(3):
        out.fill_(99), acc.fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(acc.cpu().numpy(), n)
