"""The refusals of prompt attention, the 4-bit cache and token log probabilities, on the host: every argument check comes before any
device work. Also the oracle's own pins against closed forms."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
bpw = pytest.importorskip("bit_plane_weight_amd")
from bit_plane_weight_amd import _lib  # noqa: E402
from oracle import request_ops  # noqa: E402
from test_decode_host import FakeGpu, fake, no_device, status_of  # noqa: E402, F401

F32, BF16, F16, I32, U8 = torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8


def workspace(n):
    ws = FakeGpu(torch.zeros(n + 256, dtype=U8))
    ws.t = ws.t[-ws.t.data_ptr() % 256:][:n]
    return ws


def refused(make, field, value, on="_args"):
    p = make()
    target = p._args if on == "_args" else getattr(p._args, on)
    setattr(target, field, value)
    return status_of(lambda: p.run(0))


def test_struct_sizes_match_the_header():
    sizes = {"BpwPromptAttnArgs": 160, "BpwPagedKv4": 144, "BpwKv4AppendArgs": 400, "BpwKv4AttnArgs": 272, "BpwTokenLogprobsArgs": 80}
    assert {n: ctypes.sizeof(getattr(_lib, n)) for n in sizes} == sizes


# ------------------------------------------------------------------------------ whole prompts


def prompt_plan(T=5, Hq=4, Hk=2, D=64, dt=BF16, seqs=2, out=None, **kw):
    return bpw.PromptAttnPlan(fake(T, Hq, D, dtype=dt), fake(T, Hk, D, dtype=dt), fake(T, Hk, D, dtype=dt),
                              out or fake(T, Hq, D, dtype=dt), fake(seqs + 1, dtype=I32), **kw)


def test_prompt_refusals():
    for ok in ({}, {"T": 0}, {"D": 8}, {"D": 256}, {"dt": F16, "seqs": 1}, {"lse": fake(5, 4, dtype=F32)}, {"Hq": 1, "Hk": 1}):
        assert status_of(lambda: prompt_plan(**ok).run(0)) is None, ok
    assert status_of(lambda: prompt_plan(D=12).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: prompt_plan(D=264).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: prompt_plan(dt=F32).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: prompt_plan(Hq=5).run(0)) == _lib.E_INVAL
    assert status_of(lambda: prompt_plan(out=fake(5, 4, 64, dtype=F16)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: prompt_plan(out=fake(5, 3, 64)).run(0)) == _lib.E_INVAL
    for scale in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert status_of(lambda: prompt_plan(scale=scale).run(0)) == _lib.E_INVAL, scale
    for field, value, want in (("n_tokens", -1, _lib.E_INVAL), ("n_seqs", 0, _lib.E_UNSUPPORTED), ("n_seqs", (1 << 20) + 1, _lib.E_UNSUPPORTED),
                               ("d_starts", None, _lib.E_INVAL), ("d_lse", 2, _lib.E_INVAL), ("n_tokens", 1 << 30, _lib.E_UNSUPPORTED)):
        assert refused(prompt_plan, field, value) == want, field
    for on in ("q", "k", "v", "out"):
        assert refused(prompt_plan, "token_stride", 132, on) == _lib.E_INVAL
        assert refused(prompt_plan, "d", None, on) == _lib.E_INVAL
        assert refused(prompt_plan, "d", 8, on) == _lib.E_INVAL
        assert refused(prompt_plan, "head_stride", -8, on) == _lib.E_INVAL
    assert refused(prompt_plan, "token_stride", (1 << 24) + 8, "k") == _lib.E_UNSUPPORTED
    assert refused(prompt_plan, "heads", 1, "v") == _lib.E_INVAL
    assert _lib.lib().bpw_prompt_attn(None, None) == _lib.E_INVAL
    with pytest.raises(ValueError, match="starts"):
        bpw.PromptAttnPlan(fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), fake(1, dtype=I32))
    with pytest.raises(TypeError, match="starts"):
        bpw.PromptAttnPlan(fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), fake(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="k must be"):
        bpw.PromptAttnPlan(fake(2, 1, 8), fake(1, 1, 8), fake(2, 1, 8), fake(2, 1, 8), fake(2, dtype=I32))
    with pytest.raises(ValueError, match="lse"):
        prompt_plan(lse=fake(5, 5, dtype=F32))
    with pytest.raises(ValueError, match="expanded"):
        prompt_plan(out=FakeGpu(torch.zeros(1, 4, 64, dtype=BF16).expand(5, 4, 64)))


def test_tensors_of_several_devices_are_refused():
    elsewhere = fake(2, dtype=I32)
    elsewhere.device = torch.device("meta")
    with pytest.raises(ValueError, match="several devices"):
        bpw.PromptAttnPlan(fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), fake(1, 1, 8), elsewhere)


# ------------------------------------------------------------------------------ a cache held in 4 bits


def kv4(pages=4, heads=2, page=16, dim=64):
    return bpw.PagedKv4(*(fake(pages, heads, page, dim // n, dtype=U8) for n in (2, 2, 32, 32)))


def append_plan(kv=None, T=3, Hk=2, D=64, R=64, src=F32, **kw):
    return bpw.Kv4AppendPlan(kv or kv4(), fake(T, Hk, D, dtype=src), fake(T, Hk, D, dtype=src), fake(T, dtype=torch.int64),
                             fake(T, dtype=I32), fake(R // 2, dtype=torch.float64), **kw)


def test_paged_kv4_refusals():
    with pytest.raises(TypeError, match="k_scales"):
        bpw.PagedKv4(fake(1, 1, 16, 32, dtype=U8), fake(1, 1, 16, 32, dtype=U8), fake(1, 1, 16, 2, dtype=I32), fake(1, 1, 16, 2, dtype=U8))
    with pytest.raises(ValueError, match="v_scales must be"):
        bpw.PagedKv4(fake(1, 1, 16, 32, dtype=U8), fake(1, 1, 16, 32, dtype=U8), fake(1, 1, 16, 2, dtype=U8), fake(1, 1, 16, 1, dtype=U8))
    with pytest.raises(ValueError, match="multiple of 32"):
        kv4(dim=40)
    with pytest.raises(ValueError, match="contiguous"):
        bpw.PagedKv4(FakeGpu(torch.zeros(1, 1, 32, 16, dtype=U8).transpose(2, 3)), fake(1, 1, 16, 32, dtype=U8), fake(1, 1, 16, 2, dtype=U8),
                     fake(1, 1, 16, 2, dtype=U8))
    with pytest.raises(ValueError, match="expanded"):
        bpw.PagedKv4(FakeGpu(torch.zeros(1, 1, 16, 32, dtype=U8).expand(2, 1, 16, 32)), *(fake(2, 1, 16, n, dtype=U8) for n in (32, 2, 2)))


def test_append_refusals():
    values = {"k_values": fake(3, 2, 64), "v_values": fake(3, 2, 64)}
    queries = {"q": fake(3, 8, 64, dtype=F32), "q_out": fake(3, 8, 64)}
    for ok in ({}, values, {**values, **queries}, {"T": 0}, {"src": F16}, {"v_values": fake(3, 2, 64, dtype=F16)},
               {"kv": kv4(dim=256), "D": 256, "R": 0}, {"kv": kv4(dim=32), "D": 32, "R": 6}):
        assert status_of(lambda: append_plan(**ok).run(0)) is None, ok
    for page in (8, 24, 2048):
        assert status_of(lambda: append_plan(kv4(page=page)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(kv4(dim=288), D=288).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(Hk=1).run(0)) == _lib.E_INVAL
    assert status_of(lambda: append_plan(k_values=fake(3, 1, 64)).run(0)) == _lib.E_INVAL
    assert status_of(lambda: append_plan(v_values=fake(3, 2, 64, dtype=F32)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(k_values=fake(3, 2, 64), v_values=fake(3, 2, 64, dtype=F16)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(q=fake(3, 8, 64), q_out=fake(3, 8, 64)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(q=fake(3, 8, 64, dtype=F32)).run(0)) == _lib.E_INVAL
    assert status_of(lambda: append_plan(R=66).run(0)) == _lib.E_INVAL
    assert status_of(lambda: append_plan(eps=-1.0).run(0)) == _lib.E_INVAL
    assert refused(append_plan, "d_slots", None) == _lib.E_INVAL
    for field, value in (("d_k", None), ("d_v", 8), ("d_k_scale", None), ("n_pages", -1), ("k_row_stride", 16), ("k_row_stride", 40),
                         ("k_row_stride", 1 << 25), ("v_page_stride", -16), ("ks_row_stride", 1), ("vs_head_stride", -1), ("kv_heads", 0)):
        assert refused(append_plan, field, value, "kv") == _lib.E_INVAL, field
    assert _lib.lib().bpw_kv4_append(None, None) == _lib.E_INVAL
    with pytest.raises(ValueError, match="slots"):
        bpw.Kv4AppendPlan(kv4(), fake(2, 2, 64), fake(2, 2, 64), fake(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots"):
        bpw.Kv4AppendPlan(kv4(), fake(2, 2, 64), fake(2, 2, 64), None)
    with pytest.raises(ValueError, match="expanded"):
        append_plan(k_values=FakeGpu(torch.zeros(1, 2, 64, dtype=BF16).expand(3, 2, 64)))


def attn_plan(T=3, Hq=4, kv=None, n_seqs=2, max_pages=4, max_q=2, dt=BF16, out=None, **kw):
    kv = kv or kv4()
    q = fake(T, Hq, kv.head_dim, dtype=dt)
    ws = workspace(bpw.bpw_kv4_attn_workspace_bytes(kv, q, n_seqs, max_q, max_pages))
    return bpw.Kv4AttnPlan(kv, q, out or fake(T, Hq, kv.head_dim, dtype=dt), fake(n_seqs, max_pages, dtype=I32), fake(n_seqs, dtype=I32),
                           fake(n_seqs + 1, dtype=I32), max_q, ws, **kw)


def test_attention_refusals():
    for ok in ({}, {"T": 0}, {"kv": kv4(dim=256), "Hq": 40}, {"kv": kv4(dim=32)}, {"dt": F16}, {"max_pages": 0}, {"max_pages": 5000}):
        assert status_of(lambda: attn_plan(**ok).run(0)) is None, ok
    assert status_of(lambda: attn_plan(kv=kv4(page=8)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(Hq=5).run(0)) == _lib.E_INVAL
    assert status_of(lambda: attn_plan(max_q=0).run(0)) == _lib.E_INVAL
    assert status_of(lambda: attn_plan(n_seqs=1025).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(dt=F32).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(out=fake(3, 4, 64, dtype=F16)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(out=fake(3, 2, 64)).run(0)) == _lib.E_INVAL
    for scale in (0.0, math.inf, math.nan):
        assert status_of(lambda: attn_plan(scale=scale).run(0)) == _lib.E_INVAL
    for field, value in (("d_lens", None), ("d_q_starts", None), ("d_table", None), ("table_stride", 3), ("max_pages", -1), ("n_tokens", -1),
                         ("d_lse", 2)):
        assert refused(attn_plan, field, value) == _lib.E_INVAL, field
    assert refused(attn_plan, "head_stride", 60, "q") == _lib.E_INVAL
    for n, at, want in ((-1, 0, _lib.E_SIZE), (0, 16, _lib.E_INVAL)):
        p = attn_plan()
        p._ws = (p._ws[0] + at, p._ws[1] + n)
        assert status_of(lambda: p.run(0)) == want
    p = attn_plan()
    p._ws = (None, 0)
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    assert _lib.lib().bpw_kv4_attn(None, None, 0, None) == _lib.E_INVAL
    assert _lib.lib().bpw_kv4_attn_workspace_bytes(None) == 0
    with pytest.raises(ValueError, match="lse"):
        attn_plan(lse=fake(3, 3, dtype=F32))
    with pytest.raises(ValueError, match="required"):
        bpw.Kv4AttnPlan(kv4(), fake(1, 2, 64), fake(1, 2, 64), fake(1, 1, dtype=I32), None, fake(2, dtype=I32), 1, workspace(8))


# ------------------------------------------------------------------------------ log probabilities


def logprobs_plan(T=3, V=100, K=4, dt=F32, tokens="some", ws=None, **kw):
    given = tokens == "some"
    ws = ws or workspace(bpw.bpw_token_logprobs_workspace_bytes(T, V, K))
    return bpw.TokenLogprobsPlan(fake(T, V, dtype=dt), fake(T, dtype=I32) if given else None, fake(T, dtype=F32) if given else None, ws,
                                 top_tokens=fake(T, K, dtype=I32) if K else None, top_logprobs=fake(T, K, dtype=F32) if K else None, **kw)


def test_logprobs_refusals():
    for ok in ({}, {"T": 0}, {"K": 0}, {"K": 32, "dt": F16}, {"V": 1}, {"tokens": None}, {"V": 200000}, {"entropy": fake(3, dtype=F32)}):
        assert status_of(lambda: logprobs_plan(**ok).run(0)) is None, ok
    assert status_of(lambda: logprobs_plan(K=33).run(0)) == _lib.E_UNSUPPORTED
    for scale in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert status_of(lambda: logprobs_plan(scale=scale).run(0)) == _lib.E_INVAL
    for field, value, want in (("vocab", 0, _lib.E_UNSUPPORTED), ("vocab", (1 << 24) + 1, _lib.E_UNSUPPORTED), ("n_tokens", -1, _lib.E_INVAL),
                               ("dtype", 3, _lib.E_INVAL), ("row_stride", -1, _lib.E_INVAL), ("d_logits", None, _lib.E_INVAL),
                               ("d_logits", 2, _lib.E_INVAL), ("d_tokens", None, _lib.E_INVAL), ("d_logprobs", None, _lib.E_INVAL),
                               ("d_top_tokens", None, _lib.E_INVAL), ("d_top_logprobs", None, _lib.E_INVAL)):
        assert refused(logprobs_plan, field, value) == want, field
    p = logprobs_plan(V=200000)
    assert p._ws[1] > 0
    p._ws = (p._ws[0], p._ws[1] - 1)
    assert status_of(lambda: p.run(0)) == _lib.E_SIZE
    p._ws = (None, 0)
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    assert bpw.bpw_token_logprobs_workspace_bytes(5000, 200000, 4) == 0 == bpw.bpw_token_logprobs_workspace_bytes(1, 100, 33)
    assert _lib.lib().bpw_token_logprobs(None, None, 0, None) == _lib.E_INVAL
    with pytest.raises(ValueError, match="together"):
        bpw.TokenLogprobsPlan(fake(3, 9, dtype=F32), fake(3, dtype=I32), None, workspace(8))
    with pytest.raises(ValueError, match="n_top"):
        bpw.TokenLogprobsPlan(fake(3, 9, dtype=F32), None, None, workspace(8), top_tokens=fake(3, 2, dtype=I32), top_logprobs=fake(3, 1, dtype=F32))
    with pytest.raises(TypeError, match="logits"):
        bpw.TokenLogprobsPlan(fake(3, 9, dtype=torch.float64), None, None, workspace(8))
    with pytest.raises(ValueError, match="entropy"):
        logprobs_plan(entropy=fake(2, dtype=F32))


# ------------------------------------------------------------------------------ the oracle


def test_oracle_prompt_closed_forms():
    """Equal scores average the values up to a token's own, by sequence; tokens outside stay out."""
    v = np.arange(6 * 4, dtype=np.float64).reshape(6, 1, 4)
    out, lse, _ = request_ops.prompt(np.ones((6, 2, 4)), np.zeros((6, 1, 4)), v, [1, 4, 5], 1.0)
    assert np.isnan(out[[0, 5]]).all() and np.allclose(out[1, 0], v[1, 0]) and np.allclose(out[3, 1], v[1:4, 0].mean(0))
    assert np.allclose(out[4, 0], v[4, 0]) and np.allclose(lse[1:5, 0], np.log([1, 2, 3, 1]))


def test_oracle_four_bit_closed_forms():
    x = np.zeros((1, 64))
    x[0, :10] = [7.0, -6.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, 5.0, -0.1]  # borders go to the even code; 7 to 6
    x[0, 40] = 7.001
    codes, power, near = request_ops.to_codes(x)
    assert codes[0, :10].tolist() == [7, 15, 0, 2, 10, 4, 4, 6, 6, 8] and power.tolist() == [[127, 128]]
    back = request_ops.from_codes(codes, power)
    assert back[0, :10].tolist() == [6, -6, 0, 1, -1, 2, 2, 4, 4, 0] and back[0, 40] == 8.0 and near[0, 2] == 0
    x[0, 33] = np.inf
    codes, power, _ = request_ops.to_codes(x)
    assert power.tolist() == [[127, 255]] and np.isnan(request_ops.from_codes(codes, power)[0, 32:]).all()
    assert request_ops.to_codes(np.zeros((1, 32)))[1].tolist() == [[2]]
    assert request_ops.unpacked(np.array([[0x21, 0xF3]], np.uint8)).tolist() == [[1, 2, 3, 15]]


def test_oracle_logprobs_closed_forms():
    lp, ent, top, top_lp = request_ops.logprobs(np.array([[0.0, math.log(3), -np.inf], [1.0, 1.0, 1.0], [-np.inf] * 3, [1.0, np.nan, np.inf]]),
                                                np.array([0, 3, 1, 0]), 2, 1.0)
    assert np.allclose(lp[0], math.log(0.25)) and lp[1] == lp[2] == -np.inf and np.isnan(lp[3])
    assert np.allclose(ent[:3], [-0.25 * math.log(0.25) - 0.75 * math.log(0.75), math.log(3), 0])
    assert top.tolist() == [[1, 0], [0, 1], [-1, -1], [2, 0]] and np.allclose(top_lp[0], [math.log(0.75), math.log(0.25)])
