"""The decode-step operators' refusals, on the host: every argument check comes before any device work, so
the statuses can be seen without a GPU (a call whose arguments pass ends at the device check). Also the
oracle's own pins against closed forms."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
bpw = pytest.importorskip("bit_plane_weight_amd")
from bit_plane_weight_amd import _lib  # noqa: E402
from oracle import decode_ops  # noqa: E402


class FakeGpu:
    """A CPU tensor that says it is on the GPU: enough for checks that launch nothing."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return FakeGpu(torch.zeros(*shape, dtype=dtype))


def status_of(call):
    """The status a call is refused with; None where all of its arguments pass (the device check, which
    fails here and passes on a GPU, comes last)."""
    try:
        call()
    except bpw.BpwError as e:
        return None if e.status in (_lib.E_HIP, _lib.E_ARCH) else e.status
    return None


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setenv("BPW_FORCE_ARCH_MISMATCH", "1")


def cache(pages=4, heads=2, page=16, dim=64, dtype=torch.bfloat16):
    return bpw.PagedKv(fake(pages, heads, page, dim, dtype=dtype), fake(pages, heads, page, dim, dtype=dtype))


def rope_plan(T=3, Hq=4, Hk=2, D=64, R=64, src=torch.float32, dst=torch.bfloat16, **kw):
    return bpw.QkNormRopePlan(fake(T, Hq, D, dtype=src), fake(T, Hk, D, dtype=src), fake(T, Hq, D, dtype=dst),
                              fake(T, Hk, D, dtype=dst), fake(T, dtype=torch.int32), fake(R // 2, dtype=torch.float64), **kw)


def test_struct_sizes_match_the_header():
    sizes = {"BpwHeads": 32, "BpwPagedKv": 88, "BpwRotation": 24, "BpwQkNormRopeArgs": 184, "BpwKvAppendArgs": 280,
             "BpwAttnArgs": 232, "BpwVerifyArgs": 112}
    assert {n: ctypes.sizeof(getattr(_lib, n)) for n in sizes} == sizes


def test_norm_rope_refusals():
    assert status_of(lambda: rope_plan().run(0)) is None
    assert status_of(lambda: rope_plan(D=2, R=2).run(0)) is None
    assert status_of(lambda: rope_plan(T=0).run(0)) is None
    assert status_of(lambda: rope_plan(D=63, R=2).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: rope_plan(D=1026, R=2).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: rope_plan(D=64, R=66).run(0)) == _lib.E_INVAL
    assert status_of(lambda: rope_plan(eps=-1.0).run(0)) == _lib.E_INVAL
    assert status_of(lambda: rope_plan(eps=math.nan).run(0)) == _lib.E_INVAL
    p = rope_plan()
    p._args.k_out.heads = 1
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    for field, value in (("d", None), ("token_stride", -1), ("dtype", 7), ("heads", -1)):
        p = rope_plan()
        setattr(p._args.q, field, value)
        assert status_of(lambda: p.run(0)) == _lib.E_INVAL, field
    p = rope_plan()
    p._args.q.d += 2  # not an element's alignment for float32
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = rope_plan()
    p._args.rot.d_positions = None
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = rope_plan()
    p._args.rot.interleaved = 2
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = rope_plan()
    p._args.k.dtype = _lib.F16
    assert status_of(lambda: p.run(0)) == _lib.E_UNSUPPORTED
    assert _lib.lib().bpw_qk_norm_rope(None, None) == _lib.E_INVAL


def test_binding_refuses_what_the_abi_cannot_see():
    with pytest.raises(TypeError, match="GPU"):
        bpw.QkNormRopePlan(torch.zeros(1, 1, 8), None, torch.zeros(1, 1, 8), None, None, None)
    with pytest.raises(TypeError, match="q"):
        rope_plan(src=torch.float64)
    with pytest.raises(ValueError, match="q_gain"):
        rope_plan(q_gain=fake(63, dtype=torch.float32))
    with pytest.raises(TypeError, match="positions"):
        bpw.QkNormRopePlan(fake(2, 1, 8), None, fake(2, 1, 8), None, fake(2, dtype=torch.int64),
                           fake(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="positions"):
        bpw.QkNormRopePlan(fake(2, 1, 8), None, fake(2, 1, 8), None, None, fake(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous"):
        bpw.QkNormRopePlan(FakeGpu(torch.zeros(2, 8, 4).transpose(1, 2)), None, fake(2, 4, 8), None, None, None)
    with pytest.raises(ValueError, match="expanded"):
        bpw.QkNormRopePlan(fake(2, 3, 8), None, FakeGpu(torch.zeros(1, 3, 8, dtype=torch.bfloat16).expand(2, 3, 8)),
                           None, None, None)
    with pytest.raises(TypeError, match="cache"):
        cache(dtype=torch.float32)
    with pytest.raises(ValueError, match="slots"):
        bpw.KvAppendPlan(cache(), fake(2, 2, 64), fake(2, 2, 64), fake(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots"):
        bpw.KvAppendPlan(cache(), fake(2, 2, 64), fake(2, 2, 64), None)
    with pytest.raises(ValueError, match="prefix_pages"):
        attn_plan(prefix=17, prefix_pages=fake(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="table"):
        attn_plan(table=fake(2, 4, dtype=torch.int64))
    with pytest.raises(ValueError, match="q_starts"):
        attn_plan(q_starts=fake(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="lse"):
        attn_plan(lse=fake(3, 3, dtype=torch.float32))
    with pytest.raises(ValueError, match="draft"):
        verify_plan(draft=fake(2, 3, 99, dtype=torch.float32))
    with pytest.raises(TypeError, match="different"):
        verify_plan(draft=fake(2, 3, 100, dtype=torch.float16))
    with pytest.raises(ValueError, match="out_tokens"):
        verify_plan(out_tokens=fake(2, 3, dtype=torch.int32))


def test_binding_refuses_rows_of_another_length():
    """Enough elements, but in rows that the kernels would not find; flat tensors and more rows are taken."""
    f32, i32 = torch.float32, torch.int32
    for shape in ((5, 3), (3, 5), (3, 4, 2)):
        with pytest.raises(ValueError, match=r"lse must be \[3, 4\]"):
            attn_plan(lse=fake(*shape, dtype=f32))
    with pytest.raises(ValueError, match=r"out_tokens must be \[2, 4\]"):
        verify_plan(out_tokens=fake(2, 9, dtype=i32))
    args = lambda **k: {"tokens": fake(2, 3, dtype=i32), "accept_u": fake(2, 3, dtype=f32), **k}  # noqa: E731
    plan = lambda a: bpw.DraftVerifyPlan(fake(2, 4, 100, dtype=f32), None, a["tokens"], a["accept_u"], fake(2, dtype=f32),  # noqa: E731
                                         fake(2, 4, dtype=i32), fake(2, dtype=i32), fake(4096, dtype=torch.uint8))
    plan(args())
    plan(args(tokens=fake(7, dtype=i32), accept_u=fake(5, 3, dtype=f32)))
    plan(args(tokens=fake(1, 2, 3, dtype=i32)))
    with pytest.raises(ValueError, match=r"tokens must be \[2, 3\]"):
        plan(args(tokens=fake(2, 8, dtype=i32)))
    with pytest.raises(ValueError, match=r"accept_u must be \[2, 3\]"):
        plan(args(accept_u=fake(2, 4, dtype=f32)))
    for shape in ((12,), (3, 2, 2), (9, 4)):
        assert status_of(lambda: attn_plan(lse=fake(*shape, dtype=f32)).run(0)) is None
    assert status_of(lambda: attn_plan(T=0, lse=fake(3, 4, dtype=f32)).run(0)) is None


def append_plan(kv=None, T=3, Hk=2, D=64, R=64, src=torch.float32, **kw):
    return bpw.KvAppendPlan(kv or cache(), fake(T, Hk, D, dtype=src), fake(T, Hk, D, dtype=src), fake(T, dtype=torch.int64),
                            fake(T, dtype=torch.int32), fake(R // 2, dtype=torch.float64), **kw)


def test_append_refusals():
    assert status_of(lambda: append_plan().run(0)) is None
    assert status_of(lambda: append_plan(q=fake(3, 8, 64, dtype=torch.float32), q_out=fake(3, 8, 64)).run(0)) is None
    assert status_of(lambda: append_plan(cache(page=24)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(cache(page=8)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(cache(page=2048)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(Hk=1).run(0)) == _lib.E_INVAL
    assert status_of(lambda: append_plan(q=fake(3, 8, 64), q_out=fake(3, 8, 64)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: append_plan(q=fake(3, 8, 64, dtype=torch.float32),
                                         q_out=fake(3, 8, 64, dtype=torch.float16)).run(0)) == _lib.E_UNSUPPORTED
    p = append_plan()
    p._args.d_slots = None
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    for field, value in (("d_k", None), ("n_pages", -1), ("k_row_stride", 1 << 25), ("v_page_stride", -8), ("dtype", 0)):
        p = append_plan()
        setattr(p._args.kv, field, value)
        assert status_of(lambda: p.run(0)) == _lib.E_INVAL, field
    assert _lib.lib().bpw_kv_append(None, None) == _lib.E_INVAL


def attn_plan(T=3, Hq=4, kv=None, prefix=0, prefix_pages=None, n_seqs=2, max_pages=4, max_q=2, ws=None, table=None,
              q_starts=None, **kw):
    kv = kv or cache()
    D, dt = kv.c.head_dim, kv.k_pages.dtype
    q = fake(T, Hq, D, dtype=dt)
    if ws is None:
        n = bpw.bpw_attn_shared_prefix_workspace_bytes(kv, q, prefix, n_seqs, max_q, max_pages)
        ws = FakeGpu(torch.zeros(n + 256, dtype=torch.uint8))
        ws.t = ws.t[-ws.t.data_ptr() % 256:][:n]
    if prefix and prefix_pages is None:
        prefix_pages = fake(-(-prefix // kv.page_size), dtype=torch.int32)
    return bpw.SharedPrefixAttnPlan(kv, q, fake(T, Hq, D, dtype=dt), prefix_pages, prefix,
                                    table or fake(n_seqs, max_pages, dtype=torch.int32), fake(n_seqs, dtype=torch.int32),
                                    q_starts or fake(n_seqs + 1, dtype=torch.int32), max_q, ws, **kw)


def test_attention_refusals():
    assert status_of(lambda: attn_plan().run(0)) is None
    assert status_of(lambda: attn_plan(prefix=100, T=200, max_q=200).run(0)) is None
    assert status_of(lambda: attn_plan(T=0).run(0)) is None
    assert status_of(lambda: attn_plan(kv=cache(dim=256), Hq=40).run(0)) is None
    assert status_of(lambda: attn_plan(kv=cache(dim=68)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(kv=cache(dim=264)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(kv=cache(page=8)).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(Hq=5).run(0)) == _lib.E_INVAL
    assert status_of(lambda: attn_plan(max_q=0).run(0)) == _lib.E_INVAL
    assert status_of(lambda: attn_plan(n_seqs=1025).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: attn_plan(scale=0.0).run(0)) == _lib.E_INVAL
    assert status_of(lambda: attn_plan(scale=math.inf).run(0)) == _lib.E_INVAL
    for field, value in (("d_lens", None), ("d_q_starts", None), ("d_table", None), ("table_stride", 3), ("prefix_len", -1),
                         ("prefix_len", 1 << 31), ("max_pages", -1)):
        p = attn_plan()
        setattr(p._args, field, value)
        assert status_of(lambda: p.run(0)) == _lib.E_INVAL, field
    p = attn_plan(prefix=5)
    p._args.d_prefix_pages = None
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = attn_plan()
    p._args.q.head_stride = 60
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = attn_plan()
    p._args.q.dtype = _lib.F16
    assert status_of(lambda: p.run(0)) == _lib.E_UNSUPPORTED
    p = attn_plan()
    p._ws = (p._ws[0], p._ws[1] - 1)
    assert status_of(lambda: p.run(0)) == _lib.E_SIZE
    p = attn_plan()
    p._ws = (p._ws[0] + 16, p._ws[1])
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    p = attn_plan()
    p._ws = (None, 0)
    assert status_of(lambda: p.run(0)) == _lib.E_INVAL
    assert _lib.lib().bpw_attn_shared_prefix(None, None, 0, None) == _lib.E_INVAL
    assert _lib.lib().bpw_attn_shared_prefix_workspace_bytes(None) == 0


def verify_plan(B=2, K=3, V=100, dtype=torch.float32, draft="same", out_tokens=None, **kw):
    d = fake(B, K, V, dtype=dtype) if draft == "same" else draft
    ws = FakeGpu(torch.zeros(max(1, bpw.bpw_verify_draft_workspace_bytes(B, V)) + 256, dtype=torch.uint8))
    ws.t = ws.t[-ws.t.data_ptr() % 256:]
    return bpw.DraftVerifyPlan(fake(B, K + 1, V, dtype=dtype), d, fake(B, K, dtype=torch.int32),
                               fake(B, K, dtype=torch.float32), fake(B, dtype=torch.float32),
                               out_tokens or fake(B, K + 1, dtype=torch.int32), fake(B, dtype=torch.int32), ws, **kw)


def test_verify_refusals():
    assert status_of(lambda: verify_plan().run(0)) is None
    assert status_of(lambda: verify_plan(draft=None, dtype=torch.float16).run(0)) is None
    assert status_of(lambda: verify_plan(K=65).run(0)) == _lib.E_UNSUPPORTED
    assert status_of(lambda: verify_plan(K=0, draft=None).run(0)) == _lib.E_UNSUPPORTED
    for field, value in (("d_target", None), ("d_tokens", None), ("d_out_tokens", None), ("dtype", 9), ("n_seqs", -1),
                         ("target_seq_stride", -1)):
        p = verify_plan()
        setattr(p._args, field, value)
        assert status_of(lambda: p.run(0)) == _lib.E_INVAL, field
    p = verify_plan()
    p._args.vocab = (1 << 24) + 1
    assert status_of(lambda: p.run(0)) == _lib.E_UNSUPPORTED
    p = verify_plan()
    p._ws = (p._ws[0], 8)
    assert status_of(lambda: p.run(0)) == _lib.E_SIZE
    assert bpw.bpw_verify_draft_workspace_bytes(0, 10) == 0
    assert _lib.lib().bpw_verify_draft(None, None, 0, None) == _lib.E_INVAL


def test_oracle_rotation_closed_forms():
    """A quarter turn swaps a pair's elements, a full turn changes nothing, and the norm of all-equal
    elements is the gain with their sign."""
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8) + 1
    y, _ = decode_ops.norm_rope(x, None, [1], [math.pi / 2, 2 * math.pi], 0.0, False)
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-12)
    y, _ = decode_ops.norm_rope(x, None, [1], [math.pi / 2, 2 * math.pi], 0.0, True)
    assert np.allclose(y[0, 0], [-2, 1, 3, 4, 5, 6, 7, 8], atol=1e-12)
    y, _ = decode_ops.norm_rope(np.full((1, 1, 4), -3.0), np.arange(4), [0], [], 0.0, False)
    assert np.allclose(y[0, 0], [0, -1, -2, -3])


def test_oracle_attention_closed_forms():
    """Equal scores average the values; a causal tail hides later positions; nothing seen gives zeros."""
    k = np.zeros((2, 1, 16, 4))
    v = np.arange(2 * 16 * 4, dtype=np.float64).reshape(2, 1, 16, 4)
    q = np.ones((2, 1, 4))
    out, lse, _ = decode_ops.attention(q, k, v, [1], 3, np.array([[0]]), [2], [0, 2], 2, 1.0)
    want = np.concatenate([v[1, 0, :3], v[0, 0, :2]])
    assert np.allclose(out[1, 0], want.mean(0)) and np.allclose(out[0, 0], want[:4].mean(0))
    assert np.allclose(lse[:, 0], [math.log(4), math.log(5)])
    out, lse, _ = decode_ops.attention(q, k, v, [], 0, np.array([[0]]), [1], [0, 2], 2, 1.0)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and np.allclose(out[1, 0], v[0, 0, 0])


def test_oracle_verification_closed_forms():
    p = np.array([[[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]]])
    q = np.array([[[1.0, 0.0, 0.0]]])
    toks, acc = decode_ops.verify(p, q, np.array([[0]]), None, np.array([[0.49]]), np.array([0.25]))
    assert toks.tolist() == [[0, 2]] and acc.tolist() == [1]
    toks, acc = decode_ops.verify(p, q, np.array([[0]]), None, np.array([[0.5]]), np.array([0.9]))
    assert toks.tolist() == [[1, -1]] and acc.tolist() == [0]  # 0.5 is not below 0.5; only token 1 has mass left
