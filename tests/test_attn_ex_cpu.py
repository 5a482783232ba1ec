"""Attention with modified scores, without a GPU: the 64-bit reference against differences and closed
forms, the refusals of the four calls and their workspace sizes."""
import ctypes as ct
import math

import pytest
import torch

import attn_ref


def test_reference_gradients_match_differences():
    """Central differences of a scalar of o, with cap, bias, prefix, documents, shared heads and an empty row."""
    g = torch.Generator().manual_seed(1)
    B, Hq, Hkv, Nq, Nk, d = 2, 4, 2, 5, 7, 3
    q, k, v, w = (torch.randn(B, n, h, d, generator=g, dtype=torch.float64)
                  for n, h in ((Nq, Hq), (Nk, Hkv), (Nk, Hkv), (Nq, Hq)))
    doc_k = torch.tensor([[0, 0, 0, 1, 1, 1, 1], [0, 0, 5, 5, 5, 0, -1]], dtype=torch.int32)
    doc_q = torch.tensor([[0, 1, 1, 1, 7], [5, 5, 0, 5, -1]], dtype=torch.int32)
    valid = attn_ref.valid_mask(B, Nq, Nk, True, torch.tensor([2, 4]), doc_q, doc_k)
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0])
    kw = dict(cap=1.5, slopes=slopes, valid=valid)
    r = attn_ref.attn(q, k, v, w, **kw)
    assert torch.isneginf(r["lse"][0]).any() and torch.isfinite(r["lse"][0]).any()

    def f(*a):
        return float((attn_ref.attn(*a, **kw)["o"][0] * w).sum())

    h = 1e-5
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        for _ in range(12):
            a = [q.clone(), k.clone(), v.clone()]
            i = int(torch.randint(a[at].numel(), (1,), generator=g))
            a[at].view(-1)[i] += h
            up = f(*a)
            a[at].view(-1)[i] -= 2 * h
            diff = (up - f(*a)) / (2 * h)
            # the differences' own error: h^2 times a third derivative of order 10, and rounding 1e-15 / h
            assert abs(diff - float(r[name][0].reshape(-1)[i])) <= 1e-8, name


def test_reference_closed_forms():
    q = torch.zeros(1, 3, 2, 4)
    k, v = torch.randn(1, 3, 1, 4), torch.arange(12.).view(1, 3, 1, 4)
    r = attn_ref.attn(q, k, v, valid=attn_ref.valid_mask(1, 3, 3, True))
    assert torch.allclose(r["o"][0][0, :, 0], torch.stack([v[0, :i + 1, 0].double().mean(0) for i in range(3)]))
    assert torch.allclose(r["lse"][0][0, 0], torch.tensor([1., 2., 3.]).log().double())
    # a bias alone: weights fall by exp(-slope) per step of distance
    r = attn_ref.attn(q, k, v, slopes=torch.tensor([math.log(2.0), 0.0]), valid=attn_ref.valid_mask(1, 3, 3, True))
    assert torch.allclose(r["o"][0][0, 2, 0], (v[0, 0, 0] / 4 + v[0, 1, 0] / 2 + v[0, 2, 0]).double() / 1.75)
    # one token over a cache equals the last row of the causal pass
    q, k, v = torch.randn(1, 6, 2, 4), torch.randn(1, 6, 1, 4), torch.randn(1, 6, 1, 4)
    full = attn_ref.attn(q, k, v, cap=2.0, slopes=torch.tensor([.3, .1]), valid=attn_ref.valid_mask(1, 6, 6, True))
    one = attn_ref.decode(q[:, 5], k[:, 2:], v[:, 2:], torch.tensor([4]), k[0, :2], v[0, :2], cap=2.0,
                          slopes=torch.tensor([.3, .1]))
    assert torch.allclose(one["o"][0], full["o"][0][:, 5]) and torch.allclose(one["lse"][0], full["lse"][0][..., 5])


@pytest.fixture(scope="module")
def mcs():
    from free_sparse_attention_pddp_b200 import build

    build.build()
    import free_sparse_attention_pddp_b200 as m

    m.load()
    return m


GOOD = dict(B=2, Hq=8, Hkv=4, Nq=100, Nk=300, d=128)


@pytest.mark.parametrize("bad", [dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(Nq=0), dict(Nk=0), dict(Nk=-5),
                                 dict(d=96), dict(d=0), dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf),
                                 dict(scale=math.nan), dict(scale=1e-20), dict(scale=1e20), dict(cap=1e-9), dict(Hq=129, Hkv=1), dict(Nq=1 << 28),
                                 dict(B=4, Nk=1 << 27)])
def test_attn_shapes_are_refused(mcs, bad):
    s = mcs.AttnShape(**{**GOOD, **bad})
    for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD):
        assert mcs.mcs_attn_workspace_bytes(s, op) == 0
        with pytest.raises(mcs.MCSError):
            mcs.attn_workspace(s, op, "cpu")
    p = ct.cast((ct.c_uint8 * 4096)(), ct.c_void_p)
    want = (1, 2)  # invalid or unsupported, before any device call
    assert mcs.load().mcs_dense_ex(ct.byref(s), None, p, p, p, p, None, p, 1 << 40, None) in want
    assert mcs.load().mcs_dense_bwd(ct.byref(s), None, p, p, p, p, p, p, p, p, p, p, 1 << 40, None) in want


def test_attn_workspace_sizes(mcs):
    s = mcs.AttnShape(**GOOD)
    assert mcs.mcs_attn_workspace_bytes(s, mcs.MCS_OP_DENSE_EX) >= 256
    assert mcs.mcs_attn_workspace_bytes(s, mcs.MCS_OP_DENSE_BWD) >= 256 + 4 * 2 * 8 * 100
    assert mcs.mcs_attn_workspace_bytes(s, mcs.MCS_OP_DENSE) == 0
    assert mcs.mcs_workspace_bytes(mcs.Shape(1, 2, 300, 128, topk=3), mcs.MCS_OP_DENSE_EX) == 0
    assert mcs.mcs_decode_workspace_bytes(mcs.DecodeShape(2, 8, 4, 100, 128)) >= 256
    for bad in (dict(B=0), dict(C=0), dict(P=-1), dict(d=80), dict(Hkv=3), dict(cap=-2.0), dict(C=1 << 29)):
        kw = {**dict(B=2, Hq=8, Hkv=4, C=100, d=128), **bad}
        assert mcs.mcs_decode_workspace_bytes(mcs.DecodeShape(**kw)) == 0, bad


def test_attn_arguments_are_refused(mcs):
    lib = mcs.load()
    raw = (ct.c_uint8 * 8192)()
    base = (ct.addressof(raw) + 255) // 256 * 256
    p, odd = ct.c_void_p(base), ct.c_void_p(base + 8)
    big = 1 << 40
    s = mcs.AttnShape(**GOOD)

    def fwd(opts=None, ws=p, n=big, **kw):
        a = {**dict(q=p, k=p, v=p, o=p, lse=None), **kw}
        return lib.mcs_dense_ex(ct.byref(kw.get("s", s)), opts, a["q"], a["k"], a["v"], a["o"], a["lse"], ws, n, None)

    def bwd(opts=None, ws=p, n=big, **kw):
        names = ("q", "k", "v", "o", "lse", "d_o", "dq", "dk", "dv")
        return lib.mcs_dense_bwd(ct.byref(s), opts, *(kw.get(x, p) for x in names), ws, n, None)

    for call, names in ((fwd, "q k v o ws"), (bwd, "q k v o lse d_o dq dk dv ws")):
        for name in names.split():
            assert call(**{name: None}) == 1, name
            if name != "lse":
                assert call(**{name: odd}) == 1, name
        assert call(n=16) == 1
    assert fwd(lse=ct.c_void_p(base + 2)) == 1
    # options: one document array without the other, a prefix without the causal flag, misaligned arrays
    doc = ct.cast(p, ct.c_void_p).value
    for o in (mcs.AttnOpts(None, None, doc, None), mcs.AttnOpts(None, None, None, doc), mcs.AttnOpts(None, doc, None, None),
              mcs.AttnOpts(doc + 2, None, None, None)):
        assert fwd(ct.byref(o)) == 1 and bwd(ct.byref(o)) == 1
    # more document tiles than the bitmaps hold: 2^12 of 128 keys, 2^16 of one token (128 heads to a KV head)
    docs = mcs.AttnOpts(None, None, doc, doc)
    assert fwd(ct.byref(docs), s=mcs.AttnShape(1, 1, 1, 1, (1 << 19) + 1, 64)) == 2
    assert fwd(ct.byref(docs), s=mcs.AttnShape(1, 128, 1, (1 << 16) + 1, 10, 64)) == 2


def test_decode_arguments_are_refused(mcs):
    lib = mcs.load()
    raw = (ct.c_uint8 * 8192)()
    base = (ct.addressof(raw) + 255) // 256 * 256
    p, odd = ct.c_void_p(base), ct.c_void_p(base + 8)
    names = ("q", "kp", "vp", "k", "v", "lens", "slopes", "o", "lse")
    plain, shared = mcs.DecodeShape(2, 8, 4, 100, 64), mcs.DecodeShape(2, 8, 4, 100, 64, P=50)

    def one(s=plain, n=1 << 40, ws=p, **kw):
        a = [kw.get(x, None if x in ("slopes", "lse") else p) for x in names if x not in ("kp", "vp")]
        return lib.mcs_decode(ct.byref(s), *a, ws, n, None)

    def sh(s=shared, n=1 << 40, ws=p, **kw):
        a = [kw.get(x, None if x in ("slopes", "lse") else p) for x in names]
        return lib.mcs_decode_shared(ct.byref(s), *a, ws, n, None)

    assert one(s=shared) == 1 and sh(s=plain) == 1  # the prefix belongs to mcs_decode_shared alone
    for call, which in ((one, "q k v lens o ws"), (sh, "q kp vp k v lens o ws")):
        for x in which.split():
            assert call(**{x: None}) == 1, x
        for x in which.replace("lens ", "").split():
            assert call(**{x: odd}) == 1, x
        assert call(lens=ct.c_void_p(base + 2)) == 1 and call(n=100) == 1


def test_wrappers_refuse_tensors_that_do_not_fit(mcs):
    s = mcs.AttnShape(1, 4, 2, 6, 8, 64)
    q, k = torch.zeros(1, 6, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    lse, ws = torch.zeros(1, 4, 6), torch.zeros(4096, dtype=torch.uint8)
    for a in ((q.float(), k, k, q), (q[:, :5], k, k, q), (q, k.transpose(1, 2), k, q), (q, k, k[..., ::2], q),
              (q, k, k, q)):  # the last: everything fits, but lies on the CPU
        with pytest.raises(mcs.MCSError) as e:
            mcs.mcs_dense_ex(s, *a, lse, ws)
        assert e.value.code == 1
    d = mcs.DecodeShape(2, 4, 2, 8, 64)
    qd, kd = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(mcs.MCSError):
        mcs.mcs_decode(d, qd, kd, kd, torch.zeros(2, dtype=torch.int64), qd, None, ws)


def test_caps_beyond_their_range_are_refused(mcs):
    """Scores near such a cap have no probabilities in fp32."""
    for cap, ok in ((1e20, True), (2e20, False), (1e36, False), (1e-6, True), (5e-7, False)):
        s, d = mcs.AttnShape(1, 2, 1, 10, 10, 64, cap=cap), mcs.DecodeShape(1, 2, 1, 10, 64, cap=cap)
        assert (mcs.mcs_attn_workspace_bytes(s, mcs.MCS_OP_DENSE_EX) > 0) == ok
        assert (mcs.mcs_decode_workspace_bytes(d) > 0) == ok


def test_flags(mcs):
    for flags, ok in ((0, True), (1, True), (2, True), (3, True), (4, False), (-1, False)):
        s = mcs.AttnShape(1, 2, 1, 10, 10, 64)
        s.flags = flags
        assert (mcs.mcs_attn_workspace_bytes(s, mcs.MCS_OP_DENSE_BWD) > 0) == ok
    assert mcs.AttnShape(1, 2, 1, 10, 10, 64, causal=True, d_from_o=True).flags == 3
