"""mcs_dense_ex and mcs_dense_bwd against the 64-bit reference, element by element within derived bounds."""
import pytest

import attn_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mcs():
    import free_sparse_attention_pddp_b200 as m

    m.load()
    return m


def inputs(B, Hq, Hkv, Nq, Nk, d, seed=0, gain=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return r(B, Nq, Hq, d) * gain, r(B, Nk, Hkv, d), r(B, Nk, Hkv, d), r(B, Nq, Hq, d)


def guarded(t):
    """An uninitialised-looking buffer of t's shape inside a larger one: (view, whole buffer)."""
    pad = 512
    whole = torch.full((t.numel() + 2 * pad,), 12345.0, dtype=t.dtype, device="cuda")
    return whole[pad:pad + t.numel()].view(t.shape), whole


def untouched(whole):
    return bool((whole[:512] == whole[0]).all()) and bool((whole[-512:] == whole[0]).all()) and float(whole[0]) > 12000


def run(mcs, shape, q, k, v, d_o=None, **opts):
    """Forward and, with d_o, backward into guarded buffers."""
    o, wo = guarded(q)
    lse, wl = guarded(torch.empty(shape.B, shape.Hq, shape.Nq, device="cuda"))
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_EX)
    mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws, **opts)
    assert mcs.mcs_poll_status(ws)[0] == 0
    got, guards = {"o": o, "lse": lse}, [wo, wl]
    if d_o is not None:
        (dq, w1), (dk, w2), (dv, w3) = guarded(q), guarded(k), guarded(v)
        ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD)
        mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, ws, **opts)
        assert mcs.mcs_poll_status(ws)[0] == 0
        got.update(dq=dq, dk=dk, dv=dv)
        guards += [w1, w2, w3]
    assert all(untouched(w) for w in guards)
    return got


def both(mcs, B, Hq, Hkv, Nq, Nk, d, cap=0.0, scale=0.0, slopes=None, causal=False, prefix=None, doc_q=None,
         doc_k=None, seed=0, gain=2.0, tensors=None):
    q, k, v, d_o = tensors or inputs(B, Hq, Hkv, Nq, Nk, d, seed, gain)
    dev = lambda x, t: None if x is None else torch.as_tensor(x, dtype=t).cuda().contiguous()  # noqa: E731
    slopes, prefix = dev(slopes, torch.float32), dev(prefix, torch.int32)
    doc_q, doc_k = dev(doc_q, torch.int32), dev(doc_k, torch.int32)
    shape = mcs.AttnShape(B, Hq, Hkv, Nq, Nk, d, scale=scale, cap=cap, causal=causal)
    got = run(mcs, shape, q, k, v, d_o, slopes=slopes, prefix=prefix, doc_q=doc_q, doc_k=doc_k)
    valid = attn_ref.valid_mask(B, Nq, Nk, causal, prefix, doc_q, doc_k, "cuda")
    want = attn_ref.attn(q, k, v, d_o, scale=scale or None, cap=cap, slopes=slopes, valid=valid, exact_d=Nk <= 256)
    for name in ("lse", "o", "dv", "dk", "dq"):
        attn_ref.check(got[name], want[name], name)
    return got


SIZES = [  # B, Hq, Hkv, Nq, Nk
    (1, 1, 1, 1, 1), (2, 3, 3, 1, 130), (1, 2, 1, 127, 127), (1, 2, 2, 128, 128), (2, 4, 2, 129, 129),
    (1, 8, 1, 70, 257), (1, 6, 2, 300, 640), (3, 5, 1, 33, 200), (1, 12, 1, 45, 129), (1, 128, 1, 3, 140),
    (2, 2, 2, 513, 385), (1, 4, 4, 600, 600),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plain(mcs, size, d):
    both(mcs, *size, d, seed=sum(size))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_causal_cap_and_bias(mcs, size, d):
    """Nq > Nk among the sizes: the first rows see nothing."""
    Hq = size[1]
    both(mcs, *size, d, cap=15.0, slopes=[2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], causal=True, seed=sum(size))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,gain", [(50.0, 2.0), (5.0, 8.0), (0.5, 4.0), (1000.0, 4.0)])
def test_caps_from_nearly_linear_to_saturated(mcs, cap, gain, d):
    both(mcs, 1, 4, 2, 200, 333, d, cap=cap, gain=gain, seed=5)


@pytest.mark.parametrize("slopes", [[0.0, 3.0], [-0.01, 0.2]])
def test_bias_without_a_mask_is_symmetric_in_distance(mcs, slopes):
    both(mcs, 1, 2, 1, 150, 290, 64, slopes=slopes, seed=6)


@pytest.mark.parametrize("Nq,Nk,prefix", [(257, 257, [0, 100, 257]), (40, 600, [561, 599, 10000]), (300, 200, [-7, 1, 128]),
                                          (1, 1, [0, 1, 2])])
def test_prefix(mcs, Nq, Nk, prefix):
    both(mcs, 3, 4, 2, Nq, Nk, 128, causal=True, prefix=prefix, cap=20.0, slopes=[.1, .2, .3, .4], seed=Nq)


def packed_ids(B, N, mean, seed, pad=0, shuffle=False):
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(B, N, generator=g) < 1.0 / mean).cumsum(1)
    if shuffle:  # ids in no order: documents that interleave
        ids = torch.randint(0, max(2, N // mean), (B, N), generator=g)
    for b in range(B):
        n = pad * (b + 1) // B
        if n:
            ids[b, N - n:] = -1
    return ids.int()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 3, 8])
@pytest.mark.parametrize("mean,pad,shuffle,causal", [(40, 0, False, False), (200, 90, False, True), (3000, 130, False, False),
                                                     (150, 20, True, True)])
def test_documents(mcs, mean, pad, shuffle, causal, g, d):
    ids = packed_ids(2, 700, mean, mean + g, pad, shuffle)
    both(mcs, 2, 2 * g, 2, 700, 700, d, causal=causal, doc_q=ids, doc_k=ids, cap=30.0 if g == 3 else 0.0, seed=g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hkv,N,lengths,causal", [(1, 16, 1250, (900, 20, 330), False), (1, 16, 1210, (70, 1000), True),
                                                    (2, 10, 1170, (1100, 40), False), (1, 38, 1100, (900, 60, 70), False)])
def test_documents_of_very_different_lengths(mcs, B, Hkv, N, lengths, causal, d):
    """More pairs of query tiles than SMs, some of which are cut into their tiles; odd numbers of tiles."""
    ids = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    ids = torch.cat([ids, torch.full((N - len(ids),), -1)])[None].repeat(B, 1)
    if B > 1:
        ids[1] = ids[1].flip(0)
    both(mcs, B, 2 * Hkv, Hkv, N, N, d, causal=causal, doc_q=ids, doc_k=ids, seed=N)


def test_documents_of_queries_and_keys_differ(mcs):
    """Cross-attention: a query document without keys, a key document without queries, large and negative ids."""
    dq = torch.full((1, 260), 7)
    dk = torch.full((1, 500), 7)
    dq[0, 100:180], dq[0, 200:] = 2 ** 31 - 1, -2 ** 31
    dk[0, 250:300], dk[0, 300:] = 0, -5
    r = both(mcs, 1, 4, 2, 260, 500, 64, doc_q=dq, doc_k=dk, prefix=[3], causal=True, seed=9)
    assert torch.isneginf(r["lse"][0, :, 100:180]).all() and (r["o"][0, 100:180] == 0).all()


def test_nothing_is_valid(mcs):
    r = both(mcs, 2, 2, 1, 140, 300, 128, doc_q=torch.zeros(2, 140), doc_k=torch.ones(2, 300), seed=3)
    assert torch.isneginf(r["lse"]).all() and all((r[n] == 0).all() for n in ("o", "dq", "dk", "dv"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_padded_rows_may_hold_anything(mcs, bad, g, d):
    ids = packed_ids(2, 420, 150, 4, pad=165)
    ids[0, 10:13] = -1  # and padding inside a row
    q, k, v, d_o = inputs(2, 2 * g, 2, 420, 420, d, seed=11)
    for t in (q, k, v, d_o):
        t[ids.cuda() < 0] = bad
    r = both(mcs, 2, 2 * g, 2, 420, 420, d, doc_q=ids, doc_k=ids, cap=25.0, tensors=(q, k, v, d_o))
    pad = ids.cuda() < 0
    assert all((r[n][pad] == 0).all() for n in ("o", "dq", "dk", "dv"))


def test_a_batch_does_not_read_its_neighbour(mcs):
    """The last key tile of request 0 is ragged and request 1 starts with NaN."""
    q, k, v, d_o = inputs(2, 2, 2, 200, 200, 128, seed=12)
    for t in (q, k, v, d_o):
        t[1] = float("nan")
    shape = mcs.AttnShape(2, 2, 2, 200, 200, 128)
    r = run(mcs, shape, q, k, v, d_o)
    want = attn_ref.attn(q[:1], k[:1], v[:1], d_o[:1])
    for name in want:
        attn_ref.check(r[name][:1], want[name], name)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hkv,Nq,Nk", [(2, 2, 100, 90), (4, 2, 300, 300), (2, 2, 130, 5000), (40, 40, 700, 256)])
def test_a_bad_query_shows_in_its_row_alone(mcs, Hq, Hkv, Nq, Nk, bad):
    """One slot, both slots with one tile, split keys, both slots with tiles of their own."""
    q, k, v, _ = inputs(1, Hq, Hkv, Nq, Nk, 64, seed=22)
    shape = mcs.AttnShape(1, Hq, Hkv, Nq, Nk, 64)
    good = run(mcs, shape, q, k, v)
    q[0, 77, 1, 5] = bad
    r = run(mcs, shape, q, k, v)
    assert r["o"][0, 77, 1].isnan().all() and r["lse"][0, 1, 77].isnan()
    r["o"][0, 77, 1], r["lse"][0, 1, 77] = good["o"][0, 77, 1], good["lse"][0, 1, 77]
    assert torch.equal(r["o"], good["o"]) and torch.equal(r["lse"], good["lse"])


def test_scale_and_large_scores(mcs):
    both(mcs, 1, 2, 2, 100, 300, 64, scale=1.0, gain=1.0, seed=13)
    both(mcs, 1, 2, 2, 100, 300, 64, scale=1e-4, gain=1.0, seed=14)


def test_a_row_of_equal_scores(mcs):
    """q = 0: every probability is 1 / n."""
    q, k, v, d_o = inputs(1, 2, 1, 130, 1000, 64, seed=15)
    both(mcs, 1, 2, 1, 130, 1000, 64, causal=True, tensors=(torch.zeros_like(q), k, v, d_o))


def test_long_rows(mcs):
    """Few queries over many keys, and many queries over few keys (shared heads)."""
    both(mcs, 1, 2, 1, 5, 20011, 128, causal=True, prefix=[77], seed=16)
    both(mcs, 1, 4, 1, 3001, 40, 64, slopes=[.01, .02, .03, .04], seed=17)
    both(mcs, 1, 2, 2, 2050, 2050, 128, causal=True, cap=30.0, seed=18)


def test_runs_repeat_bit_for_bit(mcs):
    q, k, v, d_o = inputs(2, 6, 2, 500, 500, 128, seed=19)
    ids = packed_ids(2, 500, 120, 2, 40).cuda()
    shape = mcs.AttnShape(2, 6, 2, 500, 500, 128, cap=30.0, causal=True)
    a, b = (run(mcs, shape, q, k, v, d_o, doc_q=ids, doc_k=ids) for _ in range(2))
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_no_lse_and_dirty_workspace(mcs):
    """lse is optional, and a workspace that held another call's data (its status block apart) gives the same."""
    q, k, v, d_o = inputs(1, 4, 2, 300, 300, 64, seed=20)
    ids = packed_ids(1, 300, 90, 3, 33).cuda()
    shape = mcs.AttnShape(1, 4, 2, 300, 300, 64)
    want = run(mcs, shape, q, k, v, d_o, doc_q=ids, doc_k=ids)
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_EX)
    wb = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD)
    ws[256:], wb[256:] = 0xff, 0xff
    o, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    mcs.mcs_dense_ex(shape, q, k, v, o, None, ws, doc_q=ids, doc_k=ids)
    mcs.mcs_dense_bwd(shape, q, k, v, o, want["lse"], d_o, dq, dk, dv, wb, doc_q=ids, doc_k=ids)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, want[n]), n
    assert mcs.mcs_poll_status(ws)[0] == 0 and mcs.mcs_poll_status(wb)[0] == 0


def test_streams_and_graphs(mcs):
    """On a side stream, and captured once and replayed on new contents of the same buffers."""
    shape = mcs.AttnShape(2, 4, 2, 260, 260, 64, cap=30.0, causal=True)
    q, k, v, d_o = inputs(2, 4, 2, 260, 260, 64, seed=21)
    ids = packed_ids(2, 260, 80, 5, 30).cuda()
    opts = dict(doc_q=ids, doc_k=ids)
    first = run(mcs, shape, q, k, v, d_o, **opts)
    o, lse = torch.empty_like(q), torch.empty(2, 4, 260, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws, wb = (mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD))

    def step():
        mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws, **opts)
        mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, wb, **opts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    got = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(got[n], first[n]) for n in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q2, k2, v2, d2 = inputs(2, 4, 2, 260, 260, 64, seed=22)
    want = run(mcs, shape, q2, k2, v2, d2, **opts)
    for t, n in ((q, q2), (k, k2), (v, v2), (d_o, d2)):
        t.copy_(n)
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in got)


def test_one_pass_equals_mcs_dense(mcs):
    """Without options the operator is the framework's dense attention."""
    q, k, v, _ = inputs(1, 3, 3, 400, 400, 128, seed=23)
    got = run(mcs, mcs.AttnShape(1, 3, 3, 400, 400, 128), q, k, v)
    s = mcs.Shape(1, 3, 400, 128)
    o, lse = torch.empty_like(q), torch.empty(1, 3, 400, device="cuda")
    mcs.mcs_dense(s, q, k, v, o, lse, mcs.workspace(s, mcs.MCS_OP_DENSE))
    want = attn_ref.attn(q, k, v)
    for n, t in (("o", o), ("lse", lse)):  # both lie within the same bound of the exact value
        attn_ref.check(got[n], want[n], n)
        attn_ref.check(t, want[n], n)


def test_queries_split_among_key_tiles(mcs):
    """Many query heads to one KV head, and few key tiles: dK and dV come as parts that are added."""
    both(mcs, 1, 8, 1, 2100, 300, 128, causal=True, cap=30.0, seed=24)
    both(mcs, 1, 24, 1, 1500, 1500, 64, causal=True, slopes=[.01 * h for h in range(24)], seed=25)
    ids = packed_ids(2, 900, 300, 7, 100)
    both(mcs, 2, 6, 1, 900, 900, 64, doc_q=ids, doc_k=ids, seed=26)


def test_documents_in_many_jobs(mcs):
    """More jobs than SMs, so that they run in the order of their tiles."""
    ids = packed_ids(3, 1300, 500, 8, 250)
    both(mcs, 3, 8, 8, 1300, 1300, 64, doc_q=ids, doc_k=ids, causal=True, prefix=[0, 700, 1300], seed=27)
    both(mcs, 3, 9, 3, 1300, 1300, 128, doc_q=ids, doc_k=ids, cap=20.0, seed=28)


@pytest.mark.parametrize("gain", [2.0, 6.0])
@pytest.mark.parametrize("N", [2, 3, 5, 17, 60, 256])
def test_few_keys_and_sharp_scores(mcs, N, gain):
    """dP - D cancels where a row has few keys: D must not carry o's rounding."""
    both(mcs, 2, 6, 3, N, N, 64, causal=True, gain=gain, seed=N)
    both(mcs, 1, 4, 4, N, N, 128, gain=gain, cap=30.0, slopes=[.1, .2, .3, .4], seed=N + 1)


@pytest.mark.parametrize("d", [64, 128])
def test_extreme_caps_and_scales(mcs, d):
    both(mcs, 1, 2, 1, 70, 150, d, cap=1e-6, seed=29)
    both(mcs, 1, 2, 1, 70, 150, d, cap=1e20, seed=30)
    both(mcs, 1, 2, 1, 70, 150, d, scale=1e-12, slopes=[.5, .01], seed=31)


def test_many_short_requests_with_documents(mcs):
    """More requests than a grid's second dimension holds."""
    B = 66000
    ids = torch.tensor([[0, 0, 1]], dtype=torch.int32).repeat(B, 1)
    both(mcs, B, 1, 1, 3, 3, 64, doc_q=ids, doc_k=ids, seed=32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("docs", [False, True])
def test_a_load_that_never_arrives_is_reported(mcs, docs, d):
    """The producer withholds its first tile (debug flag bit 0): the bounded waits run out, the status says so, and
    the next call computes."""
    from free_sparse_attention_pddp_b200.binding import debug_set_flags

    q, k, v, d_o = inputs(1, 2, 1, 140, 300, d, seed=33)
    shape = mcs.AttnShape(1, 2, 1, 140, 300, d)
    ids = dict(doc_q=torch.zeros(1, 140, dtype=torch.int32, device="cuda"),
               doc_k=torch.zeros(1, 300, dtype=torch.int32, device="cuda")) if docs else {}
    want = run(mcs, shape, q, k, v, d_o, **ids)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 140, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws, wb = (mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD))
    debug_set_flags(1)
    try:
        mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws, **ids)
        assert mcs.mcs_poll_status(ws)[0] == 4  # MCS_ERR_TIMEOUT
        mcs.mcs_dense_bwd(shape, q, k, v, want["o"], want["lse"], d_o, dq, dk, dv, wb, **ids)
        assert mcs.mcs_poll_status(wb)[0] == 4
    finally:
        debug_set_flags(0)
    again = run(mcs, shape, q, k, v, d_o, **ids)
    assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2])
def test_neighbouring_query_tiles_of_different_documents(mcs, g, d):
    """Pairs of query tiles whose documents need different keys, of equal and of very different number, with padding
    between and inside them."""
    for lengths in ([128, 900, 128, 300], [500, 140, 500, 30, 400], [256] * 6):
        ids = torch.cat([torch.full((n,), i if n != 30 else -1) for i, n in enumerate(lengths)])[None].int()
        ids[0, 200:203] = -1
        N = ids.shape[1]
        both(mcs, 1, 2 * g, 2, N, N, d, doc_q=ids, doc_k=ids, cap=30.0 * (g - 1), seed=N + g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lengths,pads", [(1, 1, (2300,), ()), (1, 1, (2100,), (150, 2099)), (40, 40, (500, 900, 260), (0, 700)),
                                                 (6, 2, (1300, 30, 760), (1299,))])
def test_a_slow_clearing_warp_changes_nothing(mcs, Hq, Hkv, lengths, pads, d):
    """The warp that clears padded rows falls ten steps behind in every tile (debug flag bit 3): the rings wait for it,
    whether tiles hold padding or not. One tile in both slots, pairs, slots with lists of their own."""
    from free_sparse_attention_pddp_b200.binding import debug_set_flags

    ids = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))[None].int()
    ids[0, list(pads)] = -1
    N = ids.shape[1]
    q, k, v, d_o = inputs(1, Hq, Hkv, N, N, d, seed=34)
    for t in (q, k, v, d_o):
        t[ids.cuda() < 0] = float("nan")
    ids = ids.cuda()
    shape = mcs.AttnShape(1, Hq, Hkv, N, N, d)
    want = run(mcs, shape, q, k, v, d_o, doc_q=ids, doc_k=ids)
    assert all(torch.isfinite(want[n]).all() for n in ("o", "dq", "dk", "dv"))
    debug_set_flags(8)
    try:
        got = run(mcs, shape, q, k, v, d_o, doc_q=ids, doc_k=ids)
    finally:
        debug_set_flags(0)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("opts", [dict(), dict(slopes=[.5, .01]), dict(cap=20.0)], ids=["plain", "biased", "capped"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_key_shows_in_every_row_that_sees_it(mcs, bad, opts, d):
    """Request b's key b holds a bad element: NaN in o and lse of the rows from b on, whatever column of a tile it
    lies in, and the rows before it as they were. An infinite score without a cap is such a row too."""
    if bad == float("inf") and "cap" in opts:
        pytest.skip("a cap makes a finite score of an infinite product")
    N = 200
    q, k, v, _ = inputs(N, 2, 1, N, N, d, seed=35)
    q[..., 3] = q[..., 3].abs() + 0.5  # so that an infinite element gives +inf
    slopes = None if "slopes" not in opts else torch.tensor(opts["slopes"], device="cuda")
    shape = mcs.AttnShape(N, 2, 1, N, N, d, cap=opts.get("cap", 0.0), causal=True)
    good = run(mcs, shape, q, k, v, slopes=slopes)
    at = torch.arange(N, device="cuda")
    k[at, at, 0, 3] = bad
    got = run(mcs, shape, q, k, v, slopes=slopes)
    sees = at[None] >= at[:, None]  # [request, row]
    assert got["o"][sees].isnan().all() and got["lse"].transpose(1, 2)[sees].isnan().all()
    assert torch.equal(got["o"][~sees], good["o"][~sees])
    assert torch.equal(got["lse"].transpose(1, 2)[~sees], good["lse"].transpose(1, 2)[~sees])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("N", [200, 600])
def test_a_bad_row_shows_in_its_gradients(mcs, N, docs, d):
    """A row whose o and lse are NaN is not an empty row: its dq is NaN, and dk and dv of the keys that it sees."""
    q, k, v, d_o = inputs(1, 2, 2, N, N, d, seed=36)
    ids = torch.repeat_interleave(torch.arange(2), torch.tensor([90, N - 90]))[None].int().cuda()
    opts = dict(doc_q=ids, doc_k=ids) if docs else {}
    shape = mcs.AttnShape(1, 2, 2, N, N, d, causal=True)
    good = run(mcs, shape, q, k, v, d_o, **opts)
    o, lse = good["o"].clone(), good["lse"].clone()
    o[0, 150, 1], lse[0, 1, 150] = float("nan"), float("nan")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD)
    mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, ws, **opts)
    assert mcs.mcs_poll_status(ws)[0] == 0
    seen = torch.zeros(N, dtype=torch.bool, device="cuda")
    seen[90 if docs else 0:151] = True
    assert dq[0, 150, 1].isnan().all() and dk[0, seen, 1].isnan().all() and dv[0, seen, 1].isnan().all()
    dq[0, 150, 1] = good["dq"][0, 150, 1]
    assert torch.equal(dq, good["dq"])
    for n, t in (("dk", dk), ("dv", dv)):
        t[0, seen, 1] = good[n][0, seen, 1]
        assert torch.equal(t, good[n]), n


def few_keys(mcs, B, Hq, Hkv, Nq, Nk, d, gain, seed, causal=False, prefix=None, ids=None, cap=0.0, slopes=None):
    """The gradients of rows that see at most 256 keys are held to the bound without o's rounding, row by row."""
    q, k, v, d_o = inputs(B, Hq, Hkv, Nq, Nk, d, seed, gain)
    dev = lambda x, t: None if x is None else torch.as_tensor(x, dtype=t).cuda().contiguous()  # noqa: E731
    prefix, slopes, doc_k = dev(prefix, torch.int32), dev(slopes, torch.float32), dev(ids, torch.int32)
    doc_q = None if ids is None else doc_k[:, Nk - Nq:].contiguous()
    shape = mcs.AttnShape(B, Hq, Hkv, Nq, Nk, d, cap=cap, causal=causal)
    got = run(mcs, shape, q, k, v, d_o, slopes=slopes, prefix=prefix, doc_q=doc_q, doc_k=doc_k)
    valid = attn_ref.valid_mask(B, Nq, Nk, causal, prefix, doc_q, doc_k, "cuda")
    few = valid.sum(-1) <= 256
    assert few.any()
    want = attn_ref.attn(q, k, v, d_o, cap=cap, slopes=slopes, valid=valid, exact_d=few)
    for name in ("lse", "o", "dv", "dk", "dq"):
        attn_ref.check(got[name], want[name], name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [2.0, 6.0])
def test_few_keys_of_a_row_in_a_long_call(mcs, gain, d):
    """Short documents packed into long rows, alone, beside long ones in one tile and interleaved; the first rows of
    causal masks; prefixes on both sides of 256."""
    few_keys(mcs, 1, 6, 2, 1500, 1500, d, gain, 41, ids=packed_ids(1, 1500, 16, 5, 40))
    mixed = torch.repeat_interleave(torch.arange(9), torch.tensor([3, 900, 7, 1, 500, 260, 16, 256, 257]))[None]
    few_keys(mcs, 1, 2, 2, mixed.shape[1], mixed.shape[1], d, gain, 42, ids=mixed)
    few_keys(mcs, 1, 3, 1, mixed.shape[1], mixed.shape[1], d, gain, 43, ids=mixed, causal=True, cap=30.0)
    few_keys(mcs, 2, 2, 1, 1900, 2000, d, gain, 44, ids=packed_ids(2, 2000, 40, 6, 70, shuffle=True))
    few_keys(mcs, 1, 4, 4, 1100, 1100, d, gain, 45, causal=True)
    few_keys(mcs, 3, 5, 1, 700, 700, d, gain, 46, causal=True, prefix=[0, 255, 257], slopes=[.01 * h for h in range(5)])
    few_keys(mcs, 1, 2, 2, 300, 500, d, gain, 47, causal=True)
    few_keys(mcs, 1, 2, 1, 800, 300, d, gain, 48, causal=True, cap=30.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("flag,Nk", [(16, 300), (32, 300), (64, 200)], ids=["key_tiles", "query_tiles", "few_keys"])
def test_a_load_that_never_arrives_in_one_kind_of_gradient_cta(mcs, flag, Nk, docs, d):
    """Only one kind of CTA misses its tile: it reports, and what the others compute is right."""
    from free_sparse_attention_pddp_b200.binding import debug_set_flags

    q, k, v, d_o = inputs(1, 2, 1, 140, Nk, d, seed=37)
    shape = mcs.AttnShape(1, 2, 1, 140, Nk, d)
    ids = dict(doc_q=torch.zeros(1, 140, dtype=torch.int32, device="cuda"),
               doc_k=torch.zeros(1, Nk, dtype=torch.int32, device="cuda")) if docs else {}
    want = run(mcs, shape, q, k, v, d_o, **ids)
    dq, dk, dv = (torch.full_like(t, 7.0) for t in (q, k, v))
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD)
    debug_set_flags(flag)
    try:
        mcs.mcs_dense_bwd(shape, q, k, v, want["o"], want["lse"], d_o, dq, dk, dv, ws, **ids)
        assert mcs.mcs_poll_status(ws)[0] == 4  # MCS_ERR_TIMEOUT
    finally:
        debug_set_flags(0)
    if flag == 16:
        assert torch.equal(dq, want["dq"]) and (dk == 7).all() and (dv == 7).all()
    if flag == 32:
        assert torch.equal(dk, want["dk"]) and torch.equal(dv, want["dv"]) and (dq == 7).all()
    again = run(mcs, shape, q, k, v, d_o, **ids)
    assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,mean", [(False, 0), (True, 0), (False, 1), (True, 5), (False, 90)])
def test_steep_slopes(mcs, causal, mean, d):
    """Slopes up to the bound, with rows that see near keys only. A score may be off by 2^-15 of the slope: in a tile of
    128 rows or 64 keys slope times row (or key) and slope times base are rounded by themselves, at most four
    roundings of 2^-24 of 128 slopes."""
    N, slopes = 300, torch.tensor([64.0, -64.0, 30.0, -7.0], device="cuda")
    q, k, v, d_o = inputs(1, 4, 2, N, N, d, seed=38)
    ids = packed_ids(1, N, mean, 9).cuda() if mean else None
    shape = mcs.AttnShape(1, 4, 2, N, N, d, causal=causal)
    got = run(mcs, shape, q, k, v, d_o, slopes=slopes, doc_q=ids, doc_k=ids)
    valid = attn_ref.valid_mask(1, N, N, causal, None, ids, ids, "cuda")
    want = attn_ref.attn(q, k, v, d_o, slopes=slopes, valid=valid, exact_d=valid.sum(-1) <= 256, slope_error=2.0 ** -15)
    for name in ("lse", "o", "dv", "dk", "dq"):
        attn_ref.check(got[name], want[name], name)


@pytest.mark.parametrize("bad", [65.0, -1e38, float("inf"), float("nan")])
def test_a_slope_out_of_range_is_reported(mcs, bad):
    q, k, v, d_o = inputs(1, 2, 2, 100, 300, 64, seed=39)
    slopes = torch.tensor([0.5, bad], device="cuda")
    shape = mcs.AttnShape(1, 2, 2, 100, 300, 64)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 100, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws, wb = (mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD))
    mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws, slopes=slopes)
    mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, wb, slopes=slopes)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    one, shared = mcs.DecodeShape(1, 2, 2, 300, 64), mcs.DecodeShape(1, 2, 2, 300, 64, P=300)
    w1, w2 = mcs.decode_workspace(one), mcs.decode_workspace(shared)
    qt, ot = q[:, 0].contiguous(), torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    mcs.mcs_decode(one, qt, k, v, lens, ot, None, w1, slopes=slopes)
    mcs.mcs_decode_shared(shared, qt, k[0], v[0], k, v, lens, ot, None, w2, slopes=slopes)
    for w in (ws, wb, w1, w2):
        status, info = mcs.mcs_poll_status(w)
        assert (status, info[1]) == (1, 1)  # MCS_ERR_INVALID_ARG, head 1
    assert torch.isfinite(o).all() and torch.isfinite(ot).all()


def test_missing_tensors_are_refused(mcs):
    """None in the place of a tensor that a call needs is refused like any other argument."""
    q, k, v, d_o = inputs(1, 2, 2, 10, 30, 64, seed=40)
    lse = torch.empty(1, 2, 10, device="cuda")
    shape = mcs.AttnShape(1, 2, 2, 10, 30, 64)
    ws, wb = (mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD))
    lens = torch.tensor([30], dtype=torch.int32, device="cuda")
    one, shared = mcs.DecodeShape(1, 2, 2, 30, 64), mcs.DecodeShape(1, 2, 2, 30, 64, P=30)
    qt, wd = q[:, 0].contiguous(), mcs.decode_workspace(shared)
    for call, args, tail in ((lambda *a: mcs.mcs_dense_ex(shape, *a), (q, k, v, q), (lse, ws)),
                             (lambda *a: mcs.mcs_dense_bwd(shape, *a), (q, k, v, q, lse, d_o, q, k, v), (wb,)),
                             (lambda *a: mcs.mcs_decode(one, *a), (qt, k, v, lens, qt), (None, wd)),
                             (lambda *a: mcs.mcs_decode_shared(shared, *a), (qt, k[0], v[0], k, v, lens, qt), (None, wd))):
        for i in range(len(args)):
            with pytest.raises(mcs.MCSError) as e:
                call(*args[:i], None, *args[i + 1:], *tail)
            assert e.value.code == 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,cap", [(0.125, 1e5), (1e-4, 1000.0), (1e-8, 100.0), (1e-12, 1e6), (1e12, 1e6), (1e12, 1e-6)])
def test_caps_far_from_the_scale(mcs, scale, cap, d):
    """Scores on both sides of the cap where scale / cap is far from 1. Each query has one element, so that a product is
    exact and the bound is the cap's own."""
    N, B = 150, 2
    q, k, v, d_o = inputs(B, 2, 1, N, N, d, seed=41)
    size = torch.linspace(0, 2.5, N, device="cuda")[None, :, None] * (cap / scale) * torch.tensor([1.0, -1.0], device="cuda")
    q.zero_()
    q[..., 5] = size.bfloat16()
    k[..., 5] = torch.tensor([0.125, 0.5, 1.0, 1.5], device="cuda")[torch.arange(N, device="cuda") % 4][None, :, None]
    both(mcs, B, 2, 1, N, N, d, scale=scale, cap=cap, tensors=(q, k, v, d_o))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [2.0, 6.0])
@pytest.mark.parametrize("opts", [dict(), dict(cap=20.0, causal=True), dict(slopes=True), dict(slopes=True, docs=700, causal=True)],
                         ids=["plain", "capped", "biased", "documents"])
def test_row_sums_in_long_calls(mcs, opts, gain, d):
    """The gradients of every row are held to the bound without o's rounding, whatever carries its P: all keys, a few
    (sharp scores), the near ones (a distance bias)."""
    N, Hq, Hkv = 1315, 6, 2
    q, k, v, d_o = inputs(1, Hq, Hkv, N, N, d, 51, gain)
    slopes = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device="cuda") if "slopes" in opts else None
    ids = packed_ids(1, N, opts["docs"], 3, 50).cuda() if "docs" in opts else None
    cap, causal = opts.get("cap", 0.0), opts.get("causal", False)
    got = run(mcs, mcs.AttnShape(1, Hq, Hkv, N, N, d, cap=cap, causal=causal), q, k, v, d_o, slopes=slopes, doc_q=ids,
              doc_k=ids)
    valid = attn_ref.valid_mask(1, N, N, causal, None, ids, ids, "cuda")
    want = attn_ref.attn(q, k, v, d_o, cap=cap, slopes=slopes, valid=valid, exact_d=True)
    for name in ("lse", "o", "dv", "dk", "dq"):
        attn_ref.check(got[name], want[name], name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,causal,mean", [(1, 4, 2, 200, 200, False, 0), (2, 6, 2, 601, 601, True, 0), (1, 5, 1, 300, 900, True, 0),
                                                        (2, 4, 4, 700, 700, False, 90), (1, 2, 1, 600, 130, True, 0)])
def test_row_sums_from_the_given_o(mcs, B, Hq, Hkv, Nq, Nk, causal, mean, d):
    """MCS_ATTN_D_FROM_O: the gradients within the bound that counts o's rounding, at every length; the forward is the
    same with the flag."""
    q, k, v, d_o = inputs(B, Hq, Hkv, Nq, Nk, d, seed=52)
    slopes = torch.tensor([.1 * (h + 1) for h in range(Hq)], device="cuda")
    ids = packed_ids(B, Nq, mean, 4, 40).cuda() if mean else None
    kw = dict(cap=30.0, causal=causal)
    a, b = (run(mcs, mcs.AttnShape(B, Hq, Hkv, Nq, Nk, d, **kw, d_from_o=f), q, k, v, d_o, slopes=slopes, doc_q=ids, doc_k=ids)
            for f in (False, True))
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"]) and not torch.equal(a["dq"], b["dq"])
    valid = attn_ref.valid_mask(B, Nq, Nk, causal, None, ids, ids, "cuda")
    want = attn_ref.attn(q, k, v, d_o, cap=30.0, slopes=slopes, valid=valid)
    for name in ("dv", "dk", "dq"):
        attn_ref.check(b[name], want[name], name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("parts", [(500, 400), (700, 60, 140)])
def test_gradients_of_a_joined_pair(mcs, parts, d):
    """Keys in parts: (o, lse) of each, joined, gives each part its gradients (MCS_ATTN_D_FROM_O); dq is their sum.

    o's parts are rounded, each by at most U of its share of sum P |v|, and the joined o once more, so D is off by at most twice
    what the bound counts; every part of dq is rounded by itself."""
    N, Hq, Hkv = 300, 4, 2
    q, k, v, d_o = inputs(1, Hq, Hkv, N, sum(parts), d, seed=53)
    pieces = list(zip([x.contiguous() for x in k.split(parts, 1)], [x.contiguous() for x in v.split(parts, 1)]))
    shapes = [mcs.AttnShape(1, Hq, Hkv, N, n, d, d_from_o=True) for n in parts]
    each = [run(mcs, s, q, kk, vv) for s, (kk, vv) in zip(shapes, pieces)]
    lse = torch.logsumexp(torch.stack([e["lse"] for e in each]), 0)
    o = sum(e["o"].float() * (e["lse"] - lse).exp().transpose(1, 2)[..., None] for e in each).bfloat16()
    dq, dk, dv = [], [], []
    for s, (kk, vv) in zip(shapes, pieces):
        out = [torch.empty_like(t) for t in (q, kk, vv)]
        ws = mcs.attn_workspace(s, mcs.MCS_OP_DENSE_BWD)
        mcs.mcs_dense_bwd(s, q, kk, vv, o, lse, d_o, *out, ws)
        assert mcs.mcs_poll_status(ws)[0] == 0
        for t, x in zip((dq, dk, dv), out):
            t.append(x)
    want = attn_ref.attn(q, k, v, d_o)
    twice = lambda n, more=0.0: (want[n][0], 2 * want[n][1] + more)  # noqa: E731
    attn_ref.check(torch.cat(dv, 1), twice("dv"), "dv")
    attn_ref.check(torch.cat(dk, 1), twice("dk"), "dk")
    attn_ref.check(sum(x.double() for x in dq), twice("dq", attn_ref.U * sum(x.double().abs() for x in dq)), "dq")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 3])
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(slopes=True)], ids=["plain", "capped", "biased"])
def test_a_single_key_has_no_score_gradient(mcs, kw, g, d):
    """A row with one key has P = 1 whatever its score: dq is 0 to the bit, and the row adds nothing to dk; in calls with one
    key, under a causal mask, and in documents of one token, alone or among others."""
    slopes = torch.tensor([.3 * (h + 1) for h in range(2 * g)], device="cuda") if "slopes" in kw else None
    shape = lambda n, nk, **k: mcs.AttnShape(2, 2 * g, 2, n, nk, d, cap=kw.get("cap", 0.0), **k)  # noqa: E731
    for n, nk in ((1, 1), (130, 1)):
        t = inputs(2, 2 * g, 2, n, nk, d, seed=61)
        got = run(mcs, shape(n, nk), *t, slopes=slopes)
        assert not got["dq"].any() and not got["dk"].any() and got["dv"].any()
    t = inputs(2, 2 * g, 2, 300, 300, d, seed=62)
    got = run(mcs, shape(300, 300, causal=True), *t, slopes=slopes)
    assert not got["dq"][:, 0].any() and got["dq"][:, 1].any()
    ids = torch.arange(300, dtype=torch.int32, device="cuda")[None].repeat(2, 1)
    got = run(mcs, shape(300, 300), *t, slopes=slopes, doc_q=ids, doc_k=ids)
    assert not got["dq"].any() and not got["dk"].any()
    ids[:, 100:250] = 100
    got = run(mcs, shape(300, 300), *t, slopes=slopes, doc_q=ids, doc_k=ids)
    alone = torch.ones(300, dtype=torch.bool, device="cuda")
    alone[100:250] = False
    assert not got["dq"][:, alone].any() and not got["dk"][:, alone].any() and got["dq"][:, ~alone].any()
