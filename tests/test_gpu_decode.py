"""mcs_decode and mcs_decode_shared against the 64-bit reference, and a run of all four calls together."""
import pytest

import attn_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mcs():
    import free_sparse_attention_pddp_b200 as m

    m.load()
    return m


def rand(g, *s):
    return torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)


def run(mcs, B, Hq, Hkv, C, d, lens, P=0, cap=0.0, scale=0.0, slopes=None, seed=0, gain=2.0, junk=float("nan"), status=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = rand(g, B, Hq, d) * gain, rand(g, B, C, Hkv, d), rand(g, B, C, Hkv, d)
    kp, vp = (rand(g, P, Hkv, d), rand(g, P, Hkv, d)) if P else (None, None)
    lens = torch.as_tensor(lens, dtype=torch.int32).cuda()
    unused = torch.arange(C, device="cuda")[None] >= lens[:, None]
    for t in (k, v):
        t[unused] = junk  # the cache behind a request's last key may hold anything
    slopes = None if slopes is None else torch.as_tensor(slopes, dtype=torch.float32).cuda()
    shape = mcs.DecodeShape(B, Hq, Hkv, C, d, P=P, scale=scale, cap=cap)
    ws = mcs.decode_workspace(shape)
    ws[256:] = 0xff
    whole = torch.full((q.numel() + 1024,), 12345.0, dtype=torch.bfloat16, device="cuda")
    o, lse = whole[512:-512].view_as(q), torch.full((B, Hq), 7.0, device="cuda")
    for _ in range(2):  # the second call finds the first one's workspace
        if P:
            mcs.mcs_decode_shared(shape, q, kp, vp, k, v, lens, o, lse, ws, slopes=slopes)
        else:
            mcs.mcs_decode(shape, q, k, v, lens, o, lse, ws, slopes=slopes)
        assert mcs.mcs_poll_status(ws)[0] == status
    assert (whole[:512] == whole[0]).all() and (whole[-512:] == whole[0]).all()
    want = attn_ref.decode(q, k, v, lens, kp, vp, scale=scale or None, cap=cap, slopes=slopes)
    attn_ref.check(lse, want["lse"], "lse")
    attn_ref.check(o, want["o"], "o")
    return o, lse


HEADS = [(1, 1), (4, 4), (8, 2), (5, 1), (12, 4), (16, 1), (34, 2), (128, 1), (40, 8)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_ragged_lengths(mcs, Hq, Hkv, d):
    lens = [1, 0, 63, 64, 65, 127, 128, 129, 500, 333]
    run(mcs, len(lens), Hq, Hkv, 500, d, lens, cap=20.0, slopes=[2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], seed=Hq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_ragged_lengths_behind_a_prefix(mcs, Hq, Hkv, d):
    lens = [1, 0, 63, 64, 200, 130, 17]
    run(mcs, len(lens), Hq, Hkv, 200, d, lens, P=257, slopes=[2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], seed=Hq)


@pytest.mark.parametrize("P", [1, 127, 128, 129, 1000])
@pytest.mark.parametrize("B", [1, 3, 40, 130])
def test_prefix_lengths_and_batches(mcs, P, B):
    run(mcs, B, 4, 2, 9, 64, [b % 10 for b in range(B)], P=P, cap=30.0, seed=P + B)


@pytest.mark.parametrize("B", [1, 2, 300])
@pytest.mark.parametrize("C", [1, 2, 7000])
def test_batches_and_capacities(mcs, B, C):
    run(mcs, B, 2, 1, C, 64, [max(1, (C * (7 * b + 3)) % (C + 1)) for b in range(B)], seed=B + C)


def test_long_and_short_requests_together(mcs):
    run(mcs, 4, 8, 2, 60000, 128, [60000, 3, 0, 41], seed=1)
    run(mcs, 1, 8, 8, 60000, 64, [59999], slopes=[.001] * 8, seed=2)


@pytest.mark.parametrize("P", [0, 300])
def test_nothing_cached(mcs, P):
    o, lse = run(mcs, 3, 4, 2, 16, 128, [0, 0, 0], P=P, seed=3)
    assert P or (torch.isneginf(lse).all() and (o == 0).all())


@pytest.mark.parametrize("P", [0, 150])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_cache_behind_the_last_key_may_hold_anything(mcs, junk, P):
    run(mcs, 3, 8, 2, 200, 128, [1, 70, 199], P=P, junk=junk, seed=4)


@pytest.mark.parametrize("B,C,P", [(200, 40, 0), (1, 400, 0), (3, 60000, 0), (3, 40, 130)])
def test_a_bad_query_shows_in_its_row_alone(mcs, B, C, P):
    """Whole requests, chunks joined within a cluster and by a second launch, a shared prefix."""
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = rand(g, B, 8, 64), rand(g, B, C, 2, 64), rand(g, B, C, 2, 64)
    kp, vp = rand(g, P or 1, 2, 64), rand(g, P or 1, 2, 64)
    lens = torch.full((B,), C, dtype=torch.int32, device="cuda")
    shape = mcs.DecodeShape(B, 8, 2, C, 64, P=P)
    ws = mcs.decode_workspace(shape)

    def call():
        o, lse = torch.empty_like(q), torch.empty(B, 8, device="cuda")
        if P:
            mcs.mcs_decode_shared(shape, q, kp, vp, k, v, lens, o, lse, ws)
        else:
            mcs.mcs_decode(shape, q, k, v, lens, o, lse, ws)
        return o, lse

    good = call()
    q[0, 3, 9] = float("nan")
    o, lse = call()
    assert o[0, 3].isnan().all() and lse[0, 3].isnan()
    o[0, 3], lse[0, 3] = good[0][0, 3], good[1][0, 3]
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("P", [0, 64])
def test_a_length_out_of_range_is_reported_and_bounded(mcs, P):
    run(mcs, 3, 4, 2, 50, 64, [12, 51, -3], P=P, junk=0.5, seed=5, status=5)


def test_caps_and_scales(mcs):
    for cap, gain, scale in ((0.5, 4.0, 0.0), (1000.0, 4.0, 0.0), (5.0, 8.0, 1.0), (0.0, 1.0, 1.0)):
        run(mcs, 2, 8, 2, 300, 64, [300, 111], P=140, cap=cap, gain=gain, scale=scale, seed=6)


def test_repeats_streams_and_graphs(mcs):
    g = torch.Generator(device="cuda").manual_seed(7)
    B, Hq, Hkv, C, P, d = 5, 8, 2, 700, 400, 128
    q, kp, vp = rand(g, B, Hq, d), rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    k, v = rand(g, B, C, Hkv, d), rand(g, B, C, Hkv, d)
    lens = torch.tensor([700, 5, 0, 320, 64], dtype=torch.int32, device="cuda")
    shape = mcs.DecodeShape(B, Hq, Hkv, C, d, P=P, cap=30.0)
    ws = mcs.decode_workspace(shape)
    o = torch.empty_like(q)

    def call():
        mcs.mcs_decode_shared(shape, q, kp, vp, k, v, lens, o, None, ws)

    call()
    first = o.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o.zero_()
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lens.copy_(torch.tensor([1, 699, 128, 0, 63]))  # lengths are read at replay
    q.copy_(rand(g, B, Hq, d))
    graph.replay()
    replayed = o.clone()
    call()
    assert torch.equal(replayed, o) and not torch.equal(o, first)
    want = attn_ref.decode(q, k, v, lens, kp, vp, cap=30.0)
    attn_ref.check(o, want["o"], "o")


def test_prefill_then_tokens_then_gradients(mcs):
    """A shared context, per-request continuations, then tokens one by one: every path gives the same attention.

    The rows of one causal pass over [context, continuation] equal, row by row, what the
    single-token calls give on the growing caches, and its gradients match the reference."""
    g = torch.Generator(device="cuda").manual_seed(8)
    B, Hq, Hkv, P, S, d, cap = 3, 8, 4, 200, 6, 64, 20.0
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(Hq)], device="cuda")
    kp, vp = rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    q, k, v = rand(g, B, S, Hq, d), rand(g, B, S, Hkv, d), rand(g, B, S, Hkv, d)
    kk = torch.cat([kp[None].expand(B, -1, -1, -1), k], 1).contiguous()
    vv = torch.cat([vp[None].expand(B, -1, -1, -1), v], 1).contiguous()
    shape = mcs.AttnShape(B, Hq, Hkv, S, P + S, d, cap=cap, causal=True)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, S, device="cuda")
    mcs.mcs_dense_ex(shape, q, kk, vv, o, lse, mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_EX), slopes=slopes)
    d_o = rand(g, B, S, Hq, d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(kk), torch.empty_like(vv)
    mcs.mcs_dense_bwd(shape, q, kk, vv, o, lse, d_o, dq, dk, dv, mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD),
                      slopes=slopes)
    valid = attn_ref.valid_mask(B, S, P + S, True, device="cuda")
    want = attn_ref.attn(q, kk, vv, d_o, cap=cap, slopes=slopes, valid=valid)
    for n, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        attn_ref.check(t, want[n], n)
    ds, dl = mcs.DecodeShape(B, Hq, Hkv, S, d, P=P, cap=cap), mcs.DecodeShape(B, Hq, Hkv, P + S, d, cap=cap)
    ws, wl = mcs.decode_workspace(ds), mcs.decode_workspace(dl)
    for t in range(S):
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        one, l1 = torch.empty(B, Hq, d, device="cuda", dtype=torch.bfloat16), torch.empty(B, Hq, device="cuda")
        two, l2 = torch.empty_like(one), torch.empty_like(l1)
        qt = q[:, t].contiguous()
        mcs.mcs_decode_shared(ds, qt, kp, vp, k, v, lens, one, l1, ws, slopes=slopes)
        mcs.mcs_decode(dl, qt, kk, vv, lens + P, two, l2, wl, slopes=slopes)
        for x, l in ((one, l1), (two, l2)):
            attn_ref.check(x, tuple(y[:, t] for y in want["o"]), f"token {t}")
            attn_ref.check(l, tuple(y[..., t] for y in want["lse"]), f"lse of token {t}")
    assert mcs.mcs_poll_status(ws)[0] == 0 and mcs.mcs_poll_status(wl)[0] == 0


@pytest.mark.parametrize("C", [65, 128, 300, 512, 4000])
def test_few_requests_whose_keys_are_split(mcs, C):
    """One to three requests, chunks joined within a cluster or by a second launch, some of them empty."""
    for B, Hq, Hkv in ((1, 12, 12), (3, 20, 1), (2, 40, 1)):
        run(mcs, B, Hq, Hkv, C, 64, [C, 1, 0][:B], cap=20.0, slopes=[.02] * Hq, seed=C + B)
        run(mcs, B, Hq, Hkv, C, 128, [C - 1, min(70, C - 1), 33][:B], seed=C)


@pytest.mark.parametrize("graph", [False, True])
def test_calls_back_to_back(mcs, graph):
    """Calls of several kernels each, one behind the other on one workspace, give what they give alone."""
    g = torch.Generator(device="cuda").manual_seed(9)
    Hq, Hkv, N, d, R, P, C = 32, 16, 1250, 64, 6, 700, 90
    q, k, v, d_o = rand(g, 1, N, Hq, d), rand(g, 1, N, Hkv, d), rand(g, 1, N, Hkv, d), rand(g, 1, N, Hq, d)
    ids = torch.repeat_interleave(torch.arange(3), torch.tensor([900, 20, 330]))[None].int().cuda()
    q1, kp, vp = rand(g, R, Hq, d), rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    kc, vc = rand(g, R, C, Hkv, d), rand(g, R, C, Hkv, d)
    lens = torch.tensor([90, 1, 0, 33, 64, 65], dtype=torch.int32, device="cuda")
    shape, step = mcs.AttnShape(1, Hq, Hkv, N, N, d), mcs.DecodeShape(R, Hq, Hkv, C, d, P=P)
    few = mcs.AttnShape(1, Hq, Hkv, 100, N, d)  # keys split, parts joined
    need = [mcs.mcs_attn_workspace_bytes(shape, mcs.MCS_OP_DENSE_EX), mcs.mcs_attn_workspace_bytes(few, mcs.MCS_OP_DENSE_EX),
            mcs.mcs_attn_workspace_bytes(shape, mcs.MCS_OP_DENSE_BWD), mcs.mcs_decode_workspace_bytes(step)]
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")

    def outputs():
        return {"o": torch.empty_like(q), "lse": torch.empty(1, Hq, N, device="cuda"), "dq": torch.empty_like(q),
                "dk": torch.empty_like(k), "dv": torch.empty_like(v), "o1": torch.empty_like(q1),
                "l1": torch.empty(R, Hq, device="cuda"), "of": torch.empty_like(q[:, :100]).contiguous()}

    q_few = q[:, :100].contiguous()

    def calls(r):
        return [lambda: mcs.mcs_dense_ex(shape, q, k, v, r["o"], r["lse"], ws, doc_q=ids, doc_k=ids),
                lambda: mcs.mcs_dense_ex(few, q_few, k, v, r["of"], None, ws),
                lambda: mcs.mcs_dense_bwd(shape, q, k, v, r["o"], r["lse"], d_o, r["dq"], r["dk"], r["dv"], ws,
                                          doc_q=ids, doc_k=ids),
                lambda: mcs.mcs_decode_shared(step, q1, kp, vp, kc, vc, lens, r["o1"], r["l1"], ws)]

    alone = outputs()
    for call in calls(alone):
        call()
        torch.cuda.synchronize()
    runs = [outputs() for _ in range(8)]

    def run_all():
        for r in runs:
            for call in calls(r):
                call()

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run_all()
        for r in runs:
            for t in r.values():
                t.zero_()
        captured.replay()
    else:
        run_all()
    assert mcs.mcs_poll_status(ws)[0] == 0
    for r in runs:
        for name, t in r.items():
            assert torch.equal(t.view(torch.uint8), alone[name].view(torch.uint8)), name


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (40, 40), (33, 1)])
@pytest.mark.parametrize("C,n", [(20000, 20000), (20000, 19937), (20000, 301), (20000, 1), (20000, 0), (5000, 4990)])
def test_a_single_request_of_any_length(mcs, Hq, Hkv, C, n):
    """Its keys are cut by its length, not by the cache's capacity."""
    run(mcs, 1, Hq, Hkv, C, 64, [n], P=130 if n == 301 else 0, seed=n)


@pytest.mark.parametrize("d", [64, 128])
def test_a_load_of_the_prefix_that_never_arrives_is_reported(mcs, d):
    """The prefix's producer withholds its first tile (debug flag bit 0): the bounded waits run out, the status says
    so, and the next call computes."""
    from free_sparse_attention_pddp_b200.binding import debug_set_flags

    g = torch.Generator(device="cuda").manual_seed(10)
    B, Hq, Hkv, C, P = 3, 4, 2, 40, 300
    q, kp, vp = rand(g, B, Hq, d), rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    k, v = rand(g, B, C, Hkv, d), rand(g, B, C, Hkv, d)
    lens = torch.tensor([40, 0, 7], dtype=torch.int32, device="cuda")
    shape = mcs.DecodeShape(B, Hq, Hkv, C, d, P=P)
    ws = mcs.decode_workspace(shape)

    def call(status):
        o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
        mcs.mcs_decode_shared(shape, q, kp, vp, k, v, lens, o, lse, ws)
        assert mcs.mcs_poll_status(ws)[0] == status
        return o, lse

    want = call(0)
    debug_set_flags(1)
    try:
        call(4)  # MCS_ERR_TIMEOUT
    finally:
        debug_set_flags(0)
    assert all(torch.equal(x, y) for x, y in zip(call(0), want))


def test_calls_side_by_side(mcs):
    """Two streams, each with workspaces and outputs of its own, run all four calls at the same time; one of them also
    from a captured graph."""
    g = torch.Generator(device="cuda").manual_seed(11)
    Hq, Hkv, N, d, R, P, C = 12, 4, 700, 128, 5, 500, 300
    q, k, v, d_o = rand(g, 2, N, Hq, d), rand(g, 2, N, Hkv, d), rand(g, 2, N, Hkv, d), rand(g, 2, N, Hq, d)
    ids = torch.repeat_interleave(torch.arange(3), torch.tensor([30, 600, 70]))[None].repeat(2, 1).int().cuda()
    q1, kp, vp = rand(g, R, Hq, d), rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    kc, vc = rand(g, R, C, Hkv, d), rand(g, R, C, Hkv, d)
    lens = torch.tensor([300, 1, 0, 133, 64], dtype=torch.int32, device="cuda")
    shape = mcs.AttnShape(2, Hq, Hkv, N, N, d, cap=20.0, causal=True)
    step, one = mcs.DecodeShape(R, Hq, Hkv, C, d, P=P), mcs.DecodeShape(R, Hq, Hkv, C, d)

    class Caller:
        def __init__(self):
            self.ws = [mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD)]
            self.ws += [mcs.decode_workspace(s) for s in (step, one)]
            self.out = [torch.empty_like(t) for t in (q, q, k, v, q1, q1)]
            self.lse = torch.empty(2, Hq, N, device="cuda")

        def __call__(self):
            o, dq, dk, dv, o1, o2 = self.out
            mcs.mcs_dense_ex(shape, q, k, v, o, self.lse, self.ws[0], doc_q=ids, doc_k=ids)
            mcs.mcs_decode_shared(step, q1, kp, vp, kc, vc, lens, o1, None, self.ws[2])
            mcs.mcs_dense_bwd(shape, q, k, v, o, self.lse, d_o, dq, dk, dv, self.ws[1], doc_q=ids, doc_k=ids)
            mcs.mcs_decode(one, q1, kc, vc, lens, o2, None, self.ws[3])

    want = Caller()
    want()
    torch.cuda.synchronize()
    callers, streams = [Caller(), Caller()], [torch.cuda.Stream(), torch.cuda.Stream()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        callers[1]()
    for c in callers:
        for t in c.out:
            t.zero_()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            callers[0]()
        with torch.cuda.stream(streams[1]):
            graph.replay()
    torch.cuda.synchronize()
    for c in callers:
        assert all(mcs.mcs_poll_status(w)[0] == 0 for w in c.ws)
        assert all(torch.equal(x, y) for x, y in zip(c.out, want.out))


def test_streams_as_arguments(mcs):
    """A stream given to the call, as torch's object or its handle, is the one that it runs on."""
    g = torch.Generator(device="cuda").manual_seed(12)
    N, Hq, Hkv, d, P = 300, 4, 2, 64, 200
    q, k, v, d_o = rand(g, 1, N, Hq, d), rand(g, 1, N, Hkv, d), rand(g, 1, N, Hkv, d), rand(g, 1, N, Hq, d)
    q1, kp, vp = rand(g, 1, Hq, d), rand(g, P, Hkv, d), rand(g, P, Hkv, d)
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    shape, one, behind = mcs.AttnShape(1, Hq, Hkv, N, N, d), mcs.DecodeShape(1, Hq, Hkv, N, d), mcs.DecodeShape(1, Hq, Hkv, N, d, P=P)
    ws = [mcs.attn_workspace(shape, op) for op in (mcs.MCS_OP_DENSE_EX, mcs.MCS_OP_DENSE_BWD)]
    ws += [mcs.decode_workspace(s) for s in (one, behind)]

    def call(stream, inputs):
        q, k, v, d_o, q1 = inputs
        o, dq, dk, dv, a, b = (torch.zeros_like(t) for t in (q, q, k, v, q1, q1))
        lse = torch.zeros(1, Hq, N, device="cuda")
        return [o, dq, dk, dv, a, b], [
            lambda: mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws[0], stream=stream),
            lambda: mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, ws[1], stream=stream),
            lambda: mcs.mcs_decode(one, q1, k, v, lens, a, None, ws[2], stream=stream),
            lambda: mcs.mcs_decode_shared(behind, q1, kp, vp, k, v, lens, b, None, ws[3], stream=stream)]

    want, calls = call(None, (q, k, v, d_o, q1))
    for f in calls:
        f()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        late = [torch.zeros_like(t) for t in (q, k, v, d_o, q1)]
        got, calls = call(stream, late)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # the inputs come late on that stream: another one would read zeros
            torch.cuda._sleep(20_000_000)
            for t, s in zip(late, (q, k, v, d_o, q1)):
                t.copy_(s)
        for f in calls:
            f()
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
