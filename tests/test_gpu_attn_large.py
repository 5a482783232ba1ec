"""Attention with modified scores where offsets pass 32 bits: values from closed forms, every element compared.

With q = 0 a row's probabilities are 1 / n, and with v the same for all of a request's keys o is that value exactly up
to P's rounding, one half bf16 step (2^-8), and o's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mcs():
    import free_sparse_attention_pddp_b200 as m

    m.load()
    yield m
    torch.cuda.empty_cache()


def by_request(B, *shape):
    """bf16 [B, *shape]: request b holds b + 1, exact up to 256."""
    t = torch.empty(B, *shape, dtype=torch.bfloat16, device="cuda")
    return t.copy_((torch.arange(B, device="cuda") + 1).view(B, *[1] * len(shape)))


def near(t, want):
    """Within two half steps; the difference is taken request by request, so that no copy doubles the tensor."""
    return all(float((t[b].float() - want[b]).abs().max()) <= 2.0 ** -7 * abs(want[b]) for b in range(t.shape[0]))


def test_a_cache_of_more_than_2_31_elements(mcs):
    B, Hq, Hkv, C, d = 3, 16, 8, 750000, 128
    k, v = torch.zeros(B, C, Hkv, d, dtype=torch.bfloat16, device="cuda"), by_request(B, C, Hkv, d)
    assert k.numel() > 2 ** 31
    lens = torch.tensor([17, C, C - 1], dtype=torch.int32, device="cuda")
    q, o = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Hq, device="cuda")
    shape = mcs.DecodeShape(B, Hq, Hkv, C, d)
    ws = mcs.decode_workspace(shape)
    v[0, 17:], k[0, 17:] = float("nan"), float("nan")
    mcs.mcs_decode(shape, q, k, v, lens, o, lse, ws)
    assert mcs.mcs_poll_status(ws)[0] == 0
    assert near(o, [1.0, 2.0, 3.0])
    # lse = log n: fp32 sums of up to 750000 equal terms, joined, and a logarithm
    assert float((lse - lens.float().log()[:, None]).abs().max()) < 1e-5
    # the prefix as long as the cache
    P = B * C - 5
    shape = mcs.DecodeShape(2, Hq, Hkv, 9, d, P=P)
    ws = mcs.decode_workspace(shape)
    kp, vp = k.view(-1, Hkv, d)[:P], v.view(-1, Hkv, d)[:P]
    kp[:17 + C], vp[:] = 0, 3.0
    mcs.mcs_decode_shared(shape, q[:2], kp, vp, k[2, :18].view(2, 9, Hkv, d), v[2, :18].view(2, 9, Hkv, d),
                          torch.tensor([9, 0], dtype=torch.int32, device="cuda"), o[:2], lse[:2], ws)
    assert mcs.mcs_poll_status(ws)[0] == 0
    assert near(o[:2], [3.0, 3.0])
    want = torch.tensor([P + 9.0, P], dtype=torch.float64).log()
    assert float((lse[:2].double().cpu() - want[:, None]).abs().max()) < 1e-5


@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("Nq,Nk,Hq,Hkv", [(8200, 60, 64, 64), (60, 8200, 64, 64)])
def test_tensors_of_more_than_2_31_elements(mcs, Nq, Nk, Hq, Hkv, docs):
    """Queries, or keys, past 2^31 elements, and their gradients: q = 0, so dk = 0, dv is d_o's sum over the rows by 1 / n;
    v and d_o are constant, so dP - D = 0 up to the rounding of D's parts."""
    B, d = 33, 128
    q = torch.zeros(B, Nq, Hq, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(B, Nk, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v, d_o = by_request(B, Nk, Hkv, d), by_request(B, Nq, Hq, d)
    assert max(q.numel(), k.numel()) > 2 ** 31
    opts = {}
    if docs:
        opts = dict(doc_q=torch.zeros(B, Nq, dtype=torch.int32, device="cuda"),
                    doc_k=torch.zeros(B, Nk, dtype=torch.int32, device="cuda"))
    shape = mcs.AttnShape(B, Hq, Hkv, Nq, Nk, d)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, Nq, device="cuda")
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_EX)
    mcs.mcs_dense_ex(shape, q, k, v, o, lse, ws, **opts)
    assert mcs.mcs_poll_status(ws)[0] == 0
    size = [b + 1.0 for b in range(B)]
    assert near(o, size) and float((lse - torch.tensor(float(Nk)).log()).abs().max()) < 1e-5
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ws = mcs.attn_workspace(shape, mcs.MCS_OP_DENSE_BWD)
    mcs.mcs_dense_bwd(shape, q, k, v, o, lse, d_o, dq, dk, dv, ws, **opts)
    assert mcs.mcs_poll_status(ws)[0] == 0
    assert not dq.any() and not dk.any()  # k = 0 and q = 0
    assert near(dv, [x * Nq / Nk for x in size])
