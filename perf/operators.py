"""Cases of the attention operators with modified scores: what is measured, and the operators' plain forms.

Operators: `mcs_dense_ex` (forward: cap, distance bias, causal, prefix and
document masks, shared KV heads), `mcs_dense_bwd` (its gradients), `mcs_decode`
(one token per request over a cache) and `mcs_decode_shared` (the same with a
prefix that all requests share).
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------------- cases

def _attn(name, op, B, Hq, Hkv, Nq, Nk, d, cap=0.0, slopes=False, causal=False, prefix=0, docs=0, pad=0):
    """docs: mean document length of a packed row (0: no documents); pad: padded tokens at a row's end;
    prefix: longest prefix of the batch (0: no prefix mask)."""
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, cap=cap, slopes=slopes, causal=causal,
                prefix=prefix, docs=docs, pad=pad)


def _decode(name, op, B, Hq, Hkv, C, shortest, d, P=0, cap=0.0, slopes=False):
    """C: the cache's capacity and its longest request; shortest: the shortest request; P: shared prefix."""
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, C=C, shortest=shortest, d=d, P=P, cap=cap, slopes=slopes)


def listed():
    return [
        # a short prompt of two requests, capped scores, odd length: latency counts
        _attn("fwd_prompt", "fwd", 2, 8, 4, 333, 333, 64, cap=30.0, causal=True),
        # an ordinary causal pass with a distance bias and shared KV heads
        _attn("fwd_bias", "fwd", 1, 16, 4, 4096, 4096, 128, slopes=True, causal=True),
        # a chunk of new frames that follows a long context: few rows, many keys, prefix visible to all
        _attn("fwd_chunk", "fwd", 1, 12, 12, 390, 32760, 128, causal=True, prefix=1560),
        # clips packed into one row of the 480p video length, with a padded tail
        _attn("fwd_packed", "fwd", 1, 2, 2, 32760, 32760, 128, docs=6000, pad=700),
        # training on a small ragged batch: padded rows, capped scores, three query heads to a KV head
        _attn("train_ragged", "train", 2, 6, 2, 601, 601, 64, cap=20.0, docs=150, pad=90),
        # training, ordinary: causal with a bidirectional prefix (conditioning frames)
        _attn("train_prefix", "train", 1, 16, 8, 4096, 4096, 128, causal=True, prefix=1024),
        # training, the largest: full attention over 8192 tokens with capped scores
        _attn("train_full", "train", 1, 12, 12, 8192, 8192, 128, cap=50.0),
        # one request's next token over a short cache: the smallest call
        _decode("decode_one", "decode", 1, 12, 12, 512, 480, 64, cap=30.0),
        # a batch of requests of very different lengths
        _decode("decode_ragged", "decode", 64, 40, 8, 8192, 100, 128, slopes=True),
        # one long context, the 720p video length
        _decode("decode_long", "decode", 1, 40, 8, 75600, 75600, 128),
        # a few samples that share a short prompt
        _decode("shared_few", "shared", 8, 16, 4, 128, 1, 128, P=4096, cap=50.0),
        # a large batch of samples that share a long conditioning context
        _decode("shared_many", "shared", 64, 40, 8, 1024, 0, 128, P=32760, slopes=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "train", "decode", "shared"])
    Hkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
    cap, slopes = rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.4
    while True:
        if op in ("fwd", "train"):
            Nk = _spread(rng, 1, 32760 if op == "fwd" else 8192)
            Nq = Nk if op == "train" or rng.random() < 0.6 else _spread(rng, 1, Nk)
            B = rng.choice([1, 1, 2, 3])
            causal = rng.random() < 0.6
            docs = _spread(rng, 16, Nk) if Nq == Nk and Nk > 16 and rng.random() < 0.4 else 0
            c = _attn("drawn", op, B, Hkv * g, Hkv, Nq, Nk, d, cap, slopes, causal,
                      prefix=rng.randint(1, Nk) if causal and rng.random() < 0.4 else 0,
                      docs=docs, pad=rng.randint(0, Nk // 4) if docs else 0)
            if B * Hkv * g * Nq * Nk <= (2 * 32760 ** 2 if op == "fwd" else 12 * 8192 ** 2):
                break
        else:
            C = _spread(rng, 1, 75600 if op == "decode" else 4096)
            P = 0 if op == "decode" else _spread(rng, 16, 32760)
            c = _decode("drawn", op, _spread(rng, 1, 96), Hkv * g, Hkv, C, rng.randint(0, C), d, P, cap, slopes)
            if c["B"] * Hkv * C * d <= 64 * 8 * 8192 * 128:
                break
    del c["name"]
    return c


# --------------------------------------------------------------------------- layouts (from the case alone)

def _doc_ids(case):
    """int32 [B, N]: documents one after the other, the padded tail -1."""
    rng = np.random.RandomState(case["docs"] + case["Nk"])
    B, N = case["B"], case["Nk"]
    starts = rng.random_sample((B, N)) < 1.0 / case["docs"]
    ids = np.cumsum(starts, axis=1)
    pad = (case["pad"] * (1 + np.arange(B))) // B
    ids[np.arange(N)[None] >= N - pad[:, None]] = -1
    return ids.astype(np.int32)


def _prefixes(case):
    B = case["B"]
    return ((case["prefix"] * (1 + np.arange(B))) // B).astype(np.int32)


def _lens(case):
    """int32 [B]: request lengths from `shortest` to C, the first one C."""
    B, C, lo = case["B"], case["C"], min(case["shortest"], case["C"])
    lens = np.random.RandomState(C + B).randint(lo, C + 1, B)
    lens[0] = C
    return lens.astype(np.int32)


def _pairs(case):
    """Valid (query, key) pairs of one query head, summed over the batch."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    pos = np.arange(Nq) + Nk - Nq
    total = 0
    ids = _doc_ids(case) if case["docs"] else None
    for b in range(B):
        if case["causal"]:
            most = np.maximum(pos + 1, _prefixes(case)[b] if case["prefix"] else 0)
        else:
            most = np.full(Nq, Nk)
        most = np.clip(most, 0, Nk)
        if ids is None:
            total += int(most.sum())
            continue
        live = ids[b] >= 0
        first = np.searchsorted(ids[b][live], ids[b][live], side="left")
        last = np.searchsorted(ids[b][live], ids[b][live], side="right")
        total += int(np.maximum(0, np.minimum(last, most[live]) - first).sum())
    return total


def work(case):
    Hq, Hkv, d, B = case["Hq"], case["Hkv"], case["d"], case["B"]
    if case["op"] in ("fwd", "train"):
        Nq, Nk = case["Nq"], case["Nk"]
        q, kv, lse = 2 * B * Nq * Hq * d, 2 * B * Nk * Hkv * d, 4 * B * Hq * Nq
        pairs = _pairs(case) * Hq
        if case["op"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * pairs}
        # forward and gradients: 2 + 5 products; q, k, v, do in, o, lse, dq, dk, dv out
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * d * pairs}
    keys = int(_lens(case).sum())
    return {"bytes": 4 * Hkv * d * (keys + case["P"]) + 4 * B * Hq * d + 4 * B * Hq,
            "flops": 4 * d * Hq * (keys + B * case["P"])}


# --------------------------------------------------------------------------- inputs

def _dev(a):
    return torch.from_numpy(a).cuda()


def _inputs(case, seed):
    """The tensors of a case, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) * gain).contiguous()

    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    # queries twice as long as after a plain norm: scores with a spread of 2, as learned gains give
    s = {"case": case}
    if case["op"] in ("fwd", "train"):
        s["q"] = normal(B, case["Nq"], Hq, d, gain=2.0)
        s["k"], s["v"] = normal(B, case["Nk"], Hkv, d), normal(B, case["Nk"], Hkv, d)
        if case["op"] == "train":
            s["do"] = normal(B, case["Nq"], Hq, d)
        s["docs"] = _dev(_doc_ids(case)) if case["docs"] else None
        s["prefix"] = _dev(_prefixes(case)) if case["prefix"] else None
    else:
        s["q"] = normal(B, Hq, d, gain=2.0)
        s["k"], s["v"] = normal(B, case["C"], Hkv, d), normal(B, case["C"], Hkv, d)
        if case["op"] == "shared":
            s["kp"], s["vp"] = normal(case["P"], Hkv, d), normal(case["P"], Hkv, d)
        s["lens"] = _dev(_lens(case))
    # one slope to a head, falling geometrically
    s["slopes"] = _dev((2.0 ** (-8.0 * (1 + np.arange(Hq)) / Hq)).astype(np.float32)) if case["slopes"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    # what a program that uses the framework keeps: output buffers (the workspace comes with the first call)
    s["o"] = torch.empty_like(s["q"])
    if case["op"] in ("fwd", "train"):
        s["lse"] = torch.empty(case["B"], case["Hq"], case["Nq"], dtype=torch.float32, device="cuda")
        if case["op"] == "train":
            s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        s["lse"] = torch.empty(case["B"], case["Hq"], dtype=torch.float32, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms

def _mask(s):
    """Valid pairs, bool, broadcast over [B, Hkv, g, Nq, Nk]; None where every pair is valid."""
    case = s["case"]
    Nq, Nk = case["Nq"], case["Nk"]
    valid = None
    if case["causal"]:
        pos = torch.arange(Nq, device="cuda") + (Nk - Nq)
        key = torch.arange(Nk, device="cuda")
        valid = (key[None, :] <= pos[:, None])[None]
        if s["prefix"] is not None:
            valid = valid | (key[None, None, :] < s["prefix"][:, None, None])
    if s["docs"] is not None:
        doc = s["docs"]
        same = (doc[:, Nk - Nq:, None] == doc[:, None, :]) & (doc >= 0)[:, None, :]
        valid = same if valid is None else valid & same
    return None if valid is None else valid[:, None, None]


def _softmax(x):
    """Probabilities and lse over the last axis; a row without a valid score gives 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    return e.div_(l.clamp_min(1e-37)), (m + l.log()).squeeze(-1)


def _heads(x, Hkv):
    """[B, N, H, d] -> fp32 [B, Hkv, g N, d], g = H / Hkv: the rows that meet one KV head"""
    B, N, H, d = x.shape
    return x.float().view(B, N, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)


def _tokens(x, like):
    """[B, Hkv, g N, d] -> the type and layout [B, N, H, d] of `like`"""
    B, N, H, d = like.shape
    return x.view(B, x.shape[1], -1, N, d).permute(0, 3, 1, 2, 4).reshape(like.shape).to(like.dtype)


def _plain_attn(s):
    case = s["case"]
    B, Hq, Hkv, Nq, Nk, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    scale, cap = 1.0 / math.sqrt(d), case["cap"]
    q, k, v = _heads(s["q"], Hkv), _heads(s["k"], Hkv), _heads(s["v"], Hkv)
    x = (q @ k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, Nq, Nk)
    x *= scale
    t = None
    if cap:
        t = torch.tanh_(x / cap)
        x = t * cap
    if s["slopes"] is not None:
        pos = torch.arange(Nq, device="cuda") + (Nk - Nq)
        dist = (pos[:, None] - torch.arange(Nk, device="cuda")[None, :]).abs().float()
        x -= s["slopes"].view(1, Hkv, Hq // Hkv, 1, 1) * dist
    valid = _mask(s)
    if valid is not None:
        x = x.masked_fill_(~valid, -math.inf)
    p, lse = _softmax(x)
    p = p.view(B, Hkv, -1, Nk)
    out = {"o": _tokens(p @ v, s["o"]), "lse": lse.reshape(B, Hq, Nq)}
    if case["op"] == "train":
        do = _heads(s["do"], Hkv)
        ds = do @ v.transpose(-1, -2)
        ds -= (p * ds).sum(-1, keepdim=True)
        ds *= p
        if cap:
            ds *= (1 - t * t).view(ds.shape)
        out["dv"] = _tokens(p.transpose(-1, -2) @ do, s["dv"])
        out["dq"] = _tokens((ds @ k) * scale, s["dq"])
        out["dk"] = _tokens((ds.transpose(-1, -2) @ q) * scale, s["dk"])
    return out


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hkv, C, P, d = (case[n] for n in ("B", "Hq", "Hkv", "C", "P", "d"))
    cap, lens = case["cap"], s["lens"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)  # [B, Hkv, C, d]
    x = q @ k.transpose(-1, -2)
    key = torch.arange(C, device="cuda")
    if P:
        kp, vp = s["kp"].float().transpose(0, 1), s["vp"].float().transpose(0, 1)  # [Hkv, P, d]
        rows = q.transpose(0, 1).reshape(Hkv, -1, d)  # every request's rows meet the prefix in one product
        x = torch.cat([(rows @ kp.transpose(-1, -2)).view(Hkv, B, -1, P).transpose(0, 1), x], -1)
        key = torch.arange(P + C, device="cuda")
    x /= math.sqrt(d)
    if cap:
        x = torch.tanh(x / cap) * cap
    if s["slopes"] is not None:
        dist = (P + lens[:, None] - 1 - key[None, :]).abs().float()
        x = x - s["slopes"].view(1, Hkv, Hq // Hkv, 1) * dist[:, None, None, :]
    x = x.masked_fill_((key[None, :] >= P + lens[:, None])[:, None, None, :], -math.inf)
    p, lse = _softmax(x)
    o = p[..., P:] @ v
    if P:
        rows = p[..., :P].transpose(0, 1).reshape(Hkv, -1, P)
        o = o + (rows @ vp).view(Hkv, B, -1, d).transpose(0, 1)
    return {"o": o.view(B, Hq, d).to(s["o"].dtype), "lse": lse.reshape(B, Hq)}


# --------------------------------------------------------------------------- the framework's calls

def _own_attn(s):
    import free_sparse_attention_pddp_b200 as mcs

    case = s["case"]
    if "shape" not in s:
        s["shape"] = mcs.AttnShape(case["B"], case["Hq"], case["Hkv"], case["Nq"], case["Nk"], case["d"],
                                   cap=case["cap"], causal=case["causal"])
        s["ws"] = mcs.attn_workspace(s["shape"], mcs.MCS_OP_DENSE_EX)
        if case["op"] == "train":
            s["ws_bwd"] = mcs.attn_workspace(s["shape"], mcs.MCS_OP_DENSE_BWD)
    opts = dict(slopes=s["slopes"], prefix=s["prefix"], doc_q=s["docs"], doc_k=s["docs"])
    mcs.mcs_dense_ex(s["shape"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["ws"], **opts)
    out = {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "train":
        mcs.mcs_dense_bwd(s["shape"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"],
                          s["ws_bwd"], **opts)
        out.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return out


def _own_decode(s):
    import free_sparse_attention_pddp_b200 as mcs

    case = s["case"]
    if "shape" not in s:
        s["shape"] = mcs.DecodeShape(case["B"], case["Hq"], case["Hkv"], case["C"], case["d"], P=case["P"],
                                     cap=case["cap"])
        s["ws"] = mcs.decode_workspace(s["shape"])
    if case["op"] == "decode":
        mcs.mcs_decode(s["shape"], s["q"], s["k"], s["v"], s["lens"], s["o"], s["lse"], s["ws"], slopes=s["slopes"])
    else:
        mcs.mcs_decode_shared(s["shape"], s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], s["o"], s["lse"],
                              s["ws"], slopes=s["slopes"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    if state["case"]["op"] in ("fwd", "train"):
        return _own_attn(state) if own else _plain_attn(state)
    return _own_decode(state) if own else _plain_decode(state)


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    g, cap, scale = Hq // Hkv, case["cap"], d ** -0.5

    def row_block(q, k, h, pos, valid):
        """Scores, d(score)/d(scaled product), probabilities and lse of some rows of head h, fp64."""
        z = torch.einsum("id,jd->ij", q, k) * scale
        slope = 1.0
        if cap:
            w = torch.tanh(z / cap)
            z, slope = cap * w, 1.0 - w.square()
        if s["slopes"] is not None:
            at = torch.arange(k.shape[0], device="cuda", dtype=torch.float64)
            z = z - s["slopes"][h].double() * (pos.double()[:, None] - at[None, :]).abs()
        z = torch.where(valid, z, torch.full_like(z, -math.inf))
        lse = torch.logsumexp(z, dim=1)
        live = torch.isfinite(lse)
        prob = torch.where(live[:, None], torch.exp(z - torch.where(live, lse, torch.zeros_like(lse))[:, None]),
                           torch.zeros_like(z))
        return slope, prob, lse

    if case["op"] in ("decode", "shared"):
        P = case["P"]
        o = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["lens"][b])
            for kv in range(Hkv):
                k, v = s["k"][b, :n, kv].double(), s["v"][b, :n, kv].double()
                if P:
                    k, v = torch.cat([s["kp"][:, kv].double(), k]), torch.cat([s["vp"][:, kv].double(), v])
                if k.shape[0] == 0:
                    lse[b, kv * g:(kv + 1) * g] = -math.inf
                    continue
                at = torch.tensor([P + n - 1], device="cuda")
                for h in range(kv * g, (kv + 1) * g):
                    every = torch.ones(1, k.shape[0], dtype=torch.bool, device="cuda")
                    _, prob, lse[b, h] = row_block(s["q"][b, h][None].double(), k, h, at, every)
                    o[b, h] = (prob @ v)[0]
        return {"o": o, "lse": lse}

    Nq, Nk = case["Nq"], case["Nk"]
    o = torch.zeros(B, Nq, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, Nq, dtype=torch.float64, device="cuda")
    train = case["op"] == "train"
    if train:
        dq = torch.zeros_like(o)
        dk, dv = (torch.zeros(B, Nk, Hkv, d, dtype=torch.float64, device="cuda") for _ in range(2))
    key = torch.arange(Nk, device="cuda")
    for b in range(B):
        for h in range(Hq):
            k, v = s["k"][b, :, h // g].double(), s["v"][b, :, h // g].double()
            for i0 in range(0, Nq, 8192):
                i1 = min(Nq, i0 + 8192)
                pos = torch.arange(i0, i1, device="cuda") + (Nk - Nq)
                valid = torch.ones(i1 - i0, Nk, dtype=torch.bool, device="cuda")
                if case["causal"]:
                    reach = pos + 1
                    if s["prefix"] is not None:
                        reach = torch.maximum(reach, s["prefix"][b].expand_as(reach))
                    valid &= key[None] < reach[:, None]
                if s["docs"] is not None:
                    mine = s["docs"][b][pos]
                    valid &= (mine[:, None] == s["docs"][b][None]) & (mine >= 0)[:, None]
                q = s["q"][b, i0:i1, h].double()
                slope, prob, lse[b, h, i0:i1] = row_block(q, k, h, pos, valid)
                o[b, i0:i1, h] = prob @ v
                if train:
                    up = s["do"][b, i0:i1, h].double()
                    delta = (up * o[b, i0:i1, h]).sum(1, keepdim=True)
                    grad = prob * (up @ v.T - delta) * slope * scale
                    dq[b, i0:i1, h] = grad @ k
                    dk[b, :, h // g] += grad.T @ q
                    dv[b, :, h // g] += prob.T @ up
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=dq, dk=dk, dv=dv)
    return out
