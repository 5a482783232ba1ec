"""Attention with modified scores in 64 bits, from its formulas, with elementwise error bounds.

The bounds follow the kernels' arithmetic. u = 2^-8 is half a bf16 step
relative to the value, e = 2^-24 half an fp32 step.
  x = scale q.k in fp32: |dx| <= (d + 8) e scale sum |q||k|. The cap, the bias
  and the exponential add at most 2^-20 (1 + |s|) to the score (a few fp32
  roundings of values of that size, and approximate instructions good to
  2^-21). Es_i is the largest score error of row i.
  P: relative error <= 2 Es_i (its own score and the row's sum), then u where it
  is rounded to bf16; every sum over n terms adds n e of the terms' sizes.
  o: u |o| + (u + 2 Es_i + n e) sum P |v|.
  dS = P (dP - D) (1 - t^2): dP like x; D = d_o.o with the o that was rounded, or
  summed from P dP in fp32.
  dq, dk, dv: u of the value, plus the terms' errors times |k|, |q|, |d_o|.
  Underflow: a probability below 2^-126, fp32's and bf16's smallest normal
  number, may become 0, and so may a result. With at most 2^17 terms of size
  below 2^9 (the scaled rows of these tests) that is off by at most 2^-100.
"""
import math

import torch

U = 2.0 ** -8
E = 2.0 ** -24
TINY = 2.0 ** -100


def valid_mask(B, Nq, Nk, causal=False, prefix=None, doc_q=None, doc_k=None, device="cpu"):
    """bool [B, Nq, Nk]"""
    pos = torch.arange(Nq, device=device) + Nk - Nq
    key = torch.arange(Nk, device=device)
    ok = torch.ones(B, Nq, Nk, dtype=torch.bool, device=device)
    if causal:
        reach = (key[None] <= pos[:, None])[None].expand(B, -1, -1)
        if prefix is not None:
            reach = reach | (key[None, None] < prefix[:, None, None])
        ok = ok & reach
    if doc_q is not None:
        ok = ok & (doc_q[:, :, None] == doc_k[:, None, :]) & (doc_q[:, :, None] >= 0)
    return ok


def attn(q, k, v, d_o=None, scale=None, cap=0.0, slopes=None, pos=None, valid=None, exact_d=False, slope_error=0.0):
    """q [B,Nq,Hq,d], k, v [B,Nk,Hkv,d] of any type; pos [B or 1, Nq] query positions; valid bool [B,Nq,Nk].

    Returns a dict of (value, bound) pairs, fp64: o [B,Nq,Hq,d], lse [B,Hq,Nq] and,
    with d_o, dq, dk, dv. Rows that no pair needs may hold NaN. exact_d: D is summed from P dP in fp32, in
    all rows (True) or in those of a mask [B, Nq].
    slope_error: what a score may be off by, times its head's slope."""
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1:3]
    g = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    if pos is None:
        pos = torch.arange(Nq, device=q.device)[None] + Nk - Nq
    if valid is None:
        valid = torch.ones(B, Nq, Nk, dtype=torch.bool, device=q.device)
    clean = lambda x: torch.nan_to_num(x.double(), nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
    Q = clean(q).permute(0, 2, 1, 3)
    K = clean(k).permute(0, 2, 1, 3).repeat_interleave(g, 1)
    V = clean(v).permute(0, 2, 1, 3).repeat_interleave(g, 1)
    x = scale * Q @ K.transpose(-1, -2)
    ex = (d + 8) * E * abs(scale) * (Q.abs() @ K.abs().transpose(-1, -2))
    t = torch.tanh(x / cap) if cap else torch.zeros_like(x)
    s = cap * t if cap else x
    if slopes is not None:
        dist = (pos[:, :, None] - torch.arange(Nk, device=q.device)[None, None]).abs().double()
        s = s - slopes.double()[None, :, None, None] * dist[:, None]
    ok = valid[:, None]
    es = ex + 2.0 ** -20 * (1 + s.abs())
    if slope_error:
        es = es + slope_error * slopes.double().abs()[None, :, None, None]
    s = s.masked_fill(~ok, -math.inf)
    Es = es.masked_fill(~ok, 0.0).amax(-1)
    lse = torch.logsumexp(s, -1)
    live = ~torch.isneginf(lse)
    P = torch.where(ok & live[..., None], torch.exp(s - torch.where(live, lse, 0.0)[..., None]), 0.0)
    tol_lse = Es + Nk * E + 2 * E * lse.abs().nan_to_num(posinf=0.0, neginf=0.0) + 2.0 ** -21
    tol_lse = torch.where(live, tol_lse, torch.zeros_like(tol_lse))
    Ep = (2 * Es + tol_lse + (Nk + 16) * E)[..., None]
    o = P @ V
    tol_o = U * o.abs() + (U + Ep) * (P @ V.abs())
    back = lambda y: y.permute(0, 2, 1, 3)  # noqa: E731
    out = {"o": (back(o), back(tol_o)), "lse": (lse, tol_lse)}
    if d_o is not None:
        G = clean(d_o).permute(0, 2, 1, 3)
        dP = G @ V.transpose(-1, -2)
        D = (G * o).sum(-1, keepdim=True)
        w = 1 - t * t
        dS = P * (dP - D) * w
        edp = (d + 8) * E * (G.abs() @ V.abs().transpose(-1, -2))
        ed = (G.abs() * (tol_o + (d + 8) * E * o.abs())).sum(-1, keepdim=True)
        if exact_d is not False:  # dP's and P's errors, and the sum's
            rows = torch.as_tensor(exact_d, device=q.device).expand(B, Nq)[:, None, :, None]
            ed = torch.where(rows, (P * (edp + Ep * dP.abs())).sum(-1, keepdim=True), ed)
        et = 2.0 ** -20 + (es / cap if cap else 0.0)  # of t
        tol_dS = U * dS.abs() + P * w * (edp + ed + Ep * (dP - D).abs()) + P * (dP - D).abs() * 2 * t.abs() * et
        if not cap:
            tol_dS = U * dS.abs() + P * (edp + ed + Ep * (dP - D).abs())
        n = (Nk + Nq * g + 16) * E
        shared = lambda y: y.reshape(B, Hkv, g, Nk, d).sum(2).permute(0, 2, 1, 3)  # noqa: E731
        dq = scale * dS @ K
        out["dq"] = (back(dq), back(U * dq.abs() + scale * (tol_dS + n * dS.abs()) @ K.abs()))
        dk = shared(scale * dS.transpose(-1, -2) @ Q)
        out["dk"] = (dk, U * dk.abs() + shared(scale * (tol_dS + n * dS.abs()).transpose(-1, -2) @ Q.abs()))
        dv = shared(P.transpose(-1, -2) @ G)
        out["dv"] = (dv, U * dv.abs() + shared((P * (U + Ep + n)).transpose(-1, -2) @ G.abs()))
    return out


def decode(q, k, v, lens, kp=None, vp=None, scale=None, cap=0.0, slopes=None):
    """q [B,Hq,d], caches [B,C,Hkv,d], lens [B], prefix [P,Hkv,d]: (value, bound) of o [B,Hq,d] and lse [B,Hq]."""
    B, C = k.shape[:2]
    P = 0 if kp is None else kp.shape[0]
    n = lens.clamp(0, C).long()
    if P:
        k = torch.cat([kp[None].expand(B, -1, -1, -1), k], 1)
        v = torch.cat([vp[None].expand(B, -1, -1, -1), v], 1)
    pos = (P + n - 1)[:, None]
    valid = (torch.arange(P + C, device=q.device)[None] < P + n[:, None])[:, None]
    r = attn(q[:, None], k, v, scale=scale, cap=cap, slopes=slopes, pos=pos, valid=valid)
    return {"o": tuple(y[:, 0] for y in r["o"]), "lse": tuple(y[..., 0] for y in r["lse"])}


def check(got, want, what):
    """`got` lies within the bound of `want` = (value, bound) everywhere; infinities are equal."""
    value, bound = want
    got = got.double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    inf = torch.isinf(value)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], value[inf]), f"{what}: infinities differ"
    err = (got - value)[~inf].abs()
    over = err - bound[~inf] - TINY
    assert not torch.isnan(err).any(), f"{what}: NaN"
    if over.numel():
        i = int(over.argmax())
        assert over.flatten()[i] <= 0, (f"{what}: off by {float(err.flatten()[i]):.3e}, bound "
                                        f"{float(bound[~inf].flatten()[i]):.3e}, {int((over > 0).sum())} of "
                                        f"{over.numel()} values over")
