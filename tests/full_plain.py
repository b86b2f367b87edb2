"""Plain 64-bit forms of the full-attention and paged-cache operators for the
parity tests, with elementwise error bounds derived from what the kernels
round.

Bounds, per element (u = half a step of the type: bf16 2^-8, fp32 2^-24):
  scores     products of bf16 are exact in fp32; summing d of them in fp32
             errs by at most es = (d + 4) 2^-24 scale sum |q||k|, + 2^-22 |s| for
             the scaling and the conversion to base 2
  weights    p = exp(s - m): relative ep = 2 es + 2^-21 (exp2's and expf's own
             errors are below 2^-21), the factor 2 for s and for the row's m
  out        (u_out |out|) + (u_P + ep + n 2^-23) sum_j p_j |v_j|: the output's
             rounding, the weight's rounding (bf16 only), the sums of n terms
             (numerator and denominator)
  lse        es + 2^-21 + n 2^-24 + 2^-23 |lse|
  gradients  P errs by ep (from the given lse); dP by (d + 4) 2^-24 sum |dout||v|;
             delta by (d + 4) 2^-24 sum |dout||out|; so dS errs by
             eds = |dS| (ep + 2^-22) + P (ddP + ddelta), and the product rounds
             P and dS (bf16 only): dq errs by u|dq| + scale sum_j (u_P |dS| +
             eds + n 2^-24 |dS|) |k_j|, dk and dv alike.
"""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U_P = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}  # weights before their product


def _attend(q, k, v, scale, u_dtype):
    """One sequence: q [Lq, Hq, d], k, v [Lk, Hkv, d] in 64 bits -> out, lse, bounds."""
    Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[:2]
    kk, vv = (x.repeat_interleave(Hq // Hkv, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    mag = torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()) * scale
    seen = torch.arange(Lk)[None] <= torch.arange(Lq)[:, None] + (Lk - Lq)
    es = (d + 4) * 2.0 ** -24 * mag + 2.0 ** -22 * s.abs()
    es = es.masked_fill(~seen, 0.0).amax(-1) if Lk else torch.zeros(Hq, Lq, dtype=torch.float64)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if Lk else torch.full((Hq, Lq), -math.inf, dtype=torch.float64)
    p = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hij,jhd->ihd", p, vv)
    ep = 2 * es + 2.0 ** -21
    tol = U[u_dtype] * out.abs() + torch.einsum("hij,jhd->ihd", p, vv.abs()) * (
        U_P[u_dtype] + ep + Lk * 2.0 ** -23).T[..., None]
    ltol = es + 2.0 ** -21 + Lk * 2.0 ** -24 + 2.0 ** -23 * torch.where(lse.isinf(), 0.0, lse.abs())
    return out, lse.T, tol, ltol.T, p, s, es


def prefill(q, k, v, spans, scale, dtype):
    """q [Tq, Hq, d], keys per sequence: spans (q0, Lq) and k, v lists [Lk, Hkv, d].
    Returns out, lse and their bounds; rows of no sequence are NaN in all."""
    res = [torch.full(q.shape, math.nan, dtype=torch.float64), torch.full(q.shape[:2], math.nan, dtype=torch.float64)]
    res += [x.clone() for x in res]
    for (q0, Lq), kb, vb in zip(spans, k, v):
        got = _attend(q[q0:q0 + Lq].double(), kb.double(), vb.double(), scale, dtype)
        for r, x in zip(res, got):
            r[q0:q0 + Lq] = x
    return res


def backward(q, k, v, out, dout, lse, scale, dtype):
    """One sequence's dq, dk, dv and their bounds (all inputs in 64 bits)."""
    Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[:2]
    hpg = Hq // Hkv
    kk, vv = (x.repeat_interleave(hpg, 1) for x in (k, v))
    seen = torch.arange(Lk)[None] <= torch.arange(Lq)[:, None] + (Lk - Lq)
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    mag = torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()) * scale
    l = torch.where(lse.isinf(), torch.zeros_like(lse), lse).T[..., None]
    p = torch.exp(s - l) * seen
    delta = (dout * out).sum(-1).T[..., None]
    dp = torch.einsum("ihd,jhd->hij", dout, vv)
    ds = p * (dp - delta)
    e = (d + 4) * 2.0 ** -24
    ep = e * mag + 2.0 ** -22 * (s.abs() + l.abs()) + 2.0 ** -21
    eds = ds.abs() * (ep + 2.0 ** -22) + p * (
        e * torch.einsum("ihd,jhd->hij", dout.abs(), vv.abs()) + e * (dout.abs() * out.abs()).sum(-1).T[..., None])
    fold = lambda x: x.reshape(Lk, Hkv, hpg, d).sum(2)  # noqa: E731  heads of a group into their key/value head
    dq = scale * torch.einsum("hij,jhd->ihd", ds, kk)
    dk = scale * fold(torch.einsum("hij,ihd->jhd", ds, q))
    dv = fold(torch.einsum("hij,ihd->jhd", p, dout))
    u, up = U[dtype], U_P[dtype]
    n = Lk
    wq = ds.abs() * (up + n * 2.0 ** -24) + eds
    tq = u * dq.abs() + scale * torch.einsum("hij,jhd->ihd", wq, kk.abs())
    n = Lq * hpg
    wk = ds.abs() * (up + n * 2.0 ** -24) + eds
    tk = u * dk.abs() + scale * fold(torch.einsum("hij,ihd->jhd", wk, q.abs()))
    tv = u * dv.abs() + fold(torch.einsum("hij,ihd->jhd", p * (up + ep + n * 2.0 ** -24), dout.abs()))
    return (dq, dk, dv), (tq, tk, tv)


def rotate(x, rope, pos, rot, interleaved):
    """x [n, heads, d] in 64 bits, rotated at positions pos [n]."""
    y = x.clone()
    c, s = (rope[pos, :, i].double()[:, None] for i in (0, 1))
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def rope_table(max_pos, rot, base=10000.0):
    half = rot // 2
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * base ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def paged(seqs_k, seqs_v, page, gen, spare=2, max_pages=None, fill=math.nan):
    """Lists of [Lk, Hkv, d] laid into shuffled pages; every other row of the
    cache holds `fill`, unused table entries a page number out of range."""
    Hkv, d = seqs_k[0].shape[1:]
    need = [-(-x.shape[0] // page) for x in seqs_k]
    num = sum(need) + spare
    order = torch.randperm(num, generator=gen).tolist()
    mp = max_pages or max(need + [1])
    table = torch.full((len(need), mp), 1 << 30, dtype=torch.int32)
    kc = torch.full((num, page, Hkv, d), fill, dtype=seqs_k[0].dtype)
    vc = kc.clone()
    at = 0
    for b, (n, kb, vb) in enumerate(zip(need, seqs_k, seqs_v)):
        mine = order[at:at + n]
        at += n
        table[b, :n] = torch.tensor(mine, dtype=torch.int32)
        for i, p in enumerate(mine):
            m = min(page, kb.shape[0] - i * page)
            kc[p, :m], vc[p, :m] = kb[i * page:i * page + m], vb[i * page:i * page + m]
    return kc, vc, table


def offsets(lens, start=0):
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def assert_within(got, want, tol, what):
    """|got - want| <= tol elementwise; infinities equal; NaN in `want` marks elements not compared."""
    got, keep = got.double().cpu(), ~want.isnan()
    g, w, t = got[keep], want[keep], tol[keep]
    inf = w.isinf()
    assert torch.equal(g[inf], w[inf]), f"{what}: infinities differ"
    bad = ~((g - w).abs() <= t) & ~inf
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {g.numel()} beyond the bound, worst |err| "
                           f"{(g - w)[bad].abs().max():.3g} against {t[bad].max():.3g}")
