"""Plain forms of the 8-bit caches and their decode, in 64 bits, with bounds.

An e4m3 row is exact: the same codes and scales are expected bit for bit (a
rotated key counts as its 64-bit rotation rounded to fp32). Decode, on top of
full_plain.py's bounds (u = half a step; log2 units: s2 = s log2 e):
  scores   es as there, + 2^-22 |s| for the two scales' products; fp32 queries
           are two f16 terms, 2^-22 of each: + 2^-22 scale sum |q||k|
  weights  w = exp2((s2 - mw) + log2 vs): roundings of both sums, of log2 and of
           the final exp2(mw - m), 2^-22 (max|s2| + max|log2 vs| + 16) in all;
           then f16: 2^-11 (bf16), two terms 2^-22 (fp32), and what lies below
           f16's least step, 2^-31 of the largest weight, per key
"""
from __future__ import annotations

import math

import torch

import full_plain as fp

U_W = {torch.bfloat16: 2.0 ** -11, torch.float32: 2.0 ** -22}
E4M3 = torch.float8_e4m3fn


def quantise(y):
    """Rows [..., d] of fp32 values -> e4m3 codes, scales [...] fp32."""
    y = y.double()
    top = y.abs().amax(-1)
    exp = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    exp = torch.where(top > torch.exp2(exp) * 448, exp + 1, exp)  # should log2 have rounded
    exp = torch.where((exp > -126) & (top <= torch.exp2(exp - 1) * 448), exp - 1, exp).clamp_min(-126)
    scale = torch.where(top > 0, torch.exp2(exp), torch.zeros_like(top))
    codes = (y * torch.exp2(-exp)[..., None]).float().to(E4M3)  # exact but for what is far below a code
    bad = ~y.isfinite().all(-1)
    return codes, torch.where(bad, torch.full_like(scale, math.nan), scale).float()


def paged(codes_k, codes_v, scale_k, scale_v, page, gen, max_pages=None):
    """Lists of codes [L, Hkv, d] and scales [L, Hkv] laid into shuffled pages;
    all else is NaN, in codes and scales."""
    as_int = lambda xs: [x.view(torch.uint8) for x in xs]  # noqa: E731
    state = gen.get_state()
    kc, vc, table = fp.paged(as_int(codes_k), as_int(codes_v), page, gen, max_pages=max_pages, fill=0x7f)
    gen.set_state(state)
    ks, vs, _ = fp.paged([x[..., None] for x in scale_k], [x[..., None] for x in scale_v], page, gen,
                         max_pages=max_pages)
    laid = lambda x: x[..., 0].transpose(1, 2).contiguous()  # noqa: E731
    return kc.view(E4M3), vc.view(E4M3), laid(ks), laid(vs), table


def decode(q, codes_k, codes_v, scale_k, scale_v, scale, dtype):
    """q [B, Hq, d]; lists per sequence. out, lse and their bounds, all 64-bit."""
    B, Hq, d = q.shape
    out, tol = torch.zeros(B, Hq, d, dtype=torch.float64), torch.zeros(B, Hq, d, dtype=torch.float64)
    lse, ltol = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b, (kc, vc, ks, vs) in enumerate(zip(codes_k, codes_v, scale_k, scale_v)):
        n, Hkv = ks.shape
        if n == 0:
            continue
        rep = lambda x: x.repeat_interleave(Hq // Hkv, 1)  # noqa: E731
        k, v = (rep(c.double() * s.double()[..., None]) for c, s in ((kc, ks), (vc, vs)))
        x = torch.einsum("hd,jhd->hj", q[b].double(), k) * scale
        mag = torch.einsum("hd,jhd->hj", q[b].double().abs(), k.abs()) * scale
        es = (d + 4) * 2.0 ** -24 * mag + 2.0 ** -21 * x.abs()
        if dtype == torch.float32:
            es = es + 2.0 ** -22 * mag
        es = es.amax(-1)
        lse[b] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[b][:, None])
        out[b] = torch.einsum("hj,jhd->hd", p, v)
        lv = torch.where(vs > 0, torch.log2(vs.double()).abs(), torch.zeros_like(vs).double())
        ew = 2.0 ** -22 * (x.abs().amax(-1) / math.log(2) + rep(lv).amax(0) + 16)
        ep = 2 * es + 2.0 ** -21 + ew
        size = torch.einsum("hj,jhd->hd", p, v.abs())
        least = n * 2.0 ** -31 * (p.T[..., None] * rep(vs.double())[..., None]).amax(0) * 448
        tol[b] = fp.U[dtype] * out[b].abs() + size * (U_W[dtype] + ep + n * 2.0 ** -23)[:, None] + least
        ltol[b] = es + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -23 * lse[b].abs()
    return out, lse, tol, ltol
