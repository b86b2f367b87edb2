"""Rows whose visible scores are all -inf; long prompts, whose items are handed
out whole, and the gradients of long documents."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp
from test_gpu_full_attn import BF16, DEV, FP32

pytestmark = pytest.mark.gpu


def _case(dtype, Hq=8, Hkv=2, d=64, L=(300, 200, 260)):
    """The scores of the first sequence's keys and of the second's first 130
    overflow to -inf (-2^130, of finite inputs): no row of the first and the
    second's first 130 have anything to divide by."""
    g = torch.Generator().manual_seed(1)
    T = sum(L)
    q, k, v = (torch.randn(T, h, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    q, k = (q.abs() + 1) * 2.0 ** 60, k * 2.0 ** -60
    k[:L[0] + 130] = -2.0 ** 70
    cu = fp.offsets(L)
    undefined = torch.zeros(T, dtype=torch.bool)
    undefined[:L[0] + 130] = True
    return q, k, v, cu, L, undefined, g


def _want(q, k, v, cu, dtype):
    """Plain attention of the rows that have a finite score: the others' keys left out."""
    a, m, e = int(cu[1]), int(cu[1]) + 130, int(cu[2])
    spans = [(m, e - m), (e, int(cu[3]) - e)]
    return fp.prefill(q, [k[m:e], k[e:]], [v[m:e], v[e:]], spans, q.shape[-1] ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_without_a_finite_score(dtype):
    """exp(-inf) over a sum of zeros is undefined: NaN, and -inf as the sum's
    logarithm, in every form; 0 is for rows that see no key."""
    q, k, v, cu, L, undefined, g = _case(dtype)
    want = _want(q, k, v, cu, dtype)
    on = cu.to(DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = msa.msa_full_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), on, on, lse=lse)
    assert out.cpu()[undefined].isnan().all() and (lse.cpu()[undefined] == -math.inf).all()
    fp.assert_within(out, want[0], want[2], "out")
    fp.assert_within(lse, want[1], want[3], "lse")
    # the same over pages, and each sequence's last row as a decode step
    page = 16
    ks, vs = ([x[int(a):int(b)] for a, b in zip(cu[:-1], cu[1:])] for x in (k, v))
    kc, vc, table = (x.to(DEV) for x in fp.paged(ks, vs, page, g))
    kv = torch.tensor(L, dtype=torch.int32, device=DEV)
    out = msa.msa_full_attn_prefill_paged(q.to(DEV), kc, vc, table, on, kv, lse=lse)
    assert out.cpu()[undefined].isnan().all() and (lse.cpu()[undefined] == -math.inf).all()
    fp.assert_within(out, want[0], want[2], "paged")
    last = (cu[1:] - 1).long()
    lse = torch.empty(3, q.shape[1], device=DEV)
    out = msa.msa_full_attn_decode(q[last].to(DEV), kc, vc, table, kv, lse=lse)
    assert out[0].isnan().all() and (lse[0] == -math.inf).all()
    fp.assert_within(out[1:], want[0][last[1:]], want[2][last[1:]], "decode")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_split_rows_without_a_finite_score(dtype):
    """The same where few rows walk many keys and their parts are joined."""
    g = torch.Generator().manual_seed(2)
    Hq, Hkv, d, Lk = 4, 1, 64, 6000
    q, k, v = (torch.randn(n, h, d, generator=g).to(dtype) for n, h in ((3, Hq), (Lk, Hkv), (Lk, Hkv)))
    q, k = (q.abs() + 1) * 2.0 ** 60, k * 2.0 ** -60
    k[:Lk - 1] = -2.0 ** 70  # -inf as a score; the last row alone sees the one key with a finite one
    cu_q, cu_k = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([0, Lk], dtype=torch.int32)
    lse = torch.empty(3, Hq, device=DEV)
    out = msa.msa_full_attn_prefill(*[x.to(DEV) for x in (q, k, v, cu_q, cu_k)], lse=lse)
    assert out[:2].isnan().all() and (lse[:2] == -math.inf).all()
    assert torch.equal(out[2].cpu(), v[-1].expand(Hq, d))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_of_rows_without_a_finite_score(dtype):
    """Their weights are undefined, and so is every gradient that they enter;
    the other sequences' stay right."""
    q, k, v, cu, L, undefined, g = _case(dtype)
    on = cu.to(DEV)
    lse = torch.empty(q.shape[:2], device=DEV)
    dev = [x.to(DEV) for x in (q, k, v)]
    out = msa.msa_full_attn_prefill(*dev, on, on, lse=lse)
    dout = torch.randn(q.shape, generator=g).to(dtype)
    dq, dk, dv = (x.cpu() for x in msa.msa_full_attn_backward(*dev, out, dout.to(DEV), lse, on, on))
    a, e = int(cu[1]), int(cu[2])
    for x in (dq, dk, dv):
        assert x[:a].isnan().all() and x[a:a + 130].isnan().all()
    sl = slice(e, int(cu[3]))
    w, t = fp.backward(*[x[sl].double() for x in (q, k, v, out.cpu(), dout, lse.cpu())], q.shape[-1] ** -0.5, dtype)
    for name, got, x, y in zip(("dq", "dk", "dv"), (dq, dk, dv), w, t):
        fp.assert_within(got[sl], x, y, name)


@pytest.mark.parametrize("heads,lens", [((32, 8, 128), [8192]), ((16, 16, 64), [5000, 1, 3333])])
def test_long_prompts(heads, lens):
    """Whole prompts of thousands of tokens: many items of many key tiles each,
    handed out whole. Rows all over the prompt against the plain form."""
    Hq, Hkv, d = heads
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(T, h, d, generator=g).to(BF16) for h in (Hq, Hkv, Hkv))
    cu = fp.offsets(lens).to(DEV)
    lse = torch.empty(T, Hq, device=DEV)
    out = msa.msa_full_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu, cu, lse=lse).cpu()
    lse = lse.cpu()
    q0 = 0
    for n in lens:
        for i in sorted({0, min(1, n - 1), n // 3, n // 2, max(n - 130, 0), n - 1} | set(range(min(n, 64) - 1, n, 511))):
            kk, vv = k[q0:q0 + i + 1], v[q0:q0 + i + 1]
            w = fp.prefill(q[q0 + i:q0 + i + 1], [kk], [vv], [(0, 1)], d ** -0.5, BF16)
            fp.assert_within(out[q0 + i:q0 + i + 1], w[0], w[2], f"row {i} of {n}")
            fp.assert_within(lse[q0 + i:q0 + i + 1], w[1], w[3], f"lse of row {i} of {n}")
        q0 += n


@pytest.mark.parametrize("heads,lens", [((4, 1, 128), [4100]), ((2, 2, 64), [3000, 77, 1500])])
def test_gradients_of_long_documents(heads, lens):
    """Walks of dozens of tiles, on key and row tiles alike, against the formula."""
    Hq, Hkv, d = heads
    g = torch.Generator().manual_seed(4)
    q, k, v, dout = (torch.randn(sum(lens), h, d, generator=g).to(BF16).to(DEV) for h in (Hq, Hkv, Hkv, Hq))
    cu = fp.offsets(lens).to(DEV)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = msa.msa_full_attn_prefill(q, k, v, cu, cu, lse=lse)
    got = msa.msa_full_attn_backward(q, k, v, out, dout, lse, cu, cu)
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        with torch.device(DEV):  # 64-bit matrices of n x n scores
            want, tol = fp.backward(*[x[sl].double() for x in (q, k, v, out, dout, lse)], d ** -0.5, BF16)
        for name, x, w, t in zip(("dq", "dk", "dv"), got, want, tol):
            fp.assert_within(x[sl], w.cpu(), t.cpu(), f"{name} of {n}")
        at += n
