"""Packed offsets that are out of order or out of range, at every place of a
batch and for batches of every size: reported, and each sequence that the
header calls in range still gets its results, every other row stays.

A sequence is in range if 0 <= cu[b] <= cu[b + 1] <= T and cu[b] is not below an
earlier offset within [0, T]."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, FP32 = torch.bfloat16, torch.float32
SIZES = [3, 40, 300]


def in_range(cu, T):
    """(b, first row, rows) of the sequences in range."""
    cu, floor, res = cu.tolist(), 0, []
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        if 0 <= a <= e <= T and a >= floor:
            res.append((b, a, e - a))
        if 0 <= a <= T:
            floor = max(floor, a)
    return res


def damaged(cu, T):
    """What a batch's offsets may look like when something went wrong."""
    n = cu.numel() - 1
    for at in (0, 1, n // 2, n - 1, n):
        for value in (T + 1, 1_000_000, -1, -1000, int(cu[min(at + 4, n)]) + (at == n)):
            yield at, value
        if at > 0:
            yield at, int(cu[at - 1]) - 1  # one below the offset before it


def cases(lens, T):
    cu, res = fp.offsets(lens), []
    for at, value in damaged(cu, T):
        bad = cu.clone()
        bad[at] = value
        if bad.min() < 0 or bad.max() > T or (bad[1:] < bad[:-1]).any():
            res.append(bad)
    return res if len(lens) < 300 else res[::3]


def _lens(B, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 40, (B,), generator=g) + torch.tensor([150 if b % 17 == 1 else 0 for b in range(B)])).tolist()


def _rand(g, n, h, d, dtype):
    return torch.randn(n, h, d, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_no_keys_or_no_rows_at_all(dtype):
    """Calls without any key, or any row, look at both sides' offsets as well."""
    g = torch.Generator().manual_seed(5)
    x, y = _rand(g, 30, 4, 64, dtype).to(DEV), _rand(g, 0, 4, 64, dtype).to(DEV)
    lse, none = torch.zeros(30, 4, device=DEV), torch.zeros(0, 4, device=DEV)
    ws = msa.workspace(1 << 20, DEV)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    # own side's offsets, the other's, rows that become zero
    for own, other, zero in [((0, 10, 20, 30), (0, 0, 5, 0), (0, 30)), ((0, 10, 20, 31), (0, 0, 0, 0), (0, 20)),
                             ((0, 10, -3, 30), (0, 0, 0, 0), (0, 10)), ((0, 99, 20, 30), (0, 0, 0, 0), (20, 30)),
                             ((-1, 10, 20, 30), (0, 0, 0, 0), (10, 30))]:
        keep = torch.ones(30, dtype=torch.bool)
        keep[slice(*zero)] = False
        filled = lambda: torch.full_like(x, 7.0)  # noqa: E731
        out, l2 = filled(), torch.full_like(lse, 7.0)
        msa.msa_full_attn_prefill(x, y, y, ints(*own), ints(*other), out=out, lse=l2, ws=ws)
        assert msa.msa_read_status(ws) == 6
        dq = filled()
        msa.msa_full_attn_backward(x, y, y, x, x, lse, ints(*own), ints(*other), dq=dq, ws=ws)
        assert msa.msa_read_status(ws) == 6
        dk, dv = filled(), filled()
        msa.msa_full_attn_backward(y, x, x, y, y, none, ints(*other), ints(*own), dk=dk, dv=dv, ws=ws)
        assert msa.msa_read_status(ws) == 6
        for t in (out, dq, dk, dv):
            assert (t.cpu()[keep] == 7.0).all() and (t.cpu()[~keep] == 0).all()
        assert (l2.cpu()[keep] == 7.0).all() and (l2.cpu()[~keep] == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B", SIZES)
def test_append(B, dtype):
    Hq, Hkv, d, page = 4, 2, 64, 16
    lens = [n % 31 for n in _lens(B, B)]
    T = sum(lens)
    g = torch.Generator().manual_seed(6)
    q, k, v = (_rand(g, T, h, d, dtype) for h in (Hq, Hkv, Hkv))
    per = 14  # pages of a sequence: room for any span that the offsets give in range
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
    ws = msa.workspace(256, DEV)
    dev, td = [x.to(DEV) for x in (q, k, v)], table.to(DEV)
    for bad in cases(lens, T):
        rows = in_range(bad, T)
        n_new = (bad[1:].long() - bad[:-1].long()).clamp(0, 200)
        kv = (n_new + torch.arange(B) % 7).to(torch.int32)
        kc, vc = (torch.full((B * per, page, Hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        qo = torch.full_like(dev[0], 7.0)
        msa.msa_paged_append(*dev, None, bad.to(DEV), kv.to(DEV), td, kc, vc, q_out=qo, ws=ws)
        what = f"{bad.tolist()[:8]}"
        assert msa.msa_read_status(ws) == 6, what
        wq = torch.full_like(q, 7.0)
        wk, wv = (torch.full((B * per * page, Hkv, d), 7.0, dtype=dtype) for _ in range(2))
        for b, a, n in rows:
            pos = torch.arange(n) + int(kv[b]) - n
            at = table[b].long()[pos // page] * page + pos % page
            wq[a:a + n], wk[at], wv[at] = q[a:a + n], k[a:a + n], v[a:a + n]
        assert torch.equal(qo.cpu(), wq), f"q_out, {what}"
        assert torch.equal(kc.cpu().flatten(0, 1), wk) and torch.equal(vc.cpu().flatten(0, 1), wv), f"cache, {what}"
