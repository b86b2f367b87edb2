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


def _workspace(op, B, Nq, Nk, Hkv, Hq, d, dtype):
    return msa.workspace(msa.msa_workspace_size(op, B, Nq, Nk, Hkv, Hq, d, 0, 0, 0, 0 if dtype == BF16 else 1), DEV)


def _want(q, k, v, cu_q, cu_k, dtype):
    """out, lse and bounds, and the sequences in range on either side."""
    rows, keys = in_range(cu_q, q.shape[0]), {b: (a, n) for b, a, n in in_range(cu_k, k.shape[0])}
    spans, ks, vs = [], [], []
    for b, a, n in rows:
        k0, m = keys.get(b, (0, 0))  # keys out of range: as without any
        spans.append((a, n))
        ks.append(k[k0:k0 + m])
        vs.append(v[k0:k0 + m])
    return fp.prefill(q, ks, vs, spans, q.shape[-1] ** -0.5, dtype), rows, keys


def _check_prefill(call, want, shape, dtype, ws, what):
    out, lse = torch.full(shape, 7.0, dtype=dtype, device=DEV), torch.full(shape[:2], 7.0, device=DEV)
    call(out, lse)
    assert msa.msa_read_status(ws) == 6, what
    none = want[1].isnan()
    assert (out.cpu()[none] == 7.0).all() and (lse.cpu()[none] == 7.0).all(), f"{what}: rows of no sequence"
    fp.assert_within(out, want[0], want[2], f"out, {what}")
    fp.assert_within(lse, want[1], want[3], f"lse, {what}")


@pytest.mark.parametrize("side", ["rows", "keys", "both"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B", SIZES)
def test_prefill(B, dtype, side):
    Hq, Hkv, d = 4, 2, 64
    lens = _lens(B, B)
    T = sum(lens)
    g = torch.Generator().manual_seed(1)
    q, k, v = (_rand(g, T, h, d, dtype) for h in (Hq, Hkv, Hkv))
    dev, fine = [x.to(DEV) for x in (q, k, v)], fp.offsets(lens)
    ws = _workspace(msa.MSA_OP_FULL_PREFILL, B, T, T, Hkv, Hq, d, dtype)
    for bad in cases(lens, T):
        cu_q, cu_k = (bad if side in ("rows", "both") else fine), (bad if side in ("keys", "both") else fine)
        want, _, _ = _want(q, k, v, cu_q, cu_k, dtype)
        on = [x.to(DEV) for x in (cu_q, cu_k)]
        if side == "both":
            on[1] = on[0]
        _check_prefill(lambda out, lse: msa.msa_full_attn_prefill(*dev, *on, out=out, lse=lse, ws=ws), want, q.shape, dtype,
                       ws, f"{side} {bad.tolist()[:8]}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B", SIZES)
def test_prefill_paged(B, dtype):
    Hq, Hkv, d, page = 8, 2, 64, 16
    lens = [n % 23 for n in _lens(B, B)]
    T = sum(lens)
    g = torch.Generator().manual_seed(2)
    kv = [n + (7 * b) % 50 for b, n in enumerate(lens)]
    q, ks, vs = _rand(g, T, Hq, d, dtype), *([_rand(g, n, Hkv, d, dtype) for n in kv] for _ in range(2))
    kc, vc, table = fp.paged(ks, vs, page, g)
    dev = [x.to(DEV) for x in (q, kc, vc, table)]
    kvd = torch.tensor(kv, dtype=torch.int32, device=DEV)
    ws = _workspace(msa.MSA_OP_FULL_PREFILL, B, T, table.shape[1] * page, Hkv, Hq, d, dtype)
    for bad in cases(lens, T):
        rows = in_range(bad, T)
        want = fp.prefill(q, [ks[b] for b, _, _ in rows], [vs[b] for b, _, _ in rows], [r[1:] for r in rows], d ** -0.5, dtype)
        cu = bad.to(DEV)
        _check_prefill(lambda out, lse: msa.msa_full_attn_prefill_paged(*dev, cu, kvd, out=out, lse=lse, ws=ws), want,
                       q.shape, dtype, ws, f"{bad.tolist()[:8]}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_long_sequences(dtype):
    """Few long sequences, whose work is divided into equal shares when the offsets are in order."""
    Hq, Hkv, d, lens = 2, 1, 64, [900, 40, 1700]
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    q, k, v = (_rand(g, T, h, d, dtype) for h in (Hq, Hkv, Hkv))
    dev = [x.to(DEV) for x in (q, k, v)]
    ws = _workspace(msa.MSA_OP_FULL_PREFILL, 3, T, T, Hkv, Hq, d, dtype)
    for cu in ([0, 900, 940, T + 1], [0, -1, 940, T], [0, 900, 850, T], [-5, 900, 940, T], [0, 1_000_000, 940, T]):
        cu = torch.tensor(cu, dtype=torch.int32)
        want, _, _ = _want(q, k, v, cu, cu, dtype)
        on = cu.to(DEV)
        _check_prefill(lambda out, lse: msa.msa_full_attn_prefill(*dev, on, on, out=out, lse=lse, ws=ws), want, q.shape, dtype,
                       ws, f"{cu.tolist()}")


@pytest.mark.parametrize("side", ["rows", "keys", "both"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B", SIZES)
def test_backward(B, dtype, side):
    Hq, Hkv, d = 4, 2, 64
    lens = _lens(B, B)
    T = sum(lens)
    g = torch.Generator().manual_seed(4)
    q, k, v, dout = (_rand(g, T, h, d, dtype) for h in (Hq, Hkv, Hkv, Hq))
    fine = fp.offsets(lens)
    ws = _workspace(msa.MSA_OP_FULL_BACKWARD, B, T, T, Hkv, Hq, d, dtype)
    for bad in cases(lens, T)[::1 if B < 300 else 2]:
        cu_q, cu_k = (bad if side in ("rows", "both") else fine), (bad if side in ("keys", "both") else fine)
        what = f"{side} {bad.tolist()[:8]}"
        want, rows, keys = _want(q, k, v, cu_q, cu_k, dtype)
        out, lse = want[0].nan_to_num(0.0).to(dtype), want[1].nan_to_num(0.0, neginf=-math.inf).float()
        grads = [torch.full(x.shape, 7.0, dtype=dtype, device=DEV) for x in (q, k, v)]
        on = [x.to(DEV) for x in (cu_q, cu_k)]
        if side == "both":
            on[1] = on[0]
        msa.msa_full_attn_backward(*[x.to(DEV) for x in (q, k, v, out, dout, lse)], *on, *grads, ws=ws)
        assert msa.msa_read_status(ws) == 6, what
        ref = [torch.full(x.shape, 7.0, dtype=torch.float64) for x in (q, k, v)]
        tol = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
        for b, a, n in rows:
            ref[0][a:a + n] = 0
        for b, (a, n) in keys.items():
            ref[1][a:a + n] = ref[2][a:a + n] = 0
        for b, a, n in rows:
            if b not in keys or n == 0 or keys[b][1] == 0:
                continue
            k0, m = keys[b]
            r, c = slice(a, a + n), slice(k0, k0 + m)
            w, t = fp.backward(*[x.double() for x in (q[r], k[c], v[c], out[r], dout[r], lse[r])], d ** -0.5, dtype)
            for dst, src, sl in zip(ref + tol, w + t, (r, c, c) * 2):
                dst[sl] = src
        for name, got, w, t in zip(("dq", "dk", "dv"), grads, ref, tol):
            fp.assert_within(got, w, t, f"{name}, {what}")


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


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B", [40, 300])
def test_captured(B, dtype):
    """A graph of append, prefill and backward replayed over offsets that are in
    order, then not, then again: every replay looks at them anew."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    lens = [1 + n % 31 for n in _lens(B, B)]
    T = sum(lens)
    g = torch.Generator().manual_seed(7)
    q, k, v, dout = (_rand(g, T, h, d, dtype).to(DEV) for h in (Hq, Hkv, Hkv, Hq))
    fine = fp.offsets(lens)
    broken = fine.clone()
    broken[B // 2] = T + 5
    cu, kv = fine.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    kc, vc = (torch.zeros(2 * B, page, Hkv, d, dtype=dtype, device=DEV) for _ in range(2))
    out, lse, qo = torch.empty_like(q), torch.empty(T, Hq, device=DEV), torch.empty_like(q)
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = [_workspace(op, B, T, T, Hkv, Hq, d, dtype)
          for op in (msa.MSA_OP_PAGED_APPEND, msa.MSA_OP_FULL_PREFILL, msa.MSA_OP_FULL_BACKWARD)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_paged_append(q, k, v, None, cu, kv, table, kc, vc, q_out=qo, ws=ws[0])
        msa.msa_full_attn_prefill(q, k, v, cu, cu, out=out, lse=lse, ws=ws[1])
        msa.msa_full_attn_backward(q, k, v, out, dout, lse, cu, cu, *grads, ws=ws[2])
    first = None
    for now, status in ((fine, 0), (broken, 6), (fine, 0)):
        cu.copy_(now)
        everything = [qo, kc, vc, out, lse, *grads]
        for x in everything:
            x.fill_(7.0)
        graph.replay()
        assert [msa.msa_read_status(w) for w in ws] == [status] * 3
        if first is None:
            first = [x.clone() for x in everything]
        elif status == 0:
            assert all(torch.equal(a, b) for a, b in zip(first, everything))
        else:
            a, e = int(fine[B // 2 - 1]), int(fine[B // 2 + 1])  # rows of the two sequences at the broken offset
            for x, y in zip((qo, out, lse, *grads), (first[0], first[3], first[4], *first[5:])):
                assert (x[a:e] == 7.0).all() and torch.equal(x[:a], y[:a]) and torch.equal(x[e:], y[e:])
            b = B // 2
            for x, y in zip((kc, vc), first[1:3]):
                assert (x[2 * b - 2:2 * b + 2] == 7.0).all()
                assert torch.equal(x[:2 * b - 2], y[:2 * b - 2]) and torch.equal(x[2 * b + 2:], y[2 * b + 2:])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_very_many_sequences(dtype):
    """More than 65536 sequences: served where their offsets are in order, left alone where not."""
    B, d = 65600, 64
    q, k, v, dout = (torch.randn(B, 1, d, device=DEV).to(dtype) for _ in range(4))
    lse = torch.empty(B, 1, device=DEV)
    fine = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    bad = fine.clone()
    bad[40000] = -1
    kv, table = torch.ones(B, dtype=torch.int32, device=DEV), fine[:B, None].contiguous()
    ws = max((_workspace(op, B, B, B, 1, 1, d, dtype) for op in (msa.MSA_OP_FULL_PREFILL, msa.MSA_OP_FULL_BACKWARD)),
             key=torch.numel)
    for cu, status in ((fine, 0), (bad, 6)):
        out, qo, dq, dk, dv = (torch.full_like(q, 7.0) for _ in range(5))
        kc, vc = (torch.full((B, 16, 1, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        msa.msa_full_attn_prefill(q, k, v, cu, cu, out=out, lse=lse, ws=ws)
        assert msa.msa_read_status(ws) == status
        msa.msa_full_attn_backward(q, k, v, v, dout, lse, cu, cu, dq, dk, dv, ws=ws)
        assert msa.msa_read_status(ws) == status
        msa.msa_paged_append(q, k, v, None, cu, kv, table, kc, vc, q_out=qo, ws=ws)
        assert msa.msa_read_status(ws) == status
        if status == 0:  # one key each: its weight is 1, in the backward within 2^-17 (|s| < 8, fp32 exponent)
            assert torch.equal(out, v) and torch.equal(qo, q)
            assert ((dv - dout).abs() <= 2.0 ** -17 * dout.abs()).all()
            assert torch.equal(kc[:, 0], k) and torch.equal(vc[:, 0], v)
        else:
            assert all((x == 7.0).all() for x in (out, qo, dq, dk, dv, kc, vc))
