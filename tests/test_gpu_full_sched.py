"""GPU tests of how full attention divides its work: items handed out whole,
items split over CTAs and joined, clusters, caches beyond 32-bit offsets, and
one workspace under all operations. Values against the plain 64-bit forms
(full_plain.py) within their bounds."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp
from test_gpu_full_attn import BF16, DEV, FP32, _decode_case, check_backward, check_decode, check_prefill, make

pytestmark = pytest.mark.gpu


def _lens(n, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, hi, (n,), generator=g).tolist()


@pytest.mark.parametrize("heads", [(16, 2, 64), (4, 4, 64), (6, 2, 128)])
def test_many_short_sequences(heads):
    """More items than CTAs, all short: handed out whole."""
    lens = _lens(150, 260, 1)
    check_prefill([(n, n) for n in lens], *heads, BF16, seed=2)
    old = _lens(150, 200, 3)
    check_prefill([(n % 40, n % 40 + o) for n, o in zip(lens, old)], *heads, BF16, paged=32, seed=3)


def test_many_sequences_with_rows_without_keys():
    spans = [(n % 90, (n * 7) % 60) for n in range(200)]
    check_prefill(spans, 4, 2, 64, BF16, seed=23)
    check_prefill(spans, 4, 2, 64, BF16, paged=16, seed=24)


def test_many_sequences_of_one_token():
    check_prefill([(1, 1 + (7 * b) % 40) for b in range(600)], 8, 2, 64, BF16, paged=16, seed=4)
    check_prefill([(1, 1)] * 300, 8, 2, 64, FP32, seed=5)


@pytest.mark.parametrize("spans", [[(70, 5000), (3, 9000)], [(1, 20000)], [(300, 2500), (2, 40), (0, 0), (1, 3300)],
                                   [(1500, 1500)]])
def test_split_items(spans):
    """Few long items: split over CTAs, each part's rows joined in the order of the keys."""
    check_prefill(spans, 8, 1, 64, BF16, seed=6)
    check_prefill(spans, 4, 2, 128, BF16, paged=64, seed=7)


def test_split_items_with_rows_without_keys():
    check_prefill([(2500, 1800), (10, 4)], 2, 1, 64, BF16, seed=8)


def test_split_items_same_bits():
    """Whoever arrives last joins the parts in the same order: runs are equal bit for bit."""
    q, k, v, cu_q, cu_k, *_ = make([(40, 6000), (100, 3000)], 16, 2, 128, BF16, 9)
    d = [x.to(DEV) for x in (q, k, v, cu_q, cu_k)]
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_PREFILL, 2, q.shape[0], k.shape[0], 2, 16, 128, 0, 0, 0,
                                              msa.MSA_BF16), DEV)
    first = msa.msa_full_attn_prefill(*d, ws=ws)
    for _ in range(20):
        assert torch.equal(first, msa.msa_full_attn_prefill(*d, ws=ws))
    assert msa.msa_read_status(ws) == 0


def test_split_items_bad_page():
    """A page out of range in a sequence whose items are split: its rows zero, the other's right."""
    g = torch.Generator().manual_seed(10)
    lens = [4000, 3500]
    q = torch.randn(20, 8, 64, generator=g).to(BF16)
    ks, vs = ([torch.randn(n, 2, 64, generator=g).to(BF16) for n in lens] for _ in range(2))
    kc, vc, table = fp.paged(ks, vs, 32, g)
    table[0, 60] = -1
    cu, kv = torch.tensor([0, 8, 20], dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_PREFILL, 2, 20, table.shape[1] * 32, 2, 8, 64, 0, 0, 0,
                                              msa.MSA_BF16), DEV)
    lse = torch.empty(20, 8, device=DEV)
    for _ in range(2):
        out = msa.msa_full_attn_prefill_paged(*[x.to(DEV) for x in (q, kc, vc, table, cu, kv)], lse=lse, ws=ws)
        assert msa.msa_read_status(ws) == 6
        assert (out[:8] == 0).all() and (lse[:8] == -math.inf).all()
        want = fp.prefill(q, ks, vs, [(0, 8), (8, 12)], 0.125, BF16)
        fp.assert_within(out[8:], want[0][8:], want[2][8:], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", [(16, 2, 64), (32, 8, 128), (4, 4, 64), (6, 2, 128), (40, 2, 64), (34, 1, 128)])
def test_decode_whole_items_per_warp(heads, dtype):
    """Many short sequences, some without keys, and one long one among them (units shared out)."""
    lens = [(13 * b) % 41 for b in range(650)]
    check_decode(lens, *heads, dtype, 16, seed=25)
    check_decode([0] * 200 + lens[:350] + [0] * 100, *heads, dtype, 32, seed=26)
    check_decode([0] * 600, *heads, dtype, 16, seed=27, max_pages=1)
    check_decode(lens[:400] + [1500] + lens[400:], *heads, dtype, 64, seed=28)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_whole_items_bad_pages(dtype):
    lens = [1 + (29 * b) % 60 for b in range(900)]
    q, kc, vc, table, kv, want = _decode_case(lens, 8, 2, 64, dtype, 16, 29)
    bad = [0, 17, 433, 899]
    table[0, 0], kv[17], kv[433] = -1, -1, table.shape[1] * 16 + 1
    table[899, (lens[899] - 1) // 16] = kc.shape[0]
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 900, 1, table.shape[1] * 16, 2, 8, 64, 0, 0, 0,
                                              0 if dtype == BF16 else 1), DEV)
    good = [b for b in range(900) if b not in bad]
    for _ in range(2):
        lse = torch.empty(900, 8, device=DEV)
        out = msa.msa_full_attn_decode(*[x.to(DEV) for x in (q, kc, vc, table, kv)], lse=lse, ws=ws)
        assert msa.msa_read_status(ws) == 6
        assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
        fp.assert_within(out[good], want[0][good], want[2][good], "out")
        fp.assert_within(lse[good], want[1][good], want[3][good], "lse")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_few_tiles(dtype):
    """Long walks of few tiles: shared by the CTAs of a cluster."""
    check_backward([(1100, 1100)] if dtype == BF16 else [(400, 400)], 4, 1, 64, dtype, seed=11)
    check_backward([(9, 1500)], 2, 1, 128, dtype, seed=12)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_many_sequences(dtype):
    check_backward([(n, n) for n in _lens(60, 90, 13)], 8, 4, 64, dtype, seed=13)
    check_backward([(2, 2)] * 26, 4, 4, 64, dtype, seed=14)


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^31 elements of the cache: append, prefill over pages, decode."""
    page, Hkv, d, Hq = 128, 8, 128, 32
    num = (1 << 31) // (page * Hkv * d) + 12
    kc = torch.zeros(num, page, Hkv, d, dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(15)
    n = 200
    q, k, v = (torch.randn(n, h, d, generator=g).to(BF16) for h in (Hq, Hkv, Hkv))
    table = torch.tensor([[num - 1, num - 3]], dtype=torch.int32, device=DEV)
    kv = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    msa.msa_paged_append(None, k.to(DEV), v.to(DEV), None, cu, kv, table, kc, vc)
    assert torch.equal(kc[num - 1].cpu(), k[:128]) and torch.equal(vc[num - 3, :72].cpu(), v[128:])
    want = fp.prefill(q, [k], [v], [(0, n)], d ** -0.5, BF16)
    out = msa.msa_full_attn_prefill_paged(q.to(DEV), kc, vc, table, cu, kv)
    fp.assert_within(out, want[0], want[2], "prefill")
    out = msa.msa_full_attn_decode(q[-1:].to(DEV), kc, vc, table, kv)
    fp.assert_within(out, want[0][-1:], want[2][-1:], "decode")


def test_one_workspace_for_all_operations():
    """Operations of any kind and size, one after the other on one workspace."""
    Hq, Hkv, d, page = 8, 2, 64, 16
    g = torch.Generator().manual_seed(16)
    lens = [3000, 5, 700]
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(BF16)  # noqa: E731
    qd, ks, vs = r(3, Hq), [r(n, Hkv) for n in lens], [r(n, Hkv) for n in lens]
    kc, vc, table = (x.to(DEV) for x in fp.paged(ks, vs, page, g))
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want_d = fp.prefill(qd, ks, vs, [(b, 1) for b in range(3)], d ** -0.5, BF16)
    q, k, v, cu_q, cu_k, rows, pk, pv, _ = make([(60, 2000), (30, 30)], Hq, Hkv, d, BF16, 17)
    want_p = fp.prefill(q, pk, pv, rows, d ** -0.5, BF16)
    dev = [x.to(DEV) for x in (q, k, v, cu_q, cu_k)]
    lse = torch.empty(q.shape[:2], device=DEV)
    size = max(msa.msa_workspace_size(op, 3, 100, 4000, Hkv, Hq, d, 0, 0, 0, msa.MSA_BF16)
               for op in (msa.MSA_OP_FULL_PREFILL, msa.MSA_OP_FULL_BACKWARD, msa.MSA_OP_FULL_DECODE))
    sp = [torch.randn(1, 512, h, e, generator=g).to(BF16).to(DEV) for h, e in ((Hq, d), (Hkv, d), (Hkv, d), (Hkv, 32))]
    ik = torch.randn(1, 512, 32, generator=g).to(BF16).to(DEV)
    qo = torch.zeros(1, dtype=torch.int32, device=DEV)
    kl = torch.full((1,), 512, dtype=torch.int32, device=DEV)
    ssize = msa.msa_workspace_size(msa.MSA_OP_PREFILL, 1, 512, 512, Hkv, Hq, d, 0, 64, 4, msa.MSA_BF16)
    ws = msa.workspace(max(size, ssize, 1 << 20), DEV)
    sparse = None
    for i in range(4):
        out = msa.msa_full_attn_prefill(*dev, lse=lse, ws=ws)
        fp.assert_within(out, want_p[0], want_p[2], "prefill")
        dec = msa.msa_full_attn_decode(qd.to(DEV), kc, vc, table, kv, ws=ws)
        fp.assert_within(dec, want_d[0], want_d[2], "decode")
        msa.msa_full_attn_backward(*dev[:3], out, dev[0], lse, *dev[3:], ws=ws)
        sel = msa.msa_index_select(sp[3], ik, qo, kl, 64, 4, ws=ws)
        got = msa.msa_sparse_attn_prefill(sp[0], sp[1], sp[2], sel, qo, kl, 64, 4, ws=ws)
        assert sparse is None or torch.equal(sparse, got)
        sparse = got
        dec = msa.msa_full_attn_decode(qd.to(DEV), kc, vc, table, kv, ws=ws)
        fp.assert_within(dec, want_d[0], want_d[2], "decode")
        assert msa.msa_read_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_of_no_sequence_then_another_call(dtype):
    """Rows that belong to no sequence: nothing is written, and the workspace's next user follows at once."""
    g = torch.Generator().manual_seed(30)
    q, k = torch.randn(6000, 16, 64, generator=g).to(dtype).to(DEV), torch.randn(300, 2, 64, generator=g).to(dtype).to(DEV)
    lse, none = torch.zeros(6000, 16, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    qc, kc, vc, table, kv, want = _decode_case([700, 3000, 1], 16, 2, 64, dtype, 16, 31)
    d = [x.to(DEV) for x in (qc, kc, vc, table, kv)]
    dt = 0 if dtype == BF16 else 1
    ws = msa.workspace(max(msa.msa_workspace_size(msa.MSA_OP_FULL_BACKWARD, 3, 6000, 300, 2, 16, 64, 0, 0, 0, dt),
                           msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 3, 1, table.shape[1] * 16, 2, 16, 64, 0, 0, 0,
                                                  dt)), DEV)
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    for _ in range(20):
        msa.msa_full_attn_backward(q, k, k, q, q, lse, none, none, dq=dq, dk=dk, dv=dv, ws=ws)
        out = msa.msa_full_attn_decode(*d, ws=ws)
        fp.assert_within(out, want[0], want[2], "out")
    assert msa.msa_read_status(ws) == 0
    assert (dq == 7.0).all() and (dk == 7.0).all() and (dv == 7.0).all()


def test_two_streams_at_once():
    """Two calls in flight on two streams, a workspace each."""
    q, k, v, cu_q, cu_k, rows, ks, vs, _ = make([(64, 8000), (300, 300)], 8, 2, 64, BF16, 18)
    want = fp.prefill(q, ks, vs, rows, 0.125, BF16)
    d = [x.to(DEV) for x in (q, k, v, cu_q, cu_k)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for o, s in zip(outs, streams):
            o.append(msa.msa_full_attn_prefill(*d, stream=s))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, outs[0][0])
    fp.assert_within(outs[0][0], want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_bad_offsets(dtype):
    """Offsets out of range: reported; gradients whose rows are known become zero, the others stay."""
    spans = [(40, 40), (30, 50), (20, 20)]
    q, k, v, cu_q, cu_k, rows, ks, vs, g = make(spans, 8, 2, 64, dtype, 19)
    fwd = fp.prefill(q, ks, vs, rows, 0.125, dtype)
    dout = torch.randn(q.shape, generator=g).to(dtype)
    good = [x.to(DEV) for x in (q, k, v, fwd[0].to(dtype), dout, fwd[1].float())]
    ws = msa.workspace(1 << 20, DEV)

    def run(cq, ck):
        grads = [torch.full(x.shape, 7.0, dtype=dtype, device=DEV) for x in (q, k, v)]
        msa.msa_full_attn_backward(*good, cq.to(DEV), ck.to(DEV), *grads, ws=ws)
        assert msa.msa_read_status(ws) == 6
        return grads

    want, tol = fp.backward(*[x[:40].double() for x in (q, k, v, fwd[0].to(dtype), dout)], fwd[1][:40].float().double(),
                            0.125, dtype)
    bad = cu_q.clone()
    bad[3] = 91
    dq, dk, dv = run(bad, cu_k)
    assert (dq[70:] == 7.0).all() and (dk[90:] == 0).all() and (dv[90:] == 0).all()
    fp.assert_within(dk[:40], want[1], tol[1], "dk")
    bad = cu_k.clone()
    bad[3] = 111
    dq, dk, dv = run(cu_q, bad)
    assert (dq[70:] == 0).all() and (dk[90:] == 7.0).all() and (dv[90:] == 7.0).all()
    fp.assert_within(dq[:40], want[0], tol[0], "dq")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_captured_training_step(dtype):
    """Prefill (split items among them) and backward in a graph, replayed on new inputs."""
    spans = [(200, 200), (7, 1500), (33, 33)]
    first = make(spans, 8, 2, 64, dtype, 20)
    d = [x.to(DEV) for x in first[:5]]
    dout = torch.randn(first[0].shape, generator=first[8]).to(dtype)
    out, lse, do = torch.empty_like(d[0]), torch.empty(d[0].shape[:2], device=DEV), dout.to(DEV)
    grads = [torch.empty_like(x) for x in d[:3]]
    size = max(msa.msa_workspace_size(op, 3, d[0].shape[0], d[1].shape[0], 2, 8, 64, 0, 0, 0, 0 if dtype == BF16 else 1)
               for op in (msa.MSA_OP_FULL_PREFILL, msa.MSA_OP_FULL_BACKWARD))
    ws = msa.workspace(size, DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_full_attn_prefill(*d, out=out, lse=lse, ws=ws)
        msa.msa_full_attn_backward(*d[:3], out, do, lse, d[3], d[4], *grads, ws=ws)
    for seed in (20, 21, 22):
        q, k, v, _, _, rows, ks, vs, _ = make(spans, 8, 2, 64, dtype, seed)
        for dst, src in zip(d, (q, k, v)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert msa.msa_read_status(ws) == 0
        want = fp.prefill(q, ks, vs, rows, 0.125, dtype)
        fp.assert_within(out, want[0], want[2], "out")
        k0 = 0
        for (q0, Lq), kb, vb in zip(rows, ks, vs):
            sl = slice(q0, q0 + Lq)
            w, t = fp.backward(*[x.double() for x in (q[sl], kb, vb, out[sl].cpu(), dout[sl], lse[sl].cpu())], 0.125, dtype)
            for name, gr, s2, x, y in zip(("dq", "dk", "dv"), grads, (sl, *[slice(k0, k0 + len(kb))] * 2), w, t):
                fp.assert_within(gr[s2], x, y, name)
            k0 += len(kb)
