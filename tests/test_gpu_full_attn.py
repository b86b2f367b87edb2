"""GPU parity of full attention over packed sequences and paged caches against
the plain 64-bit forms, within the bounds derived in full_plain.py."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, FP32 = torch.bfloat16, torch.float32

# (Lq, Lk) per sequence: one token, empty ones, tiles' edges, prefixes, rows without keys
SPANS = {
    "one": [(1, 1)],
    "edges": [(127, 127), (128, 128), (129, 129), (1, 1), (0, 0), (63, 63)],
    "ragged": [(300, 300), (0, 0), (5, 5), (257, 257), (33, 33)],
    "prefix": [(3, 200), (1, 129), (64, 65), (130, 520), (17, 400)],
    "no_keys": [(10, 4), (5, 0), (200, 70), (2, 2)],
}
HEADS = [(4, 4, 64), (8, 2, 64), (8, 2, 128), (6, 2, 128), (16, 2, 64), (16, 1, 128), (32, 1, 64), (10, 2, 128),
         (64, 1, 128), (9, 3, 64)]


def make(spans, Hq, Hkv, d, dtype, seed=0, before=0, behind=0, fill=math.nan):
    """Packed inputs on the CPU; rows of no sequence hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    Tq = before + sum(s[0] for s in spans) + behind
    Tk = before + sum(s[1] for s in spans) + behind
    cu_q, cu_k = fp.offsets([s[0] for s in spans], before), fp.offsets([s[1] for s in spans], before)
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(dtype)  # noqa: E731
    q, k, v = r(Tq, Hq), r(Tk, Hkv), r(Tk, Hkv)
    for x, cu in ((q, cu_q), (k, cu_k), (v, cu_k)):
        x[:before] = fill
        x[int(cu[-1]):] = fill
    rows = [(int(a), int(b - a)) for a, b in zip(cu_q[:-1], cu_q[1:])]
    ks = [k[int(a):int(b)] for a, b in zip(cu_k[:-1], cu_k[1:])]
    vs = [v[int(a):int(b)] for a, b in zip(cu_k[:-1], cu_k[1:])]
    return q, k, v, cu_q, cu_k, rows, ks, vs, g


def check_prefill(spans, Hq, Hkv, d, dtype, paged=None, before=0, behind=0, scale=0.0, seed=0):
    q, k, v, cu_q, cu_k, rows, ks, vs, g = make(spans, Hq, Hkv, d, dtype, seed, before, behind)
    want = fp.prefill(q, ks, vs, rows, scale or d ** -0.5, dtype)
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_PREFILL, len(spans), q.shape[0], max(k.shape[0], 1), Hkv,
                                              Hq, d, 0, 0, 0, 0 if dtype == BF16 else 1), DEV)
    if paged:
        kc, vc, table = fp.paged(ks, vs, paged, g)
        kv = torch.tensor([s[1] for s in spans], dtype=torch.int32)
        msa.msa_full_attn_prefill_paged(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), cu_q.to(DEV), kv.to(DEV),
                                        scale=scale, out=out, lse=lse, ws=ws)
    else:
        msa.msa_full_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_q.to(DEV), cu_k.to(DEV), scale=scale, out=out,
                                  lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert msa.msa_read_status(ws) == 0
    none = want[1].isnan()  # rows of no sequence: as they were
    assert (out.cpu()[none] == 7.0).all() and (lse.cpu()[none] == 7.0).all()
    fp.assert_within(out, want[0], want[2], "out")
    fp.assert_within(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", sorted(SPANS))
def test_prefill_spans(name, dtype):
    check_prefill(SPANS[name], 8, 2, 128, dtype)
    check_prefill(SPANS[name], 8, 2, 64, dtype, before=3, behind=50)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", HEADS)
def test_prefill_heads(heads, dtype):
    check_prefill([(70, 70), (20, 150), (1, 64)], *heads, dtype, seed=1)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_prefill_paged(page, dtype):
    for name in ("one", "edges", "prefix", "no_keys"):
        check_prefill(SPANS[name], 8, 2, 128 if page > 16 else 64, dtype, paged=page, seed=page)
    check_prefill([(40, 40), (9, 333)], 6, 2, 128, dtype, paged=page, before=2, behind=9)


def test_prefill_scale_and_long_rows():
    check_prefill([(900, 900)], 4, 1, 64, BF16, scale=0.5, seed=3)   # peaked rows: the running maximum moves
    check_prefill([(1, 3000), (40, 2900)], 4, 2, 128, BF16, paged=64, scale=0.3, seed=4)
    check_prefill([(1, 3000), (40, 2900)], 4, 2, 128, FP32, scale=0.3, seed=5)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_growing_scores(dtype):
    """Keys whose scores rise along the sequence: every tile raises the maximum."""
    spans = [(600, 600)]
    q, k, v, cu_q, cu_k, rows, ks, vs, _ = make(spans, 4, 2, 64, dtype, 6)
    q.fill_(1.0)
    k.copy_((torch.arange(600)[:, None, None] / 50.0).expand(600, 2, 64))
    want = fp.prefill(q, [k], [v], rows, 0.125, dtype)
    lse = torch.empty(600, 4, device=DEV)
    out = msa.msa_full_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_q.to(DEV), cu_k.to(DEV), lse=lse)
    fp.assert_within(out, want[0], want[2], "out")
    fp.assert_within(lse, want[1], want[3], "lse")


def _decode_case(lens, Hq, Hkv, d, dtype, page, seed=0, max_pages=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(dtype)  # noqa: E731
    q, ks, vs = r(len(lens), Hq), [r(n, Hkv) for n in lens], [r(n, Hkv) for n in lens]
    kc, vc, table = fp.paged(ks, vs, page, g, max_pages=max_pages)
    kv = torch.tensor(lens, dtype=torch.int32)
    want = fp.prefill(q, ks, vs, [(b, 1) for b in range(len(lens))], d ** -0.5, dtype)
    return q, kc, vc, table, kv, want


def check_decode(lens, Hq, Hkv, d, dtype, page, seed=0, max_pages=None, repeat=2):
    q, kc, vc, table, kv, want = _decode_case(lens, Hq, Hkv, d, dtype, page, seed, max_pages)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, len(lens), 1, table.shape[1] * page, Hkv, Hq, d,
                                              0, 0, 0, 0 if dtype == BF16 else 1), DEV)
    args = [x.to(DEV) for x in (q, kc, vc, table, kv)]
    first = None
    for _ in range(repeat):  # the workspace serves call after call
        lse = torch.full((len(lens), Hq), 7.0, device=DEV)
        out = msa.msa_full_attn_decode(*args, lse=lse, ws=ws)
        torch.cuda.synchronize()
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")
        fp.assert_within(lse, want[1], want[3], "lse")
        assert first is None or torch.equal(first, out)
        first = out


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths(page, dtype):
    check_decode([1, 15, 16, 17, 0, 127, 128, 129, 700, 0], 8, 2, 128, dtype, page, page)
    check_decode([333], 8, 2, 64, dtype, page, page + 1)
    check_decode([5, 2100], 4, 4, 64, dtype, page, page + 2, max_pages=200)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", HEADS)
def test_decode_heads(heads, dtype):
    check_decode([40, 1, 530], *heads, dtype, 16, 5)


def test_decode_many_sequences():
    lens = [(37 * b) % 90 for b in range(700)]
    check_decode(lens, 4, 2, 64, BF16, 16, 8)
    check_decode([9000, 1, 4500], 8, 1, 128, BF16, 64, 9)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bad_lengths_and_pages(dtype):
    """Lengths and pages out of range: reported, that sequence zero, the others right."""
    lens = [50, 60, 40, 100]
    q, kc, vc, table, kv, want = _decode_case(lens, 8, 2, 64, dtype, 16, 11)
    kv[0], kv[2] = table.shape[1] * 16 + 1, -3
    table[3, 4] = kc.shape[0]  # one past the last page
    bad, good = [0, 2, 3], [1]
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 4, 1, table.shape[1] * 16, 2, 8, 64, 0, 0, 0,
                                              0 if dtype == BF16 else 1), DEV)
    lse = torch.empty(4, 8, device=DEV)
    d = [x.to(DEV) for x in (q, kc, vc, table, kv)]
    out = msa.msa_full_attn_decode(*d, lse=lse, ws=ws)
    assert msa.msa_read_status(ws) == 6 and msa.msa_read_status(ws) == 0
    assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
    fp.assert_within(out[good], want[0][good], want[2][good], "out")
    cu = torch.arange(5, dtype=torch.int32, device=DEV)
    ws = msa.workspace(4096, DEV)
    out = msa.msa_full_attn_prefill_paged(d[0], d[1], d[2], d[3], cu, d[4], lse=lse, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
    fp.assert_within(out[good], want[0][good], want[2][good], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bad_offsets(dtype):
    """Offsets out of range: reported; nothing written for that sequence."""
    q, k, v, cu_q, cu_k, rows, ks, vs, _ = make([(20, 20), (30, 30), (10, 10)], 8, 2, 64, dtype, 12)
    want = fp.prefill(q, ks, vs, rows, 0.125, dtype)
    cu_bad = cu_q.clone()
    cu_bad[3] = 1000  # the last sequence ends behind the tensor
    ws = msa.workspace(4096, DEV)
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    msa.msa_full_attn_prefill(*[x.to(DEV) for x in (q, k, v, cu_bad, cu_k)], out=out, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (out[50:] == 7.0).all()
    fp.assert_within(out[:50], want[0][:50], want[2][:50], "out")
    ck = cu_k.clone()
    ck[3] = 61  # only the keys' end is wrong: the rows are known
    msa.msa_full_attn_prefill(*[x.to(DEV) for x in (q, k, v, cu_q, ck)], out=out, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (out[50:] == 0).all()


def check_backward(spans, Hq, Hkv, d, dtype, before=0, behind=0, seed=0, scale=0.0):
    q, k, v, cu_q, cu_k, rows, ks, vs, g = make(spans, Hq, Hkv, d, dtype, seed, before, behind)
    sc = scale or d ** -0.5
    fwd = fp.prefill(q, ks, vs, rows, sc, dtype)
    out, lse = fwd[0].to(dtype), fwd[1].float()  # rows of no sequence: NaN
    dout = torch.randn(q.shape, generator=g).to(dtype)
    dout[fwd[1][:, 0].isnan()] = math.nan
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_BACKWARD, len(spans), q.shape[0], k.shape[0], Hkv, Hq, d,
                                              0, 0, 0, 0 if dtype == BF16 else 1), DEV)
    grads = [torch.full(x.shape, 7.0, dtype=dtype, device=DEV) for x in (q, k, v)]
    args = [x.to(DEV) for x in (q, k, v, out, dout, lse, cu_q, cu_k)]
    msa.msa_full_attn_backward(*args, *grads, scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert msa.msa_read_status(ws) == 0
    again = msa.msa_full_attn_backward(*args, scale=scale, ws=ws)
    touched = [torch.zeros(x.shape[0], dtype=torch.bool) for x in (q, k, v)]
    for (q0, Lq), k0, Lk in zip(rows, cu_k[:-1].tolist(), [s[1] for s in spans]):
        at = (slice(q0, q0 + Lq), slice(k0, k0 + Lk), slice(k0, k0 + Lk))
        want, tol = fp.backward(q[at[0]].double(), k[at[1]].double(), v[at[2]].double(), out[at[0]].double(),
                                dout[at[0]].double(), lse[at[0]].double(), sc, dtype)
        for name, gr, gr2, w, t, sl, tc in zip(("dq", "dk", "dv"), grads, again, want, tol, at, touched):
            fp.assert_within(gr[sl], w, t, f"{name} of {(Lq, Lk)}")
            assert torch.equal(gr[sl], gr2[sl]), f"{name}: another run, other bits"
            tc[sl] = True
    for gr, tc in zip(grads, touched):
        assert (gr.cpu()[~tc] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", sorted(SPANS))
def test_backward_spans(name, dtype):
    check_backward(SPANS[name], 8, 2, 128, dtype)
    check_backward(SPANS[name], 4, 2, 64, dtype, before=2, behind=40)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", HEADS)
def test_backward_heads(heads, dtype):
    check_backward([(70, 70), (20, 150), (1, 64)], *heads, dtype, seed=2)


def test_backward_long_and_peaked():
    check_backward([(700, 700), (90, 600)], 4, 1, 64, BF16, seed=3, scale=0.4)
    check_backward([(520, 520)], 4, 2, 128, BF16, seed=4)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_no_rows(dtype):
    """Tq == 0: the keys' gradients are zero; rows of no sequence stay."""
    k = torch.randn(20, 2, 64, device=DEV).to(dtype)
    q = torch.empty(0, 8, 64, dtype=dtype, device=DEV)
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 0, 0], [0, 12, 17]))
    dk, dv = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    msa.msa_full_attn_backward(q, k, k, q, q, torch.empty(0, 8, device=DEV), cu_q, cu_k, dk=dk, dv=dv)
    for x in (dk, dv):
        assert (x[:17] == 0).all() and (x[17:] == 7.0).all()


def test_prefill_no_keys_at_all():
    q = torch.randn(6, 8, 64, device=DEV).to(BF16)
    k = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 6], [0, 0]))
    lse = torch.empty(6, 8, device=DEV)
    out = msa.msa_full_attn_prefill(q, k, k, cu_q, cu_k, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_against_differences(dtype):
    """The kernel's gradient along a direction against central differences of
    the 64-bit forward: error at most the gradient bounds summed along the
    direction, plus the difference's own (h^2, 64-bit) and, for delta, the
    rounding of the forward's output that the call is given."""
    Hq, Hkv, d, L = 4, 2, 64, 90
    q, k, v, cu, _, rows, ks, vs, g = make([(L, L)], Hq, Hkv, d, dtype, 21)
    fwd = lambda q, k, v: fp.prefill(q, [k], [v], rows, 0.125, dtype)  # noqa: E731
    x = [t.double() for t in (q, k, v)]
    out, lse = fwd(*x)[:2]
    dout = torch.randn(q.shape, generator=g).to(dtype)
    got = msa.msa_full_attn_backward(*[t.to(DEV) for t in (q, k, v, out.to(dtype), dout, lse.float(), cu, cu)])
    exact, tol = fp.backward(*x, out.to(dtype).double(), dout.double(), lse, 0.125, dtype)
    true, _ = fp.backward(*x, out, dout.double(), lse, 0.125, dtype)
    for n in range(3):
        u = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        at = lambda t: [y + t * u if m == n else y for m, y in enumerate(x)]  # noqa: E731
        diff = ((fwd(*at(h))[0] - fwd(*at(-h))[0]) * dout.double()).sum() / (2 * h)
        given = ((exact[n] - true[n]) * u).sum().abs()
        room = (tol[n] * u.abs()).sum() + given + 1e-5 * (1 + diff.abs())
        assert abs((got[n].double().cpu() * u).sum() - diff) <= room


def _append_want(q, k, v, rope, spans_new, kv, table, kc, vc, rot, il):
    """Plain append in 64 bits: rotated q, caches, and what may differ by a rounding."""
    page = kc.shape[1]
    qo, kc, vc = q.double().clone(), kc.double().clone(), vc.double().clone()
    for b, (t0, n) in enumerate(spans_new):
        pos = torch.arange(n) + int(kv[b]) - n
        if rot:
            qr, kr = (fp.rotate(x[t0:t0 + n].double(), rope, pos, rot, il) for x in (q, k))
        else:
            qr, kr = q[t0:t0 + n].double(), k[t0:t0 + n].double()
        qo[t0:t0 + n] = qr
        for i in range(n):
            p = int(table[b, pos[i] // page])
            kc[p, pos[i] % page], vc[p, pos[i] % page] = kr[i], v[t0 + i].double()
    return qo, kc, vc


def check_append(lens, old, Hq, Hkv, d, dtype, page, rot, il, seed=0, behind=0, in_place=False, with_q=True,
                 cu_given=True):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + behind
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    q, k, v = r(T, Hq, d), r(T, Hkv, d), r(T, Hkv, d)
    kv = torch.tensor([n + o for n, o in zip(lens, old)], dtype=torch.int32)
    total = [int(x) for x in kv]
    kc, vc, table = fp.paged([r(n, Hkv, d) for n in total], [r(n, Hkv, d) for n in total], page, g, fill=7.0)
    rope = fp.rope_table(max(total + [1]), rot) if rot else None
    cu = fp.offsets(lens)
    spans = list(zip(cu[:-1].tolist(), lens))
    want = _append_want(q, k, v, rope, spans, kv, table, kc, vc, rot, il)
    ws = msa.workspace(256, DEV)
    dq, dkc, dvc = q.to(DEV), kc.to(DEV), vc.to(DEV)
    q_out = dq if in_place else torch.full_like(dq, 7.0)
    got = msa.msa_paged_append(dq if with_q else None, k.to(DEV), v.to(DEV), rope.to(DEV) if rot else None,
                               cu.to(DEV) if cu_given else None, kv.to(DEV), table.to(DEV), dkc, dvc, interleaved=il,
                               q_out=q_out if with_q else None, ws=ws)
    torch.cuda.synchronize()
    assert msa.msa_read_status(ws) == 0
    # x cos - y sin in fp32: two products and a sum, rounded, then the type's rounding; |x|, |y| < 8
    u = fp.U[dtype]
    tol = lambda w: u * w.abs() + 3 * 2.0 ** -24 * 16  # noqa: E731
    if with_q:
        n = sum(lens)
        fp.assert_within(got[:n], want[0][:n], tol(want[0][:n]), "q_out")
        if not in_place:
            assert (got[n:] == 7.0).all()
        else:
            assert torch.equal(got[n:].cpu(), q[n:])
    else:
        assert got is None
    fp.assert_within(dkc, want[1], tol(want[1]), "k_cache")
    assert torch.equal(dvc.double().cpu(), want[2]), "v_cache"


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append(page, il, dtype):
    check_append([1, 0, 40, 129, 7], [0, 5, 300, 63, 16], 8, 2, 128, dtype, page, 128, il, page)
    check_append([33, 2], [1, 900], 6, 3, 64, dtype, page, 32, il, page + 1, behind=6)
    check_append([3], [0], 4, 1, 64, dtype, page, 16, il, page + 2, in_place=True, behind=2)
    check_append([5, 6], [9, 9], 4, 4, 128, dtype, page, 0, il, page + 3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_single_tokens(dtype):
    old = [0, 1, 15, 16, 17, 200, 63, 64]
    check_append([1] * 8, old, 32, 8, 128, dtype, 16, 128, False, 1, cu_given=False)
    check_append([1] * 8, old, 8, 2, 64, dtype, 64, 64, True, 2, cu_given=False, with_q=False)
    check_append([1] * 300, [(7 * b) % 50 for b in range(300)], 4, 2, 64, dtype, 16, 32, False, 3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_bad_positions(dtype):
    """Positions outside the table, past the rotation table, negative, or on a
    page out of range: reported, skipped (q row 0), the rest written."""
    T, d = 5, 64
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(T, 4, d, generator=g).to(dtype), torch.randn(T, 2, d, generator=g).to(dtype)
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 99], [7, 8]], dtype=torch.int32)
    kv = torch.tensor([33, 0, 25, 20, 3], dtype=torch.int32)  # past the table, -1, past rope (24), bad page, fine
    kc = torch.full((9, 16, 2, d), 7.0).to(dtype)
    vc = kc.clone()
    rope = fp.rope_table(24, 64)
    ws = msa.workspace(256, DEV)
    dkc, dvc = kc.to(DEV), vc.to(DEV)
    qo = msa.msa_paged_append(q.to(DEV), k.to(DEV), k.to(DEV), rope.to(DEV), None, kv.to(DEV), table.to(DEV), dkc, dvc,
                              ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (qo[:4] == 0).all() and (qo[4] != 0).any()
    changed = (dvc.cpu() != vc).flatten(2).any(-1).nonzero().tolist()
    assert changed == [[7, 2]]
    assert torch.equal(dvc.cpu()[7, 2], k[4])
    cu = torch.tensor([0, 3, 900], dtype=torch.int32, device=DEV)  # the second sequence ends behind the tensor
    dvc.fill_(7.0)
    msa.msa_paged_append(None, k.to(DEV), k.to(DEV), None, cu, torch.tensor([3, 3], dtype=torch.int32, device=DEV),
                         table[:2].contiguous().to(DEV), dkc, dvc, ws=ws)
    assert msa.msa_read_status(ws) == 6
    changed = (dvc.cpu() != 7.0).flatten(2).any(-1).nonzero().tolist()
    assert changed == [[0, 0], [0, 1], [0, 2]]


def _serve(step_decode):
    """Prompts enter the cache and attend; then single tokens, by ``step_decode``.
    What was rotated and cached is checked against the plain rotation, and every
    output against plain attention over what the cache then holds."""
    g = torch.Generator().manual_seed(31)
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 64, 16, 5
    lens = [50, 1, 130]
    total = [n + steps for n in lens]
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(BF16)  # noqa: E731
    qs, ks, vs = ([r(n, h) for n in total] for h in (Hq, Hkv, Hkv))
    rope = fp.rope_table(max(total), d)
    need = [-(-n // page) for n in total]
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    kc = torch.full((sum(need), page, Hkv, d), math.nan, dtype=BF16, device=DEV)
    vc = kc.clone()
    table, rope_d = table.to(DEV), rope.to(DEV)
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = fp.offsets(lens).to(DEV)
    cat = lambda x, a, e: torch.cat([t[a(b):e(b)] for b, t in enumerate(x)]).to(DEV)  # noqa: E731
    prompt = [cat(x, lambda b: 0, lambda b: lens[b]) for x in (qs, ks, vs)]
    q = msa.msa_paged_append(prompt[0], prompt[1], prompt[2], rope_d, cu, kv, table, kc, vc)
    outs = [(q, msa.msa_full_attn_prefill_paged(q, kc, vc, table, cu, kv))]
    step_in = [[cat(x, lambda b: lens[b] + i, lambda b: lens[b] + i + 1) for x in (qs, ks, vs)] for i in range(steps)]
    outs += step_decode(step_in, rope_d, kv, table, kc, vc)
    torch.cuda.synchronize()
    assert kv.tolist() == total
    at = 0
    for b in range(B):
        pages = table[b, :need[b]].cpu().long()
        kb, vb = (x.cpu()[pages].flatten(0, 1)[:total[b]] for x in (kc, vc))
        qb = torch.cat([outs[0][0][at:at + lens[b]]] + [o[0][b:b + 1] for o in outs[1:]]).cpu()
        ob = torch.cat([outs[0][1][at:at + lens[b]]] + [o[1][b:b + 1] for o in outs[1:]])
        at += lens[b]
        pos = torch.arange(total[b])
        for got, x in ((qb, qs[b]), (kb, ks[b])):
            w = fp.rotate(x.double(), rope, pos, d, False)
            fp.assert_within(got, w, 2.0 ** -8 * w.abs() + 3 * 2.0 ** -24 * 16, "rotated")
        assert torch.equal(vb, vs[b])
        w = fp.prefill(qb, [kb], [vb], [(0, total[b])], d ** -0.5, BF16)
        fp.assert_within(ob, w[0], w[2], f"sequence {b}")


def test_serving_run():
    def steps(step_in, rope, kv, table, kc, vc):
        outs = []
        for q, k, v in step_in:
            kv += 1
            q = msa.msa_paged_append(q, k, v, rope, None, kv, table, kc, vc)
            outs.append((q, msa.msa_full_attn_decode(q, kc, vc, table, kv)))
        return outs
    _serve(steps)


def test_serving_run_captured():
    """The step as a CUDA graph, replayed on new inputs; two graphs share one workspace."""
    def steps(step_in, rope, kv, table, kc, vc):
        q, k, v = (x.clone() for x in step_in[0])
        qo, out = torch.empty_like(q), torch.empty_like(q)
        ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 3, 1, table.shape[1] * 16, 2, 8, 64, 0, 0, 0,
                                                  msa.MSA_BF16), DEV)
        graphs = []
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = kv.clone()
        for _ in range(2):
            with torch.cuda.stream(side):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    kv += 1
                    msa.msa_paged_append(q, k, v, rope, None, kv, table, kc, vc, q_out=qo, ws=ws)
                    msa.msa_full_attn_decode(qo, kc, vc, table, kv, out=out, ws=ws)
                graphs.append(graph)
        torch.cuda.synchronize()
        assert torch.equal(kv, keep)
        outs = []
        for i, new in enumerate(step_in):
            for dst, src in zip((q, k, v), new):
                dst.copy_(src)
            graphs[i % 2].replay()
            outs.append((qo.clone(), out.clone()))
        assert msa.msa_read_status(ws) == 0
        return outs
    _serve(steps)


def test_other_stream():
    """Everything on a stream that is not the current one, workspaces made by the call."""
    q, k, v, cu_q, cu_k, rows, ks, vs, _ = make([(60, 60), (9, 200)], 8, 2, 64, BF16, 40)
    want = fp.prefill(q, ks, vs, rows, 0.125, BF16)
    d = [x.to(DEV) for x in (q, k, v, cu_q, cu_k)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse = torch.empty(q.shape[:2], device=DEV)
    out = msa.msa_full_attn_prefill(*d, lse=lse, stream=s)
    grads = msa.msa_full_attn_backward(*d[:3], out, d[0], lse, d[3], d[4], stream=s)
    s.synchronize()
    fp.assert_within(out, want[0], want[2], "out")
    assert all(x.isfinite().all() for x in grads)
