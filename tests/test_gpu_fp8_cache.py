"""GPU parity of the paged caches in 8 bits: codes and scales bit for bit, rows
read back, and decode over them within the bounds derived in fp8_plain.py."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import fp8_plain as f8
import full_plain as fp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, FP32 = torch.bfloat16, torch.float32
HEADS = [(4, 4, 64), (8, 2, 64), (8, 2, 128), (6, 2, 128), (16, 1, 128), (32, 1, 64), (10, 2, 128), (64, 1, 128),
         (9, 3, 64)]


def code(dtype):
    return msa.MSA_BF16 if dtype == BF16 else msa.MSA_FP32


def rows_in(T, H, d, g, dtype, values="normal"):
    x = torch.randn(T, H, d, generator=g)
    if values == "wide":  # rows of very unequal size, among them zeros, subnormals and the type's largest values
        x = x * torch.exp2(torch.randint(-40, 40, (T, H, 1), generator=g).float())
        x[::7] = 0.0
        x[1::7] *= 2.0 ** -90
        if T > 2:
            x[2] = torch.sign(x[2]) * torch.finfo(dtype).max
        x[..., ::5] = 0.0
    elif values == "borders":  # integers below 2^8 and a maximum that is not a power of two: many ties
        x = torch.randint(-255, 256, (T, H, d), generator=g).float()
    return x.to(dtype)


def check_append(lens, old, Hq, Hkv, d, dtype, page, rot, il, seed=0, behind=0, with_q=True, cu_given=True,
                 values="normal"):
    """Append, then read the new tokens back; every other cache row and scale stays."""
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens) + behind, sum(lens)
    q = torch.randn(T, Hq, d, generator=g).to(dtype)
    k, v = rows_in(T, Hkv, d, g, dtype, values), rows_in(T, Hkv, d, g, dtype, values)
    total = [a + b for a, b in zip(lens, old)]
    kv = torch.tensor(total, dtype=torch.int32)
    fill = [torch.randint(0, 256, (t, Hkv, d), generator=g, dtype=torch.uint8).view(f8.E4M3) for t in total * 2]
    scales = [torch.rand(t, Hkv, generator=g) for t in total * 2]
    B = len(lens)
    kc, vc, ks, vs, table = f8.paged(fill[:B], fill[B:], scales[:B], scales[B:], page, g)
    rope = fp.rope_table(max(total + [1]), rot) if rot else None
    cu = fp.offsets(lens)
    want = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    qw, rows_want = q.double().clone(), [[], []]
    for b, t0 in enumerate(cu[:-1].tolist()):
        pos = torch.arange(lens[b]) + old[b]
        mine = slice(t0, t0 + lens[b])
        kk = k[mine].double()
        if rot:
            kk = fp.rotate(kk, rope, pos, rot, il)
            qw[mine] = fp.rotate(q[mine].double(), rope, pos, rot, il)
        for x, (y, c, s) in enumerate(((kk.float(), want[0], want[2]), (v[mine].float(), want[1], want[3]))):
            codes, scale = f8.quantise(y)
            at = table[b, pos // page].long()
            c[at, pos % page] = codes.view(torch.uint8)
            s[at, :, pos % page] = scale
            rows_want[x].append((codes.double() * scale.double()[..., None]).to(dtype))
    ws = msa.workspace(256, DEV)
    dkc, dvc, dks, dvs = (x.to(DEV) for x in (kc, vc, ks, vs))
    dcu, dkv, dt = cu.to(DEV) if cu_given else None, kv.to(DEV), table.to(DEV)
    q_out = torch.full((T, Hq, d), 7.0, dtype=dtype, device=DEV)
    got = msa.msa_paged_append_fp8(q.to(DEV) if with_q else None, k.to(DEV), v.to(DEV), rope.to(DEV) if rot else None,
                                   dcu, dkv, dt, dkc, dvc, dks, dvs, interleaved=il, q_out=q_out if with_q else None,
                                   ws=ws)
    assert msa.msa_read_status(ws) == 0
    if with_q:  # as msa_paged_append
        fp.assert_within(got[:n], qw[:n], fp.U[dtype] * qw[:n].abs() + 3 * 2.0 ** -24 * 16, "q_out")
        assert (got[n:] == 7.0).all()
    for name, x, w in (("k_cache", dkc, want[0]), ("v_cache", dvc, want[1])):
        x = x.cpu().view(torch.uint8)
        same = (x == w) | (((x | w) == 0x80) & ((x & w) == 0))  # zeros of either sign
        assert same.all(), f"{name}: {int((~same).sum())} codes differ"
    for name, x, w in (("k_scale", dks, want[2]), ("v_scale", dvs, want[3])):
        assert torch.equal(x.cpu().view(torch.int32), w.view(torch.int32)), name
    out = [torch.full((T, Hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    msa.msa_paged_read_fp8(dkc, dvc, dks, dvs, dt, dcu, dkv, T, k_out=out[0], v_out=out[1], ws=ws)
    assert msa.msa_read_status(ws) == 0
    for x, w in zip(out, rows_want):
        assert torch.equal(x[:n].cpu(), torch.cat(w))
        assert (x[n:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_and_read(page, il, dtype):
    check_append([1, 0, 40, 129, 7], [0, 5, 300, 63, 16], 8, 2, 128, dtype, page, 128, il, page)
    check_append([33, 2], [1, 900], 6, 3, 64, dtype, page, 32, il, page + 1, behind=6)
    check_append([3], [0], 4, 1, 64, dtype, page, 16, il, page + 2, behind=2)
    check_append([5, 6], [9, 9], 4, 4, 128, dtype, page, 0, il, page + 3)
    check_append([17], [3], 5, 5, 128, dtype, page, 48, il, page + 4, with_q=False)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("values", ["wide", "borders"])
def test_append_values(values, dtype):
    check_append([70, 3], [0, 9], 8, 2, 64, dtype, 16, 0, False, 1, values=values)
    check_append([70, 3], [0, 9], 8, 2, 128, dtype, 32, 64, False, 2, values="borders")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_single_tokens(dtype):
    old = [0, 1, 15, 16, 17, 200, 63, 64]
    check_append([1] * 8, old, 32, 8, 128, dtype, 16, 128, False, 1, cu_given=False)
    check_append([1] * 8, old, 8, 2, 64, dtype, 64, 64, True, 2, cu_given=False, with_q=False)
    check_append([1] * 300, [(7 * b) % 50 for b in range(300)], 4, 2, 64, dtype, 16, 32, False, 3)
    check_append([3] * 300, [(7 * b) % 50 for b in range(300)], 4, 2, 64, dtype, 16, 32, False, 4)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_infinities(dtype):
    """A row with an infinity or NaN is NaN when read; its neighbours are not touched by it."""
    g = torch.Generator().manual_seed(5)
    k, v = torch.randn(3, 2, 64, generator=g).to(dtype), torch.randn(3, 2, 64, generator=g).to(dtype)
    k[1, 0, 5], v[2, 1, 63], v[0, 0, 0] = math.inf, math.nan, -math.inf
    caches = [torch.zeros(2, 16, 2, 64, device=DEV).to(f8.E4M3) for _ in range(2)]
    scales = [torch.zeros(2, 2, 16, device=DEV) for _ in range(2)]
    cu, kv, table = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 3], [3], [[1, 0]]))
    rope = fp.rope_table(8, 32).to(DEV)
    msa.msa_paged_append_fp8(None, k.to(DEV), v.to(DEV), rope, cu, kv, table, *caches, *scales)
    kr, vr = msa.msa_paged_read_fp8(*caches, *scales, table, cu, kv, 3, dtype=dtype)
    for x, bad in ((kr, [(1, 0)]), (vr, [(2, 1), (0, 0)])):
        for t in range(3):
            for h in range(2):
                assert x[t, h].isnan().all() if (t, h) in bad else x[t, h].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_and_read_bad_positions(dtype):
    """Positions outside the table, past the rotation table, negative, or on a
    page out of range: reported; append skips them, read gives zeros."""
    T, d = 5, 64
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(T, 4, d, generator=g).to(dtype), torch.randn(T, 2, d, generator=g).to(dtype)
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 99], [7, 8]], dtype=torch.int32, device=DEV)
    kv = torch.tensor([33, 0, 25, 20, 3], dtype=torch.int32, device=DEV)
    caches = [torch.full((9, 16, 2, d), 7.0, device=DEV).to(f8.E4M3) for _ in range(2)]
    scales = [torch.full((9, 2, 16), 2.0, device=DEV) for _ in range(2)]
    ws = msa.workspace(256, DEV)
    qo = msa.msa_paged_append_fp8(q.to(DEV), k.to(DEV), k.to(DEV), fp.rope_table(24, 64).to(DEV), None, kv, table,
                                  *caches, *scales, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (qo[:4] == 0).all() and (qo[4] != 0).any()
    for x in caches:
        assert (x.float() != 7.0).flatten(2).any(-1).nonzero().tolist() == [[7, 2]]
    for x in scales:
        assert (x != 2.0).any(1).nonzero().tolist() == [[7, 2]]
    kr, vr = msa.msa_paged_read_fp8(*caches, *scales, table, None, kv, T, dtype=dtype, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (kr[[0, 1, 3]] == 0).all() and (vr[[0, 1, 3]] == 0).all() and (kr[2] == 14.0).all()  # 25 is in the table
    assert torch.equal(vr[4].cpu(), (lambda c, s: (c.float() * s[..., None]).to(dtype))(*f8.quantise(k[4].float())))


def _cache(lens, Hkv, d, page, g, scales="pow2", max_pages=None):
    codes, sc = [], []
    for n in lens * 2:
        c, s = f8.quantise(torch.randn(n, Hkv, d, generator=g) * (0.25 + 2 * torch.rand(n, Hkv, 1, generator=g)))
        if scales == "any":
            s = torch.rand(n, Hkv, generator=g) * 0.02 + 1e-4
        elif scales == "wide":  # values over many binades, some rows zero
            s = s * torch.exp2(torch.randint(-30, 30, (n, Hkv), generator=g).float())
            s[::5] = 0.0
        codes.append(c)
        sc.append(s)
    B = len(lens)
    if scales == "wide":  # keys keep the softmax from being decided by one
        sc[:B] = [f8.quantise(c.float())[1] * 2.0 ** -7 for c in codes[:B]]
    parts = (codes[:B], codes[B:], sc[:B], sc[B:])
    return parts, f8.paged(*parts, page, g, max_pages=max_pages)


def check_decode(lens, Hq, Hkv, d, dtype, page, seed=0, scales="pow2", qmul=1.0, scale=0.0, max_pages=None, repeat=2):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(len(lens), Hq, d, generator=g) * qmul).to(dtype)
    parts, (kc, vc, ks, vs, table) = _cache(lens, Hkv, d, page, g, scales, max_pages)
    want = f8.decode(q, *parts, scale or d ** -0.5, dtype)
    kv = torch.tensor(lens, dtype=torch.int32)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_FP8, len(lens), 1, table.shape[1] * page, Hkv, Hq,
                                              d, 0, 0, 0, code(dtype)), DEV)
    args = [x.to(DEV) for x in (q, kc, vc, ks, vs, table, kv)]
    first = None
    for _ in range(repeat):  # the workspace serves call after call
        lse = torch.full((len(lens), Hq), 7.0, device=DEV)
        out = msa.msa_full_attn_decode_fp8(*args, scale=scale, lse=lse, ws=ws)
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


@pytest.mark.parametrize("heads", [(3, 3, 64), (8, 1, 64), (32, 1, 64), (9, 3, 128)])
def test_decode_ends_of_steps(heads):
    """Lengths about the ends of 16-key tiles and of a warp's 32- or 64-key steps, with an odd number of heads."""
    check_decode([31, 32, 33, 47, 48, 49, 63, 64, 65, 0, 79, 80, 81, 511, 512, 513, 575, 1089], *heads, BF16, 16, 14)
    check_decode([(29 * b) % 150 for b in range(500)], *heads, BF16, 32, 15)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_scales_and_sizes(d, dtype):
    check_decode([40, 1, 530], 8, 2, d, dtype, 16, 6, scales="any")
    check_decode([40, 1, 530, 3], 8, 2, d, dtype, 16, 7, scales="wide")
    check_decode([300, 7], 8, 2, d, dtype, 32, 8, qmul=2.0 ** -60)
    check_decode([300, 7], 8, 2, d, dtype, 32, 9, qmul=2.0 ** 40, scale=2.0 ** -43)
    check_decode([300, 7], 8, 2, d, dtype, 32, 10, qmul=0.0)
    check_decode([2500, 1000], 4, 1, d, dtype, 64, 11, scale=0.5)  # peaked: the running maxima move


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_many_sequences(dtype):
    check_decode([(37 * b) % 90 for b in range(700)], 4, 2, 64, dtype, 16, 8)  # whole items for single warps
    check_decode([9000, 1, 4500], 8, 1, 128, dtype, 64, 9)  # items in several CTAs


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (6, 3, 64), (16, 1, 128), (64, 2, 128), (4, 4, 64)])
def test_decode_runs_of_warps(heads, dtype):
    """More items than SMs: items that end in a warp's run, lie in several warps' or in several CTAs'; two lengths of them."""
    check_decode([(53 * b) % 300 for b in range(170)], *heads, dtype, 16, 16)
    check_decode([5000, 1, 0, 2500] + [1 + b % 40 for b in range(160)], *heads, dtype, 64, 17)
    check_decode([17] * 400, *heads, dtype, 32, 18)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_growing_scores(dtype):
    """Keys whose scores rise along the sequence while their values' scales fall, and the other way round."""
    n, d = 600, 64
    for up in (1, -1):
        g = torch.Generator().manual_seed(3)
        at = torch.arange(n).float() if up > 0 else torch.arange(n).flip(0).float()
        kcode = torch.ones(n, 1, d).to(f8.E4M3)
        vcode = torch.randn(n, 1, d, generator=g).to(f8.E4M3)
        ks, vs = (at / 50)[:, None], torch.exp2(-at / 25).floor_()[:, None] + torch.exp2(-(at / 25).floor())[:, None]
        q = torch.ones(1, 2, d).to(dtype)
        parts = ([kcode], [vcode], [ks], [vs])
        kc, vc, ksp, vsp, table = f8.paged(*parts, 16, g)
        want = f8.decode(q, *parts, 0.125, dtype)
        kv = torch.tensor([n], dtype=torch.int32)
        lse = torch.empty(1, 2, device=DEV)
        out = msa.msa_full_attn_decode_fp8(*[x.to(DEV) for x in (q, kc, vc, ksp, vsp, table, kv)], lse=lse)
        fp.assert_within(out, want[0], want[2], "out")
        fp.assert_within(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_bad_lengths_pages_and_nan_rows(dtype):
    """Out of range: reported, zero. A row of scale NaN: the heads that see it are NaN, no others."""
    lens = [50, 60, 40, 100, 30]
    g = torch.Generator().manual_seed(11)
    q = torch.randn(5, 8, 64, generator=g).to(dtype)
    parts, (kc, vc, ks, vs, table) = _cache(lens, 2, 64, 16, g)
    want = f8.decode(q, *parts, 0.125, dtype)
    kv = torch.tensor(lens, dtype=torch.int32)
    kv[0], kv[2] = table.shape[1] * 16 + 1, -3
    table[3, 4] = kc.shape[0]
    vs[int(table[4, 1]), 1, 3] = math.nan  # key 19 of sequence 4, second head
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_FP8, 5, 1, table.shape[1] * 16, 2, 8, 64, 0, 0, 0,
                                              code(dtype)), DEV)
    lse = torch.empty(5, 8, device=DEV)
    out = msa.msa_full_attn_decode_fp8(*[x.to(DEV) for x in (q, kc, vc, ks, vs, table, kv)], lse=lse, ws=ws)
    assert msa.msa_read_status(ws) == 6 and msa.msa_read_status(ws) == 0
    assert (out[[0, 2, 3]] == 0).all() and (lse[[0, 2, 3]] == -math.inf).all()
    fp.assert_within(out[1], want[0][1], want[2][1], "out")
    fp.assert_within(out[4, :4], want[0][4, :4], want[2][4, :4], "first head")
    assert out[4, 4:].isnan().all()


@pytest.mark.parametrize("bad", [[0, 30, 20, 50, 60], [0, -5, 30, 50, 60], [0, 10, 30, 70, 60]])
def test_offsets_out_of_order(bad):
    """Reported; sequences in range are written and read, nobody else's rows are."""
    g = torch.Generator().manual_seed(2)
    k = torch.randn(60, 2, 64, generator=g).to(BF16)
    caches = [torch.zeros(12, 16, 2, 64, device=DEV).to(f8.E4M3) for _ in range(2)]
    scales = [torch.zeros(12, 2, 16, device=DEV) for _ in range(2)]
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(4, 3)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    kv = torch.full((4,), 48, dtype=torch.int32, device=DEV)
    floor, fine = 0, []
    for a, e in zip(bad[:-1], bad[1:]):
        fine.append(0 <= a <= e <= 60 and a >= floor)
        floor = max(floor, a) if 0 <= a <= 60 else floor
    ws = msa.workspace(256, DEV)
    msa.msa_paged_append_fp8(None, k.to(DEV), k.to(DEV), None, cu, kv, table, *caches, *scales, ws=ws)
    assert msa.msa_read_status(ws) == 6
    out = [torch.full((60, 2, 64), 7.0, dtype=BF16, device=DEV) for _ in range(2)]
    msa.msa_paged_read_fp8(*caches, *scales, table, cu, kv, 60, k_out=out[0], v_out=out[1], ws=ws)
    assert msa.msa_read_status(ws) == 6
    codes, s = f8.quantise(k.float())
    want = (codes.float() * s[..., None]).to(BF16)
    mine = torch.zeros(60, dtype=torch.bool)
    for (a, e), ok in zip(zip(bad[:-1], bad[1:]), fine):
        if ok:
            mine[a:e] = True
    for x in out:
        assert torch.equal(x.cpu()[mine], want[mine]) and (x.cpu()[~mine] == 7.0).all()


def test_caches_past_32_bits():
    """Cache rows beyond 2^32 bytes of codes, and scales' offsets beyond theirs."""
    pages, page, Hkv, d = 40000, 128, 8, 128  # 5.2 GB a cache
    g = torch.Generator().manual_seed(1)
    caches = [torch.empty(pages, page, Hkv, d, dtype=torch.uint8, device=DEV).view(f8.E4M3) for _ in range(2)]
    scales = [torch.empty(pages, Hkv, page, device=DEV) for _ in range(2)]
    table = torch.tensor([[39999, 3, 35000]], dtype=torch.int32, device=DEV)
    n = 300
    k, v = torch.randn(n, Hkv, d, generator=g).to(BF16), torch.randn(n, Hkv, d, generator=g).to(BF16)
    cu, kv = torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    msa.msa_paged_append_fp8(None, k.to(DEV), v.to(DEV), None, cu, kv, table, *caches, *scales)
    (kc, ks), (vc, vs) = f8.quantise(k.float()), f8.quantise(v.float())
    kr, vr = msa.msa_paged_read_fp8(*caches, *scales, table, cu, kv, n)
    assert torch.equal(kr.cpu(), (kc.float() * ks[..., None]).to(BF16))
    assert torch.equal(vr.cpu(), (vc.float() * vs[..., None]).to(BF16))
    q = torch.randn(1, 16, d, generator=g).to(BF16)
    want = f8.decode(q, [kc], [vc], [ks], [vs], d ** -0.5, BF16)
    out = msa.msa_full_attn_decode_fp8(q.to(DEV), *caches, *scales, table, kv)
    fp.assert_within(out, want[0], want[2], "out")


def _serve(captured):
    """Prompts in two chunks (append, read back, attend as packed rows), then decode steps; all
    against plain attention over what the cache's codes stand for."""
    g = torch.Generator().manual_seed(31)
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 64, 16, 4
    first, second = [20, 1, 90], [30, 5, 40]
    total = [a + b + steps for a, b in zip(first, second)]
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(BF16)  # noqa: E731
    qs, ks, vs = ([r(n, h) for n in total] for h in (Hq, Hkv, Hkv))
    rope = fp.rope_table(max(total), d)
    need = [-(-n // page) for n in total]
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    table, rope_d = table.to(DEV), rope.to(DEV)
    cache = [torch.full((sum(need), page, Hkv, d), math.nan, device=DEV).to(f8.E4M3) for _ in range(2)]
    cache += [torch.full((sum(need), Hkv, page), math.nan, device=DEV) for _ in range(2)]
    cat = lambda x, a, e: torch.cat([t[a[b]:e[b]] for b, t in enumerate(x)]).to(DEV)  # noqa: E731
    kv = torch.zeros(B, dtype=torch.int32, device=DEV)
    got = [[] for _ in range(B)]  # (rotated q, out) of each sequence
    at = [0] * B
    for n in (first, second):
        to = [a + x for a, x in zip(at, n)]
        kv += torch.tensor(n, dtype=torch.int32, device=DEV)
        cu_q, cu_k = fp.offsets(n), fp.offsets(to)
        q = msa.msa_paged_append_fp8(*(cat(x, at, to) for x in (qs, ks, vs)), rope_d, cu_q.to(DEV), kv, table, *cache)
        kr, vr = msa.msa_paged_read_fp8(*cache, table, cu_k.to(DEV), kv, sum(to))
        out = msa.msa_full_attn_prefill(q, kr, vr, cu_q.to(DEV), cu_k.to(DEV))
        for b in range(B):
            got[b].append((q[cu_q[b]:cu_q[b + 1]].cpu(), out[cu_q[b]:cu_q[b + 1]].cpu()))
        at = to
    q, k, v = (cat(x, at, [a + 1 for a in at]) for x in (qs, ks, vs))
    qo, out = torch.empty_like(q), torch.empty_like(q)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_FP8, B, 1, table.shape[1] * page, Hkv, Hq, d, 0, 0,
                                              0, msa.MSA_BF16), DEV)

    def step():
        kv.add_(1)
        msa.msa_paged_append_fp8(q, k, v, rope_d, None, kv, table, *cache, q_out=qo, ws=ws)
        msa.msa_full_attn_decode_fp8(qo, *cache, table, kv, out=out, ws=ws)

    graphs = []
    if captured:  # two graphs share one workspace
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(2):
            with torch.cuda.stream(side):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            graphs.append(graph)
        torch.cuda.synchronize()
    for i in range(steps):
        for dst, src in zip((q, k, v), (qs, ks, vs)):
            dst.copy_(cat(src, at, [a + 1 for a in at]))
        graphs[i % 2].replay() if captured else step()
        at = [a + 1 for a in at]
        for b in range(B):
            got[b].append((qo[b:b + 1].cpu(), out[b:b + 1].cpu()))
    assert msa.msa_read_status(ws) == 0 and kv.tolist() == total
    cu = fp.offsets(total).to(DEV)
    kr, vr = (x.cpu() for x in msa.msa_paged_read_fp8(*cache, table, cu, kv, sum(total)))
    for b in range(B):
        mine = slice(int(cu[b]), int(cu[b + 1]))
        codes, s = f8.quantise(fp.rotate(ks[b].double(), rope, torch.arange(total[b]), d, False).float())
        assert torch.equal(kr[mine], (codes.float() * s[..., None]).to(BF16))
        qb, ob = (torch.cat([x[i] for x in got[b]]) for i in (0, 1))
        w = fp.prefill(qb, [kr[mine]], [vr[mine]], [(0, total[b])], d ** -0.5, BF16)
        fp.assert_within(ob, w[0], w[2], f"sequence {b}")


def test_serving_run():
    _serve(False)


def test_serving_run_captured():
    _serve(True)


def test_other_stream_and_workspace_of_another_operation():
    """Everything on a stream that is not the current one; one workspace under several operations."""
    g = torch.Generator().manual_seed(40)
    parts, laid = _cache([300, 5], 2, 64, 16, g)
    q = torch.randn(2, 8, 64, generator=g).to(BF16)
    want = f8.decode(q, *parts, 0.125, BF16)
    kc, vc, ks, vs, table, q, kv = (x.to(DEV) for x in (*laid, q, torch.tensor([300, 5], dtype=torch.int32)))
    plain = torch.randn(table.max().clamp_max(laid[0].shape[0] - 1) + 1, 16, 2, 64, device=DEV).to(BF16)
    full = torch.zeros(laid[0].shape[0], 16, 2, 64, device=DEV).to(BF16)
    full[:plain.shape[0]] = plain
    ws = msa.workspace(1 << 24, DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cu = torch.tensor([0, 300, 305], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(2):
        kr, vr = msa.msa_paged_read_fp8(kc, vc, ks, vs, table, cu, kv, 305, stream=s)
        out = msa.msa_full_attn_decode_fp8(q, kc, vc, ks, vs, table, kv, ws=ws, stream=s)
        msa.msa_full_attn_decode(q, full, full, table, kv, ws=ws, stream=s)
        again = msa.msa_full_attn_decode_fp8(q, kc, vc, ks, vs, table, kv, ws=ws, stream=s)
        s.synchronize()
        fp.assert_within(out, want[0], want[2], "out")
        assert torch.equal(out, again)
    assert torch.equal(kr.cpu(), torch.cat([(c.float() * x[..., None]).to(BF16) for c, x in zip(parts[0], parts[2])]))
    assert msa.msa_read_status(ws) == 0


def test_decode_timeout_then_recovers():
    """A warp of every second CTA lets a wait run out: reported, nothing hangs, the next call is right."""
    g = torch.Generator().manual_seed(50)
    lens = [5000, 1, 300]
    parts, laid = _cache(lens, 2, 64, 16, g)
    q = torch.randn(3, 8, 64, generator=g).to(BF16)
    want = f8.decode(q, *parts, 0.125, BF16)
    args = [x.to(DEV) for x in (q, *laid, torch.tensor(lens, dtype=torch.int32))]
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_FP8, 3, 1, laid[4].shape[1] * 16, 2, 8, 64, 0, 0, 0,
                                              msa.MSA_BF16), DEV)
    msa.msa_debug_inject_timeout(True)
    try:
        msa.msa_full_attn_decode_fp8(*args, ws=ws)
        assert msa.msa_read_status(ws) == 5
    finally:
        msa.msa_debug_inject_timeout(False)
    for _ in range(2):
        out = msa.msa_full_attn_decode_fp8(*args, ws=ws)
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")


def test_decode_timeout_of_many_items_then_recovers():
    """The same where warps take runs of steps and items lie in several CTAs."""
    g = torch.Generator().manual_seed(51)
    lens = [1 + (61 * b) % 400 for b in range(180)]
    parts, laid = _cache(lens, 2, 64, 16, g)
    q = torch.randn(180, 8, 64, generator=g).to(BF16)
    want = f8.decode(q, *parts, 0.125, BF16)
    args = [x.to(DEV) for x in (q, *laid, torch.tensor(lens, dtype=torch.int32))]
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_FP8, 180, 1, laid[4].shape[1] * 16, 2, 8, 64, 0, 0,
                                              0, msa.MSA_BF16), DEV)
    msa.msa_debug_inject_timeout(True)
    try:
        msa.msa_full_attn_decode_fp8(*args, ws=ws)
        assert msa.msa_read_status(ws) == 5
    finally:
        msa.msa_debug_inject_timeout(False)
    for _ in range(2):
        out = msa.msa_full_attn_decode_fp8(*args, ws=ws)
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_least_aligned_tensors(dtype):
    """Every tensor 16 bytes behind a coarser boundary, which is all that the calls ask for."""
    g = torch.Generator().manual_seed(60)

    def off(x):
        raw = torch.zeros(x.nbytes + 272, dtype=torch.uint8, device=DEV)
        at = (-raw.data_ptr()) % 256 + 16
        y = raw[at:at + x.nbytes].view(x.dtype).view(x.shape)
        y.copy_(x)
        return y

    lens = [40, 3]
    k, v = (torch.randn(43, 2, 64, generator=g).to(dtype) for _ in range(2))
    q = off(torch.randn(2, 8, 64, generator=g).to(dtype))
    cache = [off(torch.zeros(4, 16, 2, 64).to(f8.E4M3)) for _ in range(2)] + [off(torch.zeros(4, 2, 16)) for _ in range(2)]
    table, kv, cu = (off(i) for i in (torch.tensor([[3, 0, 1], [2, 9, 9]], dtype=torch.int32),
                                      torch.tensor(lens, dtype=torch.int32), fp.offsets(lens)))
    msa.msa_paged_append_fp8(None, off(k), off(v), None, cu, kv, table, *cache)
    out = [off(torch.zeros(43, 2, 64).to(dtype)) for _ in range(2)]
    msa.msa_paged_read_fp8(*cache, table, cu, kv, 43, k_out=out[0], v_out=out[1])
    parts = [f8.quantise(x.float()) for x in (k, v)]
    for x, (c, s) in zip(out, parts):
        assert torch.equal(x.cpu(), (c.float() * s[..., None]).to(dtype))
    cut = lambda x: [x[:40], x[40:]]  # noqa: E731
    want = f8.decode(q.cpu(), cut(parts[0][0]), cut(parts[1][0]), cut(parts[0][1]), cut(parts[1][1]), 0.125, dtype)
    got = msa.msa_full_attn_decode_fp8(q, *cache, table, kv, out=off(torch.zeros(2, 8, 64).to(dtype)))
    fp.assert_within(got, want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [5, 900])
def test_append_in_place(T, dtype):
    """q_out == q, with a CTA and with a warp per token: the bits of the other call."""
    g = torch.Generator().manual_seed(70)
    q = torch.randn(T, 8, 128, generator=g).to(dtype).to(DEV)
    k = torch.randn(T, 2, 128, generator=g).to(dtype).to(DEV)
    pages = -(-T // 16)
    cache = [torch.zeros(pages, 16, 2, 128, device=DEV).to(f8.E4M3) for _ in range(2)]
    cache += [torch.zeros(pages, 2, 16, device=DEV) for _ in range(2)]
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, pages)
    cu, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, T], [T]))
    rope = fp.rope_table(T, 96).to(DEV)
    want = msa.msa_paged_append_fp8(q, k, k, rope, cu, kv, table, *cache)
    got = msa.msa_paged_append_fp8(q, k, k, rope, cu, kv, table, *cache, q_out=q)
    assert got is q and torch.equal(got, want)


def check_parts(q, parts, dtype, scale, page=16, seed=0, floor=0.0, copies=1):
    """Decode over given codes and scales; `copies`: that many sequences read the same pages."""
    g = torch.Generator().manual_seed(seed)
    kc, vc, ks, vs, table = f8.paged(*parts, page, g)
    out_w, lse_w, tol, ltol = f8.decode(q, *parts, scale, dtype)
    lens = torch.tensor([x.shape[0] for x in parts[0]], dtype=torch.int32)
    q, table, lens = (x.repeat(copies, *[1] * (x.dim() - 1)) for x in (q, table, lens))
    lse = torch.empty(q.shape[:2], device=DEV)
    out = msa.msa_full_attn_decode_fp8(*[x.to(DEV) for x in (q, kc, vc, ks, vs, table, lens)], scale=scale, lse=lse)
    many = lambda x: x.repeat(copies, *[1] * (x.dim() - 1))  # noqa: E731
    fp.assert_within(out, many(out_w), many(tol) + floor, "out")
    fp.assert_within(lse, many(lse_w), many(ltol), "lse")


def subnormal_floor(n, dtype):
    """Behind the last factor each of up to n / 16 + 8 sums rounds by half of fp32's
    least step, 2^-149; a bf16 output by half of 2^-133."""
    return (n // 16 + 8) * 2.0 ** -150 + (2.0 ** -134 if dtype == BF16 else 0.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (3, 3, 64), (16, 1, 128)])
def test_decode_least_value_scales(heads, dtype):
    """Value scales down to 2^-126, which is what an append writes for the smallest
    rows: codes up to 448 make normal numbers of them."""
    Hq, Hkv, d = heads
    for top, lens, copies in ((-126, [40, 1, 530], 1), (-120, [300], 1), (-100, [40, 700], 1), (-126, [37, 5], 200)):
        g = torch.Generator().manual_seed(80 - top)
        q = torch.randn(len(lens), Hq, d, generator=g).to(dtype)
        (ck, cv, sk, sv), _ = _cache(lens, Hkv, d, 16, g)
        sv = [torch.exp2(torch.randint(-126, top + 1, x.shape, generator=g).float()) for x in sv]
        check_parts(q, (ck, cv, sk, sv), dtype, d ** -0.5, floor=subnormal_floor(max(lens), dtype), copies=copies)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_largest_weight_without_values(dtype):
    """Keys with most of the weight and values of 0, beside others with small scales."""
    n, d = 150, 64
    g = torch.Generator().manual_seed(90)
    kcode = torch.zeros(n, 1, d).to(f8.E4M3)
    kcode[:, :, 0] = torch.ones(n, 1).to(f8.E4M3)
    vcode = torch.randn(n, 1, d, generator=g).to(f8.E4M3)
    ks, vs = torch.rand(n, 1, generator=g), torch.full((n, 1), 2.0 ** -112)
    ks[::30], vs[::30] = 10.0, 0.0  # 2^-13 of theirs
    q = torch.zeros(1, 2, d)
    q[..., 0] = 1.0
    check_parts(q.to(dtype), ([kcode], [vcode], [ks], [vs]), dtype, 1.0, floor=subnormal_floor(n, dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_subnormal_value_scales(dtype):
    """Another writer's scales below 2^-126: finite and not negative, so they are taken."""
    lens, d = [40, 300], 128
    g = torch.Generator().manual_seed(91)
    q = torch.randn(2, 8, d, generator=g).to(dtype)
    (ck, cv, sk, sv), _ = _cache(lens, 2, d, 16, g)
    sv = [torch.randint(1 << 18, 1 << 23, x.shape, generator=g).double().mul(2.0 ** -149).float() for x in sv]
    assert all(((x > 0) & (x < 2.0 ** -126)).all() for x in sv)
    check_parts(q, (ck, cv, sk, sv), dtype, d ** -0.5, floor=subnormal_floor(300, dtype))


# What a weight's terms leave of it, of the largest weight (times its value's scale) that the warp has seen, which
# stands between 2^7 and 2^15: half of f16's least step, 2^-25, or that of a second term 2^11 times as large, 2^-36.
WEIGHT_FLOOR = {BF16: 2.0 ** -32, FP32: 2.0 ** -43}


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("steps", [0.4, 5.5, 32.5, 2048.5])
@pytest.mark.parametrize("n,copies", [(400, 1300), (20000, 1300)])
def test_decode_flat_tail_behind_large_weights(n, copies, steps, dtype):
    """A few keys with nearly all of the weight, whose values are 0 in half of the
    dims, and a long tail of equal small weights, each `steps` times f16's least step:
    in those dims the output is the tail's. Enough sequences that a warp walks the
    tail behind a large weight."""
    d, tail = 64, math.log(2.0 ** 7 / (steps * 2.0 ** -24))
    g = torch.Generator().manual_seed(92)
    kcode = torch.zeros(n, 1, d).to(f8.E4M3)
    kcode[:, :, 0] = torch.ones(n, 1).to(f8.E4M3)
    vcode = (1 + torch.rand(n, 1, d, generator=g)).to(f8.E4M3)
    ks, vs = torch.zeros(n, 1), torch.ones(n, 1)
    large = torch.arange(0, 256, 32)  # one for each warp of a CTA
    ks[large] = tail
    vcode[large, :, 32:] = torch.zeros(8, 1, 32).to(f8.E4M3)
    q = torch.zeros(1, 1, d)
    q[..., 0] = 1.0
    # f8.decode's bound but for what is below the weights' least steps: that is in proportion to the tail's own values
    out, lse, _, ltol = f8.decode(q.to(dtype), [kcode], [vcode], [ks], [vs], 1.0, dtype)
    x = ks[:, 0].double()
    p = torch.exp(x - lse[0, 0])
    v = vcode[:, 0].double()
    es = ((d + 4) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22) * tail
    ep = 2 * es + 2.0 ** -21 + 2.0 ** -22 * (tail / math.log(2) + 16)
    tol = fp.U[dtype] * out[0, 0].abs() + (p[:, None] * v).sum(0) * (f8.U_W[dtype] + ep + n * 2.0 ** -23)
    tol = tol + WEIGHT_FLOOR[dtype] * p.max() * v.sum(0)
    kc, vc, ksp, vsp, table = f8.paged([kcode], [vcode], [ks], [vs], 64, g)
    kv = torch.full((copies,), n, dtype=torch.int32)
    args = [x.to(DEV) for x in (q.to(dtype).repeat(copies, 1, 1), kc, vc, ksp, vsp, table.repeat(copies, 1), kv)]
    lse_got = torch.empty(copies, 1, device=DEV)
    got = msa.msa_full_attn_decode_fp8(*args, scale=1.0, lse=lse_got)
    fp.assert_within(got, out.expand(copies, 1, d), tol.expand(copies, 1, d), "out")
    fp.assert_within(lse_got, lse.expand(copies, 1), ltol.expand(copies, 1), "lse")


def test_decode_small_query_elements():
    """fp32 queries, one element 2^28 times the others, where all keys are 0: the
    others keep 22 bits (2^-50 of the largest)."""
    g = torch.Generator().manual_seed(93)
    for d in (64, 128):
        q = torch.randn(2, 8, d, generator=g)
        q[..., 7] = 2.0 ** 28
        (ck, cv, sk, sv), _ = _cache([40, 300], 2, d, 16, g)
        for x in ck:
            x.view(torch.uint8)[..., 7] = 0
        check_parts(q, (ck, cv, sk, sv), FP32, d ** -0.5)


def to_bf16_once(x):
    """64-bit values rounded to bf16, to nearest even, once (a cast goes by way of fp32)."""
    bits = x.view(torch.int64)
    y = (bits + (1 << 44) - 1 + ((bits >> 45) & 1)) & ~((1 << 45) - 1)
    y = y.view(torch.float64)
    least = 2.0 ** -133
    y = torch.where(x.abs() < 2.0 ** -126, torch.round(x / least) * least, y)
    y = torch.where(y.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(y, math.inf), y), y)
    assert torch.equal(y.float().to(BF16).double()[y.isfinite()], y[y.isfinite()])
    return y.float().to(BF16)


def _read_back(codes, scale, dtype):
    """Packed codes [T, Hkv, d] and scales [T, Hkv] as one sequence's cache, read whole."""
    T, Hkv, d = codes.shape
    g = torch.Generator().manual_seed(94)
    kc, vc, ks, vs, table = f8.paged([codes], [codes], [scale], [scale.flip(0)], 16, g)
    cu, kv = torch.tensor([0, T], dtype=torch.int32), torch.tensor([T], dtype=torch.int32)
    k, v = msa.msa_paged_read_fp8(*[x.to(DEV) for x in (kc, vc, ks, vs, table, cu, kv)], T, dtype=dtype)
    for got, s in ((k, scale), (v, scale.flip(0))):
        exact = codes.double() * s.double()[..., None]  # 28 bits
        want = to_bf16_once(exact) if dtype == BF16 else exact.float()
        got = got.cpu()
        assert torch.equal(got.isnan(), want.isnan())
        same = (got == want) | got.isnan()
        assert same.all(), f"{int((~same).sum())} of {same.numel()} are rounded twice"


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_read_rounds_once(dtype):
    """Scales that are no powers of two: 28 bits of code times scale are rounded to
    the output's type at once. Here code 9/8 times scale lies next to the middle of two
    bf16 numbers, closer to it than fp32 can tell."""
    near = []
    for k in range(128, 256):  # (2 k + 1) 2^-8: between k and k + 1
        for e in (1, 2, 3, -1, -2, -3):
            if ((2 * k + 1) * 2 ** 18 + e) % 9 == 0:
                near.append(((2 * k + 1) * 2 ** 18 + e) // 9 * 2.0 ** -23)  # 9 scale = middle + e 2^-26
    scale = torch.tensor(near, dtype=torch.float64)
    assert len(near) > 60 and torch.equal(scale.float().double(), scale)
    scale = scale.float()[:, None].repeat(1, 2)
    codes = torch.full((len(near), 2, 64), 1.125).to(f8.E4M3)
    codes[:, 1, ::2] = torch.full((len(near), 32), -1.125).to(f8.E4M3)
    for z in (0, -60, 100, -126):
        _read_back(codes, scale * 2.0 ** z, dtype)
    _read_back(codes, -scale, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_read_any_scales(dtype):
    """All codes, with scales over fp32's whole range, subnormal ones, 0, infinity and NaN."""
    g = torch.Generator().manual_seed(95)
    codes = torch.arange(256, dtype=torch.uint8).view(1, 4, 64).repeat(300, 1, 1).view(f8.E4M3)
    bits = torch.randint(-2 ** 31, 2 ** 31, (300, 4), generator=g).to(torch.int32)
    bits[:40] &= 0x007fffff
    scale = bits.view(torch.float32)
    scale[40:44, 0] = torch.tensor([0.0, math.inf, -math.inf, math.nan])
    _read_back(codes, scale, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_heads(dtype):
    """More key/value heads than a reciprocal divides exactly by, more items than warps."""
    check_append([3, 1], [14, 0], 9000, 9000, 64, dtype, 16, 32, False, 96, behind=1)
    check_append([1, 1], [14, 0], 20000, 20000, 64, dtype, 16, 0, False, 97, cu_given=False, with_q=False)
    for heads in ((1024, 1024, 64), (512, 64, 128), (2100, 700, 64), (701, 701, 64)):
        check_decode([40, 1, 130], *heads, dtype, 16, 98)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_rows_without_a_finite_score(d, dtype):
    """Scores that overflow to -inf, or are -inf by an infinite query: NaN where there are no
    others, -inf as the sum's logarithm, also where keys end inside a step."""
    g = torch.Generator().manual_seed(99)
    lens = [40, 300, 5, 64]
    q = (torch.randn(4, 8, d, generator=g).abs() + 1) * 2.0 ** 60
    (ck, cv, sk, sv), _ = _cache(lens, 2, d, 16, g)
    for b, n in ((0, 40), (1, 130)):
        ck[b][:n] = torch.full((n, 2, d), -448.0).to(f8.E4M3)
        sk[b][:n] = 2.0 ** 64  # scores of -2^130 and below
    sk[1][130:] *= 2.0 ** -60
    for b in (2, 3):  # 0 in all dims but the first, where every key is positive
        q[b] = 0.0
        q[b, 1::2, 0] = -math.inf
        ck[b][:, :, 0] = torch.ones(lens[b], 2).to(f8.E4M3)
    q = q.to(dtype)
    kc, vc, ks, vs, table = f8.paged(ck, cv, sk, sv, 16, g)
    kv = torch.tensor(lens, dtype=torch.int32)
    lse = torch.empty(4, 8, device=DEV)
    out = msa.msa_full_attn_decode_fp8(*[x.to(DEV) for x in (q, kc, vc, ks, vs, table, kv)], lse=lse)
    undefined = torch.zeros(4, 8, dtype=torch.bool)
    undefined[0], undefined[2:, 1::2] = True, True
    assert out.cpu()[undefined].isnan().all() and (lse.cpu()[undefined] == -math.inf).all()
    cut = lambda x: [x[1][130:], x[2], x[3]]  # noqa: E731
    q[2:, 1::2] = 0.0
    want = f8.decode(q[1:], cut(ck), cut(cv), cut(sk), cut(sv), d ** -0.5, dtype)
    for w in want:
        w[undefined[1:]] = math.nan
    fp.assert_within(out[1:], want[0], want[2], "out")
    fp.assert_within(lse[1:], want[1], want[3], "lse")
