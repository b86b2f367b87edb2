"""GPU parity of decode over shared prefixes against the plain 64-bit form of
each sequence's whole attention, within the bounds derived in full_plain.py."""
import math

import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, FP32 = torch.bfloat16, torch.float32
HEADS = [(4, 4, 64), (8, 2, 64), (8, 2, 128), (6, 2, 128), (16, 1, 128), (32, 1, 64), (10, 2, 128), (64, 1, 128),
         (9, 3, 64), (48, 2, 64)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def make(groups, Hq, Hkv, d, dtype, page, seed=0, before=0, scale=1.0):
    """groups: (prefix keys, [own keys or None for a padded entry, ...]) each;
    before: sequences without a group ahead of them, given by their keys."""
    g = torch.Generator().manual_seed(seed)
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(dtype)  # noqa: E731
    before = before or []
    ks, vs, need, cu, pre = [r(n, Hkv) for n in before], [r(n, Hkv) for n in before], [], [len(before)], []
    share = [0] * len(before)
    for n, own in groups:
        pk, pv = r(n, Hkv), r(n, Hkv)
        for x in own:
            ks.append(torch.cat([pk, r(x, Hkv)]) if x is not None else r(0, Hkv))
            vs.append(torch.cat([pv, r(x, Hkv)]) if x is not None else r(0, Hkv))
            share.append(n // page if x is not None else 0)
        cu.append(cu[-1] + len(own))
        pre.append(n)
    q = r(len(ks), Hq) * scale
    # every sequence laid out whole; then those behind the first of their group take its pages,
    # though their own table entries for them are no pages at all
    kc, vc, table = fp.paged(ks, vs, page, g)
    lead, lens = {}, [x.shape[0] for x in ks]
    for x, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        for b in range(a, e):
            if lens[b] == 0:
                continue
            if x in lead:
                kc[table[b, :share[b]].long()] = math.nan  # nobody's any more
                vc[table[b, :share[b]].long()] = math.nan
                table[b, :share[b]] = 1 << 30
            lead.setdefault(x, b)
    want = fp.prefill(q, ks, vs, [(b, 1 if lens[b] else 0) for b in range(len(ks))], d ** -0.5, dtype)
    for b, n in enumerate(lens):
        if n == 0:
            for w, fill in zip(want, (0.0, -math.inf, 0.0, 0.0)):
                w[b] = fill
    return q, kc, vc, table, i32(lens), i32(cu), i32(pre), want


def workspace(B, P, table, page, Hkv, Hq, d, dtype):
    return msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_SHARED, B, P, table.shape[1] * page, Hkv, Hq, d,
                                                0, 0, 0, msa.MSA_BF16 if dtype == BF16 else msa.MSA_FP32), DEV)


def check(groups, Hq, Hkv, d, dtype, page, seed=0, before=None, repeat=2):
    *args, want = make(groups, Hq, Hkv, d, dtype, page, seed, before)
    ws = workspace(args[0].shape[0], len(groups), args[3], page, Hkv, Hq, d, dtype)
    args = [x.to(DEV) for x in args]
    first = None
    for _ in range(repeat):  # the workspace serves call after call
        lse = torch.full(args[0].shape[:2], 7.0, device=DEV)
        out = msa.msa_full_attn_decode_shared(*args, lse=lse, ws=ws)
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")
        fp.assert_within(lse, want[1], want[3], "lse")
        assert first is None or torch.equal(first, out)
        first = out
    return out


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_shapes(page, dtype):
    P = page
    check([(P, [1])], 8, 2, 64, dtype, page, 1)                                  # one sequence, one page
    check([(4 * P, [1, 15, 16, 17, 0, 130])], 8, 2, 128, dtype, page, 2)          # nothing of its own, too
    check([(2 * P, [3, 9]), (0, [5, 40]), (9 * P, [0, 0, 7])], 8, 2, 128, dtype, page, 3, before=[20, 0, 300])
    check([(0, []), (3 * P, [None, 4, None, 30]), (P, [None, None]), (P, [])], 8, 2, 64, dtype, page, 4, before=[1])
    check([(640, [2, 3])], 4, 4, 64, dtype, page, 5)                              # whole key tiles


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", HEADS)
def test_heads(heads, dtype):
    check([(400, [5, 1, 64]), (144, [17])], *heads, dtype, 16, 6, before=[33])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_groups(dtype):
    """Groups of more sequences than a row tile, than two, than an item."""
    for n in (31, 32, 33, 63, 64, 65, 150):
        check([(272, [(3 * x) % 40 for x in range(n)]), (48, [1, 2])], 8, 2, 64, dtype, 16, n)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_long_prefixes(dtype):
    """Items that lie in several CTAs, with an odd and an even number of key tiles."""
    check([(5008, [1, 60])], 8, 1, 128, dtype, 16, 7)
    check([(4480, [4] * 40)], 8, 2, 64, dtype, 64, 8)
    check([(4224, [700, 3000]), (1920, [5])], 4, 2, 128, dtype, 128, 9)


def test_many_groups():
    """More groups than each CTA looks at by itself; many short sequences."""
    check([(16, [1 + x % 3, 2]) for x in range(300)], 4, 2, 64, BF16, 16, 10)
    check([(32, [(x * y) % 50 for y in range(7)]) for x in range(100)], 4, 2, 64, BF16, 16, 11)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_peaked_scores(dtype):
    """Large queries: the maximum lies with the prefix for some rows, with own keys for others."""
    *args, _ = make([(700 // 16 * 16, [300, 1, 90]), (16, [40])], 8, 2, 64, dtype, 16, 12)
    q, kc, vc, table, kv, cu, pre = args
    q = (q.float() * 8).to(dtype)
    full = table.clone()
    full[1, :43], full[2, :43] = table[0, :43], table[0, :43]
    ks, vs = ([x[full[b, :-(-int(kv[b]) // 16)].long()].flatten(0, 1)[:int(kv[b])] for b in range(4)] for x in (kc, vc))
    want = fp.prefill(q, ks, vs, [(b, 1) for b in range(4)], 0.125, dtype)
    lse = torch.empty(4, 8, device=DEV)
    out = msa.msa_full_attn_decode_shared(*[x.to(DEV) for x in (q, kc, vc, table, kv, cu, pre)], lse=lse)
    fp.assert_within(out, want[0], want[2], "out")
    fp.assert_within(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_without_groups(dtype):
    """P = 0 is msa_full_attn_decode, bit for bit; so are sequences of no group, but for the joins."""
    q, kc, vc, table, kv, _, _, want = make([], 8, 2, 64, dtype, 16, 13, before=[40, 1, 500])
    a = [x.to(DEV) for x in (q, kc, vc, table, kv)]
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    out = msa.msa_full_attn_decode_shared(*a, torch.zeros(1, dtype=torch.int32, device=DEV), none)
    assert torch.equal(out, msa.msa_full_attn_decode(*a))
    fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bad_prefixes_lengths_and_pages(dtype):
    groups = [(32, [5, 9]), (48, [7, 60]), (16, [3]), (32, [4, 8]), (64, [2, 2])]
    q, kc, vc, table, kv, cu, pre, want = make(groups, 8, 2, 64, dtype, 16, 14, before=[30])
    pre[1] = 40                   # not a multiple of the page
    pre[2] = table.shape[1] * 16 + 16
    table[6, 1] = kc.shape[0]     # group 3's prefix, in its leader's row
    kv[8] = 20                    # group 4: sequence 8 has fewer keys than the prefix; 9 leads now
    table[9, :4] = table[8, :4]
    table[8, 0] = -1              # not read any more
    bad, good = [3, 4, 5, 6, 7, 8], [0, 1, 2, 9]
    ws = workspace(10, 5, table, 16, 2, 8, 64, dtype)
    lse = torch.empty(10, 8, device=DEV)
    args = [x.to(DEV) for x in (q, kc, vc, table, kv, cu, pre)]
    out = msa.msa_full_attn_decode_shared(*args, lse=lse, ws=ws)
    assert msa.msa_read_status(ws) == 6 and msa.msa_read_status(ws) == 0
    assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
    fp.assert_within(out[good], want[0][good], want[2][good], "out")
    kv2 = args[4].clone()
    kv2[0], kv2[1] = -1, table.shape[1] * 16 + 1
    out = msa.msa_full_attn_decode_shared(*args[:4], kv2, *args[5:], lse=lse, ws=ws)
    assert msa.msa_read_status(ws) == 6
    assert (out[[0, 1]] == 0).all()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_out_of_order(dtype, many):
    """Whose keys are whose is not known: reported, every output zero."""
    groups = [(16, [2])] * (300 if many else 3)
    *args, want = make(groups, 4, 2, 64, dtype, 16, 15, before=[5])
    n = len(groups) + 1
    ws = workspace(n, len(groups), args[3], 16, 2, 4, 64, dtype)
    args = [x.to(DEV) for x in args]
    for at, to in ((0, -1), (1, n + 1), (len(groups), 0)):
        cu = args[5].clone()
        cu[at] = to
        lse = torch.full((n, 4), 7.0, device=DEV)
        out = msa.msa_full_attn_decode_shared(*args[:5], cu, args[6], lse=lse, ws=ws)
        assert msa.msa_read_status(ws) == 6
        assert (out == 0).all() and (lse == -math.inf).all()
    out = msa.msa_full_attn_decode_shared(*args, ws=ws)
    assert msa.msa_read_status(ws) == 0
    fp.assert_within(out, want[0], want[2], "out")


def test_infinite_scores_and_nan_elsewhere():
    """Prefix scores of -inf weigh nothing beside own keys; all of them -inf: 0 / 0, as the formula."""
    *args, _ = make([(160, [3, 0])], 4, 2, 64, BF16, 16, 16)
    q, kc, vc, table, kv, cu, pre = args
    q = torch.ones_like(q)
    pages = table[0, :10].long()
    kc[pages] = -math.inf
    out = msa.msa_full_attn_decode_shared(*[x.to(DEV) for x in (q, kc, vc, table, kv, cu, pre)])
    own = [x[int(table[0, 10])][:3] for x in (kc, vc)]
    want = fp.prefill(q[:1], [own[0]], [own[1]], [(0, 1)], 0.125, BF16)
    fp.assert_within(out[:1], want[0], want[2], "out")
    assert out[1].isnan().all()


def _steps(captured):
    """A prompt enters the cache once; its samples share the pages, append and attend step by step."""
    g = torch.Generator().manual_seed(17)
    B, Hq, Hkv, d, page, steps, pre, tail = 5, 8, 2, 64, 16, 5, 96, 7  # the prompt's last 7 keys are not a whole page
    r = lambda n, h: torch.randn(n, h, d, generator=g).to(BF16)  # noqa: E731
    pk, pv = r(pre + tail, Hkv), r(pre + tail, Hkv)
    rope = fp.rope_table(pre + tail + steps, d).to(DEV)
    full = pre // page
    table = torch.full((B, full + 1), -1, dtype=torch.int32)
    order = torch.randperm(full + B, generator=g).to(torch.int32)
    table[:, :full] = order[:full]
    table[:, full] = order[full:]
    table = table.to(DEV)
    kc, vc = (torch.full((full + B, page, Hkv, d), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    cu1, kv1 = i32([0, pre + tail]).to(DEV), i32([pre + tail]).to(DEV)
    msa.msa_paged_append(None, pk.to(DEV), pv.to(DEV), rope, cu1, kv1, table[:1].contiguous(), kc, vc)
    for x in (kc, vc):  # a partly filled page cannot be shared: it is copied
        x[table[1:, full].long()] = x[table[0, full].long()].clone()
    kv = torch.full((B,), pre + tail, dtype=torch.int32, device=DEV)
    cu, plen = i32([0, B]).to(DEV), i32([pre]).to(DEV)
    new = [[r(B, h).to(DEV) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    q, k, v = (x.clone() for x in new[0])
    qo, out = torch.empty_like(q), torch.empty_like(q)
    ws = workspace(B, 1, table, page, Hkv, Hq, d, BF16)

    def step():
        kv.add_(1)
        msa.msa_paged_append(q, k, v, rope, None, kv, table, kc, vc, q_out=qo, ws=ws)
        msa.msa_full_attn_decode_shared(qo, kc, vc, table, kv, cu, plen, out=out, ws=ws)

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
        for dst, src in zip((q, k, v), new[i]):
            dst.copy_(src)
        graphs[i % 2].replay() if captured else step()
        lens = kv.tolist()
        ks, vs = ([x[table[b].long()].flatten(0, 1)[:lens[b]].cpu() for b in range(B)] for x in (kc, vc))
        want = fp.prefill(qo.cpu(), ks, vs, [(b, 1) for b in range(B)], d ** -0.5, BF16)
        fp.assert_within(out, want[0], want[2], f"step {i}")
    assert msa.msa_read_status(ws) == 0 and lens == [pre + tail + steps] * B


def test_serving_run():
    _steps(False)


def test_serving_run_captured():
    _steps(True)


def test_other_stream_and_workspace_of_another_operation():
    *args, want = make([(320, [5, 70, 1]), (64, [9])], 8, 2, 128, BF16, 16, 18)
    args = [x.to(DEV) for x in args]
    ws = workspace(4, 2, args[3], 16, 2, 8, 128, BF16)
    ws = msa.workspace(max(ws.nbytes, 1 << 26), DEV)
    plain = args[3].clone()  # the whole tables, for calls without groups
    plain[1, :20], plain[2, :20] = plain[0, :20], plain[0, :20]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        out = msa.msa_full_attn_decode_shared(*args, ws=ws, stream=s)
        other = msa.msa_full_attn_decode(*args[:3], plain, args[4], ws=ws, stream=s)
        msa.msa_full_attn_prefill_paged(args[0], *args[1:3], plain, torch.arange(5, dtype=torch.int32, device=DEV), args[4],
                                        ws=ws, stream=s)
        s.synchronize()
        fp.assert_within(out, want[0], want[2], "out")
        fp.assert_within(other, want[0], want[2], "other")
    assert msa.msa_read_status(ws) == 0


def test_timeout_then_recovers():
    """Every second CTA of the prefixes' grid lets a wait run out: reported, nothing hangs, the next call is right."""
    *args, want = make([(2048, [5, 70, 1])], 8, 2, 128, BF16, 16, 19)
    args = [x.to(DEV) for x in args]
    ws = workspace(3, 1, args[3], 16, 2, 8, 128, BF16)
    msa.msa_debug_inject_timeout(True)
    try:
        msa.msa_full_attn_decode_shared(*args, ws=ws)
        assert msa.msa_read_status(ws) == 5
    finally:
        msa.msa_debug_inject_timeout(False)
    for _ in range(2):
        out = msa.msa_full_attn_decode_shared(*args, ws=ws)
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("own", [1, 3, 40])
def test_padded_batches(own):
    """Mostly padded groups, and own keys that a prefix's last key tile would outnumber."""
    check([(16, [None] * 40 + [own] * 3), (400, [own] + [None] * 70), (48, [own] * 90)], 8, 2, 64, BF16, 16, 20)
    check([(4096, [None] * 30 + [own, 2000])], 4, 2, 128, BF16, 64, 21)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_small_groups(dtype):
    """Groups too small or prefixes too short to be shared: walked by each sequence, by the leader's table."""
    for n in (1, 2, 3, 4, 9):
        for pre in (16, 128, 256, 1040):
            check([(pre, [x % 3 for x in range(n)]), (32, [None, 0, 5]), (pre, [7])], 8, 2, 64, dtype, 16, n + pre, repeat=1)
    check([(256, [100, 30, None, 5])] * 40, 4, 2, 128, dtype, 32, 30)


def test_thousands_of_sequences():
    """More sequences and groups than the plan's threads."""
    groups = [(32 if x % 3 else 512, [(x + y) % 5 for y in range(1 + x % 4)]) for x in range(1100)]
    check(groups, 2, 1, 64, BF16, 32, 31, before=[3, 0, 70])


def test_two_calls_at_once():
    """On two streams, a workspace each; and the same two as graphs replayed side by side."""
    calls = []
    for seed in (32, 33):
        *args, want = make([(1040, [5, 70, 1] * 8), (64, [9, 300])], 8, 2, 128, BF16, 16, seed)
        ws = workspace(26, 2, args[3], 16, 2, 8, 128, BF16)
        calls.append(([x.to(DEV) for x in args], want, ws, torch.empty(26, 8, 128, dtype=BF16, device=DEV),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for i in range(12):
        args, _, ws, out, s = calls[i % 2]
        msa.msa_full_attn_decode_shared(*args, out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    for args, want, ws, out, s in calls:
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "out")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                msa.msa_full_attn_decode_shared(*args, out=out, ws=ws)
        graphs.append(graph)
        out.zero_()
    torch.cuda.synchronize()
    for i in range(12):
        with torch.cuda.stream(calls[i % 2][4]):
            graphs[i % 2].replay()
    torch.cuda.synchronize()
    for args, want, ws, out, s in calls:
        assert msa.msa_read_status(ws) == 0
        fp.assert_within(out, want[0], want[2], "replayed")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_caches_past_32_bits(dtype):
    """Prefix and own pages beyond 2^32 bytes."""
    *args, want = make([(2048, [5, 300, 1] * 3)], 8, 8, 128, dtype, 128, 34)
    q, kc, vc, table, kv, cu, pre = [x.to(DEV) for x in args]
    pages = kc.shape[0] + (5 << 30) // (128 * 8 * 128 * dtype.itemsize)
    there = lambda x: torch.cat([torch.empty(pages - x.shape[0], *x.shape[1:], dtype=dtype, device=DEV), x])  # noqa: E731
    table = torch.where((table >= 0) & (table < kc.shape[0]), table + (pages - kc.shape[0]), table).to(torch.int32)
    out = msa.msa_full_attn_decode_shared(q, there(kc), there(vc), table, kv, cu, pre)
    fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128), (5, 1, 64)])
def test_infinite_values(heads, dtype):
    """Values of the prefix and of own keys that are infinite make their elements so, as
    msa_full_attn_decode's, and leave the others alone: few rows and many, whose joins differ."""
    for groups in ([(1040, [5, 0, 300])], [(272, [9, 1])] * 30, [(272, [9, 1, 40] * 40)], [(16, [700])]):
        *args, _ = make(groups, *heads, dtype, 16, 40)
        q, kc, vc, table, kv, cu, pre = args
        full = table.clone()  # every sequence's pages
        for x, (n, _) in enumerate(groups):
            a, e = int(cu[x]), int(cu[x + 1])
            full[a:e, :n // 16] = table[a, :n // 16]
            vc[table[a, n // 16 - 1].long(), 15, :, 3] = math.inf  # the prefix's last key
            for b in range(a, e, 2):
                last = int(kv[b]) - 1
                if last >= n:
                    vc[table[b, last // 16].long(), last % 16, :, 5] = -math.inf
        B = q.shape[0]
        ks, vs = ([x[full[b, :-(-int(kv[b]) // 16)].long()].flatten(0, 1)[:int(kv[b])] for b in range(B)] for x in (kc, vc))
        want = fp.prefill(q, ks, vs, [(b, 1) for b in range(B)], heads[2] ** -0.5, dtype)
        assert want[0].isinf().any() and not want[0].isnan().any()
        out = msa.msa_full_attn_decode_shared(*[x.to(DEV) for x in args])
        fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads", [(1024, 1024, 64), (512, 64, 128), (2100, 700, 64)])
def test_many_heads(heads, dtype):
    """More items of one sequence than there are CTAs or warps."""
    check([(144, [5, 1, 64]), (32, [17, None])], *heads, dtype, 16, 41, before=[33])
