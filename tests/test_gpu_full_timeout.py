"""The bounded-wait timeout path of full attention on the GPU, exercised without
a fault: with the library's test hook on (msa_debug_inject_timeout), every
second CTA waits once, behind its first copies, on a barrier that nothing
completes. The wait runs out after about a millisecond, the CTA drains what it
has in flight and returns; the others finish and leave their arrivals (and the
queue its count) in the workspace. Once the status is read the same workspace
serves every operation again."""
import pytest
import torch

import block_sparse_long_select_gb300 as msa
import full_plain as fp
from test_gpu_full_attn import BF16, DEV, _decode_case, make

pytestmark = pytest.mark.gpu
MSA_ERR_TIMEOUT = 5


@pytest.fixture(autouse=True)
def _hook_off(cuda_ok):
    yield
    msa.msa_debug_inject_timeout(False)


def _timed_out(call, ws):
    assert msa.msa_debug_inject_timeout(True) is False
    call()
    st = msa.msa_read_status(ws)  # synchronises: the kernels returned
    msa.msa_debug_inject_timeout(False)
    assert st == MSA_ERR_TIMEOUT and msa.msa_read_status(ws) == 0


# handed out whole (by slots, and up to 32 sequences by places), split and joined, one short item
SPANS = {
    "slots": [((37 * b) % 260, (37 * b) % 260) for b in range(150)],
    "places": [(300 + 40 * b, 300 + 40 * b) for b in range(20)],
    "split": [(40, 6000), (100, 3000)],
    "one": [(5, 5)],
}


@pytest.mark.parametrize("heads", [(16, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("name", sorted(SPANS))
def test_prefill_timeout_then_recovers(name, heads):
    Hq, Hkv, d = heads
    q, k, v, cu_q, cu_k, rows, ks, vs, _ = make(SPANS[name], Hq, Hkv, d, BF16, 1)
    want = fp.prefill(q, ks, vs, rows, d ** -0.5, BF16)
    qd, kc, vc, table, kv, want_d = _decode_case([900, 1, 5000], Hq, Hkv, d, BF16, 64, 2)
    ws = msa.workspace(max(
        msa.msa_workspace_size(msa.MSA_OP_FULL_PREFILL, len(rows), q.shape[0], k.shape[0], Hkv, Hq, d, 0, 0, 0, 0),
        msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 3, 1, table.shape[1] * 64, Hkv, Hq, d, 0, 0, 0, 0)), DEV)
    dev = [x.to(DEV) for x in (q, k, v, cu_q, cu_k)]
    dec = [x.to(DEV) for x in (qd, kc, vc, table, kv)]
    for _ in range(2):
        _timed_out(lambda: msa.msa_full_attn_prefill(*dev, ws=ws), ws)
        fp.assert_within(msa.msa_full_attn_decode(*dec, ws=ws), want_d[0], want_d[2], "decode")
        for _ in range(2):
            out = msa.msa_full_attn_prefill(*dev, ws=ws)
            assert msa.msa_read_status(ws) == 0
            fp.assert_within(out, want[0], want[2], "out")


@pytest.mark.parametrize("spans", [[(700, 700), (90, 600)], [(n, n) for n in (5, 130, 77, 300)] * 12])
def test_backward_timeout_then_recovers(spans):
    """One cluster per key tile, and a CTA each."""
    Hq, Hkv, d = 4, 2, 64
    q, k, v, cu_q, cu_k, rows, ks, vs, g = make(spans, Hq, Hkv, d, BF16, 3)
    fwd = fp.prefill(q, ks, vs, rows, d ** -0.5, BF16)
    dout = torch.randn(q.shape, generator=g).to(BF16)
    ws = msa.workspace(msa.msa_workspace_size(msa.MSA_OP_FULL_BACKWARD, len(rows), q.shape[0], k.shape[0], Hkv, Hq, d,
                                              0, 0, 0, 0), DEV)
    args = [x.to(DEV) for x in (q, k, v, fwd[0].to(BF16), dout, fwd[1].float(), cu_q, cu_k)]
    first = msa.msa_full_attn_backward(*args, ws=ws)
    for _ in range(2):
        _timed_out(lambda: msa.msa_full_attn_backward(*args, ws=ws), ws)
        again = msa.msa_full_attn_backward(*args, ws=ws)
        assert msa.msa_read_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(first, again))
