"""Host-side refusals of the full-attention and paged-cache entry points (no
GPU needed: every call below returns before any launch)."""
import ctypes
import os

import pytest
import torch

import block_sparse_long_select_gb300 as msa
from block_sparse_long_select_gb300 import _lib

P = ctypes.c_void_p(0x1000)  # never dereferenced
BF16, FP32 = msa.MSA_BF16, msa.MSA_FP32
OPS = (msa.MSA_OP_FULL_PREFILL, msa.MSA_OP_FULL_BACKWARD, msa.MSA_OP_FULL_DECODE, msa.MSA_OP_PAGED_APPEND)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.lib_path()):
        msa.build()
    return msa.load_library()


def append(lib, q=P, k=P, rope=P, cu=P, kv=P, table=P, B=2, T=5, Hq=8, Hkv=2, d=128, rot=64, il=0, max_pos=100,
           pages=4, page=16, maxp=2, dtype=BF16, q_out=P, kc=P, ws=P, nb=1 << 20):
    return lib.msa_paged_append(q, k, P, rope, cu, kv, table, B, T, Hq, Hkv, d, rot, il, max_pos, pages, page, maxp,
                                dtype, q_out, kc, P, ws, nb, None)


def decode(lib, q=P, kc=P, table=P, kv=P, B=2, Hq=8, Hkv=2, d=128, pages=4, page=16, maxp=2, dtype=BF16, out=P, ws=P,
           nb=1 << 30):
    return lib.msa_full_attn_decode(q, kc, P, table, kv, B, Hq, Hkv, d, pages, page, maxp, 0.0, dtype, out, None, ws,
                                    nb, None)


def prefill(lib, q=P, k=P, cu_q=P, cu_k=P, B=2, Tq=5, Tk=5, Hq=8, Hkv=2, d=128, dtype=BF16, out=P, ws=P, nb=1 << 30):
    return lib.msa_full_attn_prefill(q, k, P, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, 0.0, dtype, out, None, ws, nb, None)


def prefill_paged(lib, q=P, kc=P, table=P, cu_q=P, kv=P, B=2, Tq=5, Hq=8, Hkv=2, d=128, pages=4, page=16, maxp=2,
                  dtype=BF16, out=P, ws=P, nb=1 << 30):
    return lib.msa_full_attn_prefill_paged(q, kc, P, table, cu_q, kv, B, Tq, Hq, Hkv, d, pages, page, maxp, 0.0, dtype,
                                           out, None, ws, nb, None)


def backward(lib, q=P, k=P, lse=P, cu_q=P, B=2, Tq=5, Tk=5, Hq=8, Hkv=2, d=128, dtype=BF16, dq=P, dk=P, ws=P,
             nb=1 << 30):
    return lib.msa_full_attn_backward(q, k, P, P, P, lse, cu_q, P, B, Tq, Tk, Hq, Hkv, d, 0.0, dtype, dq, dk, P, ws,
                                      nb, None)


ALL = (append, decode, prefill, prefill_paged, backward)


@pytest.mark.parametrize("call", ALL)
def test_refusals_shared(lib, call):
    assert call(lib, Hq=6, Hkv=4) == 1          # Hq not a multiple of Hkv
    assert call(lib, Hkv=0) == 1
    assert call(lib, B=-1) == 1
    assert call(lib, dtype=2) == 1
    assert call(lib, d=96) == 2
    assert call(lib, Hq=65, Hkv=1) == 2         # beyond the built head ratios
    assert call(lib, ws=None) == 3
    assert call(lib, ws=ctypes.c_void_p(0x1010)) == 3
    assert call(lib, nb=128) == 3
    big = {"B": 1 << 28} if call is decode else {"T": 1 << 28} if call is append else {"Tq": 1 << 28}
    assert call(lib, **big) == 2                # rows x heads past 31 bits


@pytest.mark.parametrize("call", ALL)
def test_refuses_too_many_heads(lib, call):
    one = {"B": 1} if call is decode else {"B": 1, "T": 1} if call is append else {"B": 1, "Tq": 1}
    assert call(lib, Hq=(1 << 16) + 64, Hkv=(1 << 10) + 1, **one) == 2
    assert call(lib, Hq=1 << 16, Hkv=1 << 10, ws=None, **one) == 3


@pytest.mark.parametrize("call", (append, decode, prefill_paged))
def test_refusals_pages(lib, call):
    assert call(lib, page=0) == 1
    assert call(lib, page=24) == 2
    assert call(lib, page=256) == 2
    assert call(lib, pages=0) == 1
    assert call(lib, maxp=0) == 1
    assert call(lib, maxp=1 << 28) == 2         # max_pages * page_size past 31 bits
    assert call(lib, table=None) == 1
    assert call(lib, kc=None) == 1
    assert call(lib, kv=None) == 1


def test_refusals_each(lib):
    odd = ctypes.c_void_p(0x1008)               # not 16-byte aligned
    assert append(lib, rot=136) == 1            # more than d
    assert append(lib, rot=24) == 2             # not a multiple of 16
    assert append(lib, il=2) == 1
    assert append(lib, rope=None) == 1          # rot > 0 needs the table
    assert append(lib, max_pos=0) == 1
    assert append(lib, q_out=None) == 1         # q without q_out
    assert append(lib, q=None) == 1             # q_out without q
    assert append(lib, cu=None) == 1            # no offsets, but T != B
    assert append(lib, k=odd) == 1 and append(lib, rope=odd) == 1 and append(lib, kc=odd) == 1
    assert decode(lib, q=odd) == 1 and decode(lib, out=None) == 1 and decode(lib, kc=odd) == 1
    assert prefill(lib, k=None) == 1 and prefill(lib, cu_k=None) == 1 and prefill(lib, out=odd) == 1
    assert prefill(lib, Tk=-1) == 1
    assert prefill_paged(lib, cu_q=None) == 1 and prefill_paged(lib, q=odd) == 1
    assert backward(lib, lse=None) == 1 and backward(lib, dq=None) == 1 and backward(lib, dk=None) == 1
    assert backward(lib, k=odd) == 1 and backward(lib, cu_q=None) == 1


def test_empty_calls(lib):
    """No sequence or no row: nothing read, nothing enqueued, the rest still checked."""
    N = None
    assert append(lib, q=N, k=N, cu=N, kv=N, table=N, B=0, T=0, q_out=N, kc=N, ws=N, nb=0) == 0
    assert append(lib, T=0, ws=N, nb=0) == 0 and append(lib, T=0, d=96) == 2
    assert decode(lib, q=N, kc=N, table=N, kv=N, B=0, out=N, ws=N, nb=0) == 0 and decode(lib, B=0, page=8) == 2
    assert prefill(lib, q=N, k=N, cu_q=N, cu_k=N, B=0, out=N, ws=N, nb=0) == 0
    assert prefill(lib, Tq=0, ws=N, nb=0) == 0 and prefill(lib, Tq=0, d=32) == 2
    assert prefill_paged(lib, Tq=0, ws=N, nb=0) == 0
    assert backward(lib, q=N, k=N, lse=N, cu_q=N, B=2, Tq=0, Tk=0, dq=N, dk=N, ws=N, nb=0) == 0
    assert backward(lib, Tq=0, dk=N) == 1       # keys without rows get zeros: dk and dv must be given


def test_workspace_sizes(lib):
    size = lambda op, B=2, Nq=100, Nk=100, G=2, Hq=8, d=128, dt=BF16: msa.msa_workspace_size(  # noqa: E731
        op, B, Nq, Nk, G, Hq, d, 0, 0, 0, dt)
    for op in OPS:
        for dt in (BF16, FP32):
            assert size(op, dt=dt) >= 256 and size(op, dt=dt) % 256 == 0
            assert size(op, B=0, dt=dt) == 256
        assert size(op, d=96) == 0 and size(op, Hq=9) == 0 and size(op, B=-1) == 0 and size(op, dt=5) == 0
    assert size(msa.MSA_OP_FULL_PREFILL, Nq=0) == 256
    for op in (6, 7, 12):
        assert size(op) == 0


def test_binding_refuses_wrong_tensors():
    """The wrappers check before any pointer is taken: CPU tensors, shapes, dtypes."""
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.msa_full_attn_prefill(q, k, k, cu, cu)
    with pytest.raises(ValueError):
        msa.msa_full_attn_backward(q, k, k, q, q, torch.zeros(4, 8), cu, cu)
    with pytest.raises(ValueError):
        msa.msa_full_attn_decode(q, k[None], k[None], torch.zeros(4, 1, dtype=torch.int32), cu)
    with pytest.raises(ValueError):
        msa.msa_paged_append(q, k, k, None, cu, cu, torch.zeros(1, 1, dtype=torch.int32), k[None], k[None])
