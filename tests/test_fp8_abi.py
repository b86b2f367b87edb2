"""Host-side refusals of the 8-bit caches' entry points (no GPU needed: every
call below returns before any launch), and of their bindings."""
import ctypes
import os

import pytest
import torch

import block_sparse_long_select_gb300 as msa
from block_sparse_long_select_gb300 import _lib

P = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned
BF16, FP32 = msa.MSA_BF16, msa.MSA_FP32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.lib_path()):
        msa.build()
    return msa.load_library()


def append(lib, q=P, k=P, rope=P, cu=P, kv=P, table=P, B=2, T=5, Hq=8, Hkv=2, d=128, rot=64, il=0, max_pos=100,
           pages=4, page=16, maxp=2, dtype=BF16, out=P, kc=P, ks=P, vs=P, ws=P, nb=1 << 20):
    return lib.msa_paged_append_fp8(q, k, P, rope, cu, kv, table, B, T, Hq, Hkv, d, rot, il, max_pos, pages, page, maxp,
                                    dtype, out, kc, P, ks, vs, ws, nb, None)


def read(lib, kc=P, ks=P, vs=P, cu=P, kv=P, table=P, B=2, T=5, Hkv=2, d=128, pages=4, page=16, maxp=2, dtype=BF16,
         out=P, ws=P, nb=1 << 20):
    return lib.msa_paged_read_fp8(kc, P, ks, vs, cu, kv, table, B, T, Hkv, d, pages, page, maxp, dtype, out, P, ws, nb,
                                  None)


def decode(lib, q=P, kc=P, ks=P, vs=P, table=P, kv=P, B=2, Hq=8, Hkv=2, d=128, pages=4, page=16, maxp=2, dtype=BF16,
           out=P, ws=P, nb=1 << 30):
    return lib.msa_full_attn_decode_fp8(q, kc, P, ks, vs, table, kv, B, Hq, Hkv, d, pages, page, maxp, 0.0, dtype, out,
                                        None, ws, nb, None)


ALL = (append, read, decode)


@pytest.mark.parametrize("call", ALL)
def test_refusals(lib, call):
    assert call(lib, Hkv=0) == 1 and call(lib, B=-1) == 1 and call(lib, dtype=2) == 1
    assert call(lib, d=96) == 2
    assert call(lib, ws=None) == 3 and call(lib, ws=ctypes.c_void_p(0x1010)) == 3 and call(lib, nb=128) == 3
    assert call(lib, page=0) == 1 and call(lib, page=24) == 2 and call(lib, pages=0) == 1 and call(lib, maxp=0) == 1
    assert call(lib, maxp=1 << 28) == 2 and call(lib, pages=1 << 28) == 2
    for name in ("kc", "ks", "vs", "kv", "table"):
        assert call(lib, **{name: None}) == 1
    for name in ("kc", "ks", "vs", "out"):
        assert call(lib, **{name: ODD}) == 1
    big = {"B": 1 << 28} if call is decode else {"T": 1 << 30}
    assert call(lib, **big) == 2
    none = {"B": 0} if call is decode else {"T": 0}
    assert call(lib, ws=None, nb=0, kc=None, ks=None, **none) == 0 and call(lib, d=96, **none) == 2


def test_refusals_each(lib):
    for call in (append, decode):
        assert call(lib, Hq=6, Hkv=4) == 1 and call(lib, Hq=65, Hkv=1) == 2
    assert append(lib, rot=136) == 1 and append(lib, rot=24) == 2 and append(lib, il=2) == 1
    assert append(lib, rope=None) == 1 and append(lib, max_pos=0) == 1
    assert append(lib, out=None) == 1 and append(lib, q=None) == 1
    assert append(lib, cu=None) == 1 and read(lib, cu=None) == 1  # no offsets, but T != B
    assert append(lib, k=ODD) == 1 and append(lib, rope=ODD) == 1
    assert read(lib, T=-1) == 1 and read(lib, out=None) == 1 and read(lib, Hkv=(1 << 16) + 1, T=1) == 2
    assert decode(lib, q=None) == 1 and decode(lib, q=ODD) == 1 and decode(lib, out=None) == 1


def test_workspace_sizes(lib):
    size = lambda op, B=2, Nq=100, Nk=100, G=2, Hq=8, d=128, dt=BF16: msa.msa_workspace_size(  # noqa: E731
        op, B, Nq, Nk, G, Hq, d, 0, 0, 0, dt)
    for op in (msa.MSA_OP_PAGED_APPEND_FP8, msa.MSA_OP_PAGED_READ_FP8, msa.MSA_OP_FULL_DECODE_FP8):
        for dt in (BF16, FP32):
            assert size(op, dt=dt) >= 256 and size(op, dt=dt) % 256 == 0 and size(op, B=0, dt=dt) == 256
        assert size(op, d=96) == 0 and size(op, Hq=9) == 0 and size(op, B=-1) == 0 and size(op, dt=5) == 0


def test_bindings_refuse_wrong_tensors():
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    cache, scale = torch.zeros(1, 16, 2, 64).to(torch.float8_e4m3fn), torch.zeros(1, 2, 16)
    i = torch.tensor([0, 4], dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.msa_paged_append_fp8(q, k, k, None, i, i[1:], table, cache, cache, scale, scale)
    with pytest.raises(ValueError):
        msa.msa_paged_read_fp8(cache, cache, scale, scale, table, i, i[1:], 4)
    with pytest.raises(ValueError):
        msa.msa_full_attn_decode_fp8(q, cache, cache, scale, scale, table.expand(4, 1), i)
