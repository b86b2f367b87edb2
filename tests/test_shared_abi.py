"""Host-side refusals of msa_full_attn_decode_shared (no GPU needed: every call
below returns before any launch)."""
import ctypes
import os

import pytest
import torch

import block_sparse_long_select_gb300 as msa
from block_sparse_long_select_gb300 import _lib

P = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1008)
BF16, FP32 = msa.MSA_BF16, msa.MSA_FP32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.lib_path()):
        msa.build()
    return msa.load_library()


def shared(lib, q=P, kc=P, table=P, kv=P, cu=P, pre=P, B=4, G=2, Hq=8, Hkv=2, d=128, pages=4, page=16, maxp=2,
           dtype=BF16, out=P, ws=P, nb=1 << 30):
    return lib.msa_full_attn_decode_shared(q, kc, P, table, kv, cu, pre, B, G, Hq, Hkv, d, pages, page, maxp, 0.0,
                                           dtype, out, None, ws, nb, None)


def test_refusals(lib):
    assert shared(lib, Hq=6, Hkv=4) == 1 and shared(lib, Hkv=0) == 1 and shared(lib, B=-1) == 1
    assert shared(lib, dtype=2) == 1 and shared(lib, d=96) == 2 and shared(lib, Hq=65, Hkv=1) == 2
    assert shared(lib, page=24) == 2 and shared(lib, page=0) == 1 and shared(lib, maxp=1 << 28) == 2
    assert shared(lib, G=-1) == 1 and shared(lib, G=5) == 1  # more groups than sequences
    for name in ("q", "kc", "table", "kv", "cu", "pre", "out"):
        assert shared(lib, **{name: None}) == 1
    assert shared(lib, q=ODD) == 1 and shared(lib, kc=ODD) == 1 and shared(lib, out=ODD) == 1
    assert shared(lib, ws=None) == 3 and shared(lib, ws=ctypes.c_void_p(0x1010)) == 3 and shared(lib, nb=4096) == 3
    assert shared(lib, B=1 << 28) == 2
    assert shared(lib, B=0, G=0, q=None, kc=None, table=None, kv=None, cu=None, pre=None, out=None, ws=None, nb=0) == 0
    assert shared(lib, B=0, G=1) == 1 and shared(lib, B=0, G=0, d=96) == 2


def test_workspace_sizes():
    size = lambda B=4, G=2, Hkv=2, Hq=8, d=128, dt=BF16: msa.msa_workspace_size(  # noqa: E731
        msa.MSA_OP_FULL_DECODE_SHARED, B, G, 1000, Hkv, Hq, d, 0, 0, 0, dt)
    for dt in (BF16, FP32):
        assert size(dt=dt) % 256 == 0 and size(B=0, G=0, dt=dt) == 256
        assert size(G=0, dt=dt) == msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE, 4, 1, 1000, 2, 8, 128, 0, 0, 0, dt)
        # the parts of every row, and what was said of the size
        rows = 1000 * 32
        assert rows * 128 * 4 < size(B=1000, Hq=32, Hkv=8, dt=dt) <= rows * (2 * 128 + 4) * 4 + 60e6
    assert size(G=5) == 0 and size(G=-1) == 0 and size(d=96) == 0 and size(Hq=9) == 0 and size(B=-1) == 0


def test_binding_refuses_wrong_tensors():
    q, k = torch.zeros(4, 8, 64), torch.zeros(1, 16, 2, 64)
    i = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.msa_full_attn_decode_shared(q, k, k, torch.zeros(4, 1, dtype=torch.int32), i, i, i[1:])


def test_workspace_is_as_large_as_stated():
    """2 d + 4 fp32 values per query head and sequence, a key/value head's heads beyond
    16 counted in sixteens, 24 bytes per sequence, 48 per group, and up to 52 MB."""
    for dt in (BF16, FP32):
        for d in (64, 128):
            for hpg in (1, 2, 3, 4, 7, 8, 15, 16, 17, 24, 33, 48, 49, 64):
                for Hkv in (1, 3, 8):
                    for B, G in ((1, 1), (97, 3), (4000, 1000), (4000, 4000), (65536, 65536), (1 << 20, 1 << 20)):
                        n = msa.msa_workspace_size(msa.MSA_OP_FULL_DECODE_SHARED, B, G, 1000, Hkv, Hkv * hpg, d, 0, 0, 0,
                                                   dt)
                        if B * Hkv * hpg > 1 << 26 and n == 0:
                            continue  # more rows than a call takes
                        heads = Hkv * (hpg if hpg <= 16 else -(-hpg // 16) * 16)
                        assert B * heads * d * 4 < n <= B * heads * (2 * d + 4) * 4 + 24 * B + 48 * G + 52e6
