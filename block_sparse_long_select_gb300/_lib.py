"""ctypes binding of libmsa.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import os
from functools import lru_cache

MSA_BF16, MSA_FP32 = 0, 1
MSA_OP_INDEX_SELECT, MSA_OP_PREFILL, MSA_OP_DECODE, MSA_OP_DECODE_STEP, MSA_OP_KL_AUX, MSA_OP_BACKWARD = 0, 1, 2, 3, 4, 5
MSA_OP_FULL_PREFILL, MSA_OP_FULL_BACKWARD, MSA_OP_FULL_DECODE, MSA_OP_PAGED_APPEND = 8, 9, 10, 11
MSA_OP_PAGED_APPEND_FP8, MSA_OP_PAGED_READ_FP8, MSA_OP_FULL_DECODE_FP8 = 13, 14, 15
MSA_OP_FULL_DECODE_SHARED = 16
MSA_FORCE_LOCAL, MSA_FORCE_START = 1, 2
STATUS_NAMES = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_WORKSPACE",
                4: "MSA_ERR_CUDA", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_BOUNDS"}

# (name, restype, argtypes) of every symbol declared in include/msa.h
_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "msa_workspace_size": (_sz, [_i32] * 11),
    "msa_index_select": (_i32, [_vp, _vp, _vp, _vp] + [_i32] * 8 + [_vp, _vp, _vp, _sz, _vp]),
    "msa_index_select_v": (_i32, [_vp, _vp, _vp, _vp] + [_i32] * 9 + [_vp, _vp, _vp, _sz, _vp]),
    "msa_sparse_attn_prefill": (_i32, [_vp] * 6 + [_i32] * 8 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_sparse_attn_decode": (_i32, [_vp] * 5 + [_i32] * 7 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_decode_step": (_i32, [_vp] * 9 + [_i32] * 8 + [_f32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_kl_aux_forward": (_i32, [_vp] * 8 + [_i32] * 9 + [_f32, _i32, _vp, _vp, _sz, _vp]),
    "msa_sparse_attn_backward": (_i32, [_vp] * 9 + [_i32] * 8 + [_f32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_paged_append": (_i32, [_vp] * 7 + [_i32] * 12 + [_vp] * 4 + [_sz, _vp]),
    "msa_full_attn_decode": (_i32, [_vp] * 5 + [_i32] * 7 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_full_attn_decode_shared": (_i32, [_vp] * 7 + [_i32] * 8 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_paged_append_fp8": (_i32, [_vp] * 7 + [_i32] * 12 + [_vp] * 6 + [_sz, _vp]),
    "msa_paged_read_fp8": (_i32, [_vp] * 7 + [_i32] * 8 + [_vp] * 3 + [_sz, _vp]),
    "msa_full_attn_decode_fp8": (_i32, [_vp] * 7 + [_i32] * 7 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_full_attn_prefill": (_i32, [_vp] * 5 + [_i32] * 6 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_full_attn_prefill_paged": (_i32, [_vp] * 6 + [_i32] * 8 + [_f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "msa_full_attn_backward": (_i32, [_vp] * 8 + [_i32] * 6 + [_f32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_read_status": (_i32, [_vp, _vp]),
    "msa_status_string": (ctypes.c_char_p, [_i32]),
    "msa_index_select_noalloc": (_i32, [_vp, _vp, _vp, _vp] + [_i32] * 8 + [_vp, _vp, _vp]),
    "msa_profile_begin": (_i32, []),
    "msa_profile_end": (_i32, [_vp, _i32]),
    "msa_debug_inject_timeout": (_i32, [_i32]),
}


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


class MsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


def lib_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmsa.so")


@lru_cache(maxsize=None)
def load_library():
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with block_sparse_long_select_gb300.build() "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


# ---------------------------------------------------------------------------
def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return MSA_BF16
    if t.dtype == torch.float32:
        return MSA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise MsaError(code, where)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _check_select_args(iq, ik, q_offset, kv_len, Bs, K, sel, block_max):
    """Shapes, dtypes and devices of an index selection's tensors (the library
    writes sel and block_max through raw pointers: a short or mistyped buffer
    would be overrun on the device)."""
    import torch

    if iq.dim() != 4 or ik.dim() != 3:
        raise ValueError("iq must be [B, Nq, G, di] and ik [B, Nk, di]")
    B, Nq, G, di = iq.shape
    if ik.shape[0] != B or ik.shape[2] != di or ik.dtype != iq.dtype or ik.device != iq.device:
        raise ValueError("ik must be [B, Nk, di] with iq's dtype and device")
    for name, t in (("q_offset", q_offset), ("kv_len", kv_len)):
        if t is not None and (t.dtype != torch.int32 or t.numel() != B or t.device != iq.device):
            raise ValueError(f"{name} must be int32 of length B on iq's device")
    if sel is not None and (sel.dtype != torch.int32 or sel.numel() != B * Nq * G * K or sel.device != iq.device):
        raise ValueError("sel must be int32 with B * Nq * G * K elements on iq's device")
    nblk = (ik.shape[1] + Bs - 1) // Bs if Bs > 0 else 0
    if block_max is not None and (block_max.dtype != torch.float32 or block_max.numel() != B * Nq * G * nblk or
                                  block_max.device != iq.device):
        raise ValueError("block_max must be float32 with B * Nq * G * ceil(Nk / Bs) elements on iq's device")


def msa_workspace_size(op, B, Nq, Nk, G, Hq, d, di, Bs, K, dtype) -> int:
    return int(load_library().msa_workspace_size(op, B, Nq, Nk, G, Hq, d, di, Bs, K, dtype))


def workspace(nbytes: int, device="cuda"):
    """Zero-filled device scratch of ``nbytes`` (caching-allocator blocks are 512-byte aligned)."""
    import torch

    ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def msa_index_select(iq, ik, q_offset, kv_len, Bs, K, sel=None, block_max=None, ws=None, stream=None):
    """iq [B,Nq,G,di], ik [B,Nk,di] -> sel [B,Nq,G,K] int32 (see include/msa.h)."""
    return msa_index_select_v(iq, ik, q_offset, kv_len, Bs, K, MSA_FORCE_LOCAL, sel, block_max, ws, stream)


def msa_index_select_v(iq, ik, q_offset, kv_len, Bs, K, force, sel=None, block_max=None, ws=None, stream=None):
    """msa_index_select with a choice of forced blocks: force = MSA_FORCE_LOCAL,
    or MSA_FORCE_LOCAL | MSA_FORCE_START to keep block 0 as well (see include/msa.h)."""
    import torch

    _need_cuda(iq, ik, q_offset, kv_len, sel, block_max)
    _check_select_args(iq, ik, q_offset, kv_len, Bs, K, sel, block_max)
    B, Nq, G, di = iq.shape
    Nk = ik.shape[1]
    dt = _dtype_code(iq)
    if sel is None:
        sel = torch.empty((B, Nq, G, K), dtype=torch.int32, device=iq.device)
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_INDEX_SELECT, B, Nq, Nk, G, 0, 0, di, Bs, K, dt), iq.device)
    code = load_library().msa_index_select_v(_ptr(iq), _ptr(ik), _ptr(q_offset), _ptr(kv_len), B, Nq, Nk, G, di,
                                             Bs, K, dt, int(force), _ptr(sel), _ptr(block_max), _ptr(ws), ws.numel(),
                                             _stream(stream, iq.device))
    _check(code, "msa_index_select_v")
    return sel


def msa_index_select_noalloc(iq, ik, q_offset, kv_len, Bs, K, sel, block_max=None, stream=None):
    """msa_index_select on the library's static scratch (no workspace; see include/msa.h).
    ``sel`` must be given: this wrapper allocates nothing either."""
    _need_cuda(iq, ik, q_offset, kv_len, sel, block_max)
    if sel is None:
        raise ValueError("msa_index_select_noalloc needs a caller-owned sel")
    _check_select_args(iq, ik, q_offset, kv_len, Bs, K, sel, block_max)
    B, Nq, G, di = iq.shape
    Nk = ik.shape[1]
    code = load_library().msa_index_select_noalloc(_ptr(iq), _ptr(ik), _ptr(q_offset), _ptr(kv_len), B, Nq, Nk, G,
                                                   di, Bs, K, _dtype_code(iq), _ptr(sel), _ptr(block_max),
                                                   _stream(stream, iq.device))
    _check(code, "msa_index_select_noalloc")
    return sel


def msa_sparse_attn_prefill(q, k, v, sel, q_offset, kv_len, Bs, K, scale=0.0, out=None, lse=None, ws=None,
                            stream=None):
    """q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d], sel [B,Nq,Hkv,K] -> out [B,Nq,Hq,d]."""
    import torch

    _need_cuda(q, k, v, sel, q_offset, kv_len, out, lse)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_PREFILL, B, Nq, Nk, Hkv, Hq, d, 0, Bs, K, dt), q.device)
    code = load_library().msa_sparse_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(sel), _ptr(q_offset),
                                                  _ptr(kv_len), B, Nq, Nk, Hq, Hkv, d, Bs, K, float(scale), dt,
                                                  _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                                  _stream(stream, q.device))
    _check(code, "msa_sparse_attn_prefill")
    return out


def msa_sparse_attn_decode(q, k_cache, v_cache, sel, kv_len, Bs, K, scale=0.0, out=None, lse=None, ws=None,
                           stream=None):
    """q [B,Hq,d], caches [B,Lmax,Hkv,d], sel [B,Hkv,K] (or [B,1,Hkv,K]) -> out [B,Hq,d]."""
    import torch

    _need_cuda(q, k_cache, v_cache, sel, kv_len, out, lse)
    B, Hq, d = q.shape
    Lmax, Hkv = k_cache.shape[1], k_cache.shape[2]
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_DECODE, B, 1, Lmax, Hkv, Hq, d, 0, Bs, K, dt), q.device)
    code = load_library().msa_sparse_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(sel), _ptr(kv_len),
                                                 B, Lmax, Hq, Hkv, d, Bs, K, float(scale), dt, _ptr(out), _ptr(lse),
                                                 _ptr(ws), ws.numel(), _stream(stream, q.device))
    _check(code, "msa_sparse_attn_decode")
    return out


def msa_read_status(ws, stream=None) -> int:
    return int(load_library().msa_read_status(_ptr(ws), _stream(stream, ws.device)))


def msa_status_string(code: int) -> str:
    return load_library().msa_status_string(int(code)).decode()


def msa_profile_begin() -> None:
    load_library().msa_profile_begin()


def msa_profile_end() -> dict:
    """{kernel name: (launches, total device ms)} recorded since msa_profile_begin()."""
    buf = (KernelTime * 64)()
    n = load_library().msa_profile_end(ctypes.cast(buf, ctypes.c_void_p), 64)
    if n < 0:
        raise RuntimeError("msa_profile_end: event query failed")
    return {buf[k].name.decode(): (buf[k].launches, buf[k].total_ms) for k in range(min(n, 64))}


def msa_debug_inject_timeout(enable: bool) -> bool:
    """Test hook (see include/msa_profile.h): while on, the attention kernels
    make one bounded wait that runs out and report MSA_ERR_TIMEOUT. Returns the
    previous setting."""
    return bool(load_library().msa_debug_inject_timeout(1 if enable else 0))


def msa_decode_step(q, k_new, v_new, iq, ik_new, k_cache, v_cache, ik_cache, kv_len, Bs, K, sel=None, out=None,
                    lse=None, scale=0.0, ws=None, stream=None):
    """One streaming decode step (see include/msa.h): append the new token's
    k [B,Hkv,d], v, index key [B,di] at kv_len[b] of the caches, advance
    kv_len, then select and attend for q [B,Hq,d], iq [B,Hkv,di].
    Returns (sel [B,Hkv,K], out [B,Hq,d])."""
    import torch

    _need_cuda(q, k_new, v_new, iq, ik_new, k_cache, v_cache, ik_cache, kv_len, sel, out, lse)
    B, Hq, d = q.shape
    Lmax, Hkv = k_cache.shape[1], k_cache.shape[2]
    di = ik_cache.shape[2]
    dt = _dtype_code(q)
    if sel is None:
        sel = torch.empty((B, Hkv, K), dtype=torch.int32, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_DECODE_STEP, B, 0, Lmax, Hkv, Hq, d, di, Bs, K, dt), q.device)
    code = load_library().msa_decode_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(iq), _ptr(ik_new), _ptr(k_cache),
                                          _ptr(v_cache), _ptr(ik_cache), _ptr(kv_len), B, Lmax, Hq, Hkv, d, di, Bs, K,
                                          float(scale), dt, _ptr(sel), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                          _stream(stream, q.device))
    _check(code, "msa_decode_step")
    return sel, out


def msa_kl_aux_forward(q, k, iq, ik, sel, lse, q_offset, kv_len, Bs, K, kl=None, scale=0.0, ws=None, stream=None):
    """KL auxiliary forward (see include/msa.h): KL(head-averaged main-branch
    distribution || index softmax) per (row, group) -> kl [B, Nq, Hkv] fp32.
    ``lse`` is the forward's [B, Nq, Hq] output of msa_sparse_attn_prefill."""
    import torch

    _need_cuda(q, k, iq, ik, sel, lse, q_offset, kv_len, kl)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    di = iq.shape[3]
    dt = _dtype_code(q)
    if kl is None:
        kl = torch.empty((B, Nq, Hkv), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_KL_AUX, B, Nq, Nk, Hkv, Hq, d, di, Bs, K, dt), q.device)
    code = load_library().msa_kl_aux_forward(_ptr(q), _ptr(k), _ptr(iq), _ptr(ik), _ptr(sel), _ptr(lse),
                                             _ptr(q_offset), _ptr(kv_len), B, Nq, Nk, Hq, Hkv, d, di, Bs, K,
                                             float(scale), dt, _ptr(kl), _ptr(ws), ws.numel(),
                                             _stream(stream, q.device))
    _check(code, "msa_kl_aux_forward")
    return kl


def msa_sparse_attn_backward(q, k, v, out, dout, lse, sel, q_offset, kv_len, Bs, K, dq=None, dk=None, dv=None,
                             scale=0.0, ws=None, stream=None):
    """Main Branch backward (see include/msa.h): gradients of q [B,Nq,Hq,d],
    k and v [B,Nk,Hkv,d] through msa_sparse_attn_prefill, given its output
    ``out``, lse [B,Nq,Hq] and selection ``sel`` and the output gradient
    ``dout``. Returns (dq, dk, dv) in q's dtype."""
    import torch

    _need_cuda(q, k, v, out, dout, lse, sel, q_offset, kv_len, dq, dk, dv)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    dt = _dtype_code(q)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if ws is None:
        ws = workspace(msa_workspace_size(MSA_OP_BACKWARD, B, Nq, Nk, Hkv, Hq, d, 0, Bs, K, dt), q.device)
    code = load_library().msa_sparse_attn_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                                   _ptr(sel), _ptr(q_offset), _ptr(kv_len), B, Nq, Nk, Hq, Hkv, d,
                                                   Bs, K, float(scale), dt, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                                   ws.numel(), _stream(stream, q.device))
    _check(code, "msa_sparse_attn_backward")
    return dq, dk, dv


# ---- full attention and paged caches -----------------------------------------
# These calls serve single tokens too, where the host's time counts: a tensor's
# checks are one call each, and streams and devices are only switched if needed.
@lru_cache(maxsize=None)
def _torch():
    import torch

    return torch


def _need(name, t, dtype, dev, shape):
    """Raises unless ``t`` is contiguous, of this dtype, device and shape: the
    library reads and writes it through a raw pointer."""
    if t is None or t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        got = "None" if t is None else f"{t.dtype}, {tuple(t.shape)} on {t.device}"
        raise ValueError(f"{name} must be contiguous, {dtype}, of shape {tuple(shape)} on cuda:{dev}; got {got}")


def _rows(name, t, dims=3):
    """Shape of a packed-row tensor [rows, heads, d] (or a cache, dims 4)."""
    if not t.is_cuda or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor with {dims} dimensions")
    return t.shape


def _elsewhere(stream, dev):
    """None if a call on ``stream`` (None: the current one) for tensors on device
    ``dev`` can go ahead; else the context that makes that stream and device
    current, so that what the call allocates belongs to the stream as well."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        return _torch().cuda.stream(stream)
    return None if dev == _torch()._C._cuda_getDevice() else _torch().cuda.device(dev)


def _raw_stream(dev):
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _addr(t):
    return None if t is None else t.data_ptr()


def _full_ws(ws, ref, op, B, Nq, Nk, Hkv, Hq, d, dt):
    if ws is None:
        return workspace(msa_workspace_size(op, B, Nq, Nk, Hkv, Hq, d, 0, 0, 0, dt), ref.device)
    if ws.get_device() != ref.get_device() or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on {ref.device}")
    return ws


def msa_paged_append(q, k_new, v_new, rope, cu_new, kv_len, page_table, k_cache, v_cache, interleaved=False,
                     q_out=None, ws=None, stream=None):
    """Append packed new tokens to a paged cache and rotate keys and queries by
    position (see include/msa.h). q [T,Hq,d] or None, k_new, v_new [T,Hkv,d],
    rope [max_pos, rot/2, 2] fp32 or None, cu_new [B+1] or None (one token per
    sequence), kv_len [B] (the new tokens counted), page_table [B, max_pages],
    caches [num_pages, page_size, Hkv, d]. Returns the rotated queries (None
    without q); ``q_out=q`` rotates in place."""
    torch = _torch()
    shape = _rows("k_new", k_new)
    T, Hkv, d = shape
    dev, dtype, i32 = k_new.get_device(), k_new.dtype, torch.int32
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_paged_append(q, k_new, v_new, rope, cu_new, kv_len, page_table, k_cache, v_cache, interleaved,
                                    q_out, ws)
    num_pages, page_size = _rows("k_cache", k_cache, 4)[:2]
    B, max_pages = page_table.shape
    Hq = Hkv
    if q is not None:
        Hq = _rows("q", q)[1]
        _need("q", q, dtype, dev, (T, Hq, d))
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            _need("q_out", q_out, dtype, dev, q.shape)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _need("v_new", v_new, dtype, dev, shape)
    _need("k_cache", k_cache, dtype, dev, (num_pages, page_size, Hkv, d))
    _need("v_cache", v_cache, dtype, dev, k_cache.shape)
    if cu_new is not None:
        _need("cu_new", cu_new, i32, dev, (B + 1,))
    _need("kv_len", kv_len, i32, dev, (B,))
    _need("page_table", page_table, i32, dev, (B, max_pages))
    max_pos = half = 0
    if rope is not None:
        max_pos, half, _ = rope.shape
        _need("rope", rope, torch.float32, dev, (max_pos, half, 2))
    dt = _dtype_code(k_new)
    ws = _full_ws(ws, k_new, MSA_OP_PAGED_APPEND, B, T, 0, Hkv, Hq, d, dt)
    code = load_library().msa_paged_append(_addr(q), k_new.data_ptr(), v_new.data_ptr(), _addr(rope), _addr(cu_new),
                                           kv_len.data_ptr(), page_table.data_ptr(), B, T, Hq, Hkv, d, 2 * half,
                                           interleaved, max_pos, num_pages, page_size, max_pages, dt, _addr(q_out),
                                           k_cache.data_ptr(), v_cache.data_ptr(), ws.data_ptr(), ws.nbytes,
                                           _raw_stream(dev))
    _check(code, "msa_paged_append")
    return q_out


def msa_full_attn_decode(q, k_cache, v_cache, page_table, kv_len, scale=0.0, out=None, lse=None, ws=None,
                         stream=None):
    """One query row per sequence over its whole paged cache (see include/msa.h):
    q [B,Hq,d], caches [num_pages, page_size, Hkv, d] -> out [B,Hq,d]."""
    torch = _torch()
    shape = _rows("q", q)
    B, Hq, d = shape
    dev, dtype = q.get_device(), q.dtype
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_decode(q, k_cache, v_cache, page_table, kv_len, scale, out, lse, ws)
    num_pages, page_size, Hkv, _ = _rows("k_cache", k_cache, 4)
    max_pages = page_table.shape[1]
    _need("k_cache", k_cache, dtype, dev, (num_pages, page_size, Hkv, d))
    _need("v_cache", v_cache, dtype, dev, k_cache.shape)
    _need("kv_len", kv_len, torch.int32, dev, (B,))
    _need("page_table", page_table, torch.int32, dev, (B, max_pages))
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (B, Hq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, dtype, dev, shape)
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_DECODE, B, 1, max_pages * page_size, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                               page_table.data_ptr(), kv_len.data_ptr(), B, Hq, Hkv, d, num_pages,
                                               page_size, max_pages, scale, dt, out.data_ptr(), _addr(lse),
                                               ws.data_ptr(), ws.nbytes, _raw_stream(dev))
    _check(code, "msa_full_attn_decode")
    return out


def msa_full_attn_decode_shared(q, k_cache, v_cache, page_table, kv_len, cu_prefix, prefix_len, scale=0.0, out=None,
                                lse=None, ws=None, stream=None):
    """msa_full_attn_decode where group x of sequences, [cu_prefix[x], cu_prefix[x+1]),
    shares its first prefix_len[x] keys (see include/msa.h): cu_prefix [P+1], prefix_len [P]."""
    torch = _torch()
    shape = _rows("q", q)
    B, Hq, d = shape
    dev, dtype, i32 = q.get_device(), q.dtype, torch.int32
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_decode_shared(q, k_cache, v_cache, page_table, kv_len, cu_prefix, prefix_len, scale,
                                               out, lse, ws)
    num_pages, page_size, Hkv, _ = _rows("k_cache", k_cache, 4)
    max_pages, P = page_table.shape[1], prefix_len.shape[0]
    _need("k_cache", k_cache, dtype, dev, (num_pages, page_size, Hkv, d))
    _need("v_cache", v_cache, dtype, dev, k_cache.shape)
    _need("kv_len", kv_len, i32, dev, (B,))
    _need("page_table", page_table, i32, dev, (B, max_pages))
    _need("cu_prefix", cu_prefix, i32, dev, (P + 1,))
    _need("prefix_len", prefix_len, i32, dev, (P,))
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (B, Hq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, dtype, dev, shape)
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_DECODE_SHARED, B, P, max_pages * page_size, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_decode_shared(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                                      page_table.data_ptr(), kv_len.data_ptr(), cu_prefix.data_ptr(),
                                                      prefix_len.data_ptr(), B, P, Hq, Hkv, d, num_pages, page_size,
                                                      max_pages, scale, dt, out.data_ptr(), _addr(lse), ws.data_ptr(),
                                                      ws.nbytes, _raw_stream(dev))
    _check(code, "msa_full_attn_decode_shared")
    return out


def _need_fp8(k_cache, v_cache, k_scale, v_scale, dev):
    """Checks the four tensors of a cache in 8 bits; its num_pages, page_size, Hkv and d."""
    torch = _torch()
    shape = num_pages, page_size, Hkv, d = _rows("k_cache", k_cache, 4)
    _need("k_cache", k_cache, torch.float8_e4m3fn, dev, shape)
    _need("v_cache", v_cache, torch.float8_e4m3fn, dev, shape)
    _need("k_scale", k_scale, torch.float32, dev, (num_pages, Hkv, page_size))
    _need("v_scale", v_scale, torch.float32, dev, (num_pages, Hkv, page_size))
    return num_pages, page_size, Hkv, d


def msa_paged_append_fp8(q, k_new, v_new, rope, cu_new, kv_len, page_table, k_cache, v_cache, k_scale, v_scale,
                         interleaved=False, q_out=None, ws=None, stream=None):
    """msa_paged_append into a cache in 8 bits (see include/msa.h): caches
    [num_pages, page_size, Hkv, d] float8_e4m3fn, scales [num_pages, Hkv, page_size]
    fp32. Returns the rotated queries (None without q)."""
    torch = _torch()
    shape = _rows("k_new", k_new)
    T, Hkv, d = shape
    dev, dtype, i32 = k_new.get_device(), k_new.dtype, torch.int32
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_paged_append_fp8(q, k_new, v_new, rope, cu_new, kv_len, page_table, k_cache, v_cache, k_scale,
                                        v_scale, interleaved, q_out, ws)
    num_pages, page_size, *heads = _need_fp8(k_cache, v_cache, k_scale, v_scale, dev)
    if heads != [Hkv, d]:
        raise ValueError(f"k_cache must be [num_pages, page_size, {Hkv}, {d}]; got {tuple(k_cache.shape)}")
    B, max_pages = page_table.shape
    Hq = Hkv
    if q is not None:
        Hq = _rows("q", q)[1]
        _need("q", q, dtype, dev, (T, Hq, d))
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            _need("q_out", q_out, dtype, dev, q.shape)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _need("v_new", v_new, dtype, dev, shape)
    if cu_new is not None:
        _need("cu_new", cu_new, i32, dev, (B + 1,))
    _need("kv_len", kv_len, i32, dev, (B,))
    _need("page_table", page_table, i32, dev, (B, max_pages))
    max_pos = half = 0
    if rope is not None:
        max_pos, half, _ = rope.shape
        _need("rope", rope, torch.float32, dev, (max_pos, half, 2))
    dt = _dtype_code(k_new)
    ws = _full_ws(ws, k_new, MSA_OP_PAGED_APPEND_FP8, B, T, 0, Hkv, Hq, d, dt)
    code = load_library().msa_paged_append_fp8(_addr(q), k_new.data_ptr(), v_new.data_ptr(), _addr(rope),
                                               _addr(cu_new), kv_len.data_ptr(), page_table.data_ptr(), B, T, Hq, Hkv,
                                               d, 2 * half, interleaved, max_pos, num_pages, page_size, max_pages, dt,
                                               _addr(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
                                               k_scale.data_ptr(), v_scale.data_ptr(), ws.data_ptr(), ws.nbytes,
                                               _raw_stream(dev))
    _check(code, "msa_paged_append_fp8")
    return q_out


def msa_paged_read_fp8(k_cache, v_cache, k_scale, v_scale, page_table, cu, kv_len, rows, dtype=None, k_out=None,
                       v_out=None, ws=None, stream=None):
    """The last cached keys and values of each sequence as ``rows`` packed rows
    (see include/msa.h): cu [B+1] or None (one row per sequence). Returns
    (k, v) [rows, Hkv, d] of ``dtype`` (bfloat16 by default)."""
    torch = _torch()
    _rows("k_cache", k_cache, 4)
    dev, i32 = k_cache.get_device(), torch.int32
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_paged_read_fp8(k_cache, v_cache, k_scale, v_scale, page_table, cu, kv_len, rows, dtype, k_out,
                                      v_out, ws)
    num_pages, page_size, Hkv, d = _need_fp8(k_cache, v_cache, k_scale, v_scale, dev)
    B, max_pages = page_table.shape
    if dtype is None:
        dtype = torch.bfloat16 if k_out is None else k_out.dtype
    if k_out is None:
        k_out = torch.empty((rows, Hkv, d), dtype=dtype, device=k_cache.device)
    else:
        _need("k_out", k_out, dtype, dev, (rows, Hkv, d))
    if v_out is None:
        v_out = torch.empty_like(k_out)
    else:
        _need("v_out", v_out, dtype, dev, (rows, Hkv, d))
    if cu is not None:
        _need("cu", cu, i32, dev, (B + 1,))
    _need("kv_len", kv_len, i32, dev, (B,))
    _need("page_table", page_table, i32, dev, (B, max_pages))
    dt = _dtype_code(k_out)
    ws = _full_ws(ws, k_out, MSA_OP_PAGED_READ_FP8, B, rows, 0, Hkv, Hkv, d, dt)
    code = load_library().msa_paged_read_fp8(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                             v_scale.data_ptr(), _addr(cu), kv_len.data_ptr(), page_table.data_ptr(),
                                             B, rows, Hkv, d, num_pages, page_size, max_pages, dt, k_out.data_ptr(),
                                             v_out.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(dev))
    _check(code, "msa_paged_read_fp8")
    return k_out, v_out


def msa_full_attn_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, scale=0.0, out=None, lse=None,
                             ws=None, stream=None):
    """msa_full_attn_decode over a cache in 8 bits (see include/msa.h)."""
    torch = _torch()
    shape = _rows("q", q)
    B, Hq, d = shape
    dev, dtype = q.get_device(), q.dtype
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, scale, out, lse,
                                            ws)
    num_pages, page_size, Hkv, cached = _need_fp8(k_cache, v_cache, k_scale, v_scale, dev)
    if cached != d:
        raise ValueError(f"k_cache holds heads of {cached}, q of {d}")
    max_pages = page_table.shape[1]
    _need("kv_len", kv_len, torch.int32, dev, (B,))
    _need("page_table", page_table, torch.int32, dev, (B, max_pages))
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (B, Hq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, dtype, dev, shape)
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_DECODE_FP8, B, 1, max_pages * page_size, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_decode_fp8(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                                   k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
                                                   kv_len.data_ptr(), B, Hq, Hkv, d, num_pages, page_size, max_pages,
                                                   scale, dt, out.data_ptr(), _addr(lse), ws.data_ptr(), ws.nbytes,
                                                   _raw_stream(dev))
    _check(code, "msa_full_attn_decode_fp8")
    return out


def msa_full_attn_prefill(q, k, v, cu_q, cu_k, scale=0.0, out=None, lse=None, ws=None, stream=None):
    """Causal attention over packed sequences (see include/msa.h): q [Tq,Hq,d],
    k, v [Tk,Hkv,d], cu_q, cu_k [B+1] int32 -> out [Tq,Hq,d]."""
    torch = _torch()
    shape = _rows("q", q)
    Tq, Hq, d = shape
    dev, dtype = q.get_device(), q.dtype
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_prefill(q, k, v, cu_q, cu_k, scale, out, lse, ws)
    Tk, Hkv, _ = _rows("k", k)
    B = cu_q.shape[0] - 1
    _need("k", k, dtype, dev, (Tk, Hkv, d))
    _need("v", v, dtype, dev, k.shape)
    _need("cu_q", cu_q, torch.int32, dev, (B + 1,))
    _need("cu_k", cu_k, torch.int32, dev, (B + 1,))
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (Tq, Hq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, dtype, dev, shape)
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_PREFILL, B, Tq, Tk, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
                                                cu_k.data_ptr(), B, Tq, Tk, Hq, Hkv, d, scale, dt, out.data_ptr(),
                                                _addr(lse), ws.data_ptr(), ws.nbytes, _raw_stream(dev))
    _check(code, "msa_full_attn_prefill")
    return out


def msa_full_attn_prefill_paged(q, k_cache, v_cache, page_table, cu_q, kv_len, scale=0.0, out=None, lse=None,
                                ws=None, stream=None):
    """msa_full_attn_prefill with each sequence's kv_len[b] keys in a paged cache
    (see include/msa.h): q [Tq,Hq,d], cu_q [B+1], page_table [B, max_pages] -> out [Tq,Hq,d]."""
    torch = _torch()
    shape = _rows("q", q)
    Tq, Hq, d = shape
    dev, dtype = q.get_device(), q.dtype
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_prefill_paged(q, k_cache, v_cache, page_table, cu_q, kv_len, scale, out, lse, ws)
    num_pages, page_size, Hkv, _ = _rows("k_cache", k_cache, 4)
    B, max_pages = page_table.shape
    _need("k_cache", k_cache, dtype, dev, (num_pages, page_size, Hkv, d))
    _need("v_cache", v_cache, dtype, dev, k_cache.shape)
    _need("kv_len", kv_len, torch.int32, dev, (B,))
    _need("cu_q", cu_q, torch.int32, dev, (B + 1,))
    _need("page_table", page_table, torch.int32, dev, (B, max_pages))
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (Tq, Hq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, dtype, dev, shape)
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_PREFILL, B, Tq, max_pages * page_size, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_prefill_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                                      page_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), B, Tq,
                                                      Hq, Hkv, d, num_pages, page_size, max_pages, scale, dt,
                                                      out.data_ptr(), _addr(lse), ws.data_ptr(), ws.nbytes,
                                                      _raw_stream(dev))
    _check(code, "msa_full_attn_prefill_paged")
    return out


def msa_full_attn_backward(q, k, v, out, dout, lse, cu_q, cu_k, dq=None, dk=None, dv=None, scale=0.0, ws=None,
                           stream=None):
    """Gradients of msa_full_attn_prefill (see include/msa.h) from its output,
    its lse [Tq,Hq] and the output gradient ``dout``. Returns (dq, dk, dv)."""
    torch = _torch()
    shape = _rows("q", q)
    Tq, Hq, d = shape
    dev, dtype = q.get_device(), q.dtype
    other = _elsewhere(stream, dev)
    if other is not None:
        with other:
            return msa_full_attn_backward(q, k, v, out, dout, lse, cu_q, cu_k, dq, dk, dv, scale, ws)
    kshape = _rows("k", k)
    Tk, Hkv, _ = kshape
    B = cu_q.shape[0] - 1
    _need("k", k, dtype, dev, (Tk, Hkv, d))
    _need("v", v, dtype, dev, kshape)
    _need("out", out, dtype, dev, shape)
    _need("dout", dout, dtype, dev, shape)
    if dq is not None:
        _need("dq", dq, dtype, dev, shape)
    if dk is not None:
        _need("dk", dk, dtype, dev, kshape)
    if dv is not None:
        _need("dv", dv, dtype, dev, kshape)
    _need("cu_q", cu_q, torch.int32, dev, (B + 1,))
    _need("cu_k", cu_k, torch.int32, dev, (B + 1,))
    _need("lse", lse, torch.float32, dev, (Tq, Hq))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dt = _dtype_code(q)
    ws = _full_ws(ws, q, MSA_OP_FULL_BACKWARD, B, Tq, Tk, Hkv, Hq, d, dt)
    code = load_library().msa_full_attn_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                 dout.data_ptr(), lse.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), B,
                                                 Tq, Tk, Hq, Hkv, d, scale, dt, dq.data_ptr(), dk.data_ptr(),
                                                 dv.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(dev))
    _check(code, "msa_full_attn_backward")
    return dq, dk, dv
