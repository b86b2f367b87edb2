// C ABI of the full-attention and paged-cache operators: host-side checks and
// dispatch. Every entry point is asynchronous on its stream.
#include <algorithm>
#include <cmath>

#include "full_internal.cuh"

namespace msa {
namespace {

bool full_dtype_ok(int dtype) { return dtype == MSA_BF16 || dtype == MSA_FP32; }

// Heads, head dim and element type, shared by every entry point.
msa_status_t check_heads(int Hq, int Hkv, int d, int dtype) {
  if (Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0 || !full_dtype_ok(dtype)) return MSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq / Hkv > kMaxFullHpg || Hq > kMaxFullHeads) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

// rows * heads * d elements must stay countable: row and head indices are 32-bit
bool rows_ok(int64_t rows, int heads) { return rows * heads < (int64_t(1) << 31); }

msa_status_t check_pages(int num_pages, int page_size, int max_pages, PageMap* pm) {
  if (num_pages < 1 || max_pages < 1 || page_size < 1) return MSA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return MSA_ERR_UNSUPPORTED;
  // key positions and cache rows are 32-bit (TMA coordinates), with room for a tile behind the last
  if (int64_t(max_pages) * page_size > (int64_t(1) << 30) || int64_t(num_pages) * page_size > (int64_t(1) << 30))
    return MSA_ERR_UNSUPPORTED;
  pm->num_pages = num_pages;
  pm->max_pages = max_pages;
  pm->page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  return MSA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

msa_status_t check_full_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return MSA_ERR_UNSUPPORTED;  // sizes that msa_workspace_size refuses
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need) return MSA_ERR_WORKSPACE;
  return MSA_OK;
}

inline msa_status_t launched(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }
// Prefill: tensor cores for bf16, CUDA cores for fp32. With no key at all
// (Tk == 0) there is nothing to map for TMA: the rows are empty.
cudaError_t prefill(const FullArgs& a, cudaStream_t stream) {
  if (a.seq.Tk == 0)
    return launch_full_zero(a.seq, false, a.Hq, a.d, a.dtype, a.out, nullptr, a.lse, a.ws, stream);
  return a.dtype == MSA_BF16 ? launch_full_prefill_tc(a, stream) : launch_full_f32(a, stream);
}

inline float scale_or_default(float scale, int d) { return scale > 0.f ? scale : 1.0f / sqrtf(float(d)); }

// An append's checks and arguments, for caches of any element type.
msa_status_t check_append(AppendArgs& a, bool& empty, const void* q, const void* k_new, const void* v_new,
                          const float* rope, const int32_t* cu_new, const int32_t* kv_len, const int32_t* page_table,
                          int B, int T, int Hq, int Hkv, int d, int rot, int interleaved, int max_pos, int num_pages,
                          int page_size, int max_pages, int dtype, void* q_out, void* k_cache, void* v_cache, void* ws,
                          size_t ws_bytes) {
  empty = false;
  msa_status_t st = check_heads(Hq, Hkv, d, dtype);
  if (st == MSA_OK) st = check_pages(num_pages, page_size, max_pages, &a.pages);
  if (st != MSA_OK) return st;
  if (B < 0 || T < 0 || rot < 0 || rot > d || (interleaved != 0 && interleaved != 1)) return MSA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return MSA_ERR_UNSUPPORTED;
  if (!rows_ok(T, Hq)) return MSA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) {
    empty = true;
    return MSA_OK;
  }
  if (!cu_new && T != B) return MSA_ERR_INVALID_ARG;
  if (!k_new || !v_new || !kv_len || !page_table || !k_cache || !v_cache || (!q) != (!q_out)) return MSA_ERR_INVALID_ARG;
  if (rot > 0 && (!rope || max_pos < 1)) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(rope) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return MSA_ERR_INVALID_ARG;
  st = check_full_ws(ws, ws_bytes, kWsHeader);
  if (st != MSA_OK) return st;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.rope = rot > 0 ? rope : nullptr;
  a.cu_new = cu_new;
  a.kv_len = kv_len;
  a.pages.table = page_table;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.rot = rot;
  a.interleaved = interleaved;
  a.max_pos = max_pos;
  a.dtype = dtype;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ws = static_cast<WsHeader*>(ws);
  return MSA_OK;
}

// A decode's checks and arguments, but for its workspace.
msa_status_t check_decode(FullArgs& a, bool& empty, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* page_table, const int32_t* kv_len, int B, int Hq, int Hkv, int d, int num_pages,
                          int page_size, int max_pages, float scale, int dtype, void* out, float* lse) {
  empty = false;
  msa_status_t st = check_heads(Hq, Hkv, d, dtype);
  if (st == MSA_OK) st = check_pages(num_pages, page_size, max_pages, &a.pages);
  if (st != MSA_OK) return st;
  if (B < 0) return MSA_ERR_INVALID_ARG;
  if (!rows_ok(B, Hq)) return MSA_ERR_UNSUPPORTED;
  if (B == 0) {
    empty = true;
    return MSA_OK;
  }
  if (!q || !k_cache || !v_cache || !page_table || !kv_len || !out) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return MSA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.seq = {nullptr, nullptr, kv_len, B, B, max_pages * page_size};
  a.pages.table = page_table;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.dtype = dtype;
  a.scale = scale_or_default(scale, d);
  a.out = out;
  a.lse = lse;
  return MSA_OK;
}

}  // namespace

size_t full_ws_bytes(int op, int B, int Nq, int Nk, int Hkv, int Hq, int d, int dtype) {
  if (B < 1 || Nk < 0 || check_heads(Hq, Hkv, d, dtype) != MSA_OK) return 0;
  if (op == MSA_OP_FULL_DECODE) return rows_ok(B, Hq) ? kWsHeader + full_decode_ws_bytes(d) : 0;
  if (op == MSA_OP_FULL_DECODE_FP8)
    return rows_ok(B, Hq) ? kWsHeader + full_decode_fp8_ws_bytes(Hkv, Hq / Hkv, d, dtype) : 0;
  if (op == MSA_OP_FULL_DECODE_SHARED) {
    if (!rows_ok(B, Hq) || Nq < 0 || Nq > B) return 0;
    return kWsHeader + (Nq == 0 ? full_decode_ws_bytes(d) : full_shared_ws_bytes(B, Nq, Hkv, Hq / Hkv, d, dtype));
  }
  if (Nq < 0 || !rows_ok(Nq, Hq) || (op == MSA_OP_FULL_BACKWARD && !rows_ok(Nk, Hkv))) return 0;
  if (op == MSA_OP_FULL_PREFILL && dtype == MSA_BF16) return kWsHeader + full_prefill_ws_bytes(d, Nk);
  if (op == MSA_OP_FULL_BACKWARD) return kWsHeader + full_backward_ws_bytes(Nq, Hq);
  return kWsHeader;
}

}  // namespace msa

using namespace msa;

extern "C" msa_status_t msa_paged_append(const void* q, const void* k_new, const void* v_new, const float* rope,
                                         const int32_t* cu_new, const int32_t* kv_len, const int32_t* page_table,
                                         int B, int T, int Hq, int Hkv, int d, int rot, int interleaved, int max_pos,
                                         int num_pages, int page_size, int max_pages, int dtype, void* q_out,
                                         void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                                         cudaStream_t stream) {
  AppendArgs a{};
  bool empty;
  const msa_status_t st = check_append(a, empty, q, k_new, v_new, rope, cu_new, kv_len, page_table, B, T, Hq, Hkv, d, rot,
                                       interleaved, max_pos, num_pages, page_size, max_pages, dtype, q_out, k_cache,
                                       v_cache, ws, ws_bytes);
  return st != MSA_OK || empty ? st : launched(launch_paged_append(a, stream));
}

extern "C" msa_status_t msa_paged_append_fp8(const void* q, const void* k_new, const void* v_new, const float* rope,
                                             const int32_t* cu_new, const int32_t* kv_len, const int32_t* page_table,
                                             int B, int T, int Hq, int Hkv, int d, int rot, int interleaved,
                                             int max_pos, int num_pages, int page_size, int max_pages, int dtype,
                                             void* q_out, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  AppendArgs a{};
  bool empty;
  const msa_status_t st = check_append(a, empty, q, k_new, v_new, rope, cu_new, kv_len, page_table, B, T, Hq, Hkv, d, rot,
                                       interleaved, max_pos, num_pages, page_size, max_pages, dtype, q_out, k_cache,
                                       v_cache, ws, ws_bytes);
  if (st != MSA_OK || empty) return st;
  if (!k_scale || !v_scale || !aligned16(k_scale) || !aligned16(v_scale)) return MSA_ERR_INVALID_ARG;
  return launched(launch_paged_append_fp8(a, k_scale, v_scale, stream));
}

extern "C" msa_status_t msa_paged_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale,
                                           const float* v_scale, const int32_t* cu, const int32_t* kv_len,
                                           const int32_t* page_table, int B, int T, int Hkv, int d, int num_pages,
                                           int page_size, int max_pages, int dtype, void* k_out, void* v_out, void* ws,
                                           size_t ws_bytes, cudaStream_t stream) {
  ReadArgs a{};
  msa_status_t st = check_heads(Hkv, Hkv, d, dtype);
  if (st == MSA_OK) st = check_pages(num_pages, page_size, max_pages, &a.pages);
  if (st != MSA_OK) return st;
  if (B < 0 || T < 0) return MSA_ERR_INVALID_ARG;
  if (!rows_ok(T, Hkv)) return MSA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return MSA_OK;
  if (!cu && T != B) return MSA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !kv_len || !page_table || !k_out || !v_out) return MSA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale) || !aligned16(k_out) ||
      !aligned16(v_out))
    return MSA_ERR_INVALID_ARG;
  st = check_full_ws(ws, ws_bytes, kWsHeader);
  if (st != MSA_OK) return st;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.cu = cu;
  a.kv_len = kv_len;
  a.pages.table = page_table;
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.dtype = dtype;
  a.k_out = k_out;
  a.v_out = v_out;
  a.ws = static_cast<WsHeader*>(ws);
  return launched(launch_paged_read_fp8(a, stream));
}

extern "C" msa_status_t msa_full_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* page_table, const int32_t* kv_len, int B, int Hq, int Hkv,
                                             int d, int num_pages, int page_size, int max_pages, float scale,
                                             int dtype, void* out, float* lse, void* ws, size_t ws_bytes,
                                             cudaStream_t stream) {
  FullArgs a{};
  bool empty;
  const msa_status_t st = check_decode(a, empty, q, k_cache, v_cache, page_table, kv_len, B, Hq, Hkv, d, num_pages,
                                       page_size, max_pages, scale, dtype, out, lse);
  if (st != MSA_OK || empty) return st;
  const msa_status_t w = check_full_ws(ws, ws_bytes, kWsHeader + full_decode_ws_bytes(d));
  a.ws = ws;
  return w != MSA_OK ? w : launched(launch_full_decode(a, stream));
}

extern "C" msa_status_t msa_full_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                                                 const float* k_scale, const float* v_scale, const int32_t* page_table,
                                                 const int32_t* kv_len, int B, int Hq, int Hkv, int d, int num_pages,
                                                 int page_size, int max_pages, float scale, int dtype, void* out,
                                                 float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FullArgs a{};
  bool empty;
  const msa_status_t st = check_decode(a, empty, q, k_cache, v_cache, page_table, kv_len, B, Hq, Hkv, d, num_pages,
                                       page_size, max_pages, scale, dtype, out, lse);
  if (st != MSA_OK || empty) return st;
  if (!k_scale || !v_scale || !aligned16(k_scale) || !aligned16(v_scale)) return MSA_ERR_INVALID_ARG;
  const msa_status_t w = check_full_ws(ws, ws_bytes, kWsHeader + full_decode_fp8_ws_bytes(Hkv, Hq / Hkv, d, dtype));
  a.ws = ws;
  return w != MSA_OK ? w : launched(launch_full_decode_fp8(a, k_scale, v_scale, stream));
}

extern "C" msa_status_t msa_full_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                                    const int32_t* page_table, const int32_t* kv_len,
                                                    const int32_t* cu_prefix, const int32_t* prefix_len, int B, int P,
                                                    int Hq, int Hkv, int d, int num_pages, int page_size,
                                                    int max_pages, float scale, int dtype, void* out, float* lse,
                                                    void* ws, size_t ws_bytes, cudaStream_t stream) {
  FullArgs a{};
  bool empty;
  const msa_status_t st = check_decode(a, empty, q, k_cache, v_cache, page_table, kv_len, B, Hq, Hkv, d, num_pages,
                                       page_size, max_pages, scale, dtype, out, lse);
  if (st != MSA_OK) return st;
  if (P < 0 || P > B) return MSA_ERR_INVALID_ARG;
  if (empty) return MSA_OK;
  if (P > 0 && (!cu_prefix || !prefix_len)) return MSA_ERR_INVALID_ARG;
  const msa_status_t w = check_full_ws(
      ws, ws_bytes, full_ws_bytes(MSA_OP_FULL_DECODE_SHARED, B, P, max_pages * page_size, Hkv, Hq, d, dtype));
  if (w != MSA_OK) return w;
  a.ws = ws;
  return launched(P == 0 ? launch_full_decode(a, stream) : launch_decode_shared(a, cu_prefix, prefix_len, P, stream));
}

extern "C" msa_status_t msa_full_attn_prefill(const void* q, const void* k, const void* v, const int32_t* cu_q,
                                              const int32_t* cu_k, int B, int Tq, int Tk, int Hq, int Hkv, int d,
                                              float scale, int dtype, void* out, float* lse, void* ws,
                                              size_t ws_bytes, cudaStream_t stream) {
  msa_status_t st = check_heads(Hq, Hkv, d, dtype);
  if (st != MSA_OK) return st;
  if (B < 0 || Tq < 0 || Tk < 0) return MSA_ERR_INVALID_ARG;
  if (!rows_ok(Tq, Hq) || !rows_ok(Tk, Hkv)) return MSA_ERR_UNSUPPORTED;
  if (B == 0 || Tq == 0) return MSA_OK;
  if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v))) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return MSA_ERR_INVALID_ARG;
  st = check_full_ws(ws, ws_bytes, full_ws_bytes(MSA_OP_FULL_PREFILL, B, Tq, Tk, Hkv, Hq, d, dtype));
  if (st != MSA_OK) return st;
  FullArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.seq = {cu_q, cu_k, nullptr, B, Tq, Tk};
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.dtype = dtype;
  a.scale = scale_or_default(scale, d);
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  return launched(prefill(a, stream));
}

extern "C" msa_status_t msa_full_attn_prefill_paged(const void* q, const void* k_cache, const void* v_cache,
                                                    const int32_t* page_table, const int32_t* cu_q,
                                                    const int32_t* kv_len, int B, int Tq, int Hq, int Hkv, int d,
                                                    int num_pages, int page_size, int max_pages, float scale,
                                                    int dtype, void* out, float* lse, void* ws, size_t ws_bytes,
                                                    cudaStream_t stream) {
  FullArgs a{};
  msa_status_t st = check_heads(Hq, Hkv, d, dtype);
  if (st == MSA_OK) st = check_pages(num_pages, page_size, max_pages, &a.pages);
  if (st != MSA_OK) return st;
  if (B < 0 || Tq < 0) return MSA_ERR_INVALID_ARG;
  if (!rows_ok(Tq, Hq)) return MSA_ERR_UNSUPPORTED;
  if (B == 0 || Tq == 0) return MSA_OK;
  if (!q || !k_cache || !v_cache || !page_table || !cu_q || !kv_len || !out) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return MSA_ERR_INVALID_ARG;
  st = check_full_ws(ws, ws_bytes,
                     full_ws_bytes(MSA_OP_FULL_PREFILL, B, Tq, max_pages * page_size, Hkv, Hq, d, dtype));
  if (st != MSA_OK) return st;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.seq = {cu_q, nullptr, kv_len, B, Tq, max_pages * page_size};
  a.pages.table = page_table;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.dtype = dtype;
  a.scale = scale_or_default(scale, d);
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  return launched(prefill(a, stream));
}

extern "C" msa_status_t msa_full_attn_backward(const void* q, const void* k, const void* v, const void* out,
                                               const void* dout, const float* lse, const int32_t* cu_q,
                                               const int32_t* cu_k, int B, int Tq, int Tk, int Hq, int Hkv, int d,
                                               float scale, int dtype, void* dq, void* dk, void* dv, void* ws,
                                               size_t ws_bytes, cudaStream_t stream) {
  msa_status_t st = check_heads(Hq, Hkv, d, dtype);
  if (st != MSA_OK) return st;
  if (B < 0 || Tq < 0 || Tk < 0) return MSA_ERR_INVALID_ARG;
  if (!rows_ok(Tq, Hq) || !rows_ok(Tk, Hkv)) return MSA_ERR_UNSUPPORTED;
  if (B == 0 || (Tq == 0 && Tk == 0)) return MSA_OK;
  if (!cu_q || !cu_k) return MSA_ERR_INVALID_ARG;
  if (Tq > 0 && (!q || !out || !dout || !lse || !dq)) return MSA_ERR_INVALID_ARG;
  if (Tk > 0 && (!k || !v || !dk || !dv)) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv))
    return MSA_ERR_INVALID_ARG;
  st = check_full_ws(ws, ws_bytes, full_ws_bytes(MSA_OP_FULL_BACKWARD, B, Tq, Tk, Hkv, Hq, d, dtype));
  if (st != MSA_OK) return st;
  FullBwdArgs a{};
  a.f.q = q;
  a.f.k = k;
  a.f.v = v;
  a.f.seq = {cu_q, cu_k, nullptr, B, Tq, Tk};
  a.f.Hq = Hq;
  a.f.Hkv = Hkv;
  a.f.d = d;
  a.f.dtype = dtype;
  a.f.scale = scale_or_default(scale, d);
  a.f.out = const_cast<void*>(out);
  a.f.lse = const_cast<float*>(lse);
  a.f.ws = ws;
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  if (Tq == 0) return launched(launch_full_zero(a.f.seq, true, Hkv, d, dtype, dk, dv, nullptr, ws, stream));
  if (Tk == 0) return launched(launch_full_zero(a.f.seq, false, Hq, d, dtype, dq, nullptr, nullptr, ws, stream));
  return launched(dtype == MSA_BF16 ? launch_full_backward_tc(a, stream) : launch_full_f32_backward(a, stream));
}
