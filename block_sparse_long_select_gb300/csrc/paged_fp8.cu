// Paged caches in 8 bits: new tokens' keys and values written as e4m3 codes with
// a scale per (token, head), and cached rows read back.
//
//   y: a head's row of d values (keys: rotated, see paged_append.cu), in fp32
//   scale = the smallest power of two >= 2^-126 with max|y| / scale <= 448
//   code = e4m3(y / scale), to nearest even;   the row stands for code * scale
// A power of two divides exactly, so a code is one rounding of y: at most half
// a step, 2^-4 of it (2^-10 scale below 2^-6 scale). e4m3's own exponent
// covers 2^-6 to 448, so that the finest scale max|y| / 448 would not round the
// larger values of a row less. A row of zeros has scale 0; one with an infinity
// or NaN (also of the rotation) has scale NaN, so that it stands out wherever it is read.
// Whether a key lies on one side of a code's border or the other must not depend
// on the order of two roundings: keys are rotated with the products' and sums'
// errors carried along and rounded to fp32 once.
//
// Append: streaming, bound by HBM. A lane holds two 16-byte chunks of a head's
// row, which are both halves of its pairs; a lane's pairs are the same for every
// row of the token, so their cosines are loaded once, and the row's maximum takes
// log2(d e / 32) exchanges. Many tokens: a warp each, so that the search for the
// sequence and the rotation's loads are a warp's; few (a decode step): a CTA each,
// so that all loads are in flight at once. Measured (Hq 32, Hkv 8, d 128, bf16):
// 20924 tokens 82 us, 5.8 TB/s (85 % of the copy rate; 196 with a thread per pair
// of elements, 90 without rows loaded ahead); 64 single tokens 4 us, latency.
// Read: streaming, bound by HBM. A CTA has up to 16 packed rows, whose cache rows
// as many threads look up at once; a thread's unit is 16 codes, whose values it
// stores in whole 32-byte sectors. Measured (the same heads): 4 sequences of 8 K to
// 16 K rows 45 us, 5.9 TB/s; 64 single rows 3.4 us, latency.
#include <algorithm>

#include "full_internal.cuh"

namespace msa {
namespace {

// Up to kAppFewTokens tokens get a CTA each. Single tokens, a CTA : a warp for each, us:
//   tokens               64         304         608         912        1216        4864
//   bf16 32/8/128    4.0 : 6.3   8.3 : 8.1  13.9 : 8.4  19.4 : 9.3  25.1 : 9.5  102 : 26
//   fp32 8/2/64      3.4 : 4.1   5.2 : 5.6   5.4 : 5.8   5.6 : 6.1   6.0 : 6.2   14 : 9
//   fp32 32/8/128    3.8 : 9.7   6.1 : 12    9.1 : 12     12 : 13     15 : 13    65 : 44
// One limit for all; bf16 rows of many heads would be best off with about 300.
constexpr int kAppThreads = 128, kAppMostThreads = 512, kAppFewTokens = 4 * kNumSMs;
constexpr int kReadThreads = 256, kReadRows = 16;

// x / d, exact while x d is below 2^32, by the rounded-up reciprocal 2^32 / d
struct SmallDiv {
  uint32_t m, d;
  __host__ __device__ explicit SmallDiv(int n) : m(n > 1 ? uint32_t(0x100000000ull / uint32_t(n)) + 1u : 0u), d(n) {}
  __device__ __forceinline__ int of(int x) const { return d == 1 ? x : int(__umulhi(uint32_t(x), m)); }
};

// a b + c d, rounded to fp32 once but for errors below 2^-45 of the larger product:
// Dekker's exact products (by FMA) and Knuth's exact sum
__device__ __forceinline__ float dot2(float a, float b, float c, float d) {
  const float p = __fmul_rn(a, b), q = __fmul_rn(c, d);
  const float ep = __fmaf_rn(a, b, -p), eq = __fmaf_rn(c, d, -q);  // exact errors of the products
  const float s = __fadd_rn(p, q), t = __fsub_rn(s, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t));  // exact error of their sum
  return __fadd_rn(s, __fadd_rn(es, __fadd_rn(ep, eq)));
}

// two codes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// rows by cu_new; lengths are looked at token by token
__host__ __device__ SeqMap seqs_of(const AppendArgs& a) { return SeqMap{a.cu_new, nullptr, a.kv_len, a.B, a.T, 0}; }

// The cache row of a packed token: page * page_size + row, -1 if it is out of range.
__device__ __forceinline__ int64_t cache_row(const PageMap& m, int b, int64_t pos) {
  if (pos < 0 || pos >= int64_t(m.max_pages) << m.page_log2) return -1;
  const int page = m.table[int64_t(b) * m.max_pages + (pos >> m.page_log2)];
  if (page < 0 || page >= m.num_pages) return -1;
  return (int64_t(page) << m.page_log2) + (pos & ((1 << m.page_log2) - 1));
}

// A lane's two chunks of a row, as fp32.
template <typename T>
struct TwoChunks {
  static constexpr int N = 16 / int(sizeof(T));
  uint4 raw[2];
  float x[2][N];
  __device__ __forceinline__ void load(const T* row, int c0, int c1) {
    raw[0] = reinterpret_cast<const uint4*>(row)[c0];
    raw[1] = reinterpret_cast<const uint4*>(row)[c1];
  }
  __device__ __forceinline__ void clear() { raw[0] = raw[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void widen() {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const T* e = reinterpret_cast<const T*>(&raw[y]);
#pragma unroll
      for (int i = 0; i < N; ++i) x[y][i] = to_f(e[i]);
    }
  }
  // f(a, b, pair): the pair (a, b) and its number among the lane's N
  template <bool IL, typename F>
  __device__ __forceinline__ void pairs(F f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (IL)
        f(x[2 * i / N][2 * i % N], x[2 * i / N][2 * i % N + 1], i);
      else
        f(x[0][i], x[1][i], i);
    }
  }
};

template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kAppMostThreads)
    paged_append_fp8_kernel(const AppendArgs a, float* __restrict__ k_scale, float* __restrict__ v_scale, bool few) {
  constexpr int N = 16 / int(sizeof(T)), L = D / N / 2, kPer = 32 / L;  // elements of a chunk, lanes of a row, rows of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = few ? blockIdx.x : blockIdx.x * (kAppThreads / 32) + warp;
  const int me = few ? warp : 0, warps = few ? blockDim.x >> 5 : 1;  // of the token's warps
  const int sub = lane / L, j = lane % L;
  const int half = a.rot / 2 / N;  // chunks of half the rotated dims
  const int c0 = j < half ? j : 2 * j, c1 = j < half ? j + half : 2 * j + 1;
  // Passes of kPer rows: queries, keys, values. A batch is loaded while the one
  // before it is worked on, and the first while the token's place is looked up.
  const int nq = a.q ? (a.Hq + kPer - 1) / kPer : 0, nk = (a.Hkv + kPer - 1) / kPer, passes = nq + 2 * nk;
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  auto fetch = [&](TwoChunks<T>(&v)[kBatch], int p0) {
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int p = p0 + y * warps;
      const bool is_q = p < nq, is_k = !is_q && p < nq + nk;
      const int h = (p - (is_q ? 0 : is_k ? nq : nq + nk)) * kPer + sub, heads = is_q ? a.Hq : a.Hkv;
      if (p < passes && h < heads)
        v[y].load(static_cast<const T*>(is_q ? a.q : is_k ? a.k_new : a.v_new) + (int64_t(t) * heads + h) * D, c0, c1);
      else
        v[y].clear();
    }
  };
  TwoChunks<T> next[kBatch];
  if (t < a.T) fetch(next, me);
  int b = t;
  if (a.cu_new) {  // every warp finds its token's sequence itself
    const SeqMap m = seqs_of(a);
    if (cta_in_order(m, &a.ws->disorder)) {
      b = t < a.T ? find_row_seq(a.cu_new, a.B, t) : -1;
    } else {
      if (threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
      b = t < a.T ? scan_row_seq(m, false, t) : -1;
    }
  }
  if (b < 0 || t >= a.T) return;
  const int last = a.cu_new ? a.cu_new[b + 1] : t + 1;
  const int64_t pos = int64_t(a.kv_len[b]) - (last - t);
  const int64_t row = a.rot == 0 || pos < a.max_pos ? cache_row(a.pages, b, pos) : -1;
  if (row < 0 && me == 0 && lane == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);

  const bool turns = j < half && row >= 0;
  float cc[N], ss[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cc[i] = 1.f, ss[i] = 0.f;
  if (turns) {
    const float* cs = a.rope + pos * a.rot;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {  // two pairs each: c0 N + 2 i, or of either chunk
      const float4 f = __ldg(reinterpret_cast<const float4*>(cs) +
                             (!IL ? c0 * (N / 2) + i : i < N / 4 ? c0 * (N / 4) + i : c1 * (N / 4) + i - N / 4));
      cc[2 * i] = f.x;
      ss[2 * i] = f.y;
      cc[2 * i + 1] = f.z;
      ss[2 * i + 1] = f.w;
    }
  }
  const int64_t page = row >> a.pages.page_log2, in_page = row & ((1 << a.pages.page_log2) - 1);
  for (int p0 = me; p0 < passes; p0 += kBatch * warps) {
    TwoChunks<T> v[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) v[y].raw[0] = next[y].raw[0], v[y].raw[1] = next[y].raw[1];
    if (p0 + kBatch * warps < passes) fetch(next, p0 + kBatch * warps);
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int p = p0 + y * warps;  // one kind of rows for the whole warp
      if (p >= passes) break;
      if (p < nq) {  // ---- queries ----
        const int r = p * kPer + sub;
        if (r >= a.Hq) continue;
        if (row < 0) v[y].clear();
        if (turns) {
          v[y].widen();
          v[y].template pairs<IL>([&](float& p, float& q, int i) {
            const float x = p * cc[i] - q * ss[i];
            q = q * cc[i] + p * ss[i];
            p = x;
          });
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            T* w = reinterpret_cast<T*>(&v[y].raw[z]);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = from_f<T>(v[y].x[z][i]);
          }
        }
        T* dst = static_cast<T*>(a.q_out) + (int64_t(t) * a.Hq + r) * D;
        reinterpret_cast<uint4*>(dst)[c0] = v[y].raw[0];
        reinterpret_cast<uint4*>(dst)[c1] = v[y].raw[1];
        continue;
      }
      // ---- keys and values ----
      if (row < 0) return;
      const bool is_k = p < nq + nk;
      const int h = (p - (is_k ? nq : nq + nk)) * kPer + sub;
      v[y].widen();
      if (is_k && half > 0)  // the warp's; lanes that do not turn have cos 1, sin 0
        v[y].template pairs<IL>([&](float& p, float& q, int i) {
          const float x = dot2(p, cc[i], q, -ss[i]);
          q = dot2(q, cc[i], p, ss[i]);
          p = x;
        });
      uint32_t top = 0;  // as bits: a NaN is above infinity above all else
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[y].x[z][i]) & 0x7fffffffu);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (h >= a.Hkv) continue;
      // 448 = 1.75 * 2^8: the exponent field of top, one more if its fraction is above 1.75, less 8
      const uint32_t field = max(int((top + 0x1fffffu) >> 23) - 8, 1);
      const bool fine = top < 0x7f800000u;
      const float inv = fine ? __uint_as_float((254u - field) << 23) : 0.f;  // satfinite: codes of a row of scale NaN mean nothing
      uint8_t* dst = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + (row * a.Hkv + h) * D;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float* x = v[y].x[z];
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
          w[i] = e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
        uint8_t* to = dst + (z ? c1 : c0) * N;
        if constexpr (N == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(to) = w[0];
      }
      if (j == 0)
        (is_k ? k_scale : v_scale)[((page * a.Hkv + h) << a.pages.page_log2) + in_page] =
            !fine ? __uint_as_float(0x7fc00000u) : top == 0 ? 0.f : __uint_as_float(field << 23);
    }
  }
}

template <typename T, int D>
cudaError_t append(const AppendArgs& a, float* k_scale, float* v_scale, cudaStream_t stream) {
  constexpr int L = D * int(sizeof(T)) / 32, kPer = 32 / L;
  const bool few = a.T <= kAppFewTokens;
  const int total = (((a.q ? a.Hq : 0) + kPer - 1) / kPer + 2 * ((a.Hkv + kPer - 1) / kPer)) * 32;
  const int threads = !few ? kAppThreads : total < kAppMostThreads ? total : kAppMostThreads;
  if (a.cu_new)
    if (cudaError_t e = launch_order_check(seqs_of(a), a.ws, stream)) return e;
  ProfScope pf("paged_append_fp8", stream);
  auto kern = a.interleaved ? paged_append_fp8_kernel<T, D, true> : paged_append_fp8_kernel<T, D, false>;
  kern<<<few ? a.T : (a.T + kAppThreads / 32 - 1) / (kAppThreads / 32), threads, 0, stream>>>(a, k_scale, v_scale, few);
  return cudaGetLastError();
}

__host__ __device__ SeqMap seqs_of(const ReadArgs& a) { return SeqMap{a.cu, nullptr, a.kv_len, a.B, a.T, 0}; }

// Eight words to global memory: one whole sector
__device__ __forceinline__ void store8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// code * scale as bf16, rounded once. The product has up to 28 bits, so by way of fp32
// it would be rounded twice. It goes by the next fp32 number towards 0 instead, whose
// last bit is set if the product lies beyond it (rounding to odd): bf16 then rounds to
// the side on which the product is.
template <typename T>
__device__ __forceinline__ T rounded_once(float code, float scale) {
  const float a = fabsf(code), b = fabsf(scale), near = __fmul_rz(a, b);
  const uint32_t beyond = __fmaf_ru(a, b, -near) > 0.f ? 1u : 0u;  // also of what is below the least step; not of NaN
  const uint32_t sign = (__float_as_uint(code) ^ __float_as_uint(scale)) & 0x80000000u;
  return from_f<T>(__uint_as_float(__float_as_uint(near) | beyond | sign));
}

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) paged_read_fp8_kernel(const ReadArgs a, int rows, const SmallDiv by_heads, bool sectors) {
  constexpr int N = 16, L = D / N;          // codes of a unit, units of a head's row
  __shared__ int64_t row_s[kReadRows];      // cache row; -1: out of range, -2: nobody's
  const int t0 = blockIdx.x * rows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool in_order = !a.cu || cta_in_order(seqs_of(a), &a.ws->disorder);
  auto look = [&](int t, int b) {
    if (b < 0) return int64_t(-2);
    const int64_t row = cache_row(a.pages, b, int64_t(a.kv_len[b]) - ((a.cu ? a.cu[b + 1] : t + 1) - t));
    if (row < 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
    return row;
  };
  if (in_order) {
    const int t = t0 + int(threadIdx.x);
    if (threadIdx.x < rows) {
      int b = t < a.T ? t : -1;
      if (a.cu && t < a.T) {  // the last sequence that starts at or before t
        int n = a.B;
        b = 0;
        while (n > 1) {
          const int mid = n / 2;
          if (a.cu[b + mid] <= t) {
            b += mid;
            n -= mid;
          } else {
            n = mid;
          }
        }
        if (a.cu[b] > t || t >= a.cu[b + 1]) b = -1;
      }
      row_s[threadIdx.x] = look(t, b);
    }
  } else {
    if (threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
    for (int x = warp; x < rows; x += kReadThreads / 32) {
      const int t = t0 + x, b = t < a.T ? scan_row_seq(seqs_of(a), false, t) : -1;
      if (lane == 0) row_s[x] = look(t, b);
    }
  }
  __syncthreads();
  const int heads = 2 * a.Hkv, c = threadIdx.x % L;
  constexpr int kBatch = 4, kStep = kReadThreads / L;  // units in flight; head rows of a pass
  const int all = rows * heads;
  for (int r0 = threadIdx.x / L; r0 < all; r0 += kBatch * kStep) {
    uint4 code[kBatch];
    float scale[kBatch];
    T* to[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = min(r0 + y * kStep, all - 1);
      int x = by_heads.of(r);
      x -= x * heads > r;  // beyond 8192 key/value heads the reciprocal's quotient can be one too large
      const int hh = r - x * heads;
      const bool is_v = hh >= a.Hkv;
      const int h = is_v ? hh - a.Hkv : hh;
      const int64_t row = row_s[x], src = max(row, int64_t(0));
      code[y] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                                                     (src * a.Hkv + h) * D) + c);
      const int64_t s = (((src >> a.pages.page_log2) * a.Hkv + h) << a.pages.page_log2) + (src & ((1 << a.pages.page_log2) - 1));
      scale[y] = __ldg((is_v ? a.v_scale : a.k_scale) + s);
      if (row < 0) {  // out of range: zeros
        scale[y] = 0.f;
        code[y] = make_uint4(0, 0, 0, 0);
      }
      to[y] = row == -2 || r0 + y * kStep >= all
                  ? nullptr
                  : static_cast<T*>(is_v ? a.v_out : a.k_out) + (int64_t(t0 + x) * a.Hkv + h) * D + c * N;
    }
    auto store = [&](auto value) {
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (!to[y]) continue;
        const uint32_t w[4] = {code[y].x, code[y].y, code[y].z, code[y].w};
        constexpr int kWords = N * int(sizeof(T)) / 4;
        uint32_t out[kWords];
        T* o = reinterpret_cast<T*>(out);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          uint32_t f;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(uint16_t(w[i / 2] >> (16 * (i & 1)))));
          float lo, hi;
          asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(f));
          o[2 * i] = value(lo, scale[y]);
          o[2 * i + 1] = value(hi, scale[y]);
        }
#pragma unroll
        for (int i = 0; i < kWords; i += 8) {
          uint32_t* p = reinterpret_cast<uint32_t*>(to[y]) + i;
          if (sectors) {
            store8(p, out + i);
          } else {
            reinterpret_cast<uint4*>(p)[0] = make_uint4(out[i], out[i + 1], out[i + 2], out[i + 3]);
            reinterpret_cast<uint4*>(p)[1] = make_uint4(out[i + 4], out[i + 5], out[i + 6], out[i + 7]);
          }
        }
      }
    };
    // powers of two, as appends write them, have exact products (the longer way for all: 50 us in place of 46)
    uint32_t fraction = 0;
#pragma unroll
    for (int y = 0; y < kBatch; ++y) fraction |= __float_as_uint(scale[y]) << 9;
    if (sizeof(T) == 4 || fraction == 0)
      store([](float c, float s) { return from_f<T>(c * s); });
    else
      store([](float c, float s) { return rounded_once<T>(c, s); });
  }
}

template <typename T, int D>
cudaError_t read(const ReadArgs& a, cudaStream_t stream) {
  if (a.cu)
    if (cudaError_t e = launch_order_check(seqs_of(a), a.ws, stream)) return e;
  // fewer rows to a CTA where there would be fewer than two CTAs to an SM
  const int rows = std::max(1, std::min(kReadRows, a.T / (2 * kNumSMs)));
  const bool sectors = ((reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out)) & 31u) == 0;
  ProfScope pf("paged_read_fp8", stream);
  paged_read_fp8_kernel<T, D><<<(a.T + rows - 1) / rows, kReadThreads, 0, stream>>>(a, rows, SmallDiv(2 * a.Hkv), sectors);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append_fp8(const AppendArgs& a, float* k_scale, float* v_scale, cudaStream_t stream) {
  if (a.dtype == MSA_BF16)
    return a.d == 128 ? append<__nv_bfloat16, 128>(a, k_scale, v_scale, stream)
                      : append<__nv_bfloat16, 64>(a, k_scale, v_scale, stream);
  return a.d == 128 ? append<float, 128>(a, k_scale, v_scale, stream) : append<float, 64>(a, k_scale, v_scale, stream);
}

cudaError_t launch_paged_read_fp8(const ReadArgs& a, cudaStream_t stream) {
  if (a.dtype == MSA_BF16) return a.d == 128 ? read<__nv_bfloat16, 128>(a, stream) : read<__nv_bfloat16, 64>(a, stream);
  return a.d == 128 ? read<float, 128>(a, stream) : read<float, 64>(a, stream);
}

}  // namespace msa
