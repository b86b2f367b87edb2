// What a decoding warp does with 16 keys of a bf16 or fp32 cache.
#pragma once

#include "full_decode.cuh"

namespace msa {
namespace {

// Sixteen rows of K and of V of one head, 16-byte chunks, into a stage; rows from `valid` on arrive as zeros.
template <typename T, int D>
__device__ __forceinline__ void copy_rows(const void* k, const void* v, uint32_t dst, int64_t row0, int Hkv, int g, int valid) {
  constexpr int kCpr = D * int(sizeof(T)) / 16, kRow = D * int(sizeof(T)), kTile = kSub * kRow;
  const int lane = threadIdx.x & 31;
  const T* kp = static_cast<const T*>(k) + (row0 * Hkv + g) * D;
  const T* vp = static_cast<const T*>(v) + (row0 * Hkv + g) * D;
#pragma unroll
  for (int x = lane; x < kSub * kCpr; x += 32) {
    const int r = x / kCpr, c = x % kCpr;
    const bool in = r < valid;
    const int64_t off = in ? int64_t(r) * Hkv * D + c * (16 / int(sizeof(T))) : 0;
    cp16z(chunk_at(dst, kRow, r, c), kp + off, in);
  }
#pragma unroll
  for (int x = lane; x < kSub * kCpr; x += 32) {
    const int r = x / kCpr, c = x % kCpr;
    const bool in = r < valid;
    const int64_t off = in ? int64_t(r) * Hkv * D + c * (16 / int(sizeof(T))) : 0;
    cp16z(chunk_at(dst + kTile, kRow, r, c), vp + off, in);
  }
}

// ---- a warp's state: bf16 ------------------------------------------------------
// O^T (head dims along M) and the scores share the column = head layout: lane
// (gq = lane / 4, tq = lane % 4) holds heads 2 tq and 2 tq + 1 of each tile of 8.
template <typename T_, int D, int H>  // H: most heads of an item
struct Core;

template <int D, int H>
struct Core<__nv_bfloat16, D, H> {
  using T = __nv_bfloat16;
  using Params = FdParams;
  static constexpr bool kBulk = false;
  static constexpr int kD = D, kTiles = 1, kWarps = 8, kStages = D == 64 ? (H <= 8 ? 6 : 4) : H <= 8 ? 3 : 2;
  static constexpr int HN = (H + 7) / 8;
  static constexpr int kRow = D * 2, kTile = kSub * kRow, kStage = 2 * kTile, kExtra = 0;
  static constexpr int kM = 2 * HN, kAcc = HN * D / 4;
  uint32_t qf[HN][D / 16][2];
  float m[kM], l[kM], acc[kAcc];  // acc[(t * D / 16 + mt) * 4 + e]
  float nm[kM];                   // -m, 0 as long as that is -inf

  __device__ __forceinline__ static void copy(const FdParams& p, uint32_t dst, int page, int row, int g, int valid) {
    copy_rows<T, D>(p.k, p.v, dst, (int64_t(page) << p.pages.page_log2) + (valid > 0 ? row : 0), p.Hkv, g, valid);
  }
  __device__ __forceinline__ void start(const FdParams&, const T* q, int heads, uint32_t) {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < HN; ++t) {
      const T* qh = q + (t * 8 + gq) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          qf[t][ks][x] = t * 8 + gq < heads ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + 2 * tq + 8 * x) : 0u;
    }
#pragma unroll
    for (int x = 0; x < kM; ++x) m[x] = -INFINITY, l[x] = nm[x] = 0.f;
#pragma unroll
    for (int x = 0; x < kAcc; ++x) acc[x] = 0.f;
  }
  __device__ __forceinline__ void step(const Params& p, uint32_t kt, uint32_t, int, int valid) {
    const float scale_log2 = p.scale_log2;
    const int lane = threadIdx.x & 31, gq = lane >> 2;
    const uint32_t vt = kt + kTile;
    float s[HN][4];
#pragma unroll
    for (int t = 0; t < HN; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      ldm4(chunk_at(kt, kRow, (lane & 7) + 8 * ((lane >> 3) & 1), ks * 2 + (lane >> 4)), a);
#pragma unroll
      for (int t = 0; t < HN; ++t) mma16816(s[t], a, qf[t][ks][0], qf[t][ks][1]);
    }
    float mt[kM];
    bool up = false;
#pragma unroll
    for (int t = 0; t < HN; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = gq + 8 * (e >> 1) < valid ? s[t][e] * scale_log2 : -INFINITY;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mt[2 * t + x] = fmaxf(s[t][x], s[t][2 + x]);
        up |= mt[2 * t + x] > m[2 * t + x] + kFdLazy;
      }
    }
    // the maxima are only looked for across the lanes when some score is beyond 2^8 of its own
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int t = 0; t < HN; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = 2 * t + x;
          const float mn = fmaxf(m[i], qmax(mt[i]));
          const float a = mn == m[i] ? 1.f : ex2d(m[i] - mn);
          m[i] = mn;
          nm[i] = mn == -INFINITY ? 0.f : -mn;
          l[i] *= a;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            acc[(t * (D / 16) + k) * 4 + x] *= a;
            acc[(t * (D / 16) + k) * 4 + 2 + x] *= a;
          }
        }
    }
    uint32_t b[HN][2];
#pragma unroll
    for (int t = 0; t < HN; ++t) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = ex2d(s[t][e] + nm[2 * t + (e & 1)]);
        l[2 * t + (e & 1)] += p[e];  // unrounded; the product below takes bf16 weights
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(p[0], p[1]), hi = __floats2bfloat162_rn(p[2], p[3]);
      b[t][0] = trans8(reinterpret_cast<const uint32_t&>(lo));
      b[t][1] = trans8(reinterpret_cast<const uint32_t&>(hi));
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[4];
      const int mi = lane >> 3;
      ldm4t(chunk_at(vt, kRow, (lane & 7) + 8 * (mi >> 1), k * 2 + (mi & 1)), a);
#pragma unroll
      for (int t = 0; t < HN; ++t) {
        float(&c)[4] = reinterpret_cast<float(&)[4]>(acc[(t * (D / 16) + k) * 4]);
        mma16816(c, a, b[t][0], b[t][1]);
      }
    }
  }
  // f(head, index of its maximum, dim, value) for all that this lane holds
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < HN; ++t)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(t * 8 + 2 * tq + (e & 1), 2 * t + (e & 1), k * 16 + gq + 8 * (e >> 1), acc[(t * (D / 16) + k) * 4 + e]);
  }
  __device__ __forceinline__ void finish() {}  // before the state is joined with others
  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int x = 0; x < kM; ++x) l[x] = qsum(l[x]);
  }
  // f(head, index): the heads whose maximum and sum this lane reports
  template <typename F>
  __device__ __forceinline__ void each_head(F f) const {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
    if (gq == 0) {
#pragma unroll
      for (int x = 0; x < kM; ++x) f((x >> 1) * 8 + 2 * tq + (x & 1), x);
    }
  }
  __device__ __forceinline__ static int m_index(int x) { return 2 * (x / (D / 4)) + (x & 1); }  // acc[x]'s head
};

// ---- a warp's state: fp32 ------------------------------------------------------
// Scores: lane pair (lane, lane ^ 16) shares key lane & 15, half the dims each.
// Products: lane holds D / 32 dims of every head. Maxima are equal in all lanes.
template <int D, int H>
struct Core<float, D, H> {
  using T = float;
  static constexpr bool kWide = D == 128;
  using Params = FdParams;
  static constexpr bool kBulk = false;
  static constexpr int kD = D, kTiles = 1, kWarps = kWide ? 4 : 8, kStages = kWide ? 2 : H <= 4 ? 3 : 2;
  static constexpr int P = D / 32;
  static constexpr int kRow = D * 4, kTile = kSub * kRow, kStage = 2 * kTile;
  static constexpr int kExtra = (H * D + kSub * H) * 4;  // per warp: queries, weights
  static constexpr int kM = H, kAcc = H * P;
  float m[kM], l[kM], acc[kAcc];  // acc[h * P + x]

  __device__ __forceinline__ static void copy(const FdParams& p, uint32_t dst, int page, int row, int g, int valid) {
    copy_rows<T, D>(p.k, p.v, dst, (int64_t(page) << p.pages.page_log2) + (valid > 0 ? row : 0), p.Hkv, g, valid);
  }
  __device__ __forceinline__ void start(const FdParams&, const T* q, int heads, uint32_t extra) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int x = lane; x < H * D; x += 32) {
      const float v = x / D < heads ? q[x] : 0.f;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(extra + x * 4), "f"(v) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kM; ++x) m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
    for (int x = 0; x < kAcc; ++x) acc[x] = 0.f;
  }
  __device__ __forceinline__ static float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
  }
  __device__ __forceinline__ void step(const Params& p, uint32_t kt, uint32_t extra, int, int valid) {
    const float scale_log2 = p.scale_log2;
    const int lane = threadIdx.x & 31, key = lane & 15, half = lane >> 4;
    const uint32_t vt = kt + kTile, ps = extra + H * D * 4;
    float s[H];
#pragma unroll
    for (int h = 0; h < H; ++h) s[h] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const int ch = half * (D / 8) + c;
      const float4 k4 = lds4(chunk_at(kt, kRow, key, ch));
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float4 q4 = lds4(extra + (h * D + ch * 4) * 4);
        s[h] = fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, fmaf(k4.w, q4.w, s[h]))));
      }
    }
    bool up = false;
    float mt[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      s[h] += __shfl_xor_sync(0xffffffffu, s[h], 16);
      s[h] = key < valid ? s[h] * scale_log2 : -INFINITY;
      mt[h] = tc::warp_max_f32(s[h]);
      up |= mt[h] > m[h] + kFdLazy || (m[h] == -INFINITY && mt[h] > -INFINITY);
    }
    if (up) {  // equal in all lanes
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float mn = fmaxf(m[h], mt[h]);
        const float a = mn == m[h] ? 1.f : ex2d(m[h] - mn);
        m[h] = mn;
        l[h] *= a;
#pragma unroll
        for (int x = 0; x < P; ++x) acc[h * P + x] *= a;
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float p = ex2d(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      if (half == 0) {
        l[h] += p;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(ps + (key * H + h) * 4), "f"(p) : "memory");
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < kSub; ++j) {
      float v[P];
      if constexpr (P == 4) {
        const float4 v4 = lds4(chunk_at(vt, kRow, j, lane));
        v[0] = v4.x, v[1] = v4.y, v[2] = v4.z, v[3] = v4.w;
      } else {
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v[0]), "=f"(v[1])
                     : "r"(chunk_at(vt, kRow, j, lane >> 1) + (lane & 1) * 8));
      }
#pragma unroll
      for (int h4 = 0; h4 < H / 4; ++h4) {
        const float4 p4 = lds4(ps + (j * H + h4 * 4) * 4);
        const float pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < P; ++x) acc[(h4 * 4 + y) * P + x] = fmaf(pp[y], v[x], acc[(h4 * 4 + y) * P + x]);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int x = 0; x < P; ++x) f(h, h, lane * P + x, acc[h * P + x]);
  }
  __device__ __forceinline__ void finish() {}  // before the state is joined with others
  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
  }
  template <typename F>
  __device__ __forceinline__ void each_head(F f) const {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int h = 0; h < H; ++h) f(h, h);
    }
  }
  __device__ __forceinline__ static int m_index(int x) { return x / P; }
};

}  // namespace
}  // namespace msa
