// Full attention, decode over a cache in 8 bits: keys ks_j K_j, values vs_j V_j
// with e4m3 codes K, V and a scale per (token, head).
//
//   out = sum_j exp(s_j - lse) vs_j V_j,  s_j = scale ks_j (q . K_j),  j < kv_len
//
// Bound: HBM, d + 4 bytes per key and per value where bf16 takes 2 d. Walk,
// copies and joins: full_decode.cuh.
//
// Products: mma.sync m16n8k16 in f16, which holds every e4m3 code exactly (bf16
// would as well, but the hardware converts e4m3 to f16 in one instruction for
// two). Scales stay out of the matrices: ks_j is multiplied to the finished
// score; vs_j joins the weight as an exponent, w_j = exp2(s_j + log2 vs_j - mw)
// with a running maximum mw of its own, so that w fits f16 whatever the scales
// are. The sum of the weights keeps to exp2(s_j - m).
//   q: each head's row is multiplied by a power of two that takes its largest
//      element to [2^14, 2^15): bf16 values are exact in f16 within 2^-28 of
//      that; fp32 queries are two f16 terms (22 bits).
//   w: one f16 term (2^-11) for bf16, two for fp32.
// A contraction does not care for the order of its index, so each lane takes
// the bytes that lie together: 16-byte reads of K rows are the scores' operand
// as they stand, and of V rows after pairing the bytes of two keys.
#include "full_decode.cuh"

#include <cuda_fp16.h>

namespace msa {
namespace {

constexpr float kTop = 7.f;  // weights reach 2^(kTop + kFdLazy): what f16 drops below 2^-24 is 2^-39 of the largest

__device__ __forceinline__ void mma16816h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 codes (the low or the high half of x) as f16
__device__ __forceinline__ uint32_t low2(uint32_t x) {
  uint32_t y;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t high2(uint32_t x) {
  uint32_t y;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {  // -inf of 0
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// what an f16 pair leaves of a and b (nothing of an infinity)
__device__ __forceinline__ uint32_t rest_f16(uint32_t packed, float a, float b) {
  const float2 f = __half22float2(reinterpret_cast<const __half2&>(packed));
  return pack_f16(fabsf(f.x) < INFINITY ? a - f.x : 0.f, fabsf(f.y) < INFINITY ? b - f.y : 0.f);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds1(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

template <typename T_, int D, int H>
struct Core8 {
  using T = T_;
  static constexpr int kD = D, kWarps = 8, kTiles = 2, kStages = D == 64 ? 4 : H <= 8 ? 3 : 2;
  static constexpr int HN = (H + 7) / 8, kTerms = sizeof(T) == 4 ? 2 : 1;
  // two of: K codes | V codes | 16 K scales | 16 V scales
  static constexpr int kTile = kSub * D, kScales = 2 * kTile, kTileStage = 2 * kTile + 2 * kSub * 4;
  static constexpr int kStage = kTiles * kTileStage, kExtra = 0;
  static constexpr int kM = 2 * HN, kAcc = HN * D / 4, kWords = D / 16;  // 4-byte words of a lane's quarter of a row
  uint32_t qf[HN][kTerms][kWords][2];
  float qs[kM];  // the scores' factors: scale, log2 e and the queries' power of two
  float m[kM], l[kM], mw[kM], acc[kAcc];  // acc[(t * D / 16 + mt) * 4 + e]; mw: less kTop

  // 16-byte chunk c of row r: exchanged so that 8 lanes that read chunks of
  // neighbouring (K) or every second row (V) hit all banks.
  __device__ __forceinline__ static uint32_t at(uint32_t tile, int r, int c) {
    if (D == 128) return chunk_at(tile, 128, r, c);
    return tile + uint32_t((r >> 1) * 128 + ((r ^ (r >> 2)) & 1) * 64 + ((c ^ (r & 2)) << 4));
  }
  __device__ __forceinline__ static void copy(const FdParams& p, uint32_t dst, int page, int row, int g, int valid) {
    constexpr int kCpr = D / 16;
    const int lane = threadIdx.x & 31;
    if (valid <= 0) row = 0;
    const int64_t head = (int64_t(page) << p.pages.page_log2) + row;
    const uint8_t* kp = static_cast<const uint8_t*>(p.k) + (head * p.Hkv + g) * D;
    const uint8_t* vp = static_cast<const uint8_t*>(p.v) + (head * p.Hkv + g) * D;
#pragma unroll
    for (int x = lane; x < kSub * kCpr; x += 32) {
      const int r = x / kCpr, c = x % kCpr;
      const bool in = r < valid;
      cp16z(at(dst, r, c), kp + (in ? int64_t(r) * p.Hkv * D + c * 16 : 0), in);
    }
#pragma unroll
    for (int x = lane; x < kSub * kCpr; x += 32) {
      const int r = x / kCpr, c = x % kCpr;
      const bool in = r < valid;
      cp16z(at(dst + kTile, r, c), vp + (in ? int64_t(r) * p.Hkv * D + c * 16 : 0), in);
    }
    if (lane < 8) {  // scales: [page][head][row], four to a copy; those past the end arrive as zeros
      const int c = lane & 3;
      const float* src = (lane < 4 ? p.k_scale : p.v_scale) + (((int64_t(page) * p.Hkv + g) << p.pages.page_log2) + row);
      const int n = min(max(valid - 4 * c, 0), 4);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + kScales + lane * 16),
                   "l"(src + (n > 0 ? 4 * c : 0)), "r"(4 * n)
                   : "memory");
    }
  }
  // B fragments of the scores: lane (gq, tq) has dims [tq D / 4, ...) of head gq
  __device__ __forceinline__ void start(const FdParams& p, const T* q, int heads, uint32_t) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int t = 0; t < HN; ++t) {
      float x[4 * kWords], top = 0.f;
      const T* qh = q + (t * 8 + gq) * D + tq * (D / 4);
      const bool in = t * 8 + gq < heads;
#pragma unroll
      for (int i = 0; i < 4 * kWords; i += 16 / int(sizeof(T))) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (in) raw = *reinterpret_cast<const uint4*>(qh + i);
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int y = 0; y < 16 / int(sizeof(T)); ++y) x[i + y] = to_f(e[y]);
      }
#pragma unroll
      for (int i = 0; i < 4 * kWords; ++i) top = fmaxf(top, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^-e and 2^e as exponent fields, e = exponent(top) - 14, both normal; a row of zeros stays as it is
      const int f = max(int(__float_as_uint(top) >> 23) - 14, 27);
      const float down = top > 0.f ? __uint_as_float(uint32_t(254 - f) << 23) : 1.f;
      const float up = top > 0.f ? __uint_as_float(uint32_t(f) << 23) : 1.f;
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float a = x[4 * w + 2 * y] * down, b = x[4 * w + 2 * y + 1] * down;
          qf[t][0][w][y] = pack_f16(a, b);
          if constexpr (kTerms == 2) qf[t][1][w][y] = rest_f16(qf[t][0][w][y], a, b);
        }
#pragma unroll
      for (int y = 0; y < 2; ++y) qs[2 * t + y] = __shfl_sync(0xffffffffu, up, (2 * tq + y) * 4) * p.scale_log2;
    }
#pragma unroll
    for (int x = 0; x < kM; ++x) m[x] = mw[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
    for (int x = 0; x < kAcc; ++x) acc[x] = 0.f;
  }
  __device__ __forceinline__ void step(uint32_t stage, uint32_t, int valid, float) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    float s[kTiles][HN][4], lv[kTiles][2];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint32_t kt = stage + i * kTileStage, sc = kt + kScales;
#pragma unroll
      for (int t = 0; t < HN; ++t) s[i][t][0] = s[i][t][1] = s[i][t][2] = s[i][t][3] = 0.f;
#pragma unroll
      for (int c = 0; c < kWords / 4; ++c) {  // keys gq and gq + 8
        const uint4 lo = lds16(at(kt, gq, tq * (kWords / 4) + c)), hi = lds16(at(kt, gq + 8, tq * (kWords / 4) + c));
        const uint32_t r0[4] = {lo.x, lo.y, lo.z, lo.w}, r1[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a[4] = {low2(r0[w]), low2(r1[w]), high2(r0[w]), high2(r1[w])};
#pragma unroll
          for (int t = 0; t < HN; ++t)
#pragma unroll
            for (int y = 0; y < kTerms; ++y) mma16816h(s[i][t], a, qf[t][y][c * 4 + w][0], qf[t][y][c * 4 + w][1]);
        }
      }
      const float ks[2] = {lds1(sc + gq * 4), lds1(sc + gq * 4 + 32)};
      lv[i][0] = lg2(lds1(sc + 64 + gq * 4));
      lv[i][1] = lg2(lds1(sc + 64 + gq * 4 + 32));
#pragma unroll
      for (int t = 0; t < HN; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[i][t][e] = i * kSub + gq + 8 * (e >> 1) < valid ? s[i][t][e] * qs[2 * t + (e & 1)] * ks[e >> 1] : -INFINITY;
    }
    float mt[kM], mv[kM];
    bool up = false;
#pragma unroll
    for (int x = 0; x < kM; ++x) {
      const int t = x >> 1, e = x & 1;
      mt[x] = fmaxf(s[0][t][e], s[0][t][2 + e]);
      mv[x] = fmaxf(s[0][t][e] + lv[0][0], s[0][t][2 + e] + lv[0][1]);
#pragma unroll
      for (int i = 1; i < kTiles; ++i) {
        mt[x] = tc::fmax3(mt[x], s[i][t][e], s[i][t][2 + e]);
        mv[x] = tc::fmax3(mv[x], s[i][t][e] + lv[i][0], s[i][t][2 + e] + lv[i][1]);
      }
      mt[x] = qmax(mt[x]);
      mv[x] = qmax(mv[x]) - kTop;
      up |= mt[x] > m[x] + kFdLazy || (m[x] == -INFINITY && mt[x] > -INFINITY);
      up |= mv[x] > mw[x] + kFdLazy || (mw[x] == -INFINITY && mv[x] > -INFINITY);
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const float mn = fmaxf(m[i], mt[i]), wn = fmaxf(mw[i], mv[i]);
        l[i] *= mn == m[i] ? 1.f : ex2d(m[i] - mn);
        const float a = wn == mw[i] ? 1.f : ex2d(mw[i] - wn);
        m[i] = mn;
        mw[i] = wn;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          acc[((i >> 1) * (D / 16) + k) * 4 + (i & 1)] *= a;
          acc[((i >> 1) * (D / 16) + k) * 4 + 2 + (i & 1)] *= a;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint32_t vt = stage + i * kTileStage + kTile;
      uint32_t b[HN][kTerms][2];
#pragma unroll
      for (int t = 0; t < HN; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 2 * t + (e & 1);
          l[x] += ex2d(s[i][t][e] - (m[x] == -INFINITY ? 0.f : m[x]));
          w[e] = ex2d((s[i][t][e] - (mw[x] == -INFINITY ? 0.f : mw[x])) + lv[i][e >> 1]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t hi = pack_f16(w[2 * y], w[2 * y + 1]);
          b[t][0][y] = trans8(hi);
          if constexpr (kTerms == 2) b[t][1][y] = trans8(rest_f16(hi, w[2 * y], w[2 * y + 1]));
        }
      }
      // lane (gq, tq): keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9, dims [gq D / 8, ...)
      uint32_t v[4][D / 32];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int r = 2 * tq + (y & 1) + 8 * (y >> 1);
        if constexpr (D == 128) {
          const uint4 f = lds16(at(vt, r, gq));
          v[y][0] = f.x, v[y][1] = f.y, v[y][2] = f.z, v[y][3] = f.w;
        } else {
          const uint2 f = lds8(at(vt, r, gq >> 1) + (gq & 1) * 8);
          v[y][0] = f.x, v[y][1] = f.y;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // dims 4 w + 2 y (rows gq of the product) and 4 w + 2 y + 1 (rows gq + 8)
          const uint32_t lo = __byte_perm(v[0][w], v[1][w], y ? 0x7362 : 0x5140);
          const uint32_t hi = __byte_perm(v[2][w], v[3][w], y ? 0x7362 : 0x5140);
          const uint32_t a[4] = {low2(lo), high2(lo), low2(hi), high2(hi)};
#pragma unroll
          for (int t = 0; t < HN; ++t) {
            float(&c)[4] = reinterpret_cast<float(&)[4]>(acc[(t * (D / 16) + 2 * w + y) * 4]);
#pragma unroll
            for (int z = 0; z < kTerms; ++z) mma16816h(c, a, b[t][z][0], b[t][z][1]);
          }
        }
      }
    }
  }
  // the weights' own maximum is taken out again: from here on a state is as any other's
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < kM; ++i) {
      const float a = mw[i] == -INFINITY ? 1.f : ex2d(mw[i] - m[i]);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        acc[((i >> 1) * (D / 16) + k) * 4 + (i & 1)] *= a;
        acc[((i >> 1) * (D / 16) + k) * 4 + 2 + (i & 1)] *= a;
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < HN; ++t)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(t * 8 + 2 * tq + (e & 1), 2 * t + (e & 1), gq * (D / 8) + 2 * k + (e >> 1), acc[(t * (D / 16) + k) * 4 + e]);
  }
  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int x = 0; x < kM; ++x) l[x] = qsum(l[x]);
  }
  template <typename F>
  __device__ __forceinline__ void each_head(F f) const {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
    if (gq == 0) {
#pragma unroll
      for (int x = 0; x < kM; ++x) f((x >> 1) * 8 + 2 * tq + (x & 1), x);
    }
  }
  __device__ __forceinline__ static int m_index(int x) { return 2 * (x / (D / 4)) + (x & 1); }
};

template <typename T, int D>
cudaError_t run(const FdParams& p, cudaStream_t stream) {
  return p.hpg > 8 ? decode<Core8<T, D, 16>, false>(p, "full_decode_fp8", stream)
                   : decode<Core8<T, D, 8>, false>(p, "full_decode_fp8", stream);
}

}  // namespace

cudaError_t launch_full_decode_fp8(const FullArgs& a, const float* k_scale, const float* v_scale, cudaStream_t stream) {
  FdParams p = fd_params(a, 2 * fd_grid());
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  if (a.dtype == MSA_BF16) return a.d == 128 ? run<__nv_bfloat16, 128>(p, stream) : run<__nv_bfloat16, 64>(p, stream);
  return a.d == 128 ? run<float, 128>(p, stream) : run<float, 64>(p, stream);
}

}  // namespace msa
