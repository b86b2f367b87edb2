// Full attention, decode: one query row per sequence over the whole of its
// paged cache, all heads of a group per pass over its keys.
//
//   out = sum_j exp(s_j - lse) v_j,  s_j = scale q . k_j,  j < kv_len
//
// Bound: HBM (4 hpg FLOPs per element; every key and value is read once by each
// item of up to 16 query heads, so up to 4 times for the largest groups of 64).
// Measured (Hq 32, Hkv 8, d 128, bf16): 16 sequences of 4 K to 128 K keys 557 us,
// 6.55 TB/s (97 % of the measured copy rate); one of 777 keys 12 us, latency.
//
// Work: the keys of every (sequence, key/value head, group of up to 16 query
// heads) -- an item -- are cut into units of 128 (16 per warp; 64 for fp32 of d
// 128, which has four warps), the units of all items are numbered through, and
// each CTA of a fixed grid (one per SM) takes an equal run of them, so ragged
// lengths balance whatever they are, without the host knowing them.
// In a unit each warp takes 16 keys, which lie in one page, and works alone:
// its own ring of cp.async copies (keys past the end arrive as zeros), scores,
// running maximum and sum, products. Warps meet only where an item ends in the
// CTA: their states are joined in shared memory. An item that lies in several
// CTAs leaves a partial (maximum, sum, unnormalised output) per CTA, and the
// CTA that arrives last joins them in the order of the keys.
// Many short items: their ends would cost more than their keys (a join takes as
// long as a unit), so single warps take whole items instead, with nothing to join.
//
// bf16: mma.sync m16n8k16 with keys (then head dims) along M and the heads
// along N = 8: the tensor work is a fraction of the time the bytes take, so
// tcgen05's larger tiles would only pad. fp32: FMAs, one key per lane pair for
// the scores, four head dims per lane for the products.
#include "full_internal.cuh"
#include "tc_utils.cuh"

namespace msa {
namespace {

constexpr int kSub = 16, kSubLog2 = 4;    // keys of a warp's step: never across a page
constexpr int kFdMaxHeads = 16;           // query heads of an item
constexpr float kFdLog2e = 1.4426950408889634f, kFdLn2 = 0.6931471805599453f;
// The maximum only moves when a step exceeds it by 2^8: weights stay below
// 2^8 and their common factor drops out in the division by their sum.
constexpr float kFdLazy = 8.f;

__device__ __forceinline__ float ex2d(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 b16 matrix across the warp, transposed
__device__ __forceinline__ uint32_t trans8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float qmax(float x) {  // over the 8 lanes that share lane & 3
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float qsum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Address of 16-byte chunk c of row r in a [rows][row_bytes] tile whose chunks
// are exchanged within 128 bytes by the row's low bits (conflict-free ldmatrix
// and vector reads down a column).
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row_bytes, int r, int c) {
  return base + uint32_t(r * row_bytes) + (uint32_t(c ^ (r & 7)) << 4);
}

// ---- a warp's state: bf16 ------------------------------------------------------
// O^T (head dims along M) and the scores share the column = head layout: lane
// (gq = lane / 4, tq = lane % 4) holds heads 2 tq and 2 tq + 1 of each tile of 8.
template <typename T, int D, int H>  // H: most heads of an item
struct Core;

template <int D, int H>
struct Core<__nv_bfloat16, D, H> {
  using T = __nv_bfloat16;
  static constexpr int HN = (H + 7) / 8;
  static constexpr int kRow = D * 2, kTile = kSub * kRow, kStage = 2 * kTile, kExtra = 0;
  static constexpr int kM = 2 * HN, kAcc = HN * D / 4;
  uint32_t qf[HN][D / 16][2];
  float m[kM], l[kM], acc[kAcc];  // acc[(t * D / 16 + mt) * 4 + e]

  __device__ __forceinline__ void start(const T* q, int heads, uint32_t) {
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
    for (int x = 0; x < kM; ++x) m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
    for (int x = 0; x < kAcc; ++x) acc[x] = 0.f;
  }
  __device__ __forceinline__ void step(uint32_t kt, uint32_t, int valid, float scale_log2) {
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
        mt[2 * t + x] = qmax(fmaxf(s[t][x], s[t][2 + x]));
        up |= mt[2 * t + x] > m[2 * t + x] + kFdLazy || (m[2 * t + x] == -INFINITY && mt[2 * t + x] > -INFINITY);
      }
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int t = 0; t < HN; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = 2 * t + x;
          const float mn = fmaxf(m[i], mt[i]);
          const float a = mn == m[i] ? 1.f : ex2d(m[i] - mn);
          m[i] = mn;
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
        const float mm = m[2 * t + (e & 1)];
        p[e] = ex2d(s[t][e] - (mm == -INFINITY ? 0.f : mm));
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
  static constexpr int P = D / 32;
  static constexpr int kRow = D * 4, kTile = kSub * kRow, kStage = 2 * kTile;
  static constexpr int kExtra = (H * D + kSub * H) * 4;  // per warp: queries, weights
  static constexpr int kM = H, kAcc = H * P;
  float m[kM], l[kM], acc[kAcc];  // acc[h * P + x]

  __device__ __forceinline__ void start(const T* q, int heads, uint32_t extra) {
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
  __device__ __forceinline__ void step(uint32_t kt, uint32_t extra, int valid, float scale_log2) {
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

struct FdParams {
  const void *q, *k, *v;
  const int32_t* kv_len;
  PageMap pages;
  int B, Hq, Hkv, hpg, ngr, cap;  // ngr: head groups (items) per key/value head; cap: most keys
  float scale_log2;
  float* part_o;   // [2 * grid][16][D]
  float* part_ml;  // [2 * grid][16][2]: maximum (log2 units), sum; a negative sum marks a page out of range
  uint32_t* arrivals;  // a byte per CTA, zero between calls: the parts of the split item that it holds the first of
  void* out;
  float* lse;
  uint32_t* status;
};

__device__ __forceinline__ int units_of(const FdParams& p, int b, int unit_log2) {
  const int L = p.kv_len[b];
  return L > 0 && L <= p.cap ? ((L - 1) >> unit_log2) + 1 : 0;
}

// A walk over units in order: those of a CTA's run, or (SOLO) of every hop-th item.
struct Walk {
  int b, it, u, n;  // sequence, item within it, unit within the item, units of the item
  template <bool SOLO>
  __device__ __forceinline__ void next(const FdParams& p, int hop, int unit_log2) {
    if (++u < n) return;
    u = 0;
    if constexpr (SOLO) return seek(p, hop, hop);
    if (++it < p.Hkv * p.ngr) return;
    it = 0;
    do {
      n = ++b < p.B ? units_of(p, b, unit_log2) : 1;  // past the last sequence the walk is over
    } while (n == 0);
  }
  // To the first item with keys among those `by`, `by` + hop, ... further on.
  __device__ __forceinline__ void seek(const FdParams& p, int by, int hop) {
    const int items = p.Hkv * p.ngr;
    do {
      it += by;
      b += it / items;
      it %= items;
      by = hop;
      n = b < p.B ? units_of(p, b, kSubLog2) : 1;
    } while (n == 0);
  }
};

// Eight warps where their rings fit, one CTA per SM: the copies in flight are
// what covers HBM's latency.
template <typename T, int D, int H>
struct FdShape {
  using C = Core<T, D, H>;
  static constexpr bool kWide = sizeof(T) == 4 && D == 128;
  static constexpr int kWarps = kWide ? 4 : 8, kThreads = kWarps * 32;
  static constexpr int kUnit = kWarps * kSub;  // keys of a unit
  static constexpr int kStages = kWide ? 2 : sizeof(T) == 4 ? (H <= 4 ? 3 : 2) : D == 64 ? (H <= 8 ? 6 : 4) : H <= 8 ? 3 : 2;
  static constexpr int kRing = kStages * C::kStage;                                   // per warp
  static constexpr int kState = (C::kAcc + 2 * C::kM + 1) * 32;                       // floats of a warp's state
  static constexpr int kJoin = (kWarps - 1) * kState * 4;                             // a slot per hand-over
  static constexpr int kBytes = kWarps * (kRing + C::kExtra) + kJoin;
};

// SOLO: whole items for single warps; else the CTA's run of the `total` units.
template <typename T, int D, int H, bool SOLO>
__device__ __forceinline__ void decode_run(const FdParams& p, int64_t total) {
  using SH = FdShape<T, D, H>;
  using C = typename SH::C;
  constexpr int NS = SH::kStages, kFdWarps = SH::kWarps, kFdThreads = SH::kThreads, kUnit = SH::kUnit;
  constexpr int kCpr = D * int(sizeof(T)) / 16;  // 16-byte chunks of a row
  extern __shared__ __align__(128) uint8_t fd_smem[];
  __shared__ int last_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = tc::smem_u32(fd_smem) + warp * SH::kRing;
  const uint32_t extra = tc::smem_u32(fd_smem) + kFdWarps * SH::kRing + warp * C::kExtra;
  float* join = reinterpret_cast<float*>(fd_smem + kFdWarps * (SH::kRing + C::kExtra));
  const int items = p.Hkv * p.ngr;
  T* out = static_cast<T*>(p.out);

  constexpr int kUnitLog2 = kUnit == 64 ? 6 : 7;
  static_assert(1 << kUnitLog2 == kUnit, "keys of a unit");
  constexpr int ulog = SOLO ? kSubLog2 : kUnitLog2;
  const int hop = SOLO ? int(gridDim.x) * kFdWarps : 0, sub0 = SOLO ? 0 : warp * kSub;
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t run0 = SOLO ? 0 : blockIdx.x * per, run1 = SOLO ? INT64_MAX : min(run0 + per, total);
  if (run0 >= run1) return;
  Walk at{};
  int64_t first = 0;  // number of the walk's sequence's first unit
  int64_t item_first = 0;  // number of the item's first unit
  if constexpr (SOLO) {
    at.seek(p, warp * int(gridDim.x) + int(blockIdx.x), hop);
  } else {
    int ahead = lane < p.B ? units_of(p, lane, kUnitLog2) : 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int mine = ahead;
      ahead = b0 + 32 + lane < p.B ? units_of(p, b0 + 32 + lane, kUnitLog2) : 0;  // in flight during the scan
      int64_t incl = int64_t(mine) * items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, first + incl > run0);
      if (hit) {
        const int src = __ffs(hit) - 1;
        at.b = b0 + src;
        at.n = __shfl_sync(0xffffffffu, mine, src);
        first += __shfl_sync(0xffffffffu, incl, src) - int64_t(at.n) * items;
        break;
      }
      first += __shfl_sync(0xffffffffu, incl, 31);
    }
    at.it = int((run0 - first) / at.n);
    at.u = int((run0 - first) % at.n);
    item_first = first + int64_t(at.it) * at.n;
  }

  // ---- copies: the walk `ld` runs ahead of `at` ----
  Walk ld = at;
  int64_t ld_left = !SOLO || ld.b < p.B ? run1 - run0 : 0;
  uint32_t bad_ring = 0;  // stage x's page was out of range
  auto page_of = [&](const Walk& w) {
    const int key = (w.u << ulog) + sub0;
    return key < p.kv_len[w.b] ? p.pages.table[int64_t(w.b) * p.pages.max_pages + (key >> p.pages.page_log2)] : 0;
  };
  int page = ld_left > 0 ? page_of(ld) : 0;
  auto issue = [&](int st) {
    if (ld_left > 0) {
      const int L = p.kv_len[ld.b], key = (ld.u << ulog) + sub0;
      const int valid = L - key;
      const bool bad = valid > 0 && (page < 0 || page >= p.pages.num_pages);
      bad_ring = bad ? bad_ring | (1u << st) : bad_ring & ~(1u << st);
      const int g = ld.it / p.ngr;
      const int64_t row0 = bad || valid <= 0 ? 0
                                             : (int64_t(page) << p.pages.page_log2) +
                                                   (key & ((1 << p.pages.page_log2) - 1));
      const T* kp = static_cast<const T*>(p.k) + (row0 * p.Hkv + g) * D;
      const T* vp = static_cast<const T*>(p.v) + (row0 * p.Hkv + g) * D;
      const uint32_t dst = ring + st * C::kStage;
#pragma unroll
      for (int x = lane; x < kSub * kCpr; x += 32) {
        const int r = x / kCpr, c = x % kCpr;
        const bool in = r < valid && !bad;
        const int64_t off = in ? int64_t(r) * p.Hkv * D + c * (16 / int(sizeof(T))) : 0;
        cp16z(chunk_at(dst, C::kRow, r, c), kp + off, in);
      }
#pragma unroll
      for (int x = lane; x < kSub * kCpr; x += 32) {
        const int r = x / kCpr, c = x % kCpr;
        const bool in = r < valid && !bad;
        const int64_t off = in ? int64_t(r) * p.Hkv * D + c * (16 / int(sizeof(T))) : 0;
        cp16z(chunk_at(dst + C::kTile, C::kRow, r, c), vp + off, in);
      }
      if (--ld_left > 0) {
        ld.next<SOLO>(p, hop, ulog);
        if (!SOLO || ld.b < p.B)
          page = page_of(ld);
        else
          ld_left = 0;
      }
    }
    cp_commit_group();
  };
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(st);

  C c;
  bool fresh = true, bad = false;
  int st = 0;
  for (int64_t z = run0; z < run1 && (!SOLO || at.b < p.B); ++z) {
    const int g = at.it / p.ngr, h0 = g * p.hpg + (at.it % p.ngr) * kFdMaxHeads;
    const int heads = min(p.hpg - (at.it % p.ngr) * kFdMaxHeads, kFdMaxHeads);
    const int L = p.kv_len[at.b];
    if (fresh) {
      c.start(static_cast<const T*>(p.q) + (int64_t(at.b) * p.Hq + h0) * D, heads, extra);
      fresh = bad = false;
    }
    issue((st + NS - 1) % NS);
    cp_wait<NS - 1>();
    __syncwarp();
    bad |= (bad_ring >> st) & 1u;
    const int valid = L - ((at.u << ulog) + sub0);
    if (valid > 0) c.step(ring + st * C::kStage, extra, valid, p.scale_log2);
    __syncwarp();
    st = (st + 1) % NS;
    const int b = at.b, n = at.n;
    const bool ends = at.u + 1 == at.n;
    if (!ends && z + 1 < run1) {
      ++at.u;
      continue;
    }
    // ---- the item ends here: join the warps' states, halving their number ----
    fresh = true;
    constexpr int kRegs = C::kAcc + 2 * C::kM + 1;
    auto put = [&](float* to) {
#pragma unroll
      for (int x = 0; x < C::kAcc; ++x) to[x * 32 + lane] = c.acc[x];
#pragma unroll
      for (int x = 0; x < C::kM; ++x) {
        to[(C::kAcc + x) * 32 + lane] = c.m[x];
        to[(C::kAcc + C::kM + x) * 32 + lane] = c.l[x];
      }
      to[(kRegs - 1) * 32 + lane] = bad ? 1.f : 0.f;
    };
    auto take = [&](const float* from) {
      float wa[C::kM], wb[C::kM];
#pragma unroll
      for (int x = 0; x < C::kM; ++x) {
        const float mo = from[(C::kAcc + x) * 32 + lane], mn = fmaxf(c.m[x], mo);
        wa[x] = c.m[x] == mn ? 1.f : ex2d(c.m[x] - mn);
        wb[x] = mo == mn ? 1.f : ex2d(mo - mn);
        c.m[x] = mn;
        c.l[x] = c.l[x] * wa[x] + from[(C::kAcc + C::kM + x) * 32 + lane] * wb[x];
      }
#pragma unroll
      for (int x = 0; x < C::kAcc; ++x)
        c.acc[x] = c.acc[x] * wa[C::m_index(x)] + from[x * 32 + lane] * wb[C::m_index(x)];
      bad |= from[(kRegs - 1) * 32 + lane] != 0.f;
    };
    // Every hand-over has a slot of its own: the upper warps may be at the next
    // item's end while the lower ones still read this one's.
    if constexpr (!SOLO) {
#pragma unroll
      for (int half = kFdWarps / 2, slot0 = 0; half > 0; slot0 += half, half >>= 1) {
        if (warp >= half && warp < 2 * half) put(join + (slot0 + warp - half) * SH::kState);
        __syncthreads();
        if (warp < half) take(join + (slot0 + warp) * SH::kState);
      }
    }
    const bool whole = SOLO || (item_first >= run0 && ends);
    const int slot = 2 * int(blockIdx.x) + (item_first >= run0 ? 1 : 0);
    if (SOLO || warp == 0) {
      c.sum_l();
      if (__any_sync(0xffffffffu, bad)) {
        bad = true;
        if (lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
      }
      if (whole) {
        float inv[C::kM];
#pragma unroll
        for (int x = 0; x < C::kM; ++x) inv[x] = bad ? 0.f : 1.f / c.l[x];
        c.each([&](int h, int x, int dim, float val) {
          if (h < heads)
            out[(int64_t(b) * p.Hq + h0 + h) * D + dim] = from_f<T>(bad ? 0.f : val * inv[x]);
        });
        if (p.lse)
          c.each_head([&](int h, int x) {
            if (h < heads) p.lse[int64_t(b) * p.Hq + h0 + h] = bad ? -INFINITY : (c.m[x] + log2f(c.l[x])) * kFdLn2;
          });
      } else {
        float* po = p.part_o + int64_t(slot) * kFdMaxHeads * D;
        float* pm = p.part_ml + int64_t(slot) * kFdMaxHeads * 2;
        c.each([&](int h, int, int dim, float val) {
          if (h < heads) po[h * D + dim] = val;
        });
        c.each_head([&](int h, int x) {
          if (h < heads) {
            pm[2 * h] = c.m[x];
            pm[2 * h + 1] = bad ? -1.f : c.l[x];
          }
        });
      }
    }
    if (!whole) {
      // the item's units lie in CTAs c0..c1: the last to arrive joins them
      const int c0 = int(item_first / per), c1 = int((item_first + n - 1) / per);
      if (warp == 0) {
        __syncwarp();
        if (lane == 0) {
          // releases the warp's stores (ordered by __syncwarp), acquires the others'
          const int sh = 8 * (c0 & 3);
          uint32_t old;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                       : "=r"(old)
                       : "l"(p.arrivals + (c0 >> 2)), "r"(1u << sh)
                       : "memory");
          last_s = int((old >> sh) & 0xffu) == c1 - c0;
          if (last_s) atomicSub(p.arrivals + (c0 >> 2), uint32_t(c1 - c0 + 1) << sh);  // ready for the next call
        }
      }
      __syncthreads();
      if (last_s) {
        auto slot_of = [&](int cta) { return 2 * cta + (cta == c0 && item_first >= c0 * per ? 1 : 0); };
        constexpr int kBatch = 8;  // partials in flight: the loads of a batch do not wait for each other
        for (int o = threadIdx.x * 4; o < heads * D; o += kFdThreads * 4) {
          const int h = o / D;
          float M = -INFINITY, den = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
          bool spoilt = false;
          for (int cta = c0; cta <= c1; cta += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              const int64_t s = int64_t(slot_of(min(cta + x, c1))) * kFdMaxHeads + h;
              ml[x] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + s * 2));
              v[x] = __ldcg(reinterpret_cast<const float4*>(p.part_o + s * D + o % D));
            }
            float mn = M;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              spoilt |= ml[x].y < 0.f;
              mn = fmaxf(mn, ml[x].x);
            }
            const float a = M == mn ? 1.f : ex2d(M - mn);
            M = mn;
            den *= a;
#pragma unroll
            for (int y = 0; y < 4; ++y) sum[y] *= a;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              const float w = cta + x > c1 ? 0.f : ml[x].x == M ? 1.f : ex2d(ml[x].x - M);
              den = fmaf(w, ml[x].y, den);
              sum[0] = fmaf(w, v[x].x, sum[0]);
              sum[1] = fmaf(w, v[x].y, sum[1]);
              sum[2] = fmaf(w, v[x].z, sum[2]);
              sum[3] = fmaf(w, v[x].w, sum[3]);
            }
          }
          const float inv = 1.f / den;
          T* dst = out + (int64_t(b) * p.Hq + h0 + h) * D + o % D;
#pragma unroll
          for (int y = 0; y < 4; ++y) dst[y] = from_f<T>(spoilt ? 0.f : sum[y] * inv);
          if (p.lse && o % D == 0)
            p.lse[int64_t(b) * p.Hq + h0 + h] = spoilt ? -INFINITY : (M + log2f(den)) * kFdLn2;
        }
      }
      __syncthreads();  // last_s is read before the next item sets it
    }
    if (ends) item_first += n;
    const int was = at.b;
    at.next<SOLO>(p, hop, ulog);
    if (at.b != was) item_first = z + 1;
  }
  cp_wait<0>();
}

template <typename T, int D, int H>
__global__ void __launch_bounds__(FdShape<T, D, H>::kThreads, 1) full_decode_kernel(const FdParams p) {
  using SH = FdShape<T, D, H>;
  constexpr int kFdWarps = SH::kWarps, kFdThreads = SH::kThreads;
  const int lane = threadIdx.x & 31, items = p.Hkv * p.ngr;
  T* out = static_cast<T*>(p.out);

  // ---- all units (every warp counts alone) ----
  int64_t total = 0;
  int longest = 0;  // in warps' steps
#pragma unroll 8
  for (int b = lane; b < p.B; b += 32) {
    const int steps = units_of(p, b, kSubLog2);
    total += (steps + kFdWarps - 1) / kFdWarps;
    longest = max(longest, steps);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  longest = __reduce_max_sync(0xffffffffu, longest);
  total *= items;
  // Whole items for single warps, or shared-out units? A unit and a warp's step
  // both take about 1.1 us, and so does an item's end or start; single warps
  // come out ahead from 1.25 times the other count on. Measured both ways (Hq 32,
  // Hkv 8, d 128, bf16; lengths within a factor of 2):
  //   1280 items up to 64 keys   19 (single) : 29 us     2560 up to 256   65 :  70 us
  //   10240 items up to 128      99 : 177 us             2560 up to 512  119 : 109 us
  //   640 items up to 128        18 :  20 us              320 up to 128   17 :  16 us
  const int warps = int(gridDim.x) * kFdWarps;
  const int64_t all = int64_t(p.B) * items, rounds = (all + warps - 1) / warps;
  const bool solo = 4 * rounds * (1 + longest) * int64_t(gridDim.x) <= 5 * (total + all);
  // sequences without keys: nobody's run holds them
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (units_of(p, b, kSubLog2) > 0) continue;
    if (threadIdx.x == 0 && (p.kv_len[b] < 0 || p.kv_len[b] > p.cap)) set_status(p.status, MSA_ERR_BOUNDS);
    for (int x = threadIdx.x; x < p.Hq * D; x += kFdThreads) out[int64_t(b) * p.Hq * D + x] = from_f<T>(0.f);
    if (p.lse)
      for (int x = threadIdx.x; x < p.Hq; x += kFdThreads) p.lse[int64_t(b) * p.Hq + x] = -INFINITY;
  }
  if (solo)
    decode_run<T, D, H, true>(p, total);
  else
    decode_run<T, D, H, false>(p, total);
}

int fd_grid() { return kNumSMs; }

template <typename T, int D, int H>
cudaError_t decode(const FdParams& p, cudaStream_t stream) {
  auto kern = full_decode_kernel<T, D, H>;
  constexpr int bytes = FdShape<T, D, H>::kBytes;
  static_assert(bytes <= 227 * 1024 - 16, "shared memory of one CTA");
  static KernelReady ready;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), bytes)) return e;
  ProfScope pf("full_decode", stream);
  kern<<<fd_grid(), FdShape<T, D, H>::kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int head_groups(int hpg) { return (hpg + kFdMaxHeads - 1) / kFdMaxHeads; }

}  // namespace

size_t full_decode_ws_bytes(int d) {
  const size_t slots = 2 * size_t(fd_grid());
  return up256(slots * kFdMaxHeads * d * 4) + up256(slots * kFdMaxHeads * 8);
}

cudaError_t launch_full_decode(const FullArgs& a, cudaStream_t stream) {
  FdParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.kv_len = a.seq.kv_len;
  p.pages = a.pages;
  p.B = a.seq.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.hpg = a.Hq / a.Hkv;
  p.ngr = head_groups(p.hpg);
  p.cap = a.seq.Tk;
  p.scale_log2 = a.scale * kFdLog2e;
  const size_t slots = 2 * size_t(fd_grid());
  char* w = static_cast<char*>(a.ws) + kWsHeader;
  p.part_o = reinterpret_cast<float*>(w);
  w += up256(slots * kFdMaxHeads * a.d * 4);
  p.part_ml = reinterpret_cast<float*>(w);
  p.arrivals = static_cast<WsHeader*>(a.ws)->arrivals;
  p.out = a.out;
  p.lse = a.lse;
  p.status = &static_cast<WsHeader*>(a.ws)->status;
  // bf16: a tile holds 8 heads, so fewer cost the same. fp32: the FMAs and
  // shared-memory reads are those of H heads, so up to 4 get a variant of half the work.
  const bool wide = p.hpg > 8, few = p.hpg <= 4;
  if (a.dtype == MSA_BF16) {
    if (a.d == 128) return wide ? decode<__nv_bfloat16, 128, 16>(p, stream) : decode<__nv_bfloat16, 128, 8>(p, stream);
    return wide ? decode<__nv_bfloat16, 64, 16>(p, stream) : decode<__nv_bfloat16, 64, 8>(p, stream);
  }
  if (a.d == 128)
    return wide ? decode<float, 128, 16>(p, stream) : few ? decode<float, 128, 4>(p, stream) : decode<float, 128, 8>(p, stream);
  return wide ? decode<float, 64, 16>(p, stream) : few ? decode<float, 64, 4>(p, stream) : decode<float, 64, 8>(p, stream);
}

}  // namespace msa
