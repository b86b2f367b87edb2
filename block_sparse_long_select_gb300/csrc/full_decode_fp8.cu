// Full attention, decode over a cache in 8 bits: keys ks_j K_j, values vs_j V_j
// with e4m3 codes K, V and a scale per (token, head).
//
//   out = sum_j exp(s_j - lse) vs_j V_j,  s_j = scale ks_j (q . K_j),  j < kv_len
//
// Bound: HBM, d + 4 bytes per key and per value where bf16 takes 2 d. Walk,
// copies and joins: full_decode.cuh. Measured (Hq 32, Hkv 8, d 128, bf16): 16
// sequences of 4 K to 128 K keys 303 to 319 us, 6.2 to 6.6 TB/s (92 to 97 % of the
// copy rate); one of 777 keys 10.3 us, latency. fp32 queries: 422 us, the second terms'
// products; d 64: instructions (at run_bf16).
//
// Products: mma.sync m16n8k16 in f16, which holds every e4m3 code exactly (bf16
// would as well, but the hardware converts e4m3 to f16 in one instruction for
// two). Scales stay out of the matrices: ks_j is multiplied to the finished
// score; vs_j joins the weight as an exponent, w_j = exp2(s_j + log2 vs_j - mw)
// with a running maximum mw of its own, so that w fits f16 whatever the scales
// are. The sum of the weights keeps to exp2(s_j - m).
//   q: each head's row is multiplied by a power of two that takes its largest
//      element to [2^14, 2^15): bf16 values are exact in f16 down to 2^-28 of that,
//      smaller ones within 2^-39 of it; fp32 queries are two f16 terms (22 bits).
//   w: one f16 term (11 bits) for bf16, two for fp32 (22).
// A second term is held times 2^11, as it would soon be below f16's least step (fp32
// weights of 2^-18 of the largest would have 13 bits), and its products of a tile are
// added to the first term's as a whole. fp32, 16 sequences of 4 K to 128 K keys: 422 us,
// 404 with second terms as they are, 440 with the values times 2^-11 in their place.
// A contraction does not care for the order of its index, so each lane takes
// the bytes that lie together: 16-byte reads of K rows are the scores' operand
// as they stand, and of V rows after pairing the bytes of two keys.
#include "full_decode.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace msa {
namespace {

constexpr float kLeast = -100.f;  // log2 of the least factor that is taken at once
// Weights reach 2^(kTop + kFdLazy), and the largest so far is 2^kTop at least: half of
// f16's least step, 2^-25, is 2^-32 of it at most (2^-40 at best).
constexpr float kTop = 7.f;

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
__device__ __forceinline__ float lg2(float x) {  // of subnormal scales as well: their values need not be
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// What an f16 pair leaves of a and b (nothing of an infinity), times 2^11, which makes
// it no larger than the pair: as it is, f16's least step would take its bits from
// weights of 2^-10 of the largest on.
__device__ __forceinline__ uint32_t rest_f16(uint32_t packed, float a, float b) {
  const float2 f = __half22float2(reinterpret_cast<const __half2&>(packed));
  return pack_f16(fabsf(f.x) < INFINITY ? (a - f.x) * 2048.f : 0.f, fabsf(f.y) < INFINITY ? (b - f.y) * 2048.f : 0.f);
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

struct Fd8Params : FdParams {
  CUtensorMap tmK, tmV;    // codes as [rows][Hkv][d] bytes, boxes of rows of a head
  CUtensorMap tmKs, tmVs;  // scales as [pages][Hkv][page_size], boxes of the same rows of a pair of heads (d 64)
  int box_log2;            // rows of a box: those of a step, if they lie in one page
  int kv_heads, group;   // key/value heads, query heads of one: what Hkv and hpg say of pairs where those are items
  int inject_timeout;    // test hook: a warp of every second CTA waits on a barrier nothing completes
};

// H: most query heads of a key/value head in an item; KT: tiles of 16 keys in a
// step; HT: key/value heads in an item, 2 where there is an even number of them.
// Neighbouring heads' rows lie together in memory, and 256 bytes at a time come
// from HBM faster than 128 (8 key/value heads, d 128: 6.6 TB/s instead of 5.4).
template <typename T_, int D, int H, int KT, int HT>
struct Core8 {
  using T = T_;
  using Params = Fd8Params;
  static constexpr bool kBulk = true;
  static constexpr int kD = D, kWarps = 8, kTiles = KT;
  static constexpr int HN = (H + 7) / 8, kTerms = sizeof(T) == 4 ? 2 : 1, kCols = HT * HN;  // columns of 8 heads
  // a stage: for every head K codes | V codes of the step's keys; beside the ring K scales | V scales, of a box's heads in turn
  static constexpr int kTile = kSub * D, kScales = 2 * kSub * 4, kBoth = KT * HT, kHead = 2 * KT * kTile;
  static constexpr int kStage = HT * kHead, kTileBytes = HT * (2 * kTile + kScales);  // bytes of a tile with its scales
  static constexpr int kM = 2 * kCols, kAcc = kCols * D / 4, kWords = D / 16;  // 4-byte words of a lane's quarter of a row
  static constexpr int kStages = (227 * 1024 - 8 * (2 * kM + 1) * 128 - 512) / (8 * (kStage + kBoth * kScales));
  static_assert(kStages >= 2 && (H <= 8 || HT == 1) && HT * H <= kFdMaxHeads, "items");
  static constexpr int kExtra = kStages * kBoth * kScales;
  // A copy takes an instruction stream of one lane, a third of all instructions for
  // d 64, where few bytes hide them: there a copy takes the step's rows as far as
  // they lie in one page, and both heads' scales (32 sequences of 64 K keys, Hq 32, Hkv 8:
  // 355 us, 433 with 16 rows and a head's scales to a copy; pages of 16: 390). For
  // d 128 the large copies come in slower (16 sequences: 368 us, 352 with the small ones).
  static constexpr bool kBig = D == 64, kPairScales = kBig && HT == 2;
  uint32_t qf[kCols][kTerms][kWords][2];
  float qs[kM];  // the scores' factors: scale, log2 e and the queries' power of two
  float m[kM], l[kM], mw[kM], acc[kAcc];  // acc[(t * D / 16 + mt) * 4 + e]; mw: less kTop
  float nm[kM], nw[kM];  // -m and -mw, 0 as long as those are -inf
  int per;               // query heads of a key/value head

  // 16-byte chunk c of row r, as TMA exchanges them within 128 (64) bytes: 8 lanes
  // that read chunks of neighbouring rows (K) or, for d 128, of every second row (V) hit all banks.
  __device__ __forceinline__ static uint32_t at(uint32_t tile, int r, int c) {
    if (D == 128) return chunk_at(tile, 128, r, c);
    return tile + uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  __device__ __forceinline__ static void prefetch(const Params& p) {
    tc::tma_prefetch(&p.tmK);
    tc::tma_prefetch(&p.tmV);
    if constexpr (kPairScales) {
      tc::tma_prefetch(&p.tmKs);
      tc::tma_prefetch(&p.tmVs);
    }
  }
  __device__ __forceinline__ static int box_of(const Params& p) { return kBig ? p.box_log2 : 4; }
  // the box that begins with tile x of a stage (one thread); g: the item's key/value head or pair
  __device__ __forceinline__ static void copy(const Params& p, uint32_t stage, uint32_t extra, int st, int x, uint64_t* bar,
                                              int page, int row, int g) {
    const int r0 = (page << p.pages.page_log2) + row;
    extra += st * kBoth * kScales + x * HT * kSub * 4;
#pragma unroll
    for (int z = 0; z < HT; ++z) {
      const int head = g * HT + z;
      tma_tile(stage + z * kHead + x * kTile, &p.tmK, bar, 0, head, r0);
      tma_tile(stage + z * kHead + (KT + x) * kTile, &p.tmV, bar, 0, head, r0);
      if constexpr (!kPairScales) {
        const int64_t sc = ((int64_t(page) * p.kv_heads + head) << p.pages.page_log2) + row;  // scales: [page][head][row]
        const uint32_t bytes = 4 << box_of(p);
        tc::bulk_load(extra + z * bytes, p.k_scale + sc, bytes, bar);
        tc::bulk_load(extra + z * bytes + kBoth * kScales / 2, p.v_scale + sc, bytes, bar);
      }
    }
    if constexpr (kPairScales) {
      tma_tile(extra, &p.tmKs, bar, row, g * HT, page);
      tma_tile(extra + kBoth * kScales / 2, &p.tmVs, bar, row, g * HT, page);
    }
  }
  // where key k of head z of a step has its K scale
  __device__ __forceinline__ static uint32_t scale_at(const Params& p, uint32_t extra, int z, int k) {
    if constexpr (KT == 1 || HT == 1) return extra + (z * kSub * KT + k) * 4;
    return extra + (((((k >> box_of(p)) * HT) + z) << box_of(p)) + (k & ((1 << box_of(p)) - 1))) * 4;
  }
  __device__ __forceinline__ static void tma_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  }
  // B fragments of the scores: lane (gq, tq) has dims [tq D / 4, ...) of head gq
  __device__ __forceinline__ void start(const Params& p, const T* q, int heads, uint32_t) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    heads /= HT;  // of each
    per = heads;
#pragma unroll
    for (int t = 0; t < kCols; ++t) {
      float x[4 * kWords], top = 0.f;
      const int h = (t % HN) * 8 + gq;
      const T* qh = q + ((t / HN) * heads + h) * D + tq * (D / 4);
      const bool in = h < heads;
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
    for (int x = 0; x < kM; ++x) m[x] = mw[x] = -INFINITY, l[x] = nm[x] = nw[x] = 0.f;
#pragma unroll
    for (int x = 0; x < kAcc; ++x) acc[x] = 0.f;
  }
  __device__ __forceinline__ void step(const Params& p, uint32_t stage, uint32_t extra, int st, int valid) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    extra += st * kBoth * kScales;
    if (valid < KT * kSub) {
      // rows behind the end may hold anything, and weight 0 does not silence a NaN: they and their scales become zeros
      for (int x = lane; x < kBoth * kTile / 16; x += 32) {
        const int z = x / (KT * kTile / 16), in_head = x % (KT * kTile / 16);
        const uint32_t at_k = stage + z * kHead + in_head * 16;
        if (in_head / (D / 16) >= valid)
          asm volatile("st.shared.v4.b32 [%0], {%2, %2, %2, %2};\n\tst.shared.v4.b32 [%1], {%2, %2, %2, %2};" ::"r"(at_k),
                       "r"(at_k + KT * kTile), "r"(0)
                       : "memory");
      }
      for (int x = lane; x < kBoth * kSub; x += 32) {
        const int k = x % (KT * kSub);
        const uint32_t at_s = scale_at(p, extra, x / (KT * kSub), k);
        if (k >= valid)
          asm volatile("st.shared.b32 [%0], %2;\n\tst.shared.b32 [%1], %2;" ::"r"(at_s), "r"(at_s + kBoth * kScales / 2),
                       "r"(0)
                       : "memory");
      }
      tc::fence_proxy_async_smem();  // before the next copy into the stage
      __syncwarp();
    }
    float s[KT][kCols][4], lv[KT][HT][2];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int z = 0; z < HT; ++z) {
        const uint32_t kt = stage + z * kHead + i * kTile, sc = scale_at(p, extra, z, i * kSub) + gq * 4;
#pragma unroll
        for (int t = z * HN; t < (z + 1) * HN; ++t) s[i][t][0] = s[i][t][1] = s[i][t][2] = s[i][t][3] = 0.f;
        [[maybe_unused]] float rest[HN][4] = {};  // of the queries' second terms, 2^11 times as large
#pragma unroll
        for (int c = 0; c < kWords / 4; ++c) {  // keys gq and gq + 8
          const uint4 lo = lds16(at(kt, gq, tq * (kWords / 4) + c)), hi = lds16(at(kt, gq + 8, tq * (kWords / 4) + c));
          const uint32_t r0[4] = {lo.x, lo.y, lo.z, lo.w}, r1[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a[4] = {low2(r0[w]), low2(r1[w]), high2(r0[w]), high2(r1[w])};
#pragma unroll
            for (int t = z * HN; t < (z + 1) * HN; ++t) mma16816h(s[i][t], a, qf[t][0][c * 4 + w][0], qf[t][0][c * 4 + w][1]);
            if constexpr (kTerms == 2) {
#pragma unroll
              for (int t = 0; t < HN; ++t)
                mma16816h(rest[t], a, qf[z * HN + t][1][c * 4 + w][0], qf[z * HN + t][1][c * 4 + w][1]);
            }
          }
        }
        if constexpr (kTerms == 2) {
#pragma unroll
          for (int t = 0; t < HN; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][z * HN + t][e] = fmaf(rest[t][e], 1.f / 2048.f, s[i][z * HN + t][e]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          lv[i][z][y] = lg2(lds1(sc + kBoth * kScales / 2 + 32 * y));
          const float ks = lds1(sc + 32 * y);
#pragma unroll
          for (int t = z * HN; t < (z + 1) * HN; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[i][t][2 * y + e] *= qs[2 * t + e] * ks;
        }
      }
    if (valid < KT * kSub) {  // whatever an infinite query makes of the zeros behind the end
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int t = 0; t < kCols; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i * kSub + gq + 8 * (e >> 1) >= valid) s[i][t][e] = -INFINITY;
    }
    // The maxima are only looked for across the lanes when some score is beyond 2^8 of its own.
    float mt[kM], mv[kM];
    bool up = false;
#pragma unroll
    for (int x = 0; x < kM; ++x) {
      const int t = x >> 1, e = x & 1, z = t / HN;
      mt[x] = fmaxf(s[0][t][e], s[0][t][2 + e]);
      mv[x] = fmaxf(s[0][t][e] + lv[0][z][0], s[0][t][2 + e] + lv[0][z][1]);
#pragma unroll
      for (int i = 1; i < KT; ++i) {
        mt[x] = tc::fmax3(mt[x], s[i][t][e], s[i][t][2 + e]);
        mv[x] = tc::fmax3(mv[x], s[i][t][e] + lv[i][z][0], s[i][t][2 + e] + lv[i][z][1]);
      }
      up |= mt[x] > m[x] + kFdLazy || mv[x] > mw[x] + (kFdLazy + kTop);
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const float mn = fmaxf(m[i], qmax(mt[i])), wn = fmaxf(mw[i], qmax(mv[i]) - kTop);
        l[i] *= mn == m[i] ? 1.f : ex2d(m[i] - mn);
        const float a = wn == mw[i] ? 1.f : ex2d(mw[i] - wn);
        m[i] = mn;
        mw[i] = wn;
        nm[i] = mn == -INFINITY ? 0.f : -mn;
        nw[i] = wn == -INFINITY ? 0.f : -wn;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          acc[((i >> 1) * (D / 16) + k) * 4 + (i & 1)] *= a;
          acc[((i >> 1) * (D / 16) + k) * 4 + 2 + (i & 1)] *= a;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int z = 0; z < HT; ++z) {
        const uint32_t vt = stage + z * kHead + (KT + i) * kTile;
        uint32_t b[HN][kTerms][2];
#pragma unroll
        for (int n = 0; n < HN; ++n) {
          const int t = z * HN + n;
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = 2 * t + (e & 1);
            l[x] += ex2d(s[i][t][e] + nm[x]);
            w[e] = ex2d((s[i][t][e] + nw[x]) + lv[i][z][e >> 1]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t hi = pack_f16(w[2 * y], w[2 * y + 1]);
            b[n][0][y] = trans8(hi);
            if constexpr (kTerms == 2) b[n][1][y] = trans8(rest_f16(hi, w[2 * y], w[2 * y + 1]));
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
            auto sum = [&](int n) -> float(&)[4] {
              return reinterpret_cast<float(&)[4]>(acc[((z * HN + n) * (D / 16) + 2 * w + y) * 4]);
            };
#pragma unroll
            for (int n = 0; n < HN; ++n) mma16816h(sum(n), a, b[n][0][0], b[n][0][1]);
            if constexpr (kTerms == 2) {
#pragma unroll
              for (int n = 0; n < HN; ++n) {
                float rest[4] = {};
                mma16816h(rest, a, b[n][1][0], b[n][1][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum(n)[e] = fmaf(rest[e], 1.f / 2048.f, sum(n)[e]);
              }
            }
          }
        }
      }
  }
  // The weights' own maximum is taken out again: from here on a state is as any other's.
  // Scales down to 2^-126 make a factor below fp32's normal numbers of values that
  // are normal, so what is below 2^-100 of it comes second.
  __device__ __forceinline__ void finish() {
    bool low = false;
    auto times = [&](int i, float a) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        acc[((i >> 1) * (D / 16) + k) * 4 + (i & 1)] *= a;
        acc[((i >> 1) * (D / 16) + k) * 4 + 2 + (i & 1)] *= a;
      }
    };
#pragma unroll
    for (int i = 0; i < kM; ++i) {
      mw[i] = mw[i] == -INFINITY ? 0.f : mw[i] - m[i];
      low |= mw[i] < kLeast;
      times(i, ex2d(fmaxf(mw[i], kLeast)));
    }
    if (__any_sync(0xffffffffu, low)) {
#pragma unroll
      for (int i = 0; i < kM; ++i) times(i, ex2d(fminf(mw[i] - kLeast, 0.f)));
    }
  }
  // head h of column t, or -1
  __device__ __forceinline__ int head(int t, int h) const {
    const int x = (t % HN) * 8 + h;
    return HT == 1 ? x : x < per ? (t / HN) * per + x : -1;
  }
  // dims that a lane has of a head, which lie together
  static constexpr int kRunDims = D / 8;
  template <typename F>
  __device__ __forceinline__ void each_run(F f) const {
    const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < kCols; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = head(t, 2 * tq + e);
        if (HT > 1 && h < 0) continue;
        float v[kRunDims];
#pragma unroll
        for (int k = 0; k < kRunDims; ++k) v[k] = acc[(t * (D / 16) + (k >> 1)) * 4 + 2 * (k & 1) + e];
        f(h, 2 * t + e, gq * kRunDims, v);
      }
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
      for (int x = 0; x < kM; ++x) {
        const int h = head(x >> 1, 2 * tq + (x & 1));
        if (HT == 1 || h >= 0) f(h, x);
      }
    }
  }
  __device__ __forceinline__ static int m_index(int x) { return 2 * (x / (D / 4)) + (x & 1); }
};

bool map_codes(CUtensorMap* m, const void* p, uint64_t rows, int Hkv, int d, int box_rows) {
  const uint64_t D = d;
  const uint64_t dims[3] = {D, uint64_t(Hkv), rows};
  const uint64_t strides[2] = {D, D * Hkv};
  const uint32_t box[3] = {uint32_t(d), 1, uint32_t(box_rows)};
  return make_tmap_u8(m, p, 3, dims, strides, box, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}
bool map_scales(CUtensorMap* m, const float* p, const PageMap& pages, int Hkv, int box_rows) {
  const uint64_t size = uint64_t(1) << pages.page_log2;
  const uint64_t dims[3] = {size, uint64_t(Hkv), uint64_t(pages.num_pages)};
  const uint64_t strides[2] = {size * 4, size * 4 * Hkv};
  const uint32_t box[3] = {uint32_t(box_rows), 2, 1};
  return make_tmap_f32(m, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}
template <typename T, int D, int H, int KT, int HT>
cudaError_t run(Fd8Params& p, cudaStream_t stream) {
  using C = Core8<T, D, H, KT, HT>;
  p.box_log2 = C::kBig ? std::min(p.pages.page_log2, FdShape<C>::kStepLog2) : 4;
  const int box = 1 << p.box_log2;
  const uint64_t rows = uint64_t(p.pages.num_pages) << p.pages.page_log2;
  if (!map_codes(&p.tmK, p.k, rows, p.kv_heads, D, box) || !map_codes(&p.tmV, p.v, rows, p.kv_heads, D, box))
    return cudaErrorInvalidValue;
  if (C::kPairScales && (!map_scales(&p.tmKs, p.k_scale, p.pages, p.kv_heads, box) || !map_scales(&p.tmVs, p.v_scale, p.pages, p.kv_heads, box)))
    return cudaErrorInvalidValue;
  return decode<C, false>(p, "full_decode_fp8", stream);
}
// Whether items are pairs of key/value heads. fp32 queries are two terms, whose registers leave no room for them.
bool in_pairs(int Hkv, int group, int dtype) { return dtype == MSA_BF16 && group <= 8 && Hkv % 2 == 0; }
// Floats of the partials: two to a warp's run, of an item's heads
size_t part_floats(int Hkv, int group, int d, int dtype) {
  const int heads = std::min(in_pairs(Hkv, group, dtype) ? 2 * group : group, kFdMaxHeads);
  return size_t(2) * fd_grid() * 8 * heads * d;
}
// Up to 8 query heads to a key/value head: a step has two tiles, of neighbouring
// heads or of 32 keys, for d 64 four (a step's waits and look-ups cost as much as
// for d 128: one key/value head 456 us, with two tiles 559, before copies took whole steps). More: two of keys.
// d 64: 6.0 to 6.6 TB/s, bound by instructions: a key's scores and weights take as many
// as for d 128, its bytes half (four heads of one tile instead of two of two: 7 % slower).
template <int D>
cudaError_t run_bf16(Fd8Params& p, cudaStream_t stream) {
  using T = __nv_bfloat16;
  if (p.group > 8) return run<T, D, 16, 2, 1>(p, stream);
  if (!in_pairs(p.kv_heads, p.group, MSA_BF16)) return run<T, D, 8, D == 64 ? 4 : 2, 1>(p, stream);
  p.Hkv = p.kv_heads / 2;  // pairs, as the items' heads
  p.hpg = 2 * p.group;
  p.ngr = 1;
  return run<T, D, 8, D == 64 ? 2 : 1, 2>(p, stream);
}
template <int D>
cudaError_t run_f32(Fd8Params& p, cudaStream_t stream) {
  return p.group > 8 ? run<float, D, 16, 2, 1>(p, stream) : run<float, D, 8, 2, 1>(p, stream);
}

}  // namespace

size_t full_decode_fp8_ws_bytes(int Hkv, int hpg, int d, int dtype) {
  const size_t n = part_floats(Hkv, hpg, d, dtype);
  return up256(n * 4) + up256(n / d * 8);
}

cudaError_t launch_full_decode_fp8(const FullArgs& a, const float* k_scale, const float* v_scale, cudaStream_t stream) {
  Fd8Params p{};
  static_cast<FdParams&>(p) = fd_params(a, 0);
  p.part_ml = p.part_o + up256(part_floats(p.Hkv, p.hpg, a.d, a.dtype) * 4) / 4;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.kv_heads = p.Hkv;
  p.group = p.hpg;
  p.inject_timeout = debug_inject_timeout() ? 1 : 0;
  if (a.dtype == MSA_BF16) return a.d == 128 ? run_bf16<128>(p, stream) : run_bf16<64>(p, stream);
  return a.d == 128 ? run_f32<128>(p, stream) : run_f32<64>(p, stream);
}

}  // namespace msa
