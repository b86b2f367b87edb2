// The fp32 kernels' matrix engine on CUDA cores.
// A CTA of 128 threads keeps a
// tile of 32 rows in shared memory (queries x group heads; in dkv, keys) and
// streams 64 rows of the other side past it. A thread computes 4 x 4 dot
// products, 4 16-byte loads of either side for 64 FMAs (two to an instruction);
// the 32 x 64 results go through shared memory to the second product, where it
// owns 4 rows x D / 16 columns. 32 rows and not 64 because several small CTAs
// per SM hide each other's barriers, and short calls need the number of CTAs.
// Rows that belong to no pair arrive as zeros.
#pragma once

#include "full_tc.cuh"

namespace msa {
namespace {

constexpr int kF32Threads = 128, kA = 32, kB = 64;  // resident rows, streamed rows
constexpr int kPitch = kB + 4;                      // floats of a row of the 32 x 64 results
// CTAs per SM that registers are kept for: what shared memory allows, in fp32
// tiles of D columns (left to itself the compiler spills to fit a fourth: 66 us
// for prompts up to 999 tokens instead of 62).
template <int D>
constexpr int kF32Ctas = D == 64 ? 3 : 2;

// A thread's place in the 16 x 8 grid over a tile: a warp has 16 columns and 2
// rows, the lanes l and l ^ 1 share a column. A 16-byte shared load of a warp
// takes 2 cycles if within every quad no more than two addresses occur, else 4
// (measured). So the 8 loads per 64 FMAs take 16 cycles, as the FMAs do; with
// half warps as rows they took 24 (prompts up to 999 tokens 60 -> 55 us).
__device__ __forceinline__ int tile_x() { return int((threadIdx.x & 31) >> 1); }
__device__ __forceinline__ int tile_y() { return int((threadIdx.x >> 5 << 1) | (threadIdx.x & 1)); }

__device__ __forceinline__ void cp16f(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit_f() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait_f() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
struct Pairs {
  uint64_t lo, hi;  // two floats each
};
__device__ __forceinline__ Pairs lds_pairs(uint32_t a) {
  Pairs v;
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.lo), "=l"(v.hi) : "r"(a));
  return v;
}
// 16-byte chunk c of row r; chunks are exchanged within 128 bytes by the row's
// low bits, so reads down a column are free of bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t at(uint32_t base, int r, int c) {
  return base + uint32_t(r * D * 4) + (uint32_t(c ^ (r & 7)) << 4);
}

// Copies NR rows of D floats into a tile: row(r) is a row's address, or null for zeros.
template <int D, int NR, typename F>
__device__ __forceinline__ void load_tile(uint32_t dst, const float* any, F row) {
  constexpr int kC = D / 4, kStep = kF32Threads / kC;
  const int c = threadIdx.x % kC;
#pragma unroll 4
  for (int r = threadIdx.x / kC; r < NR; r += kStep) {
    const float* src = row(r);
    cp16f(at<D>(dst, r, c), src ? src + c * 4 : any, src != nullptr);
  }
}

// acc[i][k] = A row (4 ty + i) . B row (tx + 16 k)
template <int D>
__device__ __forceinline__ void dots(uint32_t a, uint32_t b, float (&acc)[4][4]) {
  const int tx = tile_x(), ty = tile_y();
  uint64_t sum[4][4];  // of even and of odd columns
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[i][k] = 0;
  // at<D>() with what is common to four chunks taken out: the low two bits of a
  // row's exchange are added to a chunk's, the third flips a group of four
  const uint32_t xa = a + uint32_t(ty * 4 * D * 4), ya = b + uint32_t(tx * D * 4);
  const int xs = (ty & 1) << 2, ys = tx & 4;
#pragma unroll 2
  for (int c0 = 0; c0 < D / 4; c0 += 4) {
    const uint32_t xc = xa + uint32_t((c0 ^ xs) << 4), yc = ya + uint32_t((c0 ^ ys) << 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t yo = yc + uint32_t((c ^ (tx & 3)) << 4);
      Pairs x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = lds_pairs(xc + uint32_t(i * D * 4 + ((c ^ i) << 4)));
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = lds_pairs(yo + uint32_t(16 * k * D * 4));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[i][k] = fma2(x[i].lo, y[k].lo, sum[i][k]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[i][k] = fma2(x[i].hi, y[k].hi, sum[i][k]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = split(sum[i][k]);
      acc[i][k] = f.x + f.y;
    }
}
// The thread's 4 x 4 results into the 32 x 64 matrix.
__device__ __forceinline__ void put(uint32_t m, const float (&v)[4][4]) {
  const int tx = tile_x(), ty = tile_y();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(m + ((ty * 4 + i) * kPitch + tx + 16 * k) * 4), "f"(v[i][k]) : "memory");
}
// acc[i][..] += sum over the 64 streamed rows of m[4 ty + i][row] * row's columns;
// the thread's columns are the 16-byte chunks tx, tx + 16, ...
// (pairs: columns 2 e and 2 e + 1 in acc[i][e]).
template <int D>
__device__ __forceinline__ void sums(uint32_t m, uint32_t b, uint64_t (&acc)[4][D / 32]) {
  const int tx = tile_x(), ty = tile_y();
#pragma unroll 2
  for (int j = 0; j < kB; j += 4) {
    float w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = lds4(m + ((ty * 4 + i) * kPitch + j) * 4);
      w[i][0] = f.x, w[i][1] = f.y, w[i][2] = f.z, w[i][3] = f.w;
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const Pairs f = lds_pairs(at<D>(b, j + y, tx + 16 * c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t ww = pair(w[i][y], w[i][y]);
          acc[i][2 * c] = fma2(ww, f.lo, acc[i][2 * c]);
          acc[i][2 * c + 1] = fma2(ww, f.hi, acc[i][2 * c + 1]);
        }
      }
  }
}
__device__ __forceinline__ float row_max(float x) {  // over the 16 threads of a row
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int D>
__device__ __forceinline__ void store_rows(float* dst, const uint64_t (&acc)[D / 32], float mul) {
  const int tx = tile_x();
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const float2 lo = split(acc[2 * c]), hi = split(acc[2 * c + 1]);
    reinterpret_cast<float4*>(dst)[tx + 16 * c] = make_float4(lo.x * mul, lo.y * mul, hi.x * mul, hi.y * mul);
  }
}

}  // namespace
}  // namespace msa
