// Shared by the tcgen05 kernels of full attention.
#pragma once

#include "full_internal.cuh"
#include "tc_utils.cuh"

namespace msa {

constexpr int kRows = 128, kKeys = 128;  // rows (tokens x group heads) and keys of a tile
constexpr uint32_t kHalfTile = 128 * 128;  // bytes of one 64-wide half of 128 rows (128B-swizzled)
constexpr float kLog2e = 1.4426950408889634f, kLn2f = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// A wait of a whole warp: every lane gets the same answer, so that none leaves
// a loop whose warp-wide operations the others still run.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort));
}
// Zeroes rows [from, to) of a [D / 64][128 rows][128 B] tile (one warp); the
// caller fences the writes towards the async proxy.
template <int NH>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to) {
  const int per = (to - from) * 8;
  for (int x = threadIdx.x & 31; x < per * NH; x += 32)
    *reinterpret_cast<uint4*>(tile + (x / per) * kHalfTile + from * 128 + (x % per) * 16) = make_uint4(0, 0, 0, 0);
}

// TMA maps: row tiles [tokens][hpg heads][64 dims] of a [Tq, Hq, d] tensor, and
// key tiles [rows][1 head][64 dims] of a [rows, Hkv, d] one.
inline bool map_rows(CUtensorMap* m, const void* p, int Tq, int Hq, int Hkv, int d, int tpt) {
  const uint64_t e = 2, D = d, hpg = Hq / Hkv;
  const uint64_t dims[4] = {D, hpg, uint64_t(Hkv), uint64_t(Tq)};
  const uint64_t strides[3] = {D * e, D * e * hpg, D * e * Hq};
  const uint32_t box[4] = {64, uint32_t(hpg), 1, uint32_t(tpt)};
  return make_tmap_bf16(m, p, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
inline bool map_keys(CUtensorMap* m, const void* p, uint64_t rows, int Hkv, int d, int box_rows) {
  const uint64_t e = 2, D = d;
  const uint64_t dims[3] = {D, uint64_t(Hkv), rows};
  const uint64_t strides[2] = {D * e, D * e * Hkv};
  const uint32_t box[3] = {64, 1, uint32_t(box_rows)};
  return make_tmap_bf16(m, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace msa
