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
// Two fp32 operations per instruction (sm_100 and up): the same rate as single
// ones, but half the issue slots, which the epilogue warps share with the
// thread that issues the matrix products.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// ---- work split over a cluster ------------------------------------------------
// A call with few tiles gives each to a cluster of CTAs: they share the walk
// over the other side, leave fp32 partials in their own shared memory, and
// each adds up a slice of everybody's in rank order (deterministic) over
// distributed shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of all CTAs of the cluster; shared memory written before is seen after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 16-byte chunk c of row r of a fp32 partial [rows][D]; chunks are exchanged by
// the row's low bits, so that a thread per row writes without bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t part_at(uint32_t base, int r, int c) {
  return base + uint32_t(r) * (D * 4) + (uint32_t(c ^ (r & 7)) << 4);
}
// One thread's row: `cols` columns of TMEM into row r of a partial, from chunk c0 on (whole warp).
template <int D>
__device__ __forceinline__ void put_partial(uint32_t base, int r, int c0, uint32_t taddr, int cols) {
  for (int c = 0; c < cols; c += 32) {
    uint32_t o[32];
    tc::tmem_ld_32x32b_x32(taddr + c, o);
    tc::tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 8; ++x)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(part_at<D>(base, r, c0 + c / 4 + x)), "r"(o[4 * x]),
                   "r"(o[4 * x + 1]), "r"(o[4 * x + 2]), "r"(o[4 * x + 3])
                   : "memory");
  }
}
// CTAs of a cluster for `ctas` tiles that walk `steps` each on average: doubled
// while the grid stays within one wave of SMs and every CTA keeps several steps
// (33 tiles of up to 512 steps: 774 us alone, 399 in twos, 210 in fours); once
// more than that into two waves where walks are long and ragged (76 tiles of up
// to 28 steps: 46.5 us alone, 39.1 in twos, 53.5 in fours; but 80 tiles of 3
// steps: 28.7 alone, 38.7 in twos, because a CTA's start and end cost about five).
inline int cluster_split(int64_t ctas, int64_t steps) {
  int c = 1;
  while (c < 8 && steps >= 8 * c && (ctas * c * 2 <= kNumSMs || (c == 1 && ctas <= kNumSMs))) c *= 2;
  return c;
}
// `early`: the grid may start while the one before it in the stream ends (it
// waits for that one's writes itself).
template <typename... P, typename... A>
cudaError_t launch_clusters(KernelReady& ready, void (*kern)(P...), int64_t ctas, int cluster, int threads, int smem,
                            bool early, cudaStream_t stream, A... args) {
  if (ctas * cluster >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), smem)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas * cluster));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
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
