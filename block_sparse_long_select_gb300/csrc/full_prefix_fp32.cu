// Decode over shared prefixes, the prefixes' part in fp32 on CUDA cores
// (formulas and parts: full_prefix_tc.cu, full_shared.cuh). An item is 32 rows:
// sequences x up to 16 heads; the engine is the prefill's (full_fp32_tiles.cuh).
// Bound: FMAs and the shared-memory reads beside them. Measured, the whole call (Hq 8,
// Hkv 2, d 64): 10 sequences behind two prefixes of up to 600 keys 20 us, the latency
// of its four grids.
#include "full_fp32_tiles.cuh"
#include "full_shared.cuh"

namespace msa {
namespace {

struct PfxParams {
  SharedParams s;
  PageMap pages;
  const float *q, *k, *v;
  int Hq, Hkv, hpg;
  float scale_log2;
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kF32Threads, 2) full_prefix_f32_kernel(const PfxParams p) {
  extern __shared__ __align__(128) uint8_t pfx_smem[];
  __shared__ PrefixPart part_s;
  __shared__ int state_s;  // 0: a part to compute, 1: one with bad pages, 2: no more
  const uint32_t sq = tc::smem_u32(pfx_smem), sk = sq + kA * D * 4, sv = sk + kB * D * 4, sp = sv + kB * D * 4;
  const int tx = tile_x(), ty = tile_y(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tc::griddep_wait();               // the plan
  tc::griddep_launch_dependents();  // behind it, so that the decode grid, which may start now, has it as well
  PrefixRuns plan{p.s, p.Hkv};
  bool some = false;
  if (warp == 0) some = plan.init(p.s.get_head(), blockIdx.x);
  const int psz = 1 << p.pages.page_log2, heads = p.s.geo.heads;
  for (;;) {
    if (warp == 0) {
      int state = 2;
      if (some && plan.at < plan.end) {
        const PrefixPart d = plan.next();
        const int32_t* row = p.pages.table + int64_t(d.leader) * p.pages.max_pages;
        const int per = kPxKeys >> p.pages.page_log2, to = min((d.jb + d.n) * per, d.Lk >> p.pages.page_log2);
        bool bad = false;
        for (int x = d.jb * per + lane; x < to; x += 32) bad |= row[x] < 0 || row[x] >= p.pages.num_pages;
        state = __any_sync(0xffffffffu, bad) ? 1 : 0;
        if (lane == 0) part_s = d;
        if (state == 1 && lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
      }
      if (lane == 0) state_s = state;
    }
    __syncthreads();
    if (state_s == 2) return;
    const PrefixPart d = part_s;
    const bool bad = state_s == 1;
    const int32_t* table = p.pages.table + int64_t(d.leader) * p.pages.max_pages;
    const int j0 = d.jb * kPxKeys, end = min((d.jb + d.n) * kPxKeys, d.Lk), n = bad ? 0 : ceil_div(end - j0, kB);
    // row r: sequence r / heads, head r % heads of the item's
    auto has = [&](int r) { return r / heads < d.count && d.hg * heads + r % heads < p.hpg; };
    auto key = [&](const float* base, int j) -> const float* {
      if (j >= end) return nullptr;
      const int64_t row = (int64_t(table[j >> p.pages.page_log2]) << p.pages.page_log2) + (j & (psz - 1));
      return base + (row * p.Hkv + d.g) * D;
    };
    load_tile<D, kA>(sq, p.q, [&](int r) {
      return has(r) ? p.q + (int64_t(d.b0 + r / heads) * p.Hq + d.g * p.hpg + d.hg * heads + r % heads) * D : nullptr;
    });
    if (n > 0) load_tile<D, kB>(sk, p.k, [&](int r) { return key(p.k, j0 + r); });
    cp_commit_f();
    if (n > 0) load_tile<D, kB>(sv, p.v, [&](int r) { return key(p.v, j0 + r); });
    cp_commit_f();
    float m[4], l[4];
    uint64_t acc[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[i][c] = 0;
    }
    for (int j = 0; j < n; ++j) {
      cp_wait_f<1>();
      __syncthreads();
      float sc[4][4];
      dots<D>(sq, sk, sc);
      __syncthreads();  // K is read
      if (j + 1 < n) load_tile<D, kB>(sk, p.k, [&](int r) { return key(p.k, j0 + (j + 1) * kB + r); });
      cp_commit_f();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[i][k] = j0 + j * kB + tx + 16 * k < end ? sc[i][k] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, sc[i][k]);
        }
        const float mn = fmaxf(m[i], row_max(mx));
        const float z = mn == -INFINITY ? 0.f : mn, a = ex2(m[i] - z);  // no branch: rows of a warp differ
        m[i] = mn;
        l[i] *= a;
        const uint64_t aa = pair(a, a);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = mul2(acc[i][c], aa);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[i][k] = ex2(sc[i][k] - z);
          l[i] += sc[i][k];
        }
      }
      put(sp, sc);
      cp_wait_f<1>();
      __syncthreads();
      sums<D>(sp, sv, acc);
      __syncthreads();  // V and P are read
      if (j + 1 < n) load_tile<D, kB>(sv, p.v, [&](int r) { return key(p.v, j0 + (j + 1) * kB + r); });
      cp_commit_f();
    }
    cp_wait_f<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float den = row_sum(l[i]);
      const int r = ty * 4 + i;
      if (!has(r)) continue;
      store_rows<D>(p.s.part + (d.row + r) * D, acc[i], 1.f);
      if (tx == 0) p.s.stat[d.row + r] = bad ? make_float2(-INFINITY, -1.f) : make_float2(m[i], den);
    }
    __syncthreads();  // Q and part_s are read before the next part's
  }
}

template <int D>
cudaError_t prefix(const SharedArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  PfxParams p{};
  p.s = a.s;
  p.pages = f.pages;
  p.q = static_cast<const float*>(f.q);
  p.k = static_cast<const float*>(f.k);
  p.v = static_cast<const float*>(f.v);
  p.Hq = f.Hq;
  p.Hkv = f.Hkv;
  p.hpg = f.Hq / f.Hkv;
  p.scale_log2 = f.scale * kLog2e;
  p.status = &static_cast<WsHeader*>(f.ws)->status;
  auto kern = full_prefix_f32_kernel<D>;
  constexpr int bytes = (kA + 2 * kB) * D * 4 + kA * kPitch * 4;
  static KernelReady ready;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), bytes)) return e;
  ProfScope pf("full_prefix", stream);
  return launch_early(kern, a.s.geo.grid, kF32Threads, bytes, stream, p);
}

}  // namespace

PrefixGeometry prefix_geometry_f32(int hpg) {
  // Every group of two or more is items. Measured (Hq 8, Hkv 2, d 64; `worth` 1, 4, 16): 1000 sequences of 100 keys in
  // 250 groups behind 128 keys 67, 61, 67 us, behind 512 112, 112, 114; 512 of 200 in 256 behind 256 67, 67, 58; 200 of
  // 100 in 50 behind 1024 61, 61, 56; ten in two groups behind up to 600 19, 19, 15; 32 of 100 behind 8 K 38 with each.
  const int heads = hpg < 16 ? hpg : 16;
  return {heads, ceil_div(hpg, heads), kA / heads, 0, kA, 2 * kNumSMs, 1, 0, 1};
}

cudaError_t launch_prefix_f32(const SharedArgs& a, cudaStream_t stream) {
  return a.f.d == 128 ? prefix<128>(a, stream) : prefix<64>(a, stream);
}

}  // namespace msa
