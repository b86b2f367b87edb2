// Decode over shared prefixes: each sequence's own keys by the decode kernel's
// walk (full_decode.cuh), and the join of its parts with those that the
// prefixes' grid left (full_prefix_tc.cu, full_prefix_fp32.cu). Each of the three
// grids behind the plan starts while the one before it ends. Bound: HBM while both
// walks run, and about 20 us of plan, first loads and joins. Measured, whole calls (Hq 32,
// Hkv 8, d 128, bf16; bytes that have to be read at the copy rate: 87, 87, 7 us): 97
// sequences of 1300 own keys behind three prefixes, 20 K keys, 108 us; 24 behind
// 128 K keys 107; 32 of up to 200 behind 8 K 28. The 20 us are there however little is
// shared: full_decode.cu's one grid is as fast up to about 16 K keys of prefix times
// sequences (16 sequences behind 1 K: 19 us both; 4 behind 8 K: 24 and 23).
#include "full_decode_cores.cuh"

namespace msa {
namespace {

// A thread per four values of a query head, or of four heads of one key/value head;
// D / 4 of them a head. All but the parts is known before the grids that leave
// them end. Bound by latency: few rows have twenty parts in flight, many rows four
// of four heads, whose places are found once (128 000 rows 62 us; a head to a thread
// took 1.4, ten parts in flight 2.1 times as long). Ten parts in 80 registers spill
// 56 bytes, a head to a thread in 40 registers 96. Small CTAs fit beside the decode grid's.
constexpr int kJoinThreads = 128;
template <typename T, int D, int BATCH, int CTAS, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, CTAS) full_join_kernel(const FdParams p) {
  constexpr int kLanes = D / 4;
  const int64_t row = (int64_t(blockIdx.x) * (kJoinThreads / kLanes) + threadIdx.x / kLanes) * ROWS;
  const int dim = (threadIdx.x % kLanes) * 4;
  if (row >= int64_t(p.B) * p.Hq) {
    tc::griddep_wait();
    return;
  }
  const int b = int(row / p.Hq), h = int(row % p.Hq), g = h / p.hpg, hg = h - g * p.hpg;
  const int64_t step0 = __ldcg(p.shared.step0 + b);  // in flight with the others
  const SharedHead head = p.shared.get_head();
  Own own = own_of<true>(p, b);
  own.ok &= !head.disorder;
  PrefixRows<D> pre{nullptr, nullptr, 0, 0};
  const int heads = min(p.hpg, kFdMaxHeads);
  int64_t part0 = 0;  // the parts of its own keys
  int parts = 0;
  if (own.ok && own.L > 0) {  // (nothing else holds where cu_prefix is out of order)
    pre = p.shared.rows<D>(own.x, b, g, hg, head.per);
    if (const int n = own.units(4)) {
      const int it = g * p.ngr + hg / heads;
      const int64_t at = step0 + int64_t(it) * (n + kOwnItemSteps) + kOwnItemSteps, c0 = at / head.own_per;
      part0 = int64_t(b) * p.Hkv * p.ngr + it + c0;
      parts = int((at + n - 1) / head.own_per - c0) + 1;
    }
  }
  tc::griddep_wait();
  if (parts + pre.n == 0) {
    if (!own.ok && dim == 0) set_status(p.status, MSA_ERR_BOUNDS);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      T* dst = static_cast<T*>(p.out) + (row + r) * D + dim;
#pragma unroll
      for (int y = 0; y < 4; ++y) dst[y] = from_f<T>(0.f);
      if (p.lse && dim == 0) p.lse[row + r] = -INFINITY;
    }
    return;
  }
  join_head<T, BATCH, ROWS>(p, row, D, dim, parts + pre.n, [&](int y) {
    if (y >= parts) return pre.part(y - parts);
    const int64_t at = (part0 + y) * heads + hg % heads;
    return PartAt{p.part_o + at * D, p.part_ml + at * 2};
  });
}

template <typename T, int D, int BATCH, int CTAS, int ROWS>
cudaError_t launch_join(const FdParams& p, cudaStream_t stream) {
  ProfScope pf("full_join", stream);
  const int64_t threads = int64_t(p.B) * p.Hq / ROWS * (D / 4);
  return launch_early(full_join_kernel<T, D, BATCH, CTAS, ROWS>, (threads + kJoinThreads - 1) / kJoinThreads, kJoinThreads, 0,
                      stream, p);
}
template <typename T, int D>
cudaError_t join(const FdParams& p, cudaStream_t stream) {
  const int64_t ctas = int64_t(p.B) * p.Hq * (D / 4) / kJoinThreads;
  if (ctas < 3 * kNumSMs) return launch_join<T, D, 20, 3, 1>(p, stream);
  if (ctas < 8 * kNumSMs) return launch_join<T, D, 10, 6, 1>(p, stream);
  return p.hpg % 4 == 0 ? launch_join<T, D, 4, 4, 4>(p, stream) : launch_join<T, D, 4, 12, 1>(p, stream);
}
template <typename T, int D, int H>
cudaError_t run(const FdParams& p, cudaStream_t stream) {
  if (cudaError_t e = decode<Core<T, D, H>, true>(p, "full_decode_shared", stream)) return e;
  return join<T, D>(p, stream);
}

PrefixGeometry geometry(int hpg, int dtype) { return dtype == MSA_BF16 ? prefix_geometry_tc(hpg) : prefix_geometry_f32(hpg); }
// The workspace behind the header.
struct Regions {
  size_t head, seqs, step0, recs, stat, part, own_stat, own_part, end;
  Regions(const PrefixGeometry& g, int B, int groups, int Hkv, int hpg, int d) {
    // every item's rows, and a block for every part beyond its first
    const size_t rows = size_t(B) * Hkv * g.groups * g.heads + size_t(prefix_most_parts(g)) * g.block;
    const size_t own_items = size_t(B) * Hkv * head_groups(hpg), own_rows = (own_items + fd_grid() * 8) * (hpg < kFdMaxHeads ? hpg : kFdMaxHeads);
    size_t at = kWsHeader;
    auto take = [&](size_t bytes) {
      const size_t r = at;
      at += up256(bytes);
      return r;
    };
    head = take(sizeof(SharedHead));
    seqs = take(size_t(B) * sizeof(SharedSeq));
    step0 = take(size_t(B) * sizeof(int64_t));
    recs = take(size_t(groups) * sizeof(PrefixRec));
    stat = take(rows * sizeof(float2));
    part = take(rows * d * sizeof(float));
    own_stat = take(own_rows * sizeof(float2));
    own_part = take(own_rows * d * sizeof(float));
    end = at;
  }
};

}  // namespace

size_t full_shared_ws_bytes(int B, int groups, int Hkv, int hpg, int d, int dtype) {
  return Regions(geometry(hpg, dtype), B, groups, Hkv, hpg, d).end - kWsHeader;
}

cudaError_t launch_decode_shared(const FullArgs& a, const int32_t* cu_prefix, const int32_t* prefix_len, int groups,
                                 cudaStream_t stream) {
  const int B = a.seq.B, hpg = a.Hq / a.Hkv;
  SharedParams s{};
  s.groups = SeqMap{cu_prefix, nullptr, prefix_len, groups, B, a.seq.Tk};
  s.prefix_len = prefix_len;
  s.geo = geometry(hpg, a.dtype);
  const Regions at(s.geo, B, groups, a.Hkv, hpg, a.d);
  char* w = static_cast<char*>(a.ws);
  s.head = reinterpret_cast<SharedHead*>(w + at.head);
  s.seqs = reinterpret_cast<SharedSeq*>(w + at.seqs);
  s.step0 = reinterpret_cast<int64_t*>(w + at.step0);
  s.recs = reinterpret_cast<PrefixRec*>(w + at.recs);
  s.stat = reinterpret_cast<float2*>(w + at.stat);
  s.part = reinterpret_cast<float*>(w + at.part);
  const SharedArgs args{a, s};
  const int warps = a.dtype == MSA_FP32 && a.d == 128 ? Core<float, 128, 4>::kWarps : Core<__nv_bfloat16, 128, 8>::kWarps;
  if (cudaError_t e = launch_shared_plan(args, warps, a.Hkv * head_groups(hpg), stream)) return e;
  if (cudaError_t e = a.dtype == MSA_BF16 ? launch_prefix_tc(args, stream) : launch_prefix_f32(args, stream)) return e;
  FdParams p = fd_params(a, 0);
  p.shared = s;
  p.part_ml = reinterpret_cast<float*>(w + at.own_stat);
  p.part_o = reinterpret_cast<float*>(w + at.own_part);
  const bool wide = hpg > 8, few = hpg <= 4;  // as in full_decode.cu
  if (a.dtype == MSA_BF16) {
    if (a.d == 128) return wide ? run<__nv_bfloat16, 128, 16>(p, stream) : run<__nv_bfloat16, 128, 8>(p, stream);
    return wide ? run<__nv_bfloat16, 64, 16>(p, stream) : run<__nv_bfloat16, 64, 8>(p, stream);
  }
  if (a.d == 128) return wide ? run<float, 128, 16>(p, stream) : few ? run<float, 128, 4>(p, stream) : run<float, 128, 8>(p, stream);
  return wide ? run<float, 64, 16>(p, stream) : few ? run<float, 64, 4>(p, stream) : run<float, 64, 8>(p, stream);
}

}  // namespace msa
