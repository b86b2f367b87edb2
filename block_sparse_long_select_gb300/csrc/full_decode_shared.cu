// Decode over shared prefixes: each sequence's own keys by the decode kernel's
// walk (full_decode.cuh), whose joins take in the parts that the prefixes' grid
// left (full_prefix_tc.cu, full_prefix_fp32.cu). The grid starts while that one
// ends and waits for it before its first join.
#include "full_decode_cores.cuh"

namespace msa {
namespace {

constexpr int kSharedSlots = kNumSMs * 8;  // a slot for every warp

template <typename T, int D, int H>
cudaError_t run(const FdParams& p, cudaStream_t stream) {
  return decode<Core<T, D, H>, true>(p, "full_decode_shared", stream);
}
PrefixGeometry geometry(int hpg, int dtype) { return dtype == MSA_BF16 ? prefix_geometry_tc(hpg) : prefix_geometry_f32(hpg); }
// most rows of all parts: every item's (an alt item's twice), and a block for every CTA that an item goes on in
size_t part_rows(const PrefixGeometry& g, int B, int Hkv) {
  return size_t(B) * Hkv * g.groups * g.heads * (g.half > 0 ? 2 : 1) + size_t(g.grid) * g.block;
}

}  // namespace

size_t full_shared_ws_bytes(int B, int groups, int Hkv, int hpg, int d, int dtype) {
  const size_t rows = part_rows(geometry(hpg, dtype), B, Hkv);
  return fd_part_bytes(kSharedSlots, d) + up256(size_t(groups) * sizeof(PrefixRec)) + up256(rows * sizeof(float2)) +
         up256(rows * d * sizeof(float));
}

cudaError_t launch_decode_shared(const FullArgs& a, const int32_t* cu_prefix, const int32_t* prefix_len, int groups,
                                 cudaStream_t stream) {
  const int B = a.seq.B, hpg = a.Hq / a.Hkv;
  SharedParams s{};
  s.groups = SeqMap{cu_prefix, nullptr, prefix_len, groups, B, a.seq.Tk};
  s.prefix_len = prefix_len;
  s.disorder = &static_cast<WsHeader*>(a.ws)->disorder;
  s.geo = geometry(hpg, a.dtype);
  char* w = static_cast<char*>(a.ws) + kWsHeader + fd_part_bytes(kSharedSlots, a.d);
  s.recs = reinterpret_cast<PrefixRec*>(w);
  w += up256(size_t(groups) * sizeof(PrefixRec));
  s.stat = reinterpret_cast<float2*>(w);
  s.part = reinterpret_cast<float*>(w + up256(part_rows(s.geo, B, a.Hkv) * sizeof(float2)));
  if (cudaError_t e = launch_order_check(s.groups, a.ws, stream)) return e;
  const SharedArgs args{a, s};
  if (cudaError_t e = a.dtype == MSA_BF16 ? launch_prefix_tc(args, stream) : launch_prefix_f32(args, stream)) return e;
  FdParams p = fd_params(a, kSharedSlots);
  p.shared = s;
  const bool wide = hpg > 8, few = hpg <= 4;  // as in full_decode.cu
  if (a.dtype == MSA_BF16) {
    if (a.d == 128) return wide ? run<__nv_bfloat16, 128, 16>(p, stream) : run<__nv_bfloat16, 128, 8>(p, stream);
    return wide ? run<__nv_bfloat16, 64, 16>(p, stream) : run<__nv_bfloat16, 64, 8>(p, stream);
  }
  if (a.d == 128) return wide ? run<float, 128, 16>(p, stream) : few ? run<float, 128, 4>(p, stream) : run<float, 128, 8>(p, stream);
  return wide ? run<float, 64, 16>(p, stream) : few ? run<float, 64, 4>(p, stream) : run<float, 64, 8>(p, stream);
}

}  // namespace msa
