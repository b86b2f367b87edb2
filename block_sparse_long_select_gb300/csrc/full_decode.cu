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
// bf16: mma.sync m16n8k16 with keys (then head dims) along M and the heads
// along N = 8: the tensor work is a fraction of the time the bytes take, so
// tcgen05's larger tiles would only pad. fp32: FMAs, one key per lane pair for
// the scores, four head dims per lane for the products.
#include "full_decode_cores.cuh"

namespace msa {

size_t full_decode_ws_bytes(int d) { return fd_part_bytes(2 * fd_grid(), d); }

namespace {
template <typename T, int D, int H>
cudaError_t run(const FdParams& p, cudaStream_t stream) {
  return decode<Core<T, D, H>, false>(p, "full_decode", stream);
}
}  // namespace

cudaError_t launch_full_decode(const FullArgs& a, cudaStream_t stream) {
  const FdParams p = fd_params(a, 2 * fd_grid());
  // bf16: a tile holds 8 heads, so fewer cost the same. fp32: the FMAs and
  // shared-memory reads are those of H heads, so up to 4 get a variant of half the work.
  const bool wide = p.hpg > 8, few = p.hpg <= 4;
  if (a.dtype == MSA_BF16) {
    if (a.d == 128) return wide ? run<__nv_bfloat16, 128, 16>(p, stream) : run<__nv_bfloat16, 128, 8>(p, stream);
    return wide ? run<__nv_bfloat16, 64, 16>(p, stream) : run<__nv_bfloat16, 64, 8>(p, stream);
  }
  if (a.d == 128) return wide ? run<float, 128, 16>(p, stream) : few ? run<float, 128, 4>(p, stream) : run<float, 128, 8>(p, stream);
  return wide ? run<float, 64, 16>(p, stream) : few ? run<float, 64, 4>(p, stream) : run<float, 64, 8>(p, stream);
}

}  // namespace msa
