// Full attention in fp32 on CUDA cores: forward over packed or paged keys, and
// the backward over packed ones (formulas at full_prefill_tc.cu and
// full_backward_tc.cu).
//
// Bound: FMAs (the tensor cores have no fp32 products; tf32 would keep 11 bits),
// which the shared-memory reads beside them just keep up with; short calls are
// bound by the walk of their longest tile. Measured (d 64): one prompt of 4096
// tokens (Hq 32, Hkv 8) 1.81 ms, 38 TFLOP/s, half of the FMA rate; (Hq 8, Hkv 2)
// three prompts of up to 999 tokens 55 us (20 TFLOP/s), the gradients of three
// documents of up to 500 tokens 43 us (dk, dv) and 27 us (dq).
// Every kernel is the same small matrix engine: full_fp32_tiles.cuh.
#include "full_fp32_tiles.cuh"

namespace msa {
namespace {

// The thread's 4 rows into a partial [rows][D] in shared memory, from row r0 on.
template <int D>
__device__ __forceinline__ void put_rows(uint32_t part, int r0, const uint64_t (&acc)[4][D / 32]) {
  const int tx = tile_x(), ty = tile_y();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at<D>(part, r0 + ty * 4 + i, tx + 16 * c)),
                   "l"(acc[i][2 * c]), "l"(acc[i][2 * c + 1])
                   : "memory");
}
// This rank's slice of `rows` rows, summed over the cluster in rank order:
// dst(row) is where a row goes (null: nowhere), mul(row) its factor.
template <int D, typename F, typename M>
__device__ __forceinline__ void sum_ranks(uint32_t part, int rows, int rank, int cl, F dst, M mul) {
  const int per = rows / cl;
  for (int x = threadIdx.x; x < per * (D / 4); x += kF32Threads) {
    const int r = rank * per + x / (D / 4), c = x % (D / 4);
    float* to = dst(r);
    if (!to) continue;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int y = 0; y < cl; ++y) {
      const float4 f = ld_peer4(peer_addr(at<D>(part, r, c), y));
      s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
    }
    const float m = mul(r);
    reinterpret_cast<float4*>(to)[c] = make_float4(s.x * m, s.y * m, s.z * m, s.w * m);
  }
}

struct F32Params {
  const float *q, *k, *v, *dout;
  SeqMap seq;
  PageMap pages;
  int Hq, Hkv, hpg, nslots;
  float scale, scale_log2;
  const float2* rows;  // [Hkv][Tq][hpg]: lse in log2 units, delta (full_common.cu)
  float *out, *lse, *dq, *dk, *dv;
  uint32_t* status;
  const uint32_t* disorder;
};

// Row x (token x / hpg, head x % hpg of group g) of a sequence in a [Tq, Hq] array.
__device__ __forceinline__ int64_t row_of(const F32Params& p, const SeqSpan& s, int g, int x) {
  return (int64_t(s.q0) + x / p.hpg) * p.Hq + g * p.hpg + x % p.hpg;
}

// The row tile of CTA (or cluster) `work` of `works`: sequence, head, tile (-1:
// none). Up to 32 sequences: tiles ordered by their place in their sequence,
// the last places (the longest walks) first, and the order turned round on
// every second lap over the SMs. These CTAs are small and most calls put all of
// them on the SMs at once, a lap after the other, so what counts is that each
// SM's laps add up alike (three prompts of up to 999 tokens: the busiest SM had
// 1.7 times the average). More sequences: by slots, late places first. Sets the
// status where offsets are out of order. Whole CTA.
__device__ __forceinline__ int find_row_tile(const F32Params& p, int work, int works, int& g, int& tile, SeqSpan& s) {
  if (p.seq.B > 32) {
    const bool in_order = cta_in_order(p.seq, p.disorder);
    if (!in_order && threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
    g = work % p.Hkv;
    return find_tile(p.seq, in_order, false, kA, p.hpg, p.nslots - 1 - work / p.Hkv, tile, s);
  }
  const int lane = threadIdx.x & 31, lap = work / kNumSMs, at = work % kNumSMs;
  const int rank = lap * kNumSMs + (lap & 1 ? min(kNumSMs, works - lap * kNumSMs) - 1 - at : at);
  // the warp has all offsets in hand: those out of order cost a prefix maximum, no second way to search
  SeqSpan own{};
  if (lane < p.seq.B) own = seq_span(p.seq, lane);
  if (__any_sync(0xffffffffu, lane < p.seq.B && !span_in_order(p.seq, own))) {
    SpanFloor floor;
    floor.apply(p.seq, own);
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
  }
  const int mine = lane < p.seq.B && own.rows_ok ? (own.Lq * p.hpg + kA - 1) / kA : 0;
  // tiles at places >= x, of all heads
  auto from = [&](int x) { return int(__reduce_add_sync(0xffffffffu, max(mine - x, 0))) * p.Hkv; };
  if (rank >= from(0)) return -1;
  int lo = 0, hi = __reduce_max_sync(0xffffffffu, mine);  // from(lo) > rank >= from(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (from(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  const int nth = (rank - from(hi)) / p.Hkv;  // of the sequences that reach place lo
  g = (rank - from(hi)) % p.Hkv;
  tile = lo;
  const uint32_t reach = __ballot_sync(0xffffffffu, mine > lo);
  const int b = __ffs(__ballot_sync(0xffffffffu, mine > lo && __popc(reach & ((1u << lane) - 1u)) == nth)) - 1;
  auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, b); };
  s = SeqSpan{of(own.q0), of(own.Lq), of(own.k0), of(own.Lk), of(own.rows_ok) != 0, of(own.keys_ok) != 0, of(own.ok) != 0};
  return b;
}

// ---------------------------------------------------------------------------------
// forward: 32 rows; smem Q | K | V | P
// ---------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kF32Threads, kF32Ctas<D>) full_f32_kernel(const F32Params p) {
  extern __shared__ __align__(128) uint8_t f32_smem[];
  const uint32_t sq = tc::smem_u32(f32_smem), sk = sq + kA * D * 4, sv = sk + kB * D * 4, sp = sv + kB * D * 4;
  const int tx = tile_x(), ty = tile_y();
  int g, tile;
  SeqSpan s;
  const int b = find_row_tile(p, blockIdx.x, gridDim.x, g, tile, s);
  if (b < 0) return;
  const int x0 = tile * kA, x1 = min(x0 + kA, s.Lq * p.hpg);
  const int32_t* table = p.pages.table ? p.pages.table + int64_t(b) * p.pages.max_pages : nullptr;
  bool bad = !s.ok;
  if (!bad && table) {  // every page of the sequence in range, for all its rows alike
    const int np = (s.Lk + (1 << p.pages.page_log2) - 1) >> p.pages.page_log2;
    for (int x = threadIdx.x; x < np; x += kF32Threads) bad |= table[x] < 0 || table[x] >= p.pages.num_pages;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
  const int n = bad ? 0 : (max(s.Lk - s.Lq + (x1 - 1) / p.hpg + 1, 0) + kB - 1) / kB;
  auto key = [&](const float* base, int j) -> const float* {
    if (j >= s.Lk) return nullptr;
    const int64_t row = table ? (int64_t(table[j >> p.pages.page_log2]) << p.pages.page_log2) +
                                    (j & ((1 << p.pages.page_log2) - 1))
                              : int64_t(s.k0) + j;
    return base + (row * p.Hkv + g) * D;
  };
  load_tile<D, kA>(sq, p.q, [&](int r) { return x0 + r < x1 ? p.q + row_of(p, s, g, x0 + r) * D : nullptr; });
  if (n > 0) load_tile<D, kB>(sk, p.k, [&](int r) { return key(p.k, r); });
  cp_commit_f();
  if (n > 0) load_tile<D, kB>(sv, p.v, [&](int r) { return key(p.v, r); });
  cp_commit_f();
  int vis[4];  // keys the thread's rows see
  float m[4], l[4];
  uint64_t acc[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    vis[i] = s.Lk - s.Lq + (x0 + ty * 4 + i) / p.hpg + 1;
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
    if (j + 1 < n) load_tile<D, kB>(sk, p.k, [&](int r) { return key(p.k, (j + 1) * kB + r); });
    cp_commit_f();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sc[i][k] = j * kB + tx + 16 * k < vis[i] ? sc[i][k] * p.scale_log2 : -INFINITY;
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
    if (j + 1 < n) load_tile<D, kB>(sv, p.v, [&](int r) { return key(p.v, (j + 1) * kB + r); });
    cp_commit_f();
  }
  cp_wait_f<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float den = row_sum(l[i]);
    const int x = x0 + ty * 4 + i;
    if (x >= x1) continue;
    const int64_t row = row_of(p, s, g, x);
    const bool some = !bad && vis[i] > 0;  // scores that are all -inf divide 0 by 0, as the formula does
    store_rows<D>(p.out + row * D, acc[i], some ? 1.f / den : 0.f);
    if (p.lse && tx == 0) p.lse[row] = some ? (m[i] + log2f(den)) * kLn2f : -INFINITY;
  }
}

// ---------------------------------------------------------------------------------
// dq: 32 rows; smem Q | dO | K | V | dS
// ---------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kF32Threads, kF32Ctas<D>) full_f32_dq_kernel(const F32Params p) {
  extern __shared__ __align__(128) uint8_t f32_smem[];
  const uint32_t sq = tc::smem_u32(f32_smem), so = sq + kA * D * 4, sk = so + kA * D * 4, sv = sk + kB * D * 4,
                 sp = sv + kB * D * 4;
  const int tx = tile_x(), ty = tile_y();
  const int cl = cluster_size(), rank = cluster_rank(), work = blockIdx.x / cl;
  int g, tile;
  SeqSpan s;
  if (find_row_tile(p, work, gridDim.x / cl, g, tile, s) < 0) return;
  const int x0 = tile * kA, x1 = min(x0 + kA, s.Lq * p.hpg);
  const int n = s.ok ? (max(s.Lk - s.Lq + (x1 - 1) / p.hpg + 1, 0) + kB - 1) / kB : 0;
  auto key = [&](const float* base, int j) -> const float* {
    return j < s.Lk ? base + ((int64_t(s.k0) + j) * p.Hkv + g) * D : nullptr;
  };
  load_tile<D, kA>(sq, p.q, [&](int r) { return x0 + r < x1 ? p.q + row_of(p, s, g, x0 + r) * D : nullptr; });
  load_tile<D, kA>(so, p.q, [&](int r) { return x0 + r < x1 ? p.dout + row_of(p, s, g, x0 + r) * D : nullptr; });
  int vis[4];
  float2 rd[4];
  uint64_t acc[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = x0 + ty * 4 + i;
    vis[i] = s.Lk - s.Lq + x / p.hpg + 1;
    rd[i] = x < x1 ? p.rows[(int64_t(g) * p.seq.Tq + s.q0) * p.hpg + x] : make_float2(INFINITY, 0.f);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[i][c] = 0;
  }
  for (int j = n * rank / cl; j < n * (rank + 1) / cl; ++j) {  // this CTA's key tiles
    load_tile<D, kB>(sk, p.k, [&](int r) { return key(p.k, j * kB + r); });
    load_tile<D, kB>(sv, p.k, [&](int r) { return key(p.v, j * kB + r); });
    cp_commit_f();
    cp_wait_f<0>();
    __syncthreads();
    float sc[4][4], dp[4][4];
    dots<D>(sq, sk, sc);
    dots<D>(so, sv, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float pr = ex2(fmaf(sc[i][k], p.scale_log2, -rd[i].x));
        sc[i][k] = j * kB + tx + 16 * k < vis[i] ? pr * (dp[i][k] - rd[i].y) : 0.f;
      }
    put(sp, sc);
    __syncthreads();
    sums<D>(sp, sk, acc);
    __syncthreads();  // K, V and dS are read
  }
  cp_commit_f();
  cp_wait_f<0>();
  if (cl == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = x0 + ty * 4 + i;
      if (x < x1) store_rows<D>(p.dq + row_of(p, s, g, x) * D, acc[i], p.scale);
    }
    return;
  }
  put_rows<D>(sk, 0, acc);  // K is read
  cluster_sync();
  sum_ranks<D>(sk, kA, rank, cl, [&](int r) { return x0 + r < x1 ? p.dq + row_of(p, s, g, x0 + r) * D : nullptr; },
               [&](int) { return p.scale; });
  cluster_sync();  // nobody leaves while its partial is read
}

// ---------------------------------------------------------------------------------
// dk, dv: 32 keys; smem K | V | Q | dO | P^T | dS^T | lse, delta
// ---------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kF32Threads, kF32Ctas<D>) full_f32_dkv_kernel(const F32Params p) {
  extern __shared__ __align__(128) uint8_t f32_smem[];
  const uint32_t sk = tc::smem_u32(f32_smem), sv = sk + kA * D * 4, sq = sv + kA * D * 4, so = sq + kB * D * 4,
                 sp = so + kB * D * 4, sd = sp + kA * kPitch * 4;
  float2* srow = reinterpret_cast<float2*>(f32_smem + (2 * kA + 2 * kB) * D * 4 + 2 * kA * kPitch * 4);
  const int tx = tile_x(), ty = tile_y();
  const int cl = cluster_size(), rank = cluster_rank(), work = blockIdx.x / cl;
  const int g = work % p.Hkv;
  int tile;
  SeqSpan s;
  const bool in_order = cta_in_order(p.seq, p.disorder);
  if (!in_order && threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
  // early keys first: most rows. Also CTAs without work wait: this grid must not
  // be over before the one that still writes the rows' data
  if (find_tile(p.seq, in_order, true, kA, 1, work / p.Hkv, tile, s) < 0) return tc::griddep_wait();
  const int j0 = tile * kA, off = s.ok ? s.Lk - s.Lq : 0, xn = s.ok ? s.Lq * p.hpg : 0;
  auto key = [&](const float* base, int j) -> const float* {
    return j < s.Lk ? base + ((int64_t(s.k0) + j) * p.Hkv + g) * D : nullptr;
  };
  load_tile<D, kA>(sk, p.k, [&](int r) { return key(p.k, j0 + r); });
  load_tile<D, kA>(sv, p.k, [&](int r) { return key(p.v, j0 + r); });
  int from[4];  // first row that sees the thread's keys
  uint64_t ak[4][D / 32], av[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    from[i] = max(j0 + ty * 4 + i - off, 0) * p.hpg;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) ak[i][c] = av[i][c] = 0;
  }
  tc::griddep_wait();  // the rows' data are the previous grid's
  const int xs = max(j0 - off, 0) * p.hpg / kB * kB, n = max(xn - xs + kB - 1, 0) / kB;
  for (int z = n * rank / cl; z < n * (rank + 1) / cl; ++z) {  // this CTA's row tiles
    const int x0 = xs + z * kB;
    load_tile<D, kB>(sq, p.k, [&](int r) { return x0 + r < xn ? p.q + row_of(p, s, g, x0 + r) * D : nullptr; });
    load_tile<D, kB>(so, p.k, [&](int r) { return x0 + r < xn ? p.dout + row_of(p, s, g, x0 + r) * D : nullptr; });
    cp_commit_f();
    if (threadIdx.x < kB)
      srow[threadIdx.x] = x0 + int(threadIdx.x) < xn
                              ? p.rows[(int64_t(g) * p.seq.Tq + s.q0) * p.hpg + x0 + threadIdx.x]
                              : make_float2(INFINITY, 0.f);
    cp_wait_f<0>();
    __syncthreads();
    float sc[4][4], dp[4][4];
    dots<D>(sk, sq, sc);
    dots<D>(sv, so, dp);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 rd = srow[tx + 16 * k];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float pr = ex2(fmaf(sc[i][k], p.scale_log2, -rd.x));
        sc[i][k] = x0 + tx + 16 * k >= from[i] ? pr : 0.f;
        dp[i][k] = sc[i][k] * (dp[i][k] - rd.y);
      }
    }
    put(sp, sc);
    put(sd, dp);
    __syncthreads();
    sums<D>(sp, so, av);
    sums<D>(sd, sq, ak);
    __syncthreads();
  }
  cp_commit_f();
  cp_wait_f<0>();
  if (cl == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + ty * 4 + i;
      if (j >= s.Lk) continue;
      const int64_t row = ((int64_t(s.k0) + j) * p.Hkv + g) * D;
      store_rows<D>(p.dk + row, ak[i], p.scale);
      store_rows<D>(p.dv + row, av[i], 1.f);
    }
    return;
  }
  put_rows<D>(sq, 0, ak);  // Q is read
  put_rows<D>(sq, kA, av);
  cluster_sync();
  sum_ranks<D>(sq, 2 * kA, rank, cl,
               [&](int r) {
                 const int j = j0 + r % kA;
                 return j < s.Lk ? (r < kA ? p.dk : p.dv) + ((int64_t(s.k0) + j) * p.Hkv + g) * D : nullptr;
               },
               [&](int r) { return r < kA ? p.scale : 1.f; });
  cluster_sync();  // nobody leaves while its partial is read
}

F32Params params(const FullArgs& a) {
  F32Params p{};
  p.q = static_cast<const float*>(a.q);
  p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.seq = a.seq;
  p.pages = a.pages;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.hpg = a.Hq / a.Hkv;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.status = &static_cast<WsHeader*>(a.ws)->status;
  p.disorder = &static_cast<WsHeader*>(a.ws)->disorder;
  return p;
}

// `split`: steps that a tile's walk may have at most, if a cluster may share it.
// About four CTAs of this size per SM hide each other's latencies, so a cluster
// is doubled until there are that many (a walk of 31 steps in 60 CTAs: 182 us
// alone).
template <typename K>
cudaError_t run(const char* name, KernelReady& ready, K kern, F32Params p, int slots, int64_t split, int bytes, bool early,
                cudaStream_t stream) {
  const int64_t ctas = int64_t(slots) * p.Hkv;
  int c = 1;
  while (c < 8 && ctas * c * 2 <= 4 * kNumSMs && split >= 4 * c) c *= 2;
  ProfScope pf(name, stream);
  p.nslots = slots;
  return launch_clusters(ready, kern, ctas, c, kF32Threads, bytes, early, stream, p);
}

template <int D>
cudaError_t forward(const FullArgs& a, cudaStream_t stream) {
  F32Params p = params(a);
  p.out = static_cast<float*>(a.out);
  p.lse = a.lse;
  if (cudaError_t e = launch_order_check(a.seq, a.ws, stream)) return e;
  static KernelReady ready;
  return run("full_f32", ready, full_f32_kernel<D>, p, int(int64_t(a.seq.Tq) * p.hpg / kA) + a.seq.B, 1,
             (kA + 2 * kB) * D * 4 + kA * kPitch * 4, false, stream);
}
template <int D>
cudaError_t backward(const FullBwdArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  F32Params p = params(f);
  p.dout = static_cast<const float*>(a.dout);
  p.rows = reinterpret_cast<float2*>(static_cast<char*>(f.ws) + kWsHeader);
  p.dq = static_cast<float*>(a.dq);
  p.dk = static_cast<float*>(a.dk);
  p.dv = static_cast<float*>(a.dv);
  if (cudaError_t e = launch_order_check(f.seq, f.ws, stream)) return e;
  if (cudaError_t e = launch_full_bwd_rows(a, stream)) return e;
  constexpr int m = kA * kPitch * 4;
  static KernelReady dkv, dq;
  if (cudaError_t e = run("full_f32_dkv", dkv, full_f32_dkv_kernel<D>, p, f.seq.Tk / kA + f.seq.B,
                          int64_t(f.seq.Tq) * p.hpg / kB,
                          (2 * kA + 2 * kB) * D * 4 + 2 * m + kB * 8, true, stream))
    return e;
  return run("full_f32_dq", dq, full_f32_dq_kernel<D>, p, int(int64_t(f.seq.Tq) * p.hpg / kA) + f.seq.B,
             f.seq.Tk / kB, (2 * kA + 2 * kB) * D * 4 + m, false, stream);
}

}  // namespace

cudaError_t launch_full_f32(const FullArgs& a, cudaStream_t stream) {
  return a.d == 128 ? forward<128>(a, stream) : forward<64>(a, stream);
}
cudaError_t launch_full_f32_backward(const FullBwdArgs& a, cudaStream_t stream) {
  return a.f.d == 128 ? backward<128>(a, stream) : backward<64>(a, stream);
}

}  // namespace msa
