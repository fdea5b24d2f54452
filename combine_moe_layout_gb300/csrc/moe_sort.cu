// Token sort: the rows of one device's tokens in expert order and back, with
// their gradients. The packed layout is the receive hook's (rows in (expert,
// source rank, token) order, region offsets, the forward map tok_packed), made
// from the tokens directly: no slots, flags or per-region bound, and half the
// bytes.
//
//   sort         packed[p(t, j)] = x[t]
//   sort_grad    dx[t] = sum_j dpacked[p(t, j)]
//   unsort       out[t] = sum_j w[t][j] y[p(t, j)]
//   unsort_grad  dy[p(t, j)] = w[t][j] dout[t],  dw[t][j] = sum_h y[p(t, j)][h] dout[t][h]
//
// p(t, j) is the rank of (expert, t, j) among the choices that name an expert,
// so it is the same on every run. All four move each row once per choice and
// are bound by HBM; the forward map lets each of them walk the tokens and read
// or write the token's own row once.
//
// Ranking: one thread-block cluster over the flattened choices, cut into one
// contiguous piece per warp. Every warp counts its piece per expert in its own
// shared-memory row, a scan over the warps, the cluster's CTAs (distributed
// shared memory) and the experts turns the counts into positions, and a second
// pass over the piece hands them out in order: the lanes of 32 choices that
// name the same expert are found with one ballot per bit of the expert's index
// (match.any slows down with the number of different experts: with it in both
// passes a CTA took 26 us for 8192 choices of 256 experts, with counting by
// shared-memory atomics and ballots 15.8 us). A warp whose piece holds the first choice
// of a source rank reads that rank's region offsets off its counters.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "moe_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kRankThreads = 1024;
// CTAs of a cluster: up to 8 are granted everywhere, more have to be allowed for
// the kernel and found room for on one part of the device.
#ifndef MOE_RANK_CLUSTER
#define MOE_RANK_CLUSTER 16
#endif
constexpr int kRankMaxCluster = MOE_RANK_CLUSTER, kRankPortableCluster = 8;
constexpr int kRankMaxExperts = 8192;
constexpr int kRankMaxBits = 13;
constexpr int kRankSmem = 200 * 1024;
constexpr int kRankBatch = 8;  // loads in flight per lane

struct RankArgs {
  const int32_t *topk_idx;
  int32_t *region_offsets;  // [E * R + 1]
  int32_t *tok_packed;      // [R * T * k]
  int32_t *err;
  uint32_t n;               // R * T * k, below 2^31
  uint32_t per_rank;        // T * k
  uint32_t per_warp;        // choices of a warp's piece: a multiple of 32
  int E, R, warps;          // warps: warps per CTA that take a piece
  int bits;                 // bits of an expert's index
};

// The expert of choice i, or -1 for a masked or invalid one.
__device__ __forceinline__ int expert_at(const RankArgs &a, uint32_t i, uint32_t end, bool *bad) {
  if (i >= end) return -1;
  const int e = __ldg(a.topk_idx + i);
  if (e >= 0 && e < a.E) return e;
  if (e != kMaskedExpert) *bad = true;
  return -1;
}

// The lanes whose expert equals this lane's (e < 0: none, and not asked for).
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
  unsigned same = __ballot_sync(0xffffffffu, e >= 0);
#pragma unroll
  for (int b = 0; b < kRankMaxBits; ++b) {
    if (b >= bits) break;
    const int bit = static_cast<int>(static_cast<unsigned>(e) << (31 - b)) >> 31;  // 0 or -1
    same &= ~(__ballot_sync(0xffffffffu, bit != 0) ^ static_cast<unsigned>(bit));
  }
  return same;
}

__global__ void __launch_bounds__(kRankThreads) rank_kernel(RankArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ int32_t rsm[];
  int32_t *hist = rsm;                      // [warps][E]: counts, then positions
  int32_t *total = hist + a.warps * a.E;    // [E]: counts of this CTA
  int32_t *base = total + a.E;              // [E]: position of this CTA's first choice of an expert
  __shared__ int32_t warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());

  grid_dependency_wait();
  grid_dependents_launch();  // the row copy may load its rows meanwhile
  for (int i = tid; i < a.warps * a.E; i += kRankThreads) hist[i] = 0;
  __syncthreads();

  const uint32_t c0 = min((static_cast<uint32_t>(cta) * a.warps + warp) * a.per_warp, a.n);
  const uint32_t c1 = warp < a.warps ? min(c0 + a.per_warp, a.n) : c0;
  int32_t *mine = hist + warp * a.E;
  bool bad = false;
  int e[kRankBatch];
  for (uint32_t i0 = c0; i0 < c1; i0 += 32 * kRankBatch) {
#pragma unroll
    for (int b = 0; b < kRankBatch; ++b) e[b] = expert_at(a, i0 + b * 32 + lane, c1, &bad);
#pragma unroll
    for (int b = 0; b < kRankBatch; ++b)
      if (e[b] >= 0) atomicAdd(mine + e[b], 1);
  }
  if (bad) latch_error(a.err, MOE_EINVAL);
  __syncthreads();

  for (int e = tid; e < a.E; e += kRankThreads) {
    int run = 0;
    for (int w0 = 0; w0 < a.warps; w0 += 8) {
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = w0 + i < a.warps ? hist[(w0 + i) * a.E + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (w0 + i < a.warps) hist[(w0 + i) * a.E + e] = run;
        run += c[i];
      }
    }
    total[e] = run;
  }
  __syncwarp();
  cluster.sync();  // every CTA's counts are visible to the cluster

  // exclusive scan over the experts of the cluster's counts: thread tid owns experts [e0, e1)
  const int per = (a.E + kRankThreads - 1) / kRankThreads;
  const int e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int all = 0, before = 0;
    for (int q = 0; q < ctas; ++q) {
      const int c = *cluster.map_shared_rank(total + e, q);
      if (q < cta) before += c;
      all += c;
    }
    base[e] = sum + before;
    sum += all;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int first = incl - sum;
  for (int w = 0; w < warp; ++w) first += warp_sums[w];
  for (int e = e0; e < e1; ++e) base[e] += first;
  if (cta == 0 && tid == kRankThreads - 1) a.region_offsets[static_cast<int64_t>(a.E) * a.R] = first + sum;
  __syncthreads();

  // the choices of the piece in order; a piece of one batch still has its experts in registers
  uint32_t src = c0 < c1 ? c0 / a.per_rank : 0;
  uint32_t bound = src * a.per_rank;  // the next first choice of a source rank
  if (bound < c0) bound += a.per_rank, ++src;
  for (uint32_t i0 = c0; i0 < c1; i0 += 32 * kRankBatch) {
    if (c1 - c0 > 32 * kRankBatch) {
#pragma unroll
      for (int b = 0; b < kRankBatch; ++b) e[b] = expert_at(a, i0 + b * 32 + lane, c1, &bad);
    }
#pragma unroll
    for (int b = 0; b < kRankBatch; ++b) {
      const uint32_t c = i0 + b * 32;
      if (c >= c1) break;  // the whole warp
      // the group's choices, cut where a source rank begins
      for (int lo = 0; lo < 32 && c + lo < c1;) {
        if (bound == c + lo) {
          for (int x = lane; x < a.E; x += 32)
            a.region_offsets[static_cast<int64_t>(x) * a.R + src] = base[x] + mine[x];
          bound += a.per_rank;
          ++src;
          __syncwarp();
        }
        const int hi = bound < c + 32 ? static_cast<int>(bound - c) : 32;
        const int x = lane >= lo && lane < hi ? e[b] : -1;
        const unsigned same = same_expert(x, a.bits);
        const int at = x >= 0 ? mine[x] : 0;
        __syncwarp();
        if (x >= 0 && lane == __ffs(same) - 1) mine[x] = at + __popc(same);
        __syncwarp();
        if (lane >= lo && lane < hi && c + lane < c1)
          a.tok_packed[c + lane] = x >= 0 ? base[x] + at + __popc(same & ((1u << lane) - 1u)) : -1;
        lo = hi;
      }
    }
  }
  __syncwarp();
  cluster.sync();  // no CTA leaves while another may still read its counts
}

__global__ void empty_offsets_kernel(int32_t *region_offsets, int64_t n) {
  grid_dependency_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n) region_offsets[i] = 0;
}

// Row copy: thread v of a token's row loads 16 bytes once and stores them to
// the token's k packed rows; the thread at the start of each 128 bytes carries
// the scale of that block too. The loads come before the dependency wait: the
// ranking, which comes before this kernel, writes no rows and lets it start only
// after its own wait. Bound by HBM: 8192 tokens of 14 KB to eight rows each
// (1.06 GB) take 157 us beside the ranking, 6.7 TB/s; 1024 tokens of
// e4m3 rows with scales (68 MB) take 16.6 us, of which the ranking is 7.6.
struct RowArgs {
  const uint8_t *x;
  const float *scales;
  const int32_t *tok_packed;
  uint8_t *packed;
  float *packed_scales;
  int64_t ntok;
  int V, k, nsc;          // V: 16-byte vectors of a row
  int tpb, chunks, vpc;   // tokens per block; chunks of vpc vectors per row
};

template <bool QUANT>
__global__ void __launch_bounds__(256) sort_rows_kernel(RowArgs a) {
  const int tl = threadIdx.x / a.vpc, vl = threadIdx.x - tl * a.vpc;
  const int64_t blk = blockIdx.x / a.chunks;
  const int v = static_cast<int>(blockIdx.x - blk * a.chunks) * a.vpc + vl;
  const int64_t t = blk * a.tpb + tl;
  const bool live = tl < a.tpb && t < a.ntok && v < a.V;
  uint4 r = make_uint4(0, 0, 0, 0);
  if (live) r = __ldcs(reinterpret_cast<const uint4 *>(a.x) + t * a.V + v);
  if constexpr (QUANT) {
    // 8 bf16 elements a thread; 16 neighbouring threads share a 128-element block
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
    float f[8];
    float amax = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(u[q] << 16);
      f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
      amax = fmaxf(amax, fmaxf(fabsf(f[2 * q]), fabsf(f[2 * q + 1])));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const BlockScale bs = block_scale(amax);
    uint32_t c[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      c[q] = static_cast<uint32_t>(e4m3x2_of_quotients(f[4 * q], f[4 * q + 1], bs)) |
             (static_cast<uint32_t>(e4m3x2_of_quotients(f[4 * q + 2], f[4 * q + 3], bs)) << 16);
    grid_dependency_wait();
    if (!live) return;
    for (int j = 0; j < a.k; ++j) {
      const int32_t p = a.tok_packed[t * a.k + j];
      if (p < 0) continue;
      reinterpret_cast<uint2 *>(a.packed)[static_cast<int64_t>(p) * a.V + v] = make_uint2(c[0], c[1]);
      if ((v & 15) == 0) a.packed_scales[static_cast<int64_t>(p) * a.nsc + (v >> 4)] = bs.s;
    }
  } else {
    float sc = 0.0f;
    const bool has = live && a.nsc > 0 && (v & 7) == 0;
    if (has) sc = a.scales[t * a.nsc + (v >> 3)];
    grid_dependency_wait();
    if (!live) return;
    for (int j = 0; j < a.k; ++j) {
      const int32_t p = a.tok_packed[t * a.k + j];
      if (p < 0) continue;
      reinterpret_cast<uint4 *>(a.packed)[static_cast<int64_t>(p) * a.V + v] = r;
      if (has) a.packed_scales[static_cast<int64_t>(p) * a.nsc + (v >> 3)] = sc;
    }
  }
}

// Gradients of unsort: one CTA per token walks the
// k choices, loading y, storing w * dout and adding up y . dout.
// The sum over the row is a shuffle tree per warp and the warps in order, the
// same on every run. dout is read again for each choice, from L1 after the
// first: with it in registers a CTA of 8 warps would hold one width of row only.
// 8192 tokens of 4096 elements, two choices (335 MB): 49 us, 6.8 TB/s, HBM. At 32
// registers a thread eight CTAs fit an SM (at 40 it took 53 us); several choices
// at a time took more registers and longer.
struct UnsortGradArgs {
  const uint16_t *y;
  const int32_t *tok_packed;
  const float *weights;
  const uint16_t *gout;
  uint16_t *gy;
  float *gw;  // may be null
  int32_t *err;
  int64_t nrows;
  int V, k;
};

__device__ __forceinline__ void unpack_bf16x8(const uint4 &r, float (&f)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(u[q] << 16);
    f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 scale_bf16x8(const float (&f)[8], float w) {
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * q] * w, f[2 * q + 1] * w);
    u[q] = *reinterpret_cast<const uint32_t *>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

constexpr int kUnsortGradMaxWarps = 8;

__global__ void __launch_bounds__(kUnsortGradMaxWarps * 32) unsort_grad_kernel(UnsortGradArgs a) {
  __shared__ float part[kMaxTopk][kUnsortGradMaxWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int64_t t = blockIdx.x;
  grid_dependency_wait();
  const uint4 *g = reinterpret_cast<const uint4 *>(a.gout) + t * a.V;
  for (int j = 0; j < a.k; ++j) {
    int32_t p = __ldg(a.tok_packed + t * a.k + j);
    const float w = __ldg(a.weights + t * a.k + j);
    if (p >= a.nrows) {
      if (tid == 0) latch_error(a.err, MOE_EINVAL);
      p = -1;
    }
    float dot = 0.0f;
    const uint4 *y = reinterpret_cast<const uint4 *>(a.y) + static_cast<int64_t>(p) * a.V;
    uint4 *gy = reinterpret_cast<uint4 *>(a.gy) + static_cast<int64_t>(p) * a.V;
    for (int v = tid; v < a.V; v += nt) {
      if (p < 0) break;
      const uint4 yv = __ldcs(y + v);
      float gf[8], yf[8];
      unpack_bf16x8(__ldg(g + v), gf);
      unpack_bf16x8(yv, yf);
#pragma unroll
      for (int q = 0; q < 8; ++q) dot = fmaf(yf[q], gf[q], dot);
      __stcs(gy + v, scale_bf16x8(gf, w));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) part[j][warp] = dot;
  }
  __syncthreads();
  if (a.gw != nullptr && tid < a.k) {
    float s = 0.0f;
    for (int w = 0; w < nt / 32; ++w) s += part[tid][w];
    a.gw[t * a.k + tid] = s;
  }
}

// The most CTAs that a cluster of the ranking may have on the current device, asked
// once with the most shared memory that one takes.
int rank_cluster_limit() {
  static std::atomic<int> known[64];
  if (kRankMaxCluster <= kRankPortableCluster) return kRankMaxCluster;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kRankPortableCluster;
  int most = known[dev].load(std::memory_order_relaxed);
  if (most != 0) return most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kRankMaxCluster, 1, 1);
  cfg.blockDim = dim3(kRankThreads, 1, 1);
  cfg.dynamicSmemBytes = kRankSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kRankMaxCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  most = kRankMaxCluster;
  if (!raise_smem_limit(rank_kernel, kRankSmem) ||
      cudaFuncSetAttribute(rank_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&clusters, rank_kernel, &cfg) != cudaSuccess || clusters < 1) {
    cudaGetLastError();  // an answer, not a failed call
    most = kRankPortableCluster;
  }
  known[dev].store(most, std::memory_order_relaxed);
  return most;
}

// Cluster shape of the ranking: a CTA per 512 choices, one a lane of 16 warps, as
// far as clusters go: handing out the positions is bound by instructions, about
// 0.8 us for a group of 32 choices in each of a CTA's warps. 8192 choices of 256
// experts: 15.8 us with one CTA, 7.6 with eight of 32 warps. A whole sort of 128
// elements a row with eight and with sixteen CTAs: 65536 choices 15.4 and 12.5
// us, a million 207 and 128 us.
moe_status launch_rank(const Sizes &s, const int32_t *topk_idx, int32_t *region_offsets, int32_t *tok_packed,
                       int32_t *err, cudaStream_t stream) {
  if (s.E > kRankMaxExperts) return MOE_EINVAL;
  const int64_t n = s.ntok * s.k;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = MOE_PDL;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (n == 0) {
    const int64_t words = static_cast<int64_t>(s.E) * s.R + 1;
    cfg.gridDim = dim3(static_cast<unsigned>((words + 255) / 256), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    if (cudaLaunchKernelEx(&cfg, empty_offsets_kernel, region_offsets, words) != cudaSuccess) return MOE_ECUDA;
    return launch_status();
  }
  int warps = kRankSmem / 4 / s.E - 2;
  if (warps > kRankThreads / 32) warps = kRankThreads / 32;
  if (warps < 1) return MOE_EINVAL;
  int64_t ctas = (n + 511) / 512;
  if (ctas > kRankPortableCluster) {
    const int most = rank_cluster_limit();
    if (ctas > most) ctas = most;
  }
  const int64_t needed = ((n + 31) / 32 + ctas - 1) / ctas;
  if (warps > needed) warps = static_cast<int>(needed);
  const int64_t pieces = ctas * warps;
  const int64_t per_warp = ((n + pieces - 1) / pieces + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(warps + 2) * s.E * sizeof(int32_t);
  if (!raise_smem_limit(rank_kernel, smem)) return MOE_ECUDA;
  int bits = 0;
  while ((1 << bits) < s.E) ++bits;
  RankArgs a{topk_idx, region_offsets, tok_packed, err, static_cast<uint32_t>(n),
             static_cast<uint32_t>(static_cast<int64_t>(s.T) * s.k), static_cast<uint32_t>(per_warp), s.E, s.R, warps, bits};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kRankThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, rank_kernel, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

moe_status launch_sort_rows(const Sizes &s, const void *x, const float *x_scales, const int32_t *tok_packed,
                            void *packed, float *packed_scales, cudaStream_t stream) {
  const int V = static_cast<int>(s.in_row_bytes / 16);
  RowArgs a{static_cast<const uint8_t *>(x), x_scales, tok_packed, static_cast<uint8_t *>(packed), packed_scales,
            s.ntok, V, s.k, s.nsc, 1, 1, V};
  // blocks of at most 256 threads, cut so that the threads of a row's last block are not idle; whole 16-lane
  // groups (a quantised block) stay together
  a.chunks = (V + 255) / 256;
  a.vpc = (V + a.chunks - 1) / a.chunks;
  if (a.chunks > 1) a.vpc = (a.vpc + 31) / 32 * 32;
  a.chunks = (V + a.vpc - 1) / a.vpc;
  a.tpb = a.chunks > 1 ? 1 : 256 / a.vpc;
  const int64_t blocks = (s.ntok + a.tpb - 1) / a.tpb * a.chunks;
  if (blocks > 0x7fffffffll) return MOE_EINVAL;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>((a.tpb * a.vpc + 31) / 32 * 32), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, s.quant ? sort_rows_kernel<true> : sort_rows_kernel<false>, a) != cudaSuccess)
    return MOE_ECUDA;
  return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_sort(const moe_desc *desc, const int32_t *topk_idx, const void *x, const float *x_scales,
                               int32_t *region_offsets, void *packed_x, float *packed_scales, int32_t *tok_packed,
                               int32_t *err, void *stream) {
  Sizes s;
  moe_status st = check_desc(desc, &s);
  if (st != MOE_OK) return st;
  if (region_offsets == nullptr || err == nullptr || !aligned4(region_offsets) || !aligned4(err)) return MOE_EINVAL;
  if (s.ntok > 0) {
    if (topk_idx == nullptr || x == nullptr || packed_x == nullptr || tok_packed == nullptr) return MOE_EINVAL;
    if (s.nsc > 0 && packed_scales == nullptr) return MOE_EINVAL;
    if (s.dtype == MOE_FP8_E4M3 && x_scales == nullptr) return MOE_EINVAL;
    if (!aligned4(topk_idx) || !aligned16(x) || !aligned4(x_scales) || !aligned16(packed_x) ||
        !aligned4(packed_scales) || !aligned4(tok_packed))
      return MOE_EINVAL;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  st = launch_rank(s, topk_idx, region_offsets, tok_packed, err, cs);
  if (st != MOE_OK || s.ntok == 0) return st;
  return launch_sort_rows(s, x, x_scales, tok_packed, packed_x, packed_scales, cs);
}

extern "C" moe_status moe_sort_grad(const moe_desc *desc, const uint16_t *grad_packed, const int32_t *tok_packed,
                                    uint16_t *grad_x, int32_t *err, void *stream) {
  Sizes s;
  const moe_status st = check_desc(desc, &s);
  if (st != MOE_OK) return st;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (s.ntok == 0) return MOE_OK;
  if (grad_packed == nullptr || tok_packed == nullptr || grad_x == nullptr) return MOE_EINVAL;
  if (!aligned16(grad_packed) || !aligned4(tok_packed) || !aligned16(grad_x)) return MOE_EINVAL;
  return launch_gather_sum(s, grad_packed, nullptr, tok_packed, grad_x, err, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_unsort(const moe_desc *desc, const uint16_t *packed_y, const int32_t *tok_packed,
                                 const float *topk_weights, uint16_t *out, int32_t *err, void *stream) {
  Sizes s;
  const moe_status st = check_desc(desc, &s);
  if (st != MOE_OK) return st;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (s.ntok == 0) return MOE_OK;
  if (packed_y == nullptr || tok_packed == nullptr || topk_weights == nullptr || out == nullptr) return MOE_EINVAL;
  if (!aligned16(packed_y) || !aligned4(tok_packed) || !aligned4(topk_weights) || !aligned16(out)) return MOE_EINVAL;
  return launch_gather_sum(s, packed_y, topk_weights, tok_packed, out, err, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_unsort_grad(const moe_desc *desc, const uint16_t *packed_y, const int32_t *tok_packed,
                                      const float *topk_weights, const uint16_t *grad_out, uint16_t *grad_packed_y,
                                      float *grad_weights, int32_t *err, void *stream) {
  Sizes s;
  const moe_status st = check_desc(desc, &s);
  if (st != MOE_OK) return st;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (s.ntok == 0) return MOE_OK;
  if (packed_y == nullptr || tok_packed == nullptr || topk_weights == nullptr || grad_out == nullptr ||
      grad_packed_y == nullptr)
    return MOE_EINVAL;
  if (!aligned16(packed_y) || !aligned4(tok_packed) || !aligned4(topk_weights) || !aligned16(grad_out) ||
      !aligned16(grad_packed_y) || !aligned4(grad_weights))
    return MOE_EINVAL;
  if (s.ntok > 0x7fffffffll) return MOE_EINVAL;
  UnsortGradArgs a{packed_y, tok_packed, topk_weights, grad_out, grad_packed_y, grad_weights, err, s.ntok * s.k,
                   s.H / 8, s.k};
  int warps = (a.V + 31) / 32;
  if (warps > kUnsortGradMaxWarps) warps = kUnsortGradMaxWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.ntok), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(warps) * 32, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, unsort_grad_kernel, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}
