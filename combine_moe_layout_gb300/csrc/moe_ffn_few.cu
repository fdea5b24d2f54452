// The gated feed-forward block for up to 16 rows (single tokens being decoded):
// bound by the weights, which are read once, straight into the registers that
// mma.sync multiplies from.
//
// Linear 1: a CTA takes 8 columns of the hidden width of one expert: the A tile of
// m16n8k16 is their 8 gate rows and 8 up rows, so that a thread's accumulator holds
// g and u of the same column and row, and act(g) u needs no exchange. Linear 2: 16
// output columns. B is the rows, 8 or 16 of them (short ones are zeros).
// The CTA's eight warps split K in chunks of 32 and add their sums through shared
// memory, in order. A lane loads 16 bytes (8 consecutive k) of a weight row and of
// a row of x; which k a lane's registers stand for is the same permutation on both
// sides, so that the product is that of the formula.
//
// Linear 2 is released as soon as linear 1 has begun. In a dense block it fetches its
// first weights before it waits for h; with offsets it waits first (which experts
// have rows it reads from them).
//
// Measured (one call among others, weights from HBM) against tiles on the tensor
// cores, whose 128 rows are then mostly empty: 7168 -> 2048 1 row 18.1 us against
// 27, 16 rows 20.6 against 26; 4096 -> 14336 58.6 (6.0 TB/s) against 82, 64.7 against
// 66.1; 2048 -> 1408 7.2 against 13, 8 against 13.5. Rows of 64 experts, 4096 -> 1408:
// 1 row 12.7 us against 18.4, 4 rows 31.4 against 34.9, 8 rows 60.2 against 65.7, 16
// rows 111 against 91 (each expert that has a row takes its own CTAs, which nearly all
// have one row). Beyond 16 rows the tiles take over.
#include <cuda_bf16.h>

#include "moe_ffn.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

struct FewArgs {
  const int32_t *offsets;
  int32_t *err;
  const __nv_bfloat16 *in;         // x or h
  const __nv_bfloat16 *w0, *w1;    // gate and up, or down
  __nv_bfloat16 *out;              // h or y
  __nv_bfloat16 *keep_gate, *keep_up;
  int rows, E, R;
  int K, N;                        // contraction and output widths
  int blocks;                      // column blocks of an expert
  int act;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  __syncwarp();
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: past L1.
__device__ __forceinline__ uint4 load_weight(const __nv_bfloat16 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// UP: linear 1; else linear 2. NT: tiles of 8 rows.
template <bool UP, int NT>
__global__ void __launch_bounds__(kFewThreads, 2) ffn_few_kernel(const FewArgs a) {
  __shared__ float part[kFewWarps][NT * 4][32];
  __shared__ int first[kFewRows], expert_of[kFewRows], rows_of[kFewRows], active_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lr = lane >> 2, lk = (lane & 3) * 8;

  int e = 0, row0 = 0, nrows = a.rows, block = blockIdx.x;
  const bool dense = a.offsets == nullptr;
  // chunks in flight: each is asked for again as soon as its registers have been multiplied, two CTAs on an SM
  constexpr int kUnroll = NT == 1 ? 7 : 4;
  uint4 wa[kUnroll], wb[kUnroll], xa[kUnroll][NT];
  const __nv_bfloat16 *ra, *rb;
  bool la, lb;
  // the lane's two weight rows: columns block * 8 + lr of gate and up, or block * 16 + lr and + 8 of down
  auto rows_at = [&]() {
    if constexpr (UP) {
      const int64_t i = static_cast<int64_t>(block) * 8 + lr;
      la = lb = i < a.N;
      const int64_t at = (static_cast<int64_t>(e) * a.N + (la ? i : 0)) * a.K + lk;
      ra = a.w0 + at;
      rb = a.w1 + at;
    } else {
      const int64_t j = static_cast<int64_t>(block) * 16 + lr;
      la = j < a.N;
      lb = j + 8 < a.N;
      ra = a.w0 + (static_cast<int64_t>(e) * a.N + (la ? j : 0)) * a.K + lk;
      rb = a.w0 + (static_cast<int64_t>(e) * a.N + (lb ? j + 8 : 0)) * a.K + lk;
    }
  };
  auto fetch = [&](int u, int chunk) {
    const int k = chunk * 32;
    const bool in = k + lk < a.K;
    wa[u] = in && la ? load_weight(ra + k) : make_uint4(0, 0, 0, 0);
    wb[u] = in && lb ? load_weight(rb + k) : make_uint4(0, 0, 0, 0);
  };
  auto fetch_rows = [&](int u, int chunk) {
    const int k = chunk * 32 + lk;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + lr;
      xa[u][n] = k < a.K && r < nrows
                     ? *reinterpret_cast<const uint4 *>(a.in + static_cast<int64_t>(row0 + r) * a.K + k)
                     : make_uint4(0, 0, 0, 0);
    }
  };

  if (UP || !dense) grid_dependency_wait();
  if (UP) grid_dependents_launch();
  if (!dense) {
    // the experts that have rows, in order: at most as many as rows
    if (tid < kFewRows) first[tid] = -1;
    __syncthreads();
    for (int x = tid; x < a.E; x += kFewThreads) {
      const int lo = a.offsets[static_cast<int64_t>(x) * a.R], hi = a.offsets[static_cast<int64_t>(x + 1) * a.R];
      if (lo < 0 || hi < lo || hi > a.rows) {
        latch_error(a.err, MOE_EINVAL);
      } else if (hi > lo) {
        first[lo] = x;
        rows_of[lo] = hi - lo;
      }
    }
    __syncthreads();
    if (tid == 0) {
      int n = 0;
      for (int r = 0; r < a.rows; ++r)
        if (first[r] >= 0) expert_of[n++] = r;
      active_s = n;
    }
    __syncthreads();
    const int which = block / a.blocks;
    block -= which * a.blocks;
    if (which >= active_s) return;
    row0 = expert_of[which];
    e = first[row0];
    nrows = rows_of[row0];
  }
  rows_at();
  const int chunks = (a.K + 31) / 32;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) fetch(u, warp + u * kFewWarps);
  if (!UP && dense) grid_dependency_wait();
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) fetch_rows(u, warp + u * kFewWarps);

  float c[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
  for (int c0 = warp; c0 < chunks; c0 += kUnroll * kFewWarps) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(c[n], wa[u].x, wb[u].x, wa[u].y, wb[u].y, xa[u][n].x, xa[u][n].y);
        mma16816(c[n], wa[u].z, wb[u].z, wa[u].w, wb[u].w, xa[u][n].z, xa[u][n].w);
      }
      const int next = c0 + (kUnroll + u) * kFewWarps;
      fetch(u, next);
      fetch_rows(u, next);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][n * 4 + i][lane] = c[n][i];
  __syncthreads();
  // thread t: accumulator lane t % 32, of row tile n its pair (0, 2) or (1, 3): the same row of B, A rows lr and lr + 8
  for (int t = tid; t < NT * 64; t += kFewThreads) {
    const int l = t & 31, n = t >> 6, odd = (t >> 5) & 1;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      s0 += part[w][n * 4 + odd][l];
      s1 += part[w][n * 4 + 2 + odd][l];
    }
    const int r = n * 8 + (l & 3) * 2 + odd;
    if (r >= nrows) continue;
    const int64_t p = static_cast<int64_t>(row0 + r) * a.N;
    if constexpr (UP) {
      const int i = block * 8 + (l >> 2);
      if (i >= a.N) continue;
      a.out[p + i] = __float2bfloat16(act_of<false>(s0, a.act, nullptr) * s1);
      if (a.keep_gate != nullptr) {
        a.keep_gate[p + i] = __float2bfloat16(s0);
        a.keep_up[p + i] = __float2bfloat16(s1);
      }
    } else {
      const int j = block * 16 + (l >> 2);
      if (j < a.N) a.out[p + j] = __float2bfloat16(s0);
      if (j + 8 < a.N) a.out[p + j + 8] = __float2bfloat16(s1);
    }
  }
}

template <bool UP>
moe_status launch_few_stage(const FewArgs &a, cudaStream_t stream) {
  const int experts = a.offsets == nullptr ? 1 : (a.E < a.rows ? a.E : a.rows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(experts) * static_cast<unsigned>(a.blocks), 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  const cudaError_t st = a.rows <= 8 ? cudaLaunchKernelEx(&cfg, ffn_few_kernel<UP, 1>, a)
                                     : cudaLaunchKernelEx(&cfg, ffn_few_kernel<UP, 2>, a);
  if (st != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

}  // namespace

moe_status launch_ffn_few(const FfnSizes &s, const int32_t *offsets, const void *x, const void *w_gate,
                          const void *w_up, const void *w_down, void *h, void *y, void *gate, void *up, int32_t *err,
                          cudaStream_t stream) {
  using bf = __nv_bfloat16;
  FewArgs a{};
  a.offsets = offsets;
  a.err = err;
  a.rows = s.rows;
  a.E = s.E;
  a.R = s.R;
  a.act = s.act;
  a.in = static_cast<const bf *>(x);
  a.w0 = static_cast<const bf *>(w_gate);
  a.w1 = static_cast<const bf *>(w_up);
  a.out = static_cast<bf *>(h);
  a.keep_gate = s.save == MOE_SAVE_BF16 ? static_cast<bf *>(gate) : nullptr;
  a.keep_up = s.save == MOE_SAVE_BF16 ? static_cast<bf *>(up) : nullptr;
  a.K = s.H;
  a.N = s.I;
  a.blocks = (s.I + 7) / 8;
  moe_status st = launch_few_stage<true>(a, stream);
  if (st != MOE_OK) return st;
  a.in = static_cast<const bf *>(h);
  a.w0 = a.w1 = static_cast<const bf *>(w_down);
  a.out = static_cast<bf *>(y);
  a.keep_gate = a.keep_up = nullptr;
  a.K = s.I;
  a.N = s.H;
  a.blocks = (s.H + 15) / 16;
  return launch_few_stage<false>(a, stream);
}

}  // namespace moe
