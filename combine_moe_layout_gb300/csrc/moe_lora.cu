// A projection shared by all requests of a batch with each request's low-rank
// adapter beside it:
//
//   y[t] = bf16( x[t] W^T + s_a (x[t] A_a^T) B_a^T ),  a = adapter[t], or no second term for a = -1
//
// x [T][in], W [out][in], A_a [rank][in], B_a [out][rank], all bf16, K-major.
// The adapters are extra K blocks of the projection's own accumulation, in fp32
// on the tensor cores: with u[t] = s_a x[t] A_a^T rounded to bf16, the tile's
// product goes on with u and B_a for every adapter a among its tokens, each time
// writing only the accumulator rows of the tokens that use it (the MMA's
// disable-output-lane mask, so no adapter's value, not even a NaN, reaches
// another request's row). y is rounded once. u is rounded to bf16 too, which is what
// the tensor cores take: up to 2^-8 of each u_i b_i, which is more than rounding y
// costs where these cancel. Over ten shapes the error of y against 64 bits
// (relative, over the whole matrix) is 1.70e-3 to 2.35e-3, where y's rounding alone
// leaves 1.63e-3 to 1.68e-3. A call may ask for u in two parts, its rounding and the
// rounding of what that left (2^-17 of u), which meet the same B_a one after the
// other, with the error of y's rounding alone (1.63e-3 to 1.70e-3). That takes
// 9.8 us for 9.7 (one token, 4096 -> 4096, rank 16), 17.3 for 15.5 (64 tokens, 7168
// -> 2048, 32 adapters), 22.2 for 20.7 (389 tokens, 2056 -> 4104) and 191 for 179
// (8192 tokens, 7168 -> 2048, rank 64): the parts share one place in shared memory,
// since a second one would leave 256-wide tiles three stages of their ring for four
// (203 us for 181).
//
// Two kernels a call:
//   lora_shrink_kernel  u[t] = s_a x[t] A_a^T. A tile is 128 tokens against the
//     stacked rows of up to 128 / rank adapters that occur among them (or one
//     adapter's, if it has more): a token's own columns are picked in the
//     epilogue. in is split over a cluster of CTAs whose partial sums meet in
//     distributed shared memory in a fixed order. Few tokens take
//     lora_shrink_small_kernel: 16 tokens of one adapter at a time.
//   lora_gemm_kernel    the projection with its extra K blocks. Tiles of 128
//     tokens x BN outputs; TMA brings x and W (then u and B_a) tiles, one lane
//     issues tcgen05.mma, four warps find the tile's adapters and their rows.
//     With few tiles in is split over a cluster as above; with many a CTA walks
//     its tiles with two accumulators, so that a tile's stores overlap the next
//     one's products. It starts on x and W while the shrink kernel is running;
//     only the loads of u wait for that.
//   lora_one_kernel     the projection of a single token, without tensor cores.
//
// Shared memory and tensor memory: a CTA that takes c of the 512 tensor-memory
// columns of an SM takes at least c / 512 of its shared memory, so that CTAs
// that share an SM never wait for one another's columns (a cluster whose CTAs
// did could wait for ever). Every other wait is bounded, as in the expert stage.
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>

#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int kLBM = 128;           // tokens of a tile
constexpr int kLBK = 64;            // K elements of a stage: one 128-byte swizzle row
constexpr int kLRow = kLBK * 2;     // bytes of a tile row
constexpr int kLPieceRow = 32;      // bytes of a row of 16 columns of a B_a
constexpr int kLMaxStages = 8;
constexpr int kLMaxRank = 256;
constexpr int kLSmemMax = 227 * 1024;
constexpr int kLStatic = 8192;      // room for a kernel's static shared memory
constexpr int kLBytesPerCol = 228 * 1024 / 512;  // shared memory that goes with one tensor-memory column
constexpr int kShrinkThreads = 192;
constexpr int kGemmLThreads = 320;
constexpr int kShrinkCols = 128;    // adapter rows of a shrink tile (or one adapter's, if it has more)
constexpr int kLMaxCluster = 8;    // of the shrink kernel
constexpr int kLMaxSplit = 4;      // of the projection
// Ranks up to 32 have several adapters' B_a in a stage, as pieces of 16 columns:
// a block of 64 columns would be half empty or more, and each would take a
// stage's way through the ring (64 tokens, 32 adapters of rank 16: eight adapters
// a stage took it from 17.1 to 16.1 us).
constexpr int kLPackedPieces = 2;

struct LoraArgs {
  const int32_t *adapter;
  const float *scales;
  __nv_bfloat16 *u;  // [T][rank]
  __nv_bfloat16 *y;  // [T][out]
  int32_t *err;
  int T, K, N, rank, adapters;
  int xrows;           // rows of an x box (a multiple of 8, at most 128)
  int xbytes;          // bytes of an x tile in a stage (a multiple of 1024)
  int stage, stages;   // bytes and number of the ring's stages (shrink: the most of them)
  int kblocks;
  // shrink
  int ring;              // bytes of the ring
  int per_pass, groups;  // adapters of one pass over K, and the CTAs that share a tile's passes
  uint32_t cols;         // tensor-memory columns
  // projection
  int lora, ntiles_n, mtiles, group_n;
  int parts;             // 1, or 2: u is followed by what its rounding left
  int whole, total;      // tiles taken whole, and tiles and halves in all
  int own;               // one token: rows of W of a CTA
  int pieces, packed;    // ranks up to 32: pieces of 16 columns of one B_a, and the B_a of a stage (0: 64 columns a stage)
};

__device__ __forceinline__ uint32_t lora_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t lora_cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// The cluster barrier, the named barriers and the tensor-memory loads below are
// instructions of a whole warp: a warp that comes from a branch or a loop that
// its lanes left at different times is brought together first.
__device__ __forceinline__ void lora_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void lora_cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void lora_cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Writes v at this shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ void peer_store(uint32_t saddr, uint32_t rank, float v) {
  uint32_t p;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(p), "f"(v) : "memory");
}

// 16 bytes at this shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 peer_load(uint32_t saddr, uint32_t rank) {
  uint32_t p;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(p)
               : "memory");
  return v;
}

// The sum over the cluster's CTAs, in their order, of 8 floats at this
// shared-memory address. All loads are issued before the first is used: one
// after the other they take a quarter of a microsecond each.
template <int MAX>
__device__ __forceinline__ void cluster_sum8(uint32_t saddr, int ctas, float (&f)[8]) {
  float4 lo[MAX], hi[MAX];
#pragma unroll
  for (int p = 0; p < MAX; ++p)
    if (p < ctas) {
      lo[p] = peer_load(saddr, p);
      hi[p] = peer_load(saddr + 16, p);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 0.0f;
#pragma unroll
  for (int p = 0; p < MAX; ++p)
    if (p < ctas) {
      f[0] += lo[p].x;
      f[1] += lo[p].y;
      f[2] += lo[p].z;
      f[3] += lo[p].w;
      f[4] += hi[p].x;
      f[5] += hi[p].y;
      f[6] += hi[p].z;
      f[7] += hi[p].w;
    }
}

template <int ID>
__device__ __forceinline__ void bar128() {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory");
}

// bar128 that also tells every thread whether v was set in all of them.
template <int ID>
__device__ __forceinline__ bool bar128_and(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(ID)
      : "memory");
  return r != 0;
}

// 8 consecutive fp32 accumulator columns of this thread's row.
__device__ __forceinline__ void tmem_load8_wait(uint32_t taddr, float (&f)[8]) {
  uint32_t r[8];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i]);
}

// The four K = 16 steps of one 64-wide K block, from the low words of the
// tiles' shared-memory descriptors (kDescHi is the high word of every
// descriptor of this layout; a step is 32 bytes, 2 in the descriptor's units).
// A block's products take 256 cycles (BN = 128); descriptors made anew for every
// step took longer than that.
constexpr uint32_t kDescHi = static_cast<uint32_t>(sw128_desc(0) >> 32);

// As sw128_desc for tiles of 16 elements a row: 32-byte rows, 8-row groups 256
// bytes apart, swizzle mode 6 = 32 bytes (tiles start on 256-byte boundaries).
__host__ __device__ constexpr uint64_t sw32_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16 >> 4) << 16) |
         (static_cast<uint64_t>(256 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(6) << 61);
}

__device__ __forceinline__ uint64_t full_desc(uint32_t lo) { return (static_cast<uint64_t>(kDescHi) << 32) | lo; }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return static_cast<uint32_t>(sw128_desc(saddr)); }

__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// mma_bf16 accumulating into the rows (tensor-memory lanes) whose bit is clear in `off` only.
__device__ __forceinline__ void mma_bf16_rows(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              const uint4 &off) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w)
      : "memory");
}

__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
    u[q] = *reinterpret_cast<const uint32_t *>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight columns of a token's u, as its one or two parts.
__device__ __forceinline__ void store_u(const LoraArgs &a, int64_t t, int c, const float (&f)[8]) {
  __nv_bfloat16 *at = a.u + t * a.rank + c;
  *reinterpret_cast<uint4 *>(at) = round8(f);
  if (a.parts > 1) {
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      rest[j] = f[j] - __bfloat162float(__float2bfloat16_rn(f[j]));
      if (!(fabsf(rest[j]) <= FLT_MAX)) rest[j] = 0.0f;  // of an infinity or a NaN the first part says all
    }
    *reinterpret_cast<uint4 *>(at + static_cast<int64_t>(a.T) * a.rank) = round8(rest);
  }
}

// A whole warp's bounded wait on an mbarrier phase: every lane gets the same
// answer, so the warp stays together. As role_wait otherwise.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = role_wait(bar, parity, abort, err) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  // the other lanes order their later accesses after the phase too
  return ok != 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
}

// One lane of a warp that is all here. The producer's and the MMA issuer's
// loops are run by the whole warp with only this lane issuing: their operands
// are then the same in every lane, and four MMAs with their commit take about
// 160 cycles to issue instead of 245 from a loop that a single lane runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e)
      :
      : "memory");
  return e != 0;
}

// Position in the ring of stages: the stage and the parity of its use. Kept by
// counting: the number of stages is a run-time value, and dividing by it in
// every K block took longer than the block's products.
struct Ring {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == static_cast<uint32_t>(stages)) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// Waits (bounded) until the last load issued into each stage has landed; r is
// the position after `it` loads.
__device__ __forceinline__ void drain_ring(uint64_t *full, Ring r, uint32_t it, int stages) {
  for (uint32_t i = 0; i < static_cast<uint32_t>(stages) && i < it; ++i) {
    if (r.s == 0) {
      r.s = stages;
      r.ph ^= 1u;
    }
    --r.s;
    mbar_wait_bounded(full + r.s, r.ph);
  }
}

// Scratch of tile_adapters.
struct AdapterScratch {
  int32_t ids[kLBM];
  int32_t pos[kLBM];
  int32_t counts[4];
};

// The distinct adapters of a tile's tokens, in order of first use, by 128
// threads (thread m: token t0 + m). Returns their number and this token's place
// in the list (-1: no adapter). An id outside [-1, adapters) counts as none and
// sets *bad.
template <int BAR>
__device__ __forceinline__ int tile_adapters(const LoraArgs &a, int t0, int m, AdapterScratch &s, int32_t *list, int *slot,
                                             bool *bad) {
  const int lane = m & 31, warp = m >> 5;
  int id = -1;
  if (t0 + m < a.T) {
    id = __ldg(a.adapter + t0 + m);
    if (id < -1 || id >= a.adapters) {
      *bad = true;
      id = -1;
    }
  }
  s.ids[m] = id;
  bar128<BAR>();
  int first = m;
  for (int j = (m & ~3); j >= 0; j -= 4) {
    const int4 v = *reinterpret_cast<const int4 *>(s.ids + j);
    if (v.w == id && j + 3 < first) first = j + 3;
    if (v.z == id && j + 2 < first) first = j + 2;
    if (v.y == id && j + 1 < first) first = j + 1;
    if (v.x == id && j < first) first = j;
  }
  const bool is_first = id >= 0 && first == m;
  const unsigned firsts = __ballot_sync(0xffffffffu, is_first);
  if (lane == 0) s.counts[warp] = __popc(firsts);
  bar128<BAR>();
  int before = 0, n = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < warp) before += s.counts[w];
    n += s.counts[w];
  }
  if (is_first) {
    const int p = before + __popc(firsts & ((1u << lane) - 1u));
    s.pos[m] = p;
    list[p] = id;
  }
  bar128<BAR>();
  *slot = id >= 0 ? s.pos[first] : -1;
  return n;
}

// ---------------------------------------------------------------------------
// u[t] = s_a x[t] A_a^T
//
// Bound by the loads of x, which every pass reads once (x's bytes at HBM's rate)
// and of A, which every tile reads from L2: 8192 tokens of 7168 inputs with
// adapters of rank 64 take about 31 us before the projection (its CTAs need all
// of an SM's shared memory and cannot start earlier); x alone is 17 us.
// ---------------------------------------------------------------------------
struct ShrinkShared {
  AdapterScratch scratch;
  int32_t list[kLBM], slot[kLBM];  // the tile's adapters, and each token's place among them (-1: none)
  uint64_t full[kLMaxStages], empty[kLMaxStages], tfull, done;
  uint32_t tmem;
  int abort, n;
};

__global__ void __launch_bounds__(kShrinkThreads)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
                       const LoraArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) ShrinkShared sh;
  uint8_t *smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  volatile int *abort = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = static_cast<int>(lora_cluster_size()), split = static_cast<int>(lora_cluster_rank());
  const int item = static_cast<int>(blockIdx.x) / splits;
  const int group = item / a.mtiles, mt = item - group * a.mtiles;
  const int t0 = mt * kLBM;

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(sh.full + s, 1);
      mbar_init(sh.empty + s, 1);
    }
    mbar_init(&sh.tfull, 1);
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&map_x);
    prefetch_tensormap(&map_a);
  }
  grid_dependency_wait();
  // The projection's CTAs may come: they find what this kernel's predecessors wrote, and by the rule on shared
  // memory they leave every CTA of this kernel its tensor memory. (A projection of several tiles a CTA lets nothing
  // start before it ends.)
  grid_dependents_launch();
  int slot = -1;
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_addr(&sh.tmem), a.cols);
    tmem_relinquish();
  }
  if (warp >= 2) {
    bool bad = false;
    const int n = tile_adapters<1>(a, t0, tid - 64, sh.scratch, sh.list, &slot, &bad);
    if (bad && group == 0 && split == 0) latch_error(a.err, MOE_EINVAL);
    if (tid == 64) sh.n = n;
    sh.slot[tid - 64] = slot;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const bool leader = elect_one();  // used by warps 0 and 1
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.kblocks) * split / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.kblocks) * (split + 1) / splits);
  const int rows = min(kLBM, a.T - t0), vecs = a.rank / 8;
  float *red = reinterpret_cast<float *>(smem);  // [128][rank]: this split's sums, once the ring is idle
  // the ring as this tile's adapters fill it: most tiles of prompts have one or two, and more stages for it
  const int stage = a.xbytes + ((min(sh.n, a.per_pass) * a.rank + 15) & ~15) * kLRow;
  const int stages = min(a.stages, a.ring / stage);
  Ring r;
  uint32_t it = 0, ph = 0;

  // the tile's adapters, per_pass at a time (the same passes in every CTA of the cluster)
  for (int first = group * a.per_pass; first < sh.n; first += a.groups * a.per_pass, ph ^= 1u) {
    const int nact = min(sh.n - first, a.per_pass);
    if (warp == 0) {
      const uint32_t bytes = static_cast<uint32_t>(a.xrows + nact * a.rank) * kLRow;
      for (int kb = kb0; kb < kb1; ++kb, ++it, r.next(stages)) {
        if (!warp_wait(sh.empty + r.s, r.ph ^ 1u, abort, a.err)) break;
        if (leader) {
          const uint32_t sx = smem_addr(smem) + r.s * stage, sa = sx + a.xbytes, fb = smem_addr(sh.full) + r.s * 8;
          mbar_arrive_expect_tx(sh.full + r.s, bytes);
          tma_load_2d(sx, &map_x, kb * kLBK, t0, fb);
          for (int i = 0; i < nact; ++i)
            tma_load_2d(sa + i * a.rank * kLRow, &map_a, kb * kLBK, sh.list[first + i] * a.rank, fb);
        }
        __syncwarp();
      }
      if (leader) drain_ring(sh.full, r, it, stages);
      __syncwarp();
    } else if (warp == 1) {
      const uint32_t idesc = idesc_bf16(kLBM, (nact * a.rank + 15) & ~15);
      const uint32_t xlo = desc_lo(smem_addr(smem)), step = stage >> 4, xstep = a.xbytes >> 4;
      const uint32_t empty = smem_addr(sh.empty);
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, r.next(stages)) {
        ok = warp_wait(sh.full + r.s, r.ph, abort, a.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t lo = xlo + r.s * step;
          mma_block(tmem, lo, lo + xstep, idesc, kb != kb0);
          mma_commit(empty + r.s * 8);
        }
        __syncwarp();
      }
      if (leader) {
        if (ok) mma_commit(smem_addr(&sh.tfull));
        mma_commit(smem_addr(&sh.done));
        mbar_wait_bounded(&sh.done, ph);
      }
      __syncwarp();
    } else {
      // each token's own columns of the tile (accumulator row m is token t0 + m)
      const int q = warp & 3, m = q * 32 + lane;
      const int mine = sh.slot[m] - first;
      if (warp_wait(&sh.tfull, ph, abort, a.err)) {
        tc_fence_after();
        for (int i = 0; i < nact; ++i) {
          if (!__any_sync(0xffffffffu, mine == i)) continue;
          for (int c = 0; c < a.rank; c += 8) {
            float f[8];
            tmem_load8_wait(tmem + (static_cast<uint32_t>(q * 32) << 16) + i * a.rank + c, f);
            if (mine == i) {
              float4 *d = reinterpret_cast<float4 *>(red + m * a.rank + c);
              d[0] = make_float4(f[0], f[1], f[2], f[3]);
              d[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
        tc_fence_before();
      }
      __syncwarp();
    }
    lora_cluster_sync();
    // the splits' sums, row m in CTA m % splits
    const int own = (rows - split + splits - 1) / splits;
    for (int i = tid; i < own * vecs; i += kShrinkThreads) {
      const int q = i / vecs, m = q * splits + split, c = (i - q * vecs) * 8;
      const int p = sh.slot[m] - first;
      if (p < 0 || p >= nact) continue;
      const float sc = a.scales != nullptr ? __ldg(a.scales + sh.list[first + p]) : 1.0f;
      float f[8];
      cluster_sum8<kLMaxCluster>(smem_addr(red + m * a.rank + c), splits, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= sc;
      store_u(a, t0 + m, c, f);
    }
    fence_proxy_async_smem();  // the ring is loaded again where the sums were
    lora_cluster_sync();       // and no CTA leaves while another may still read its sums
    tc_fence_after();
  }
  __syncthreads();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, a.cols);
}

// ---------------------------------------------------------------------------
// u for few tokens: one cluster of CTAs per (adapter in use, 16 of its rows), which
// takes its tokens 16 at a time, K split over the cluster. The tensor-core tiles
// above take 128 tokens whether they use the adapter or not; here a token's x row
// meets only its own adapter.
// With more adapters than tokens there is a cluster per token instead, and the
// first token of an adapter takes all of its tokens: clusters without work cost
// 29 us for one token and 1000 adapters.
// Bound by the latency of the loads, beside the projection's stream of W: a CTA
// asks for all of its rows' pieces at once, with one bulk copy a row into shared
// memory (two halves in turn where they do not fit). Loading them to registers,
// in two rounds, took 6 us at the sizes below, and takes 4 us so.
// Products: mma.sync, whose 16-row tiles fit a handful of tokens (a
// tensor-memory accumulator would cost a claim, a commit and a read back for
// them). Lane (g, t) reads elements 8t .. 8t + 7 of a 32-wide K piece of row g
// and gives them to two k = 16 steps as its elements (2t, 2t + 1) and (2t + 8,
// 2t + 9) of each; x and A_a are permuted alike, so the sum is the same. Rows lie
// 64 bytes past a multiple of 128 apart, so that eight lanes' reads meet every
// bank once.
// Sums: every CTA of the cluster sends its part of a sum to the CTA that owns it
// and the owner adds them in the order of the CTAs. What it receives has two
// places in turn, so one cluster barrier a pass is enough.
// 64 tokens (7168 -> 2048, 32 adapters of rank 16): the call takes 15.8 us, and 20.7
// with the tensor-memory kernel. When this one was new it took 17.3 us, where loads
// to registers and sums read from the other CTAs had taken 19.5.
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallM = 16, kSmallN = 16;
constexpr int kSmallPad = 64;  // bytes between rows in shared memory
constexpr int kSmallTokens = 64;  // of a call, at most

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  __syncwarp();  // the lanes' rows may end at different places
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// K elements (a multiple of 64) of which `bytes` hold `rows` rows.
__host__ __device__ constexpr int small_chunk(int bytes, int rows) { return (bytes / rows - kSmallPad) / 128 * 64; }

__global__ void __launch_bounds__(kSmallThreads)
    lora_shrink_small_kernel(const LoraArgs a, const __nv_bfloat16 *__restrict__ x, const __nv_bfloat16 *__restrict__ lora_a) {
  extern __shared__ __align__(128) uint8_t small_rows[];  // a.ring bytes: rows of A_a, then of x
  __shared__ float part[kSmallWarps][kSmallM][kSmallN + 1];
  __shared__ __align__(16) float recv[2][kLMaxCluster][kSmallM * kSmallN];  // the parts of the sums that this CTA owns
  __shared__ int32_t token[kSmallTokens];
  __shared__ int32_t counts[kSmallWarps];
  __shared__ uint64_t full[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = static_cast<int>(lora_cluster_size()), split = static_cast<int>(lora_cluster_rank());
  const int first_of = blockIdx.x / splits, n0 = blockIdx.y * kSmallN;
  if (tid == 0) {
    mbar_init(full, 1);
    mbar_init(full + 1, 1);
    fence_mbar_init();
  }
  lora_cluster_arrive();  // the others may be written to once they have started
  grid_dependency_wait();
  grid_dependents_launch();  // the projection finds what this kernel's predecessors wrote
  // this adapter's tokens, in token order
  const int id = tid < a.T ? __ldg(a.adapter + tid) : -1;
  if ((id < -1 || id >= a.adapters) && blockIdx.x == 0 && n0 == 0) latch_error(a.err, MOE_EINVAL);
  // a cluster per adapter, or, with more adapters than tokens, per token: the first one of its adapter takes all
  const int ad = a.adapters > a.T ? __ldg(a.adapter + first_of) : first_of;
  const bool uses = id == ad && ad >= 0 && ad < a.adapters;
  const unsigned users = __ballot_sync(0xffffffffu, uses);
  if (lane == 0) counts[warp] = __popc(users);
  const bool taken = __syncthreads_or(a.adapters > a.T && uses && tid < first_of) != 0;
  int total = 0, at = __popc(users & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kSmallWarps; ++w) {
    if (w < warp) at += counts[w];
    total += counts[w];
  }
  if (taken) total = 0;
  if (uses) token[at] = tid;
  __syncthreads();

  // this CTA's K elements, its passes of 16 tokens (the same in every CTA of the cluster) and the steps of a pass
  const int pieces = (a.K + 31) / 32;
  const int e0 = static_cast<int>(static_cast<int64_t>(pieces) * split / splits) * 32;
  const int len = max(min(static_cast<int>(static_cast<int64_t>(pieces) * (split + 1) / splits) * 32, a.K) - e0, 0);
  const int passes = (total + kSmallM - 1) / kSmallM;
  const int nr = min(kSmallN, a.rank - n0);                  // rows of A_a
  const int most = nr + min(kSmallM, total);  // and of x
  const bool whole = passes == 1 && len <= small_chunk(a.ring, most);
  const int chunk = whole ? (len + 63) / 64 * 64 : small_chunk(a.ring / 2, most);
  const int chunks = len > 0 ? (len + chunk - 1) / chunk : 0, steps = passes * chunks;
  const int pitch = chunk * 2 + kSmallPad;
  // asks for step s into half s & 1 (warp 0)
  const auto load = [&](int s) {
    const int m0 = s / chunks * kSmallM, o = s % chunks * chunk;
    const int nt = min(total - m0, kSmallM);
    const uint32_t bytes = static_cast<uint32_t>(min(chunk, len - o)) * 2;
    uint8_t *dst = small_rows + (s & 1) * (a.ring / 2);
    if (lane == 0) mbar_arrive_expect_tx(full + (s & 1), static_cast<uint32_t>(nr + nt) * bytes);
    __syncwarp();
    if (lane < kSmallN) {
      if (lane < nr)
        bulk_load(dst + lane * pitch, lora_a + (static_cast<int64_t>(ad) * a.rank + n0 + lane) * a.K + e0 + o, bytes,
                  full + (s & 1));
    } else if (lane - kSmallN < nt) {
      bulk_load(dst + (nr + lane - kSmallN) * pitch, x + static_cast<int64_t>(token[m0 + lane - kSmallN]) * a.K + e0 + o,
                bytes, full + (s & 1));
    }
    __syncwarp();
  };
  if (warp == 0) {
    if (steps > 0) load(0);
    if (steps > 1) load(1);
  }
  const int g = lane >> 2, t4 = lane & 3;
  const float sc = a.scales != nullptr && passes > 0 ? __ldg(a.scales + ad) : 1.0f;
  lora_cluster_wait();

  for (int pass = 0, s = 0; pass < passes; ++pass) {
    const int m0 = pass * kSmallM;
    const int nt = min(total - m0, kSmallM);
    float acc[2][4] = {};
    for (int c = 0; c < chunks; ++c, ++s) {
      if (!mbar_wait_bounded(full + (s & 1), (s >> 1) & 1)) latch_error(a.err, MOE_ETIMEOUT);
      const uint8_t *rows = small_rows + (s & 1) * (a.ring / 2) + t4 * 16;
      const int n = min(chunk, len - c * chunk);
#pragma unroll 2
      for (int p = warp; p * 32 < n; p += kSmallWarps) {
        const bool in = p * 32 + t4 * 8 < n;
        uint4 av[2], xv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t *q = rows + (i * 8 + g) * pitch + p * 64;
          av[i] = xv[i] = make_uint4(0, 0, 0, 0);
          if (in && i * 8 + g < nr) av[i] = *reinterpret_cast<const uint4 *>(q);
          if (in && i * 8 + g < nt) xv[i] = *reinterpret_cast<const uint4 *>(q + nr * pitch);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mma_m16n8k16(acc[j], xv[0].x, xv[1].x, xv[0].y, xv[1].y, av[j].x, av[j].y);
          mma_m16n8k16(acc[j], xv[0].z, xv[1].z, xv[0].w, xv[1].w, av[j].z, av[j].w);
        }
      }
      if (s + 2 < steps) {
        __syncthreads();  // this half has been read
        if (warp == 0) load(s + 2);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) part[warp][(c >> 1) * 8 + g][j * 8 + t4 * 2 + (c & 1)] = acc[j][c];
    __syncthreads();
    {
      const int m = tid / kSmallN, n = tid - m * kSmallN;  // one sum a thread; 8 of them have one owner
      float f = 0.0f;
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) f += part[w][m][n];
      peer_store(smem_addr(&recv[pass & 1][split][tid]), (tid >> 3) % splits, f);
    }
    lora_cluster_sync();
    // 8 columns a thread, the cluster's sums in the order of its CTAs
    const int i = tid * splits + split, m = i >> 1, c = (i & 1) * 8;
    if (m < nt && n0 + c < a.rank) {
      float f[8] = {};
      for (int p = 0; p < splits; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += recv[pass & 1][p][i * 8 + j];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= sc;
      store_u(a, token[m0 + m], n0 + c, f);
    }
  }
}

// ---------------------------------------------------------------------------
// The projection with the adapters as extra K blocks.
//
// Bound by the tensor cores for many tokens: 8192 tokens, 7168 -> 2048 with
// adapters of rank 64, 151 us, 1.6 PFLOP/s. For few by what a call has to do one
// after the other: u, W's way through one SM's ring, the last products and the
// sum over the cluster (64 tokens, 7168 -> 2048, 32 adapters of rank 16: 15.8 us
// with the shrink kernel, 12.1 without adapters, where the bytes alone are 5.7 us).
// ---------------------------------------------------------------------------
struct GemmShared {
  AdapterScratch scratch;
  int32_t list[2][kLBM];        // the adapters of a tile's tokens
  uint4 off[2][kLBM];           // for each of them, the rows that do not use it
  uint64_t full[kLMaxStages], empty[kLMaxStages];
  uint64_t tfull[2], tempty[2], lfull[2], lempty[2], ufull, uempty, done;
  int count[2];
  uint32_t tmem;
  int abort;
};

static_assert(kSmallThreads >= kSmallTokens, "a thread per token");
static_assert(kSmallThreads == kSmallM * kSmallN, "a thread per sum");
static_assert(sizeof(GemmShared) <= kLStatic && sizeof(ShrinkShared) <= kLStatic, "");

struct LTile {
  int t0, n0, cols;
};

// Tile w: groups of group_n n-tiles, each group swept over the m-tiles with its
// n-tiles innermost, so that the CTAs running at one time share both the
// group's weight tiles and each m-tile's rows in L2. The tiles from `whole` on
// are cut in halves of 128 outputs, numbered one after the other: the last,
// partial wave of whole tiles would keep less than half of the SMs busy.
template <int BN>
__device__ __forceinline__ LTile ltile_of(int w, const LoraArgs &a) {
  int half = 0, cols = BN;
  if (BN > 128 && w >= a.whole) {
    half = (w - a.whole) & 1;
    w = a.whole + ((w - a.whole) >> 1);
    cols = BN / 2;
  }
  const int per_group = a.mtiles * a.group_n;
  const int g = w / per_group, r = w - g * per_group;
  const int gw = min(a.group_n, a.ntiles_n - g * a.group_n);
  const int mt = r / gw;
  return LTile{mt * kLBM, (g * a.group_n + r - mt * gw) * BN + half * (BN / 2), cols};
}

// Whether a CTA takes several tiles: whole 256-wide ones only. All other forms have a CTA (or a cluster) for each tile.
template <int BN, bool SPLIT>
constexpr bool kLWalks = BN > 128 && !SPLIT;

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kGemmLThreads, 1)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_u, const __grid_constant__ CUtensorMap map_b,
                     const LoraArgs a) {
  constexpr int kAcc = kLWalks<BN, SPLIT> ? 2 : 1;  // accumulators
  constexpr uint32_t kCols = kAcc * BN;
  constexpr int kRedPitch = BN + 4;                 // floats of a row of partial sums
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) GemmShared sh;
  uint8_t *smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  const uint32_t ubuf = smem_addr(smem) + a.stages * a.stage;  // the tile's u, one x-shaped tile per 64 columns
  volatile int *abort = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = SPLIT ? static_cast<int>(lora_cluster_size()) : 1;
  const int split = SPLIT ? static_cast<int>(lora_cluster_rank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / splits : static_cast<int>(blockIdx.x);
  const int total = a.total;
  const int stride = kLWalks<BN, SPLIT> ? static_cast<int>(gridDim.x) : total;  // (the loops over tiles end after one)
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.kblocks) * split / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.kblocks) * (split + 1) / splits);
  const int rblocks = (a.rank + kLBK - 1) / kLBK;   // K blocks of one adapter

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(sh.full + s, 1);
      mbar_init(sh.empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sh.tfull + b, 1);
      mbar_init(sh.tempty + b, 4);
      mbar_init(sh.lfull + b, 1);
      mbar_init(sh.lempty + b, 2);
    }
    mbar_init(&sh.ufull, 1);
    mbar_init(&sh.uempty, 1);
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (tid == 32) {
    prefetch_tensormap(&map_x);
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_u);
    prefetch_tensormap(&map_b);
  }
  // With adapters the shrink kernel comes before this one: it let this grid
  // start only after its own dependency wait, so x is there, and only the warp
  // that loads u waits for it.
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_addr(&sh.tmem), kCols);
    tmem_relinquish();
  }
  if (!a.lora) grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const bool leader = elect_one();  // used by warps 0 and 1

  if (warp == 0) {
    // ---- TMA producer ----
    uint32_t it = 0;
    Ring r;
    int lt = 0;
    bool ok = true;
    const uint32_t ring = smem_addr(smem), fulls = smem_addr(sh.full);
    // asks for the tile's rows of W or of B_a in stage s
    const auto load_w = [&](const CUtensorMap *map, uint32_t s, int row, int k, int cols) {
      const uint32_t sw = ring + s * a.stage + a.xbytes, fb = fulls + s * 8;
      tma_load_2d(sw, map, k, row, fb);
      if (cols > kBoxRows) tma_load_2d(sw + kBoxRows * kLRow, map, k, row + kBoxRows, fb);
    };
    for (int w = first; ok && w < total; w += stride, ++lt) {
      const LTile t = ltile_of<BN>(w, a);
      for (int kb = kb0; kb < kb1; ++kb, ++it, r.next(a.stages)) {
        ok = warp_wait(sh.empty + r.s, r.ph ^ 1u, abort, a.err);
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(sh.full + r.s, static_cast<uint32_t>(a.xrows + t.cols) * kLRow);
          load_w(&map_w, r.s, t.n0, kb * kLBK, t.cols);
          tma_load_2d(ring + r.s * a.stage, &map_x, kb * kLBK, t.t0, fulls + r.s * 8);
        }
        __syncwarp();
      }
      if (!ok || !a.lora) continue;
      const int b = lt & 1;
      ok = warp_wait(sh.lfull + b, (lt >> 1) & 1u, abort, a.err);
      if (!ok) break;
      const int blocks = sh.count[b] * rblocks;
      for (int part = 0; ok && part < a.parts; ++part) {
        if (a.packed > 0) {  // a piece a lane
          for (int j = split; j < blocks; j += splits * a.packed, ++it, r.next(a.stages)) {
            ok = warp_wait(sh.empty + r.s, r.ph ^ 1u, abort, a.err);
            if (!ok) break;
            const int n = min(a.packed, (blocks - j + splits - 1) / splits) * a.pieces;
            if (leader) mbar_arrive_expect_tx(sh.full + r.s, static_cast<uint32_t>(n * t.cols) * kLPieceRow);
            __syncwarp();
            if (lane < n) {
              const int row = sh.list[b][j + lane / a.pieces * splits] * a.N + t.n0, k = lane % a.pieces * 16;
              const uint32_t dst = ring + r.s * a.stage + lane * (BN * kLPieceRow), fb = fulls + r.s * 8;
              tma_load_2d(dst, &map_b, k, row, fb);
              if (t.cols > kBoxRows) tma_load_2d(dst + kBoxRows * kLPieceRow, &map_b, k, row + kBoxRows, fb);
            }
            __syncwarp();
          }
        } else {
          for (int j = split; j < blocks; j += splits, ++it, r.next(a.stages)) {
            ok = warp_wait(sh.empty + r.s, r.ph ^ 1u, abort, a.err);
            if (!ok) break;
            if (leader) {
              mbar_arrive_expect_tx(sh.full + r.s, static_cast<uint32_t>(t.cols) * kLRow);
              load_w(&map_b, r.s, sh.list[b][j / rblocks] * a.N + t.n0, (j % rblocks) * kLBK, t.cols);
            }
            __syncwarp();
          }
        }
      }
      if (leader) mbar_arrive(smem_addr(sh.lempty + b));
      __syncwarp();
    }
    if (SPLIT) grid_dependents_launch();  // what comes next may be on its way during the last products and sums
    // the last loads land before the CTA may exit
    if (leader) drain_ring(sh.full, r, it, a.stages);
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer ----
    Ring r;
    int lt = 0;
    const uint32_t xlo = desc_lo(smem_addr(smem)), step = a.stage >> 4, xstep = a.xbytes >> 4;
    const uint32_t empty = smem_addr(sh.empty);
    uint32_t uphase = 0;  // parts of tiles' u that were used
    bool ok = true;
    for (int w = first; ok && w < total; w += stride, ++lt) {
      const int buf = lt % kAcc;
      ok = warp_wait(sh.tempty + buf, ((lt / kAcc) & 1) ^ 1u, abort, a.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * BN, idesc = idesc_bf16(kLBM, ltile_of<BN>(w, a).cols);
      for (int kb = kb0; kb < kb1; ++kb, r.next(a.stages)) {
        ok = warp_wait(sh.full + r.s, r.ph, abort, a.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t lo = xlo + r.s * step;
          mma_block(d, lo, lo + xstep, idesc, kb != kb0);
          mma_commit(empty + r.s * 8);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (a.lora) {
        const int b = lt & 1;
        ok = warp_wait(sh.lfull + b, (lt >> 1) & 1u, abort, a.err);
        if (!ok) break;
        const int blocks = sh.count[b] * rblocks;
        for (int part = 0; ok && part < a.parts; ++part) {
          if (split < blocks) {
            ok = warp_wait(&sh.ufull, uphase & 1u, abort, a.err);
            if (!ok) break;
            ++uphase;
          }
          if (a.packed > 0) {
            for (int j = split; j < blocks; j += splits * a.packed, r.next(a.stages)) {
              ok = warp_wait(sh.full + r.s, r.ph, abort, a.err);
              if (!ok) break;
              tc_fence_after();
              const int n = min(a.packed, (blocks - j + splits - 1) / splits);
              if (leader) {
                uint64_t piece = sw32_desc(smem_addr(smem) + r.s * a.stage);
                const uint32_t ulo = desc_lo(ubuf);
                for (int i = 0; i < n; ++i) {
                  const uint4 off = sh.off[b][j + i * splits];
                  for (int q = 0; q < a.pieces; ++q, piece += (BN * kLPieceRow) >> 4)
                    mma_bf16_rows(d, full_desc(ulo + q * 2), piece, idesc, off);
                }
                mma_commit(empty + r.s * 8);
              }
              __syncwarp();
            }
          } else {
            for (int j = split; j < blocks; j += splits, r.next(a.stages)) {
              ok = warp_wait(sh.full + r.s, r.ph, abort, a.err);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
                const uint32_t lo = xlo + r.s * step, ulo = desc_lo(ubuf) + (j % rblocks) * xstep;
                const uint4 off = sh.off[b][j / rblocks];
                // columns past the rank are zeros in both tiles, so a step's last ones add nothing
                const int cols = min(kLBK, a.rank - (j % rblocks) * kLBK);
                for (int kk = 0; kk * 16 < cols; ++kk)
                  mma_bf16_rows(d, full_desc(ulo + kk * 2), full_desc(lo + xstep + kk * 2), idesc, off);
                mma_commit(empty + r.s * 8);
              }
              __syncwarp();
            }
          }
          if (leader && split < blocks) mma_commit(smem_addr(&sh.uempty));
        }
        if (leader) mbar_arrive(smem_addr(sh.lempty + b));
      }
      if (ok && leader) mma_commit(smem_addr(sh.tfull + buf));
      __syncwarp();
    }
    // every MMA issued completes before the tensor memory is freed
    if (leader) {
      mma_commit(smem_addr(&sh.done));
      mbar_wait_bounded(&sh.done, 0);
    }
    __syncwarp();
  } else if (warp < 6) {
    // ---- epilogue: warp w reads TMEM lanes 32 * (w % 4) .. + 31 ----
    const int q = warp & 3, m = q * 32 + lane;
    int lt = 0;
    for (int w = first; w < total; w += stride, ++lt) {
      const int buf = lt % kAcc;
      if (!warp_wait(sh.tfull + buf, (lt / kAcc) & 1u, abort, a.err)) break;
      tc_fence_after();
      const LTile t = ltile_of<BN>(w, a);
      const bool valid = t.t0 + m < a.T;
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * BN;
      if constexpr (SPLIT) {
        float *red = reinterpret_cast<float *>(smem) + m * kRedPitch;
        if (__any_sync(0xffffffffu, valid)) {
          for (int c = 0; c < BN; c += 8) {
            float f[8];
            tmem_load8_wait(tb + c, f);
            if (valid) {
              *reinterpret_cast<float4 *>(red + c) = make_float4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<float4 *>(red + c + 4) = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
      } else {
        __nv_bfloat16 *row = a.y + static_cast<int64_t>(valid ? t.t0 + m : 0) * a.N + t.n0;
        for (int c = 0; c < t.cols; c += 32) {
          uint32_t r[32];
          tmem_load32_wait(tb + c, r);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (valid && t.n0 + c + v * 8 < a.N) {
              float f[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[v * 8 + j]);
              *reinterpret_cast<uint4 *>(row + c + v * 8) = round8(f);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(sh.tempty + buf));
    }
  } else if (a.lora) {
    // ---- the tile's adapters, the rows that do not use each of them, and u ----
    const int m = tid - 192;
    int lt = 0;
    uint32_t uphase = 0;  // parts of tiles' u that were loaded
    for (int w = first; w < total; w += stride, ++lt) {
      const int b = lt & 1;
      const LTile t = ltile_of<BN>(w, a);
      // the four warps go on or give up together: the barriers below take all of them
      if (!bar128_and<2>(warp_wait(sh.lempty + b, ((lt >> 1) & 1) ^ 1u, abort, a.err))) break;
      int slot = -1;
      bool bad = false;  // reported by the shrink kernel
      sh.off[b][m] = make_uint4(~0u, ~0u, ~0u, ~0u);
      const int n = tile_adapters<2>(a, t.t0, m, sh.scratch, sh.list[b], &slot, &bad);
      if (slot >= 0) atomicAnd(reinterpret_cast<uint32_t *>(&sh.off[b][slot]) + (m >> 5), ~(1u << (m & 31)));
      if (m == 0) sh.count[b] = n;
      bar128<2>();
      if (m == 0) mbar_arrive(smem_addr(sh.lfull + b));
      // The tile's u is loaded once, as soon as it is there: every CTA reads the
      // same few rows, and once per adapter (64 tokens, 32 adapters of rank 16)
      // they took 0.7 us a block.
      if (warp == 6 && split < n * rblocks) {
        grid_dependency_wait();  // u is written
        for (int part = 0; part < a.parts; ++part) {
          if (!warp_wait(&sh.uempty, (uphase & 1u) ^ 1u, abort, a.err)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh.ufull, static_cast<uint32_t>(rblocks * a.xrows) * kLRow);
            for (int q = 0; q < rblocks; ++q)
              tma_load_2d(ubuf + q * a.xbytes, &map_u, q * kLBK, part * a.T + t.t0, smem_addr(&sh.ufull));
          }
          __syncwarp();
          ++uphase;
        }
      }
    }
    // the last load lands before the CTA may exit
    if (warp == 6 && lane == 0 && uphase > 0) mbar_wait_bounded(&sh.ufull, (uphase - 1) & 1u);
  }
  __syncwarp();
  if constexpr (SPLIT) {
    lora_cluster_sync();
    if (first < total) {
      // the splits' sums, row m in CTA m % splits
      const LTile t = ltile_of<BN>(first, a);
      const int rows = min(kLBM, a.T - t.t0);
      constexpr int vecs = BN / 8;
      const int own = (rows - split + splits - 1) / splits;
      for (int i = tid; i < own * vecs; i += kGemmLThreads) {
        const int q = i / vecs, m = q * splits + split, c = (i - q * vecs) * 8;
        if (t.n0 + c >= a.N) continue;
        float f[8];
        cluster_sum8<kLMaxSplit>(smem_addr(reinterpret_cast<float *>(smem) + m * kRedPitch + c), splits, f);
        *reinterpret_cast<uint4 *>(a.y + static_cast<int64_t>(t.t0 + m) * a.N + t.n0 + c) = round8(f);
      }
    }
    lora_cluster_sync();  // no CTA leaves while another may still read its sums
  }
  // this grid ends after the shrink kernel also where no tile had an adapter:
  // what comes next in the stream waits for this grid only
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ---------------------------------------------------------------------------
// The projection of one token: a dot product of each row of W with it.
//
// Bound by the stream of W, so what counts besides it is what a call does before
// its first load and after its last: there is no ring to set up, no tensor memory
// and no cluster, only shuffles and one barrier. A CTA takes a few rows of W and
// all of K: thread tid the 16-byte vectors tid, tid + 256, ... of eight rows at a
// time, two vectors in turn, so that sixteen loads are in flight in a thread.
// Products and sums are in fp32, the sums over lanes and warps in a fixed order.
// The adapter's term is added last, from u and the rows of B_a, by eight lanes
// for each row.
// Against the tiles above, without an adapter and with one of rank 16: 4096 -> 4096
// 8.5 and 9.6 us (tiles 9.8 and 12.0), 7168 -> 2048 7.5 and 8.5 (10.3 and 12.4),
// 1024 -> 1024 4.3 and 7.2 (5.4 and 7.9), 2048 -> 7168 8.6 and 11.0 (9.3 and 11.5),
// 512 -> 7168 5.6 and 8.50 (5.8 and 8.43), 4096 -> 14336 24.1 and 26.1 (23.8 and
// 25.9): at worst 1% behind, so every single token comes here. When it was new, two
// tokens came out even with an adapter (10.8 and 11.2 us) and four behind (11.5 and
// 14.1: the sums take the
// registers that loads in flight need).
// ---------------------------------------------------------------------------
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneChunk = 8;  // rows at a time
constexpr int kOneRows = 16;  // rows of a CTA, at most

__device__ __forceinline__ void unpack8(const uint4 &r, float (&f)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(u[q] << 16);
    f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
  }
}

__global__ void __launch_bounds__(kOneThreads, 2)
    lora_one_kernel(const LoraArgs a, const uint4 *__restrict__ x, const uint4 *__restrict__ w,
                    const uint4 *__restrict__ lora_b) {
  __shared__ float part[kOneWarps][kOneRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = static_cast<int>(blockIdx.x) * a.own, rows = min(a.own, a.N - row0);
  const int kv = a.K / 8, rv = a.rank / 8;  // 16-byte vectors of a row of W and of B_a
  if (!a.lora) grid_dependency_wait();      // (as in the kernel above)
  for (int c0 = 0; c0 < rows; c0 += kOneChunk) {
    float acc[kOneChunk] = {};
    const uint4 *wr = w + static_cast<int64_t>(row0 + c0) * kv;
#pragma unroll 2
    for (int v = tid; v < kv; v += kOneThreads) {
      uint4 wv[kOneChunk];
#pragma unroll
      for (int j = 0; j < kOneChunk; ++j)
        wv[j] = c0 + j < rows ? __ldcs(wr + static_cast<int64_t>(j) * kv + v) : make_uint4(0, 0, 0, 0);
      float xf[8];
      unpack8(__ldg(x + v), xf);
#pragma unroll
      for (int j = 0; j < kOneChunk; ++j) {
        float wf[8];
        unpack8(wv[j], wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j] = fmaf(wf[e], xf[e], acc[j]);
      }
    }
    // each step halves the rows that a lane holds: in the end lane l has row l / 4 of the chunk
#pragma unroll
    for (int half = kOneChunk / 2, bit = 16; half > 0; half >>= 1, bit >>= 1) {
      const bool up = (lane & bit) != 0;
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float send = up ? acc[j] : acc[j + half], keep = up ? acc[j + half] : acc[j];
        acc[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    float f = acc[0];
    f += __shfl_xor_sync(0xffffffffu, f, 2);
    f += __shfl_xor_sync(0xffffffffu, f, 1);
    if ((lane & 3) == 0) part[warp][c0 + (lane >> 2)] = f;
  }
  grid_dependents_launch();  // what comes next may be on its way during the sums
  grid_dependency_wait();    // u is written
  __syncthreads();
  const int r = tid >> 3, sub = tid & 7;
  float f = 0.0f;
  if (r < rows) {
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < kOneWarps; ++i) f += part[i][r];
    }
    const int id = a.lora ? __ldg(a.adapter) : -1;
    if (id >= 0 && id < a.adapters) {
      const uint4 *u = reinterpret_cast<const uint4 *>(a.u);
      const uint4 *b = lora_b + (static_cast<int64_t>(id) * a.N + row0 + r) * rv;
      for (int v = sub; v < rv; v += 8) {
        float bf[8];
        unpack8(__ldg(b + v), bf);
        for (int part = 0; part < a.parts; ++part) {
          float uf[8];
          unpack8(__ldcg(u + part * rv + v), uf);
#pragma unroll
          for (int e = 0; e < 8; ++e) f = fmaf(uf[e], bf[e], f);
        }
      }
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
  if (r < rows && sub == 0) a.y[row0 + r] = __float2bfloat16_rn(f);
}

static_assert(kOneRows * 8 <= kOneThreads, "eight lanes a row");

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// 2-D map of a row-major [rows][K] bf16 matrix, boxes of box_rows x 64 (or 16) elements, 128-byte (32-byte) swizzle.
bool make_box_map(CUtensorMap *map, const void *base, int64_t K, int64_t rows, int box_rows, int box_k = kLBK) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_k), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box_k == kLBK ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_32B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's attributes, set once on a device (a call of two kernels spent 1 us
// of 6 on the host setting them anew): up to `most` bytes of dynamic shared
// memory, and the largest carve-out, so that an SM which runs one of the kernels
// has room for the other.
template <auto FN>
bool kernel_ready(int most) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if ((done.load(std::memory_order_relaxed) & bit) != 0) return true;
  if (cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
      cudaFuncSetAttribute(FN, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Launch with a cluster of `cluster` CTAs and programmatic dependent launch.
template <auto FN, class... Q>
moe_status launch_cluster(int most, dim3 grid, int threads, int cluster, int smem, cudaStream_t stream, Q &&...args) {
  if (smem > most) return MOE_EINVAL;
  if (!kernel_ready<FN>(most)) return MOE_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = MOE_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, FN, args...) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

// A launch's dynamic shared memory: what it uses, and at least its columns'
// share. (All 512 columns: the most a CTA can have, which leaves no room for
// another one's share.)
int with_columns(int smem, int cols) {
  int share = cols * kLBytesPerCol;
  if (share > kLSmemMax - kLStatic) share = kLSmemMax - kLStatic;
  return smem > share ? smem : share;
}

// Stages of a ring of at most `bytes`, no more than there are K blocks, and at least 3.
int ring_stages(int stage, int blocks, int bytes) {
  int n = bytes / stage;
  if (n > kLMaxStages) n = kLMaxStages;
  if (n > blocks) n = blocks;
  return n < 3 ? 3 : n;
}

// Rings of CTAs that are to share an SM: two shrink CTAs, one and a CTA of the
// projection, or two of the projection.
constexpr int kShrinkRing = 84 * 1024;
constexpr int kSplitRing = 84 * 1024;
constexpr int kSplitRingFew = 128 * 1024;  // up to kFewShrink tokens: their shrink CTAs leave SMs enough
constexpr int kFewShrink = 8;
// Rows of few tokens' shrink CTAs: two CTAs an SM. Where there are no more of
// them than SMs, one an SM: they come while the last call's projection is ending,
// and several on an SM that it does not use would leave no room for the next
// projection's CTA there, whose cluster then starts when they end (64 tokens: 5 to
// 7 us late for half of the clusters).
constexpr int kSmallRows = 80 * 1024;
constexpr int kSmallAlone = 90 * 1024;
constexpr int kSmallLeast = 12 * 1024;  // a half holds 64 elements of the most rows
static_assert(small_chunk(kSmallLeast / 2, kSmallM + kSmallN) >= 64 && kSmallRows % 256 == 0 && kSmallLeast % 256 == 0, "");

// Whether u is computed 16 tokens of an adapter at a time: up to 16 tokens, one
// pass each; up to 64 where they are likely to use enough adapters. Every further
// pass of an adapter's tokens costs 3 us or more, while the tensor-memory tiles
// take all of them at once. Which adapters are used is not known here, so this
// goes by how many there are. Measured, small tiles and tensor memory, 4096 ->
// 4096: 16 tokens of one adapter 12.3 and 14.4 us, 20 of one 17.4 and 14.3, 24 of
// two 12.7 and 14.7, 64 of 16 19.7 and 20.4 (four used: 21.7 and 19.6), 64 of 8
// 20.2 and 19.2 (24.5 and 18.4), 128 of 32 20.5 and 24.0 (27.4 and 21.8); 64
// tokens 7168 -> 2048 of 32: 15.9 and 20.7.
bool few_tokens(const LoraArgs &a) {
  if (a.T <= kSmallM) return true;
  return a.T <= 2 * kSmallM ? a.adapters >= 2 : a.T <= kSmallTokens && a.T <= 4 * static_cast<int64_t>(a.adapters);
}

moe_status launch_shrink_small(LoraArgs a, const void *x, const void *lora_a, int sms, cudaStream_t stream) {
  const int nchunks = (a.rank + kSmallN - 1) / kSmallN;
  const int clusters = a.adapters < a.T ? a.adapters : a.T;  // for each 16 rows
  const int64_t busy = static_cast<int64_t>(clusters) * nchunks;
  int splits = kLMaxCluster;
  while (splits > 1 && busy * splits > sms) splits >>= 1;
  const dim3 grid(static_cast<unsigned>(clusters * splits), static_cast<unsigned>(nchunks));
  const int64_t ctas = static_cast<int64_t>(grid.x) * grid.y;
  const int rows = (a.rank < kSmallN ? a.rank : kSmallN) + (a.T < kSmallM ? a.T : kSmallM);
  const int64_t slice = static_cast<int64_t>((a.K + 31) / 32 + splits - 1) / splits * 32;  // a CTA's K elements, at most
  const int64_t need = rows * ((slice + 63) / 64 * 128 + kSmallPad);
  a.ring = need < kSmallRows ? static_cast<int>((need + 255) / 256 * 256) : kSmallRows;
  if (a.ring < kSmallLeast) a.ring = kSmallLeast;
  const int least = a.T > kFewShrink && ctas <= sms ? kSmallAlone : 0;
  return launch_cluster<lora_shrink_small_kernel>(kSmallAlone, grid, kSmallThreads, splits,
                                                  a.ring > least ? a.ring : least, stream, a,
                                                  static_cast<const __nv_bfloat16 *>(x),
                                                  static_cast<const __nv_bfloat16 *>(lora_a));
}

moe_status launch_shrink(LoraArgs a, const void *x, const void *lora_a, int sms, cudaStream_t stream) {
  if (few_tokens(a)) return launch_shrink_small(a, x, lora_a, sms, stream);
  const int most = a.adapters < a.T ? (a.adapters < kLBM ? a.adapters : kLBM) : (a.T < kLBM ? a.T : kLBM);
  // up to two CTAs an SM (8192 tokens: the whole call takes 184 us so, 189 us with one)
  int splits = kLMaxCluster;
  while (splits > 1 && (a.mtiles * splits > 2 * sms || splits > a.kblocks)) splits >>= 1;
  // few tokens: their adapters are spread over the SMs that are left
  const int spread = sms / (a.mtiles * splits) > 1 ? sms / (a.mtiles * splits) : 1;
  a.per_pass = (most + spread - 1) / spread;
  if (a.per_pass > kShrinkCols / a.rank) a.per_pass = a.rank > kShrinkCols ? 1 : kShrinkCols / a.rank;
  a.groups = (most + a.per_pass - 1) / a.per_pass;
  if (a.groups > spread) a.groups = spread;
  int n = (a.per_pass * a.rank + 15) & ~15;
  a.cols = 32;
  while (static_cast<int>(a.cols) < n) a.cols <<= 1;
  // room for two stages of the widest tile; narrower ones have up to kLMaxStages
  a.ring = 2 * (a.xbytes + n * kLRow);
  if (a.ring < kShrinkRing) a.ring = kShrinkRing;
  a.stages = kLMaxStages;
  // the products take 128 rows from the x tile's place also where the tile has
  // fewer: what follows it inside the allocation is read then
  int smem = 1024 + a.ring + kLBM * kLRow - a.xbytes;
  const int red = 1024 + kLBM * a.rank * 4;
  if (smem < red) smem = red;
  smem = with_columns(smem, static_cast<int>(a.cols));
  CUtensorMap mx, ma;
  if (!make_box_map(&mx, x, a.K, a.T, a.xrows) ||
      !make_box_map(&ma, lora_a, a.K, static_cast<int64_t>(a.adapters) * a.rank, a.rank))
    return MOE_ECUDA;
  const int64_t grid = static_cast<int64_t>(a.mtiles) * a.groups * splits;
  if (grid > 0x7fffffffll) return MOE_EINVAL;
  return launch_cluster<lora_shrink_kernel>(kLSmemMax - kLStatic, dim3(static_cast<unsigned>(grid)), kShrinkThreads, splits,
                                            smem, stream, mx, ma, a);
}

// The projection's tiles: their width and the CTAs that share one's K, by the
// time they are expected to take, in ns: waves of CTAs x K blocks of one x the
// time of a block, the sum over a cluster, and an end (a tile's stores and, for
// 256-wide tiles, the shrink kernel that their CTAs have to let finish first).
// A block takes longer the more CTAs there are, and where rows of x and W do not
// begin on 128-byte lines; sums of 128 tokens or fewer take half the time. Only
// 256-wide tiles come several to a CTA, and widths of 64 are for 128 tokens.
// The constants were fitted to the times of every choice at 360 shapes (1 to 2500
// tokens, 512 to 7168 inputs and outputs): the calls take 1% longer than with the
// best choice in the geometric mean, 12% at worst but for one shape. 256 tokens
// 1024 -> 2048: 12.2 us with 128-wide tiles, 14.4 with two CTAs a tile, 16.9 with
// four; 1000 tokens 4096 -> 1024: 24.2, 19.5 and 25.3 us.
int tile_width(const LoraArgs &a, int sms, int *splits) {
  constexpr int kWidths[3] = {64, 128, 256};
  constexpr int kBlockNs[3] = {220, 290, 340}, kEndNs[3] = {1200, 1100, 4700};
  constexpr int kSum2Ns = 2800, kSum4Ns = 6700;
  const double unaligned = a.K % kLBK != 0 ? 1.35 : 1.0;
  double best = 1e300;
  int width = 256;
  *splits = 1;
  for (int i = 0; i < 3; ++i)
    for (int s = 1; s <= kLMaxSplit; s *= 2) {
      if (s > a.kblocks || (kWidths[i] == 64 && (a.mtiles > 1 || s == 1))) continue;
      const int64_t ctas = static_cast<int64_t>(a.mtiles) * ((a.N + kWidths[i] - 1) / kWidths[i]) * s;
      if ((s > 1 || kWidths[i] < 256) && ctas > sms) continue;
      const double busy = ctas < sms ? static_cast<double>(ctas) / sms : 1.0;
      const double block = kBlockNs[i] * unaligned * (0.57 + 0.43 * busy);
      const double sum = (s == 1 ? 0 : s == 2 ? kSum2Ns : kSum4Ns) * (a.T <= kLBM ? 0.5 : 1.0);
      const double ns = static_cast<double>((ctas + sms - 1) / sms) * ((a.kblocks + s - 1) / s) * block + kEndNs[i] + sum;
      if (ns < best) {
        best = ns;
        width = kWidths[i];
        *splits = s;
      }
    }
  return width;
}

template <int BN, bool SPLIT>
moe_status launch_gemm(LoraArgs a, const void *x, const void *w, const void *lora_b, int splits, int sms,
                       cudaStream_t stream) {
  a.ntiles_n = (a.N + BN - 1) / BN;
  a.stage = a.xbytes + BN * kLRow;
  const int rblocks = a.lora ? (a.rank + kLBK - 1) / kLBK : 0;
  // what follows the ring: u, and the rest of the 128 rows of x that the products take (as in the shrink kernel)
  const int tail = rblocks * a.xbytes + kLBM * kLRow - a.xbytes;
  // BN 256: four stages, or three beside a u of rank above 64. BN 128 over whole tiles: three (with six, which keep
  // the shrink kernel's CTAs off the SM, no block came sooner)
  a.stages = BN > 128 ? (rblocks <= 1 ? 4 : 3)
             : SPLIT  ? ring_stages(a.stage, (a.kblocks + splits - 1) / splits, a.T > kFewShrink ? kSplitRing : kSplitRingFew)
                      : 3;
  const int64_t tiles = static_cast<int64_t>(a.mtiles) * a.ntiles_n;
  if (tiles > 0x3fffffffll / kLMaxSplit) return MOE_EINVAL;
  a.whole = a.total = static_cast<int>(tiles);
  constexpr bool kWalks = kLWalks<BN, SPLIT>;
  const int64_t grid = kWalks ? (tiles < sms ? tiles : sms) : tiles * splits;
  const int rest = static_cast<int>(tiles % grid);
  if (kWalks && rest > 0 && 2 * rest <= grid) {
    a.whole -= rest;
    a.total += rest;
  }
  a.group_n = a.ntiles_n < 8 ? a.ntiles_n : 8;
  const int smem = with_columns(1024 + a.stages * a.stage + tail, (kWalks ? 2 : 1) * BN);
  if (smem > kLSmemMax - kLStatic) return MOE_EINVAL;
  constexpr int kBox = BN < kBoxRows ? BN : kBoxRows;
  a.pieces = (a.rank + 15) / 16;
  a.packed = a.lora && a.pieces <= kLPackedPieces ? a.stage / (BN * kLPieceRow) / a.pieces : 0;
  CUtensorMap mx, mw, mu, mb;
  if (!make_box_map(&mx, x, a.K, a.T, a.xrows) || !make_box_map(&mw, w, a.K, a.N, kBox)) return MOE_ECUDA;
  mu = mx;
  mb = mw;  // not used without adapters
  if (a.lora && (!make_box_map(&mu, a.u, a.rank, static_cast<int64_t>(a.parts) * a.T, a.xrows) ||
                 !make_box_map(&mb, lora_b, a.rank, static_cast<int64_t>(a.adapters) * a.N, kBox, a.packed > 0 ? 16 : kLBK)))
    return MOE_ECUDA;
  return launch_cluster<lora_gemm_kernel<BN, SPLIT>>(kLSmemMax - kLStatic, dim3(static_cast<unsigned>(grid)), kGemmLThreads,
                                                     SPLIT ? splits : 1, smem, stream, mx, mw, mu, mb, a);
}

// The projection of one token: two CTAs an SM, as far as their rows go.
moe_status launch_one(LoraArgs a, const void *x, const void *w, const void *lora_b, int sms, cudaStream_t stream) {
  a.own = (a.N + 2 * sms - 1) / (2 * sms);
  if (a.own > kOneRows) a.own = kOneRows;
  return launch_cluster<lora_one_kernel>(0, dim3(static_cast<unsigned>((a.N + a.own - 1) / a.own)), kOneThreads, 1, 0, stream, a,
                                         static_cast<const uint4 *>(x), static_cast<const uint4 *>(w),
                                         static_cast<const uint4 *>(lora_b));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_lora_linear(const moe_lora_desc *desc, const void *x, const void *w, const void *lora_a,
                                      const void *lora_b, const float *scales, const int32_t *adapter, void *u, void *y,
                                      int32_t *err, void *stream) {
  if (desc == nullptr) return MOE_EINVAL;
  const int T = desc->num_tokens, K = desc->in_dim, N = desc->out_dim, r = desc->rank, A = desc->num_adapters;
  if (T < 0 || K < 8 || N < 8 || A < 0 || K % 8 != 0 || N % 8 != 0 || desc->num_sms < 0) return MOE_EINVAL;
  if (A > 0 && (r < 8 || r > kLMaxRank || r % 8 != 0)) return MOE_EINVAL;
  const int parts = desc->u_parts > 1 ? desc->u_parts : 1;
  if (desc->u_parts < 0 || parts > 2) return MOE_EINVAL;
  // weight rows are 32-bit TMA coordinates, a tile's last ones may lie up to 256 past the end
  if (static_cast<int64_t>(A) * N > INT32_MAX - 256 || static_cast<int64_t>(A) * r > INT32_MAX - 256 ||
      static_cast<int64_t>(parts) * T > INT32_MAX - 256 || N > INT32_MAX - 256 || K > INT32_MAX - 256)
    return MOE_EINVAL;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (x == nullptr || w == nullptr || y == nullptr || !aligned16(x) || !aligned16(w) || !aligned16(y))
    return MOE_EINVAL;
  if (A > 0 && (lora_a == nullptr || lora_b == nullptr || adapter == nullptr || u == nullptr || !aligned16(lora_a) ||
                !aligned16(lora_b) || !aligned4(scales) || !aligned4(adapter) || !aligned16(u)))
    return MOE_EINVAL;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int sms = desc->num_sms > 0 && desc->num_sms < sm_count() ? desc->num_sms : sm_count();
  LoraArgs a{};
  a.adapter = adapter;
  a.scales = scales;
  a.u = static_cast<__nv_bfloat16 *>(u);
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.err = err;
  a.T = T;
  a.K = K;
  a.N = N;
  a.rank = A > 0 ? r : kLBK;
  a.adapters = A;
  a.lora = A > 0;
  a.parts = parts;
  a.xrows = T >= kLBM ? kLBM : (T + 7) / 8 * 8;
  a.xbytes = a.xrows * kLRow;
  a.kblocks = (K + kLBK - 1) / kLBK;
  a.mtiles = (T + kLBM - 1) / kLBM;
  if (a.lora) {
    const moe_status st = launch_shrink(a, x, lora_a, sms, cs);
    if (st != MOE_OK) return st;
  }
  if (T == 1) return launch_one(a, x, w, lora_b, sms, cs);
  int splits = 1;
  switch (tile_width(a, sms, &splits)) {
    case 256:
      return splits > 1 ? launch_gemm<256, true>(a, x, w, lora_b, splits, sms, cs)
                        : launch_gemm<256, false>(a, x, w, lora_b, 1, sms, cs);
    case 64: return launch_gemm<64, true>(a, x, w, lora_b, splits, sms, cs);
    default: break;
  }
  if (splits > 1) return launch_gemm<128, true>(a, x, w, lora_b, splits, sms, cs);
  return launch_gemm<128, false>(a, x, w, lora_b, 1, sms, cs);
}
