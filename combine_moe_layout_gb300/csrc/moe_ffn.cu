// The gated feed-forward block in training: linear 1 that keeps its projections,
// linear 2, and the gradients with respect to the rows and all three weights, for
// the packed rows of every expert (or one dense block), on the 5th-generation
// tensor cores.
//
//   g = x w_gate^T, u = x w_up^T, h = bf16(act(g) u), y = h w_down^T
//   dh = dy w_down;  dg = dh u act'(g), du = dh act(g)
//   dx = dg w_gate + du w_up
//   dw_gate = dg^T x, dw_up = du^T x, dw_down = dy^T h   (sums over an expert's rows)
//
// One persistent kernel, a CTA per SM, in five forms. Roles as in the expert
// stage: a TMA producer warp, an MMA warp with two 128 x 256 fp32 accumulators in
// tensor memory, eight epilogue warps; in the weights' form one more warp that
// clears what the last K block of an expert holds of the next one's rows.
//
//   form   D [128 x up to 256]        A                    B                     K
//   kUp    g | u (128 + 128 columns)  x          K-major   w_gate | w_up K-major H
//   kDown  y                          h          K-major   w_down  K-major       I
//   kDh    dh, made dg, du and h      dy         K-major   w_down  N-major       H
//   kDx    dx                         dg then du K-major   w_gate then w_up, N-major   2 I
//   kDw    dw (three of them)         dg, du, dy M-major   x, x, h  N-major      rows of the expert
//
// The transposed operands are read as they lie in memory: a box of 64 columns and
// 64 rows lands as 64 swizzled 128-byte lines, the M- or N-major form of the
// 128-byte swizzle (64 elements contiguous, lines of successive k 128 bytes
// apart), so that no kernel transposes anything. Weights have 3-D maps, [expert]
// outermost: a box that passes an expert's last row or column is filled with
// zeros, whatever the next expert's weights hold, and widths need only be
// multiples of 8.
//
// Measured, among others: 24576 rows of 64 uneven experts, 4096 -> 1408, kept in 8
// bits: forward 776 to 816 us on different cards (1.04 to 1.10 PFLOP/s), gradients
// 1748 to 1788 us, both 0.88 of that with 384 rows each; 4096 rows, 4096 -> 14336:
// forward 860 us (1.68 PFLOP/s) a few at a time and 930 in a loop of a second,
// gradients 2075 to 2132 us.
// Bound by the tensor cores under the power limit, less the rows that an expert's
// last tile does not have, and in dw of short experts by its results' way out.
// 512 rows of 64 experts, 4096 -> 1408 (2.2 GB of weights): 329 us, 6.7 TB/s.
//
// What is rounded: h, dg and du to bf16 between two products (each is an operand
// of bf16 tensor cores: at most 2^-8 of a term, as its output's own rounding; the
// results are 2.35e-3 off in the 2-norm, 1.66e-3 of which is their own), sums in
// fp32 throughout. The tensor cores drop what falls below a sum's last place
// instead of rounding it, so that sums of thousands of terms come out low by a
// little: the kept scales of 4096 inputs by 4.2e-6 of their value.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <initializer_list>

#include "moe_ffn.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kUK = 16;
constexpr int kBN = 256;
constexpr int kStages = 4;
constexpr int kTileA = kBM * kBK * 2;
constexpr int kTileB = kBN * kBK * 2;
constexpr int kStage = kTileA + kTileB;
constexpr int kHalfBox = 64 * kBK * 2;    // a box of 64 columns x 64 rows
constexpr int kFullBox = 128 * kBK * 2;   // a box of 64 columns x 128 rows
constexpr int kEpilogueWarps = 8;  // two for each quarter of tensor memory's lanes
constexpr int kThreads = 64 + 32 * kEpilogueWarps, kThreadsDw = kThreads + 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemFixed = 1024 + kStages * kStage + (3 * kStages + 5) * 8 + 8;
constexpr int kSmemMax = 227 * 1024;
constexpr int kPiece = 32 * 64 * 2;  // kDw: 32 rows x 64 columns of the result, on their way out of a warp
constexpr int kSmemDw = kSmemFixed + kEpilogueWarps * kPiece;
static_assert(kSmemDw <= kSmemMax, "");

// A wait for something that comes after n K blocks (a whole tile's, or those of every tile up to the next one with a
// tail) allows for each of them 10 us, ten times what one takes when its operands come from HBM: a weight's gradient over
// 2^27 rows has two million blocks in a tile and takes longer than a wait for one copy may.
__device__ __forceinline__ uint64_t blocks_ns(uint32_t n) { return kMbarWaitNs + n * 10000ull; }

enum Form { kUp = 0, kDown = 1, kDh = 2, kDx = 3, kDw = 4 };

__host__ __device__ constexpr bool a_is_mn(int form) { return form == kDw; }
__host__ __device__ constexpr bool b_is_mn(int form) { return form >= kDh; }

// Descriptor of an M- or N-major bf16 tile with the 128-byte swizzle, made of boxes
// of 64 (M or N) x 64 (K): the leading-dimension offset is the next box (8192
// bytes), the stride offset the next 8 lines of K (1024 bytes).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kHalfBox >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

struct FfnMaps {
  CUtensorMap m[5];  // operands
  CUtensorMap d[3];  // kDw: the results
  CUtensorMap zeros[4];  // kDw: boxes of 1, 2, 4 and 8 lines, unswizzled
};

struct FfnArgs {
  const int32_t *offsets;  // [E * R + 1], or null: one expert with all rows
  int32_t *err;
  void *out0, *out1, *out2;             // by form: h | y | dg, du, h | dx
  const void *gate, *up;                // kDh: what the forward kept
  const float *gate_scales, *up_scales;
  void *keep_gate, *keep_up;            // kUp: what it keeps
  float *keep_gate_scales, *keep_up_scales;
  int rows, E, R;
  int H, I;
  int kblocks;    // K blocks of a tile (kDw: by the expert's rows)
  int n_total;    // output columns
  int out_cols;   // output columns of a tile: 128 (kUp) or 256
  int ntiles_n, group_n;
  int act, save;
  int wide;       // every row that the epilogue touches begins on a 32-byte boundary
  int dw_total;   // kDw: tiles of all experts
  int first;      // the first kernel of its call
};

struct Job {
  int e, row0, rows;  // packed rows (kDw: all of the expert's)
  int m0, n0, ncols;  // kDw: first row of the weight; first output column and the tile's MMA width
  int which;          // kDw: 0 dw_gate, 1 dw_up, 2 dw_down
  int kblocks, tail;  // tail: rows of the last K block (kDw; 64 or 0: whole)
};

// First packed row of expert e; e = E: behind the last.
__device__ __forceinline__ int row_offset(const FfnArgs &a, int e) {
  return a.offsets != nullptr ? __ldg(a.offsets + static_cast<int64_t>(e) * a.R) : (e == 0 ? 0 : a.rows);
}

template <int FORM>
__device__ __forceinline__ Job job_of(int w, const int32_t *pref, const int32_t *offs, const FfnArgs &a) {
  Job j;
  if constexpr (FORM == kDw) {
    // expert by expert; in each the three weights, in groups of group_n column tiles swept by row tiles
    const int mi = (a.I + kBM - 1) / kBM, mh = (a.H + kBM - 1) / kBM;
    const int ni = (a.I + a.out_cols - 1) / a.out_cols, nh = (a.H + a.out_cols - 1) / a.out_cols;
    const int p01 = mi * nh, per = 2 * p01 + mh * ni;
    j.e = w / per;
    int r = w - j.e * per;
    j.which = r < p01 ? 0 : (r < 2 * p01 ? 1 : 2);
    r -= j.which * p01;
    const int mt = j.which == 2 ? mh : mi, nt = j.which == 2 ? ni : nh;
    const int g = r / (mt * a.group_n);
    r -= g * mt * a.group_n;
    const int gw = min(a.group_n, nt - g * a.group_n);
    const int m = r / gw;
    j.m0 = m * kBM;
    j.n0 = (g * a.group_n + r - m * gw) * a.out_cols;
    const int left = (j.which == 2 ? a.I : a.H) - j.n0;
    j.ncols = min(a.out_cols, (left + 63) & ~63);
    const int lo = row_offset(a, j.e), hi = row_offset(a, j.e + 1);
    const bool good = lo >= 0 && hi >= lo && hi <= a.rows;
    j.row0 = good ? lo : 0;
    j.rows = good ? hi - lo : 0;
    j.kblocks = (j.rows + kBK - 1) / kBK;
    j.tail = j.rows & (kBK - 1);
  } else {
    const Tile t = tile_of<kBM>(w, pref, offs, a);
    j.e = t.e;
    j.row0 = t.row0;
    j.rows = t.rows;
    j.m0 = 0;
    j.n0 = t.n0;
    j.which = 0;
    j.kblocks = a.kblocks;
    j.tail = 0;
    if constexpr (FORM == kUp)
      j.ncols = kBN;
    else if constexpr (FORM == kDown)
      j.ncols = a.n_total - t.n0 > 128 ? 256 : 128;
    else
      j.ncols = min(kBN, (a.n_total - t.n0 + 63) & ~63);
  }
  return j;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float lo_of(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_of(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void e4m3x2_to_float(uint16_t c, float *lo, float *hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  float a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(h));
  *lo = a;
  *hi = b;
}

// ---- epilogues: one thread, half of its accumulator row ----

// 32 bytes of a row: one whole sector where rows begin on such a boundary (two stores of 16 bytes each reach L2 as
// two half sectors), `left` of their elements of 1 << ELEM bytes existing.
template <int ELEM>
__device__ __forceinline__ void store32(void *dst, const uint32_t *v, bool wide, int left) {
  constexpr int per = 32 >> ELEM;  // elements
  if (wide && left >= per) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
    return;
  }
  uint4 *d = static_cast<uint4 *>(dst);
  if (left > 0) d[0] = make_uint4(v[0], v[1], v[2], v[3]);
  if (left > per / 2) d[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

template <int ELEM>
__device__ __forceinline__ void load32(const void *src, uint32_t *v, bool wide, int left) {
  constexpr int per = 32 >> ELEM;
  if (wide && left >= per) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src));
    return;
  }
  const uint4 *s = static_cast<const uint4 *>(src);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 a = left > 0 ? __ldg(s) : zero, b = left > per / 2 ? __ldg(s + 1) : zero;
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// y, dx, dw: 32 columns, rounded.
__device__ __forceinline__ void store_plain(__nv_bfloat16 *dst, const uint32_t *r, bool wide, int left) {
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t pk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      pk[i] = pack2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
    store32<1>(dst + 16 * v, pk, wide, left - 16 * v);
  }
}

// h = act(g) u for 32 columns; r: g then u.
__device__ __forceinline__ void store_hidden(__nv_bfloat16 *dst, const uint32_t (&r)[64], int act, bool wide, int left) {
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t pk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = 16 * v + 2 * i;
      const float h0 = act_of<false>(__uint_as_float(r[k]), act, nullptr) * __uint_as_float(r[32 + k]);
      const float h1 = act_of<false>(__uint_as_float(r[k + 1]), act, nullptr) * __uint_as_float(r[33 + k]);
      pk[i] = pack2(h0, h1);
    }
    store32<1>(dst + 16 * v, pk, wide, left - 16 * v);
  }
}

// 32 columns as e4m3 codes of the block's scale (library format: amax / 448 over 128 columns).
__device__ __forceinline__ void store_codes(uint8_t *dst, const uint32_t *r, const BlockScale &bs, bool wide) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q[i] = static_cast<uint32_t>(
               e4m3x2_of_quotients(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), bs)) |
           (static_cast<uint32_t>(
                e4m3x2_of_quotients(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]), bs))
            << 16);
  store32<0>(dst, q, wide, 32);
}

__device__ __forceinline__ void epilogue_up(const FfnArgs &a, const Job &t, uint32_t tb, int m, int half) {
  const bool valid = m < t.rows, wide = a.wide != 0;
  const int64_t p = t.row0 + (valid ? m : 0);
  const int left = a.I - t.n0;  // columns of the tile that exist
  const int64_t at = p * a.I + t.n0;
  BlockScale gs, us;
  if (a.save == MOE_SAVE_FP8) {  // I is a multiple of 128: the tile's 128 columns are one block
    float ga = 0.0f, ua = 0.0f;
    for (int c = 0; c < 128; c += 32) {
      uint32_t r[64];
      tmem_load32x2_wait(tb + c, tb + 128 + c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        ga = fmaxf(ga, fabsf(__uint_as_float(r[i])));
        ua = fmaxf(ua, fabsf(__uint_as_float(r[32 + i])));
      }
    }
    gs = block_scale(ga);
    us = block_scale(ua);
    if (valid) {
      const int64_t sc = p * (a.I / kScaleBlock) + t.n0 / kScaleBlock;
      if (half == 0)
        a.keep_gate_scales[sc] = gs.s;
      else
        a.keep_up_scales[sc] = us.s;
    }
  }
  for (int c = 64 * half; c < 64 * half + 64; c += 32) {
    uint32_t r[64];
    tmem_load32x2_wait(tb + c, tb + 128 + c, r);
    if (!valid) continue;
    store_hidden(static_cast<__nv_bfloat16 *>(a.out0) + at + c, r, a.act, wide, left - c);
    if (a.save == MOE_SAVE_BF16) {
      store_plain(static_cast<__nv_bfloat16 *>(a.keep_gate) + at + c, r, wide, left - c);
      store_plain(static_cast<__nv_bfloat16 *>(a.keep_up) + at + c, r + 32, wide, left - c);
    } else if (a.save == MOE_SAVE_FP8) {
      store_codes(static_cast<uint8_t *>(a.keep_gate) + at + c, r, gs, wide);
      store_codes(static_cast<uint8_t *>(a.keep_up) + at + c, r + 32, us, wide);
    }
  }
}

// dg, du and h of 16 columns, from dh and what was kept (8 words of bf16 pairs, or 4 of codes).
template <bool F8>
__device__ __forceinline__ void dh_of(const uint32_t *gq, const uint32_t *uq, float gsc, float usc, const uint32_t *dh,
                                      int act, uint32_t (&pd)[8], uint32_t (&pu)[8], uint32_t (&ph)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float g0, g1, u0, u1;
    if constexpr (F8) {
      e4m3x2_to_float(static_cast<uint16_t>(gq[k >> 1] >> (16 * (k & 1))), &g0, &g1);
      e4m3x2_to_float(static_cast<uint16_t>(uq[k >> 1] >> (16 * (k & 1))), &u0, &u1);
      g0 *= gsc, g1 *= gsc, u0 *= usc, u1 *= usc;
    } else {
      g0 = lo_of(gq[k]), g1 = hi_of(gq[k]), u0 = lo_of(uq[k]), u1 = hi_of(uq[k]);
    }
    float d0, d1;
    const float a0 = act_of<true>(g0, act, &d0), a1 = act_of<true>(g1, act, &d1);
    const float h0 = __uint_as_float(dh[2 * k]), h1 = __uint_as_float(dh[2 * k + 1]);
    pd[k] = pack2(h0 * u0 * d0, h1 * u1 * d1);
    pu[k] = pack2(h0 * a0, h1 * a1);
    ph[k] = pack2(a0 * u0, a1 * u1);
  }
}

__device__ __forceinline__ void epilogue_dh(const FfnArgs &a, const Job &t, uint32_t tb, int m, int half) {
  const bool valid = m < t.rows, wide = a.wide != 0, f8 = a.save == MOE_SAVE_FP8;
  const int64_t p = t.row0 + (valid ? m : 0);
  const int end = min(t.ncols, 128 * half + 128);
  for (int c = 128 * half; c < end; c += 32) {
    const int left = a.I - t.n0 - c;
    const int64_t at = p * a.I + t.n0 + c;
    uint32_t gq[16], uq[16];  // 32 values as bf16 pairs, or as codes in the first 8
    float gsc = 1.0f, usc = 1.0f;
    if (valid) {
      if (f8) {
        load32<0>(static_cast<const uint8_t *>(a.gate) + at, gq, wide, left);
        load32<0>(static_cast<const uint8_t *>(a.up) + at, uq, wide, left);
        if (left > 0) {
          const int64_t sc = p * (a.I / kScaleBlock) + (t.n0 + c) / kScaleBlock;
          gsc = __ldg(a.gate_scales + sc);
          usc = __ldg(a.up_scales + sc);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          load32<1>(static_cast<const uint16_t *>(a.gate) + at + 16 * v, gq + 8 * v, wide, left - 16 * v);
          load32<1>(static_cast<const uint16_t *>(a.up) + at + 16 * v, uq + 8 * v, wide, left - 16 * v);
        }
      }
    }
    uint32_t r[32];
    tmem_load32_wait(tb + c, r);
    if (!valid) continue;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint32_t pd[8], pu[8], ph[8];
      if (f8)
        dh_of<true>(gq + 4 * v, uq + 4 * v, gsc, usc, r + 16 * v, a.act, pd, pu, ph);
      else
        dh_of<false>(gq + 8 * v, uq + 8 * v, 1.0f, 1.0f, r + 16 * v, a.act, pd, pu, ph);
      store32<1>(static_cast<__nv_bfloat16 *>(a.out0) + at + 16 * v, pd, wide, left - 16 * v);
      store32<1>(static_cast<__nv_bfloat16 *>(a.out1) + at + 16 * v, pu, wide, left - 16 * v);
      store32<1>(static_cast<__nv_bfloat16 *>(a.out2) + at + 16 * v, ph, wide, left - 16 * v);
    }
  }
}

__device__ __forceinline__ void epilogue_plain(const FfnArgs &a, const Job &t, uint32_t tb, int m, int half) {
  const bool valid = m < t.rows;
  __nv_bfloat16 *dst =
      static_cast<__nv_bfloat16 *>(a.out0) + static_cast<int64_t>(t.row0 + (valid ? m : 0)) * a.n_total + t.n0;
  const int end = min(t.ncols, 128 * half + 128);
  for (int c = 128 * half; c < end; c += 64) {
    uint32_t r[64];
    tmem_load32x2_wait(tb + c, tb + c + 32, r);
    if (valid) {
      store_plain(dst + c, r, a.wide != 0, a.n_total - t.n0 - c);
      store_plain(dst + c + 32, r + 32, a.wide != 0, a.n_total - t.n0 - c - 32);
    }
  }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// A weight's gradient leaves through shared memory and TMA: with few K blocks to a tile its stores bound the kernel,
// and as stores of each thread's own row (32 lines to an instruction) they also held up the clearing of tails, whose
// shared-memory stores queue behind them (24576 rows of 64 experts, 383 each: 1168 us so, 828 without stores).
__device__ __forceinline__ void epilogue_dw(const FfnArgs &a, const FfnMaps &maps, const Job &t, uint32_t tb, int q,
                                            int half, int lane, uint8_t *piece, uint64_t *released) {
  const int width = t.which == 2 ? a.I : a.H, height = t.which == 2 ? a.H : a.I;
  const int y = t.m0 + q * 32;
  const int end = min(t.ncols, 128 * half + 128);
  for (int c = 128 * half; c < 128 * half + 128; c += 64) {
    uint32_t r[64];
    const bool some = c < end && y < height;
    if (some && t.kblocks != 0) {
      tmem_load32x2_wait(tb + c, tb + c + 32, r);
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) r[i] = 0;  // an expert without rows: its gradient is 0
    }
    if (c == 128 * half + 64) {  // the accumulator has been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(released));
    }
    if (!some) continue;
    // the piece's last store has read it
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
    uint4 *line = reinterpret_cast<uint4 *>(piece + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      line[j ^ (lane & 7)] = make_uint4(pack2(__uint_as_float(r[8 * j]), __uint_as_float(r[8 * j + 1])),
                                        pack2(__uint_as_float(r[8 * j + 2]), __uint_as_float(r[8 * j + 3])),
                                        pack2(__uint_as_float(r[8 * j + 4]), __uint_as_float(r[8 * j + 5])),
                                        pack2(__uint_as_float(r[8 * j + 6]), __uint_as_float(r[8 * j + 7])));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && t.n0 + c < width) {
      tma_store_3d(&maps.d[t.which], smem_addr(piece), t.n0 + c, y, t.e);
      bulk_commit();
    }
  }
}

// The loads of K block kb of a tile: A and B.
template <int FORM>
__device__ __forceinline__ void load_a(const FfnMaps &maps, const Job &t, int kb, uint32_t sa, uint32_t bar) {
  if constexpr (FORM == kDw) {  // maps: dg, du, dy (A), x, h (B)
    for (int c = 0; c < kBM; c += 64)
      tma_load_2d(sa + c / 64 * kHalfBox, &maps.m[t.which], t.m0 + c, t.row0 + kb * kBK, bar);
  } else if constexpr (FORM == kDx) {  // dg, du (A), w_gate, w_up (B)
    const int second = kb >= t.kblocks / 2 ? 1 : 0;
    tma_load_2d(sa, &maps.m[second], (kb - second * (t.kblocks / 2)) * kBK, t.row0, bar);
  } else {
    tma_load_2d(sa, &maps.m[0], kb * kBK, t.row0, bar);
  }
}

template <int FORM>
__device__ __forceinline__ void load_b(const FfnMaps &maps, const Job &t, int kb, uint32_t sb, uint32_t bar) {
  if constexpr (FORM == kUp) {
    tma_load_3d(sb, &maps.m[1], kb * kBK, t.n0, t.e, bar);
    tma_load_3d(sb + kFullBox, &maps.m[2], kb * kBK, t.n0, t.e, bar);
  } else if constexpr (FORM == kDown) {
    tma_load_3d(sb, &maps.m[1], kb * kBK, t.n0, t.e, bar);
    if (t.ncols > 128) tma_load_3d(sb + kFullBox, &maps.m[1], kb * kBK, t.n0 + 128, t.e, bar);
  } else if constexpr (FORM == kDh) {
    for (int c = 0; c < t.ncols; c += 64)
      tma_load_3d(sb + c / 64 * kHalfBox, &maps.m[1], t.n0 + c, kb * kBK, t.e, bar);
  } else if constexpr (FORM == kDx) {
    const int second = kb >= t.kblocks / 2 ? 1 : 0;
    const int k = (kb - second * (t.kblocks / 2)) * kBK;
    for (int c = 0; c < t.ncols; c += 64)
      tma_load_3d(sb + c / 64 * kHalfBox, &maps.m[2 + second], t.n0 + c, k, t.e, bar);
  } else {
    for (int c = 0; c < t.ncols; c += 64)
      tma_load_2d(sb + c / 64 * kHalfBox, &maps.m[t.which == 2 ? 4 : 3], t.n0 + c, t.row0 + kb * kBK, bar);
  }
}

// The MMAs of one K block; of an expert's last one (kDw) only the steps of 16 rows that hold one of its rows.
template <int FORM>
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t sa, uint32_t sb, uint32_t idesc, bool first,
                                          int steps = kBK / kUK) {
#pragma unroll
  for (int kk = 0; kk < kBK / kUK; ++kk)
    if (FORM != kDw || kk < steps)
      mma_bf16(d, a_is_mn(FORM) ? sw128_desc_mn(sa + kk * kUK * 128) : sw128_desc(sa + kk * kUK * 2),
               b_is_mn(FORM) ? sw128_desc_mn(sb + kk * kUK * 128) : sw128_desc(sb + kk * kUK * 2), idesc,
               !first || kk != 0);
}

template <int FORM>
__device__ __forceinline__ uint32_t idesc_of(const Job &t) {
  return idesc_bf16(kBM, t.ncols) | (a_is_mn(FORM) ? 1u << 15 : 0u) | (b_is_mn(FORM) ? 1u << 16 : 0u);
}

template <int FORM>
__global__ void __launch_bounds__(FORM == kDw ? kThreadsDw : kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const FfnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  // kDw: a piece of the result for each epilogue warp, behind the stages
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStage + (FORM == kDw ? kEpilogueWarps * kPiece : 0));
  uint64_t *empty = full + kStages;
  uint64_t *landed = empty + kStages;  // kDw: an expert's last K block, before its tail has been cleared
  uint64_t *tfull = landed + kStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int32_t *offs = reinterpret_cast<int32_t *>(tmem_slot + 2);
  int32_t *pref = offs + (a.E + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
      mbar_init(landed + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, kEpilogueWarps);
    }
    mbar_init(done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (tid == 32)
    for (int i = 0; i < 5; ++i) prefetch_tensormap(&maps.m[i]);
  // The first kernel of a call reads nothing before its wait; the offsets are final once it has passed its own. The
  // next one may begin early, on SMs that have run out of tiles.
  constexpr bool kFirst = FORM == kUp || FORM == kDh;
  if constexpr (kFirst) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if constexpr (FORM != kDw)
    for (int e = tid; e <= a.E; e += kThreads) offs[e] = row_offset(a, e);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if constexpr (FORM != kDw) {
    if (warp == 0) tile_prefix<kBM>(offs, pref, a, lane);
    __syncthreads();
  }
  if constexpr (!kFirst) {
    grid_dependency_wait();
    if (FORM == kDx) grid_dependents_launch();
  }
  const int total = FORM == kDw ? a.dw_total : tile_total(pref, a);

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer ----
      uint32_t it = 0, tails = 0;  // tails: bit s: the last load into stage s went to `landed`
      uint32_t landings = 0;       // bit s: parity of the next phase of landed[s]
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Job t = job_of<FORM>(w, pref, offs, a);
        const uint32_t bytes = kTileA + t.ncols * kBK * 2;
        for (int kb = 0; kb < t.kblocks; ++kb) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!role_wait(empty + s, ph ^ 1u, abort, a.err)) {
            ok = false;
            break;
          }
          uint64_t *bar = full + s;
          if (FORM == kDw && t.tail != 0 && kb == t.kblocks - 1) {
            bar = landed + s;  // the clearing warp passes it on
            tails |= 1u << s;
            landings ^= 1u << s;
          } else {
            tails &= ~(1u << s);
          }
          const uint32_t sa = smem_addr(smem + s * kStage), sb = sa + kTileA, fb = smem_addr(bar);
          mbar_arrive_expect_tx(bar, bytes);
          load_a<FORM>(maps, t, kb, sa, fb);
          load_b<FORM>(maps, t, kb, sb, fb);
          ++it;
        }
      }
      // the last load issued into each stage lands before the CTA may exit
      for (uint32_t s = 0; s < kStages && s < it; ++s) {
        const uint32_t last = s + ((it - 1 - s) / kStages) * kStages;
        if ((tails >> s) & 1u) mbar_wait_bounded(landed + s, ((landings >> s) & 1u) ^ 1u);
        mbar_wait_bounded(full + s, (last / kStages) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer ----
      uint32_t it = 0;
      int lt = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x, ++lt) {
        const Job t = job_of<FORM>(w, pref, offs, a);
        const uint32_t idesc = idesc_of<FORM>(t);
        const int buf = lt & 1;
        const uint32_t ph = (lt >> 1) & 1;
        if (!role_wait(tempty + buf, ph ^ 1u, abort, a.err)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * kBN;
        for (int kb = 0; kb < t.kblocks; ++kb) {
          const uint32_t s = it % kStages, sph = (it / kStages) & 1u;
          if (!role_wait(full + s, sph, abort, a.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_addr(smem + s * kStage), sb = sa + kTileA;
          mma_block<FORM>(d, sa, sb, idesc, kb == 0,
                          t.tail != 0 && kb == t.kblocks - 1 ? (t.tail + kUK - 1) / kUK : kBK / kUK);
          mma_commit(smem_addr(empty + s));
          ++it;
        }
        if (ok) mma_commit(smem_addr(tfull + buf));
      }
      // every MMA issued completes before the tensor memory is freed
      mma_commit(smem_addr(done));
      mbar_wait_bounded(done, 0);
    }
    __syncwarp();
  } else if (warp < 2 + kEpilogueWarps) {
    // ---- epilogue: warp w reads TMEM lanes 32 * (w % 4) .. + 31, of the first or second half of the columns ----
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int m = q * 32 + lane;
    int lt = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x, ++lt) {
      const int buf = lt & 1;
      const uint32_t ph = (lt >> 1) & 1;
      const Job t = job_of<FORM>(w, pref, offs, a);
      int ok = 0;
      if (lane == 0) ok = role_wait(tfull + buf, ph, abort, a.err, blocks_ns(t.kblocks)) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kBN;
      if constexpr (FORM == kUp)
        epilogue_up(a, t, tb, m, half);
      else if constexpr (FORM == kDh)
        epilogue_dh(a, t, tb, m, half);
      else if constexpr (FORM == kDw)
        epilogue_dw(a, maps, t, tb, q, half, lane, smem + kStages * kStage + (warp - 2) * kPiece, tempty + buf);
      else
        epilogue_plain(a, t, tb, m, half);
      if constexpr (FORM != kDw) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(tempty + buf));
      }
    }
    if (FORM == kDw && lane == 0) bulk_wait_all();
    __syncwarp();
  } else if constexpr (FORM == kDw) {
    // ---- clears the rows of the last K block that are not the expert's (they may hold anything), up to the next
    // multiple of 16, in both operands: lines of 128 bytes, one for each k and 64 columns. By TMA loads from behind the
    // array's last row, which fill them with zeros and complete on the stage's barrier: written by the warp itself
    // they needed a fence between the proxies, which took as long as two blocks (24576 rows of 64 experts, 383 each:
    // 1153 us so) ----
    if (lane == 0) {
      uint32_t it = 0, landings = 0, seen = 0;  // seen: blocks up to the last wait
      for (int w = blockIdx.x; w < total; w += gridDim.x) {
        const Job t = job_of<FORM>(w, pref, offs, a);
        it += t.kblocks;
        if (t.tail == 0) continue;
        // (a barrier of its own for each stage: the stage is not used again before this warp has passed it on, so
        // that no phase is missed, and it is cleared while the MMAs of the blocks before it run)
        const uint32_t s = (it - 1) % kStages;
        if (!role_wait(landed + s, (landings >> s) & 1u, abort, a.err, blocks_ns(it - seen))) break;
        seen = it;
        landings ^= 1u << s;
        const uint32_t box = smem_addr(smem + s * kStage) + t.tail * 128;
        const int boxes = kBM / 64 + t.ncols / 64;  // those of A, and those of B right behind them
        const int lines = -t.tail & (kUK - 1);
        const uint32_t fb = smem_addr(full + s);
        if (lines == 0) {
          mbar_arrive(fb);
          continue;
        }
        mbar_arrive_expect_tx(full + s, boxes * lines * 128);
        for (int b = 0; b < boxes; ++b) {
          uint32_t to = box + b * kHalfBox;
          for (int i = 0; i < 4; ++i)  // 1, 2, 4, 8 lines
            if ((lines >> i) & 1) {
              tma_load_2d(to, &maps.zeros[i], 0, a.rows, fb);
              to += 128u << i;
            }
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Few tiles (short batches): a cluster of S CTAs shares a tile, each with its part of K, so that every SM streams
// weights. The parts are added over the cluster: a tile is 8 slices (of 32 columns, or of 16 of g and the same 16 of
// u), slice j is CTA j % S's, and every CTA puts its sums of a slice into the owner's shared memory, where the
// stages were; the owner adds them in order and does what the form does with its columns.
//   64 rows of one expert, 7168 -> 2048: 28.8 us so, 62 with a CTA per tile (16 and 28 tiles).
// ---------------------------------------------------------------------------
constexpr int kMaxSplit = 8;
constexpr int kSlices = 8;
constexpr int kSliceBytes = kBM * 32 * 4;  // a slice's sums of one CTA: 32 columns of 128 rows
constexpr int kTops = kSlices * 2 * kBM * 8;  // largest magnitudes (of g, u) of a row's 16 parts
constexpr int kSmemSplit = kSmemFixed + kTops;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_index() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Slices that a CTA of a cluster of S owns at most, and whether their parts fit where the stages were.
__host__ __device__ constexpr int slices_of(int S) { return (kSlices + S - 1) / S; }
constexpr bool split_fits(int S) { return slices_of(S) * S * kSliceBytes <= kStages * kStage; }

// 16 columns of a row (kUp: 8 of g, then 8 of u) whose sums are v.
template <int FORM>
__device__ __forceinline__ void finish16(const FfnArgs &a, const Job &t, int64_t p, int col, const uint32_t (&v)[16],
                                         float g_top, float u_top) {
  const bool wide = a.wide != 0;
  const int left = a.n_total - t.n0 - col;
  const int64_t at = p * a.n_total + t.n0 + col;
  if (left <= 0) return;
  if constexpr (FORM == kUp) {
    uint32_t pk[4], pg[4], pu[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g0 = __uint_as_float(v[2 * i]), g1 = __uint_as_float(v[2 * i + 1]);
      const float u0 = __uint_as_float(v[8 + 2 * i]), u1 = __uint_as_float(v[9 + 2 * i]);
      pk[i] = pack2(act_of<false>(g0, a.act, nullptr) * u0, act_of<false>(g1, a.act, nullptr) * u1);
      pg[i] = pack2(g0, g1);
      pu[i] = pack2(u0, u1);
    }
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out0) + at) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (a.save == MOE_SAVE_BF16) {
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.keep_gate) + at) = make_uint4(pg[0], pg[1], pg[2], pg[3]);
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.keep_up) + at) = make_uint4(pu[0], pu[1], pu[2], pu[3]);
    } else if (a.save == MOE_SAVE_FP8) {
      const BlockScale gs = block_scale(g_top), us = block_scale(u_top);
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = static_cast<uint32_t>(e4m3x2_of_quotients(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), gs)) |
               static_cast<uint32_t>(e4m3x2_of_quotients(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]), gs))
                   << 16;
        q[2 + i] =
            static_cast<uint32_t>(e4m3x2_of_quotients(__uint_as_float(v[8 + 4 * i]), __uint_as_float(v[9 + 4 * i]), us)) |
            static_cast<uint32_t>(e4m3x2_of_quotients(__uint_as_float(v[10 + 4 * i]), __uint_as_float(v[11 + 4 * i]), us))
                << 16;
      }
      *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.keep_gate) + at) = make_uint2(q[0], q[1]);
      *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.keep_up) + at) = make_uint2(q[2], q[3]);
      if (col == 0) {
        const int64_t sc = p * (a.I / kScaleBlock) + t.n0 / kScaleBlock;
        a.keep_gate_scales[sc] = gs.s;
        a.keep_up_scales[sc] = us.s;
      }
    }
  } else if constexpr (FORM == kDh) {
    uint32_t gq[8], uq[8], pd[8], pu[8], ph[8];
    if (a.save == MOE_SAVE_FP8) {
      const int64_t sc = p * (a.I / kScaleBlock) + (t.n0 + col) / kScaleBlock;
      const uint4 g = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.gate) + at));
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.up) + at));
      gq[0] = g.x, gq[1] = g.y, gq[2] = g.z, gq[3] = g.w;
      uq[0] = u.x, uq[1] = u.y, uq[2] = u.z, uq[3] = u.w;
      dh_of<true>(gq, uq, __ldg(a.gate_scales + sc), __ldg(a.up_scales + sc), v, a.act, pd, pu, ph);
    } else {
      load32<1>(static_cast<const uint16_t *>(a.gate) + at, gq, wide, left);
      load32<1>(static_cast<const uint16_t *>(a.up) + at, uq, wide, left);
      dh_of<false>(gq, uq, 1.0f, 1.0f, v, a.act, pd, pu, ph);
    }
    store32<1>(static_cast<__nv_bfloat16 *>(a.out0) + at, pd, wide, left);
    store32<1>(static_cast<__nv_bfloat16 *>(a.out1) + at, pu, wide, left);
    store32<1>(static_cast<__nv_bfloat16 *>(a.out2) + at, ph, wide, left);
  } else {
    uint32_t pk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) pk[i] = pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    store32<1>(static_cast<__nv_bfloat16 *>(a.out0) + at, pk, wide, left);
  }
}

template <int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_split_kernel(const __grid_constant__ FfnMaps maps, const FfnArgs a, int S) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  float2 *tops = reinterpret_cast<float2 *>(smem + kStages * kStage);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStage + kTops);
  uint64_t *empty = full + kStages;
  uint64_t *done = empty + kStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int32_t *offs = reinterpret_cast<int32_t *>(tmem_slot + 2);
  int32_t *pref = offs + (a.E + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (tid == 32)
    for (int i = 0; i < 5; ++i) prefetch_tensormap(&maps.m[i]);
  // The first kernel of a call reads nothing before its wait. The second one runs once the first has passed its own:
  // offsets and weights are final then, and the rows alone are waited for.
  if (a.first) grid_dependency_wait();
  grid_dependents_launch();
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kBN);
    tmem_relinquish();
  }
  for (int e = tid; e <= a.E; e += kThreads) offs[e] = row_offset(a, e);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0) tile_prefix<kBM>(offs, pref, a, lane);
  __syncthreads();
  const int w = static_cast<int>(cluster_index());
  const bool some = w < tile_total(pref, a);  // the same in the whole cluster
  Job t{};
  int kb0 = 0, kb1 = 0;
  if (some) {
    t = job_of<FORM>(w, pref, offs, a);
    kb0 = t.kblocks * rank / S;
    kb1 = t.kblocks * (rank + 1) / S;
  }
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bytes = kTileA + t.ncols * kBK * 2;
      int early = kb0;  // K blocks whose weights have been asked for before the wait
      if (!a.first) {
        for (; early < kb1 && early < kb0 + kStages; ++early) {
          const int s = early - kb0;
          mbar_arrive_expect_tx(full + s, bytes);
          load_b<FORM>(maps, t, early, smem_addr(smem + s * kStage) + kTileA, smem_addr(full + s));
        }
        grid_dependency_wait();
      }
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        const uint32_t sa = smem_addr(smem + s * kStage), fb = smem_addr(full + s);
        if (kb >= early) {
          if (!role_wait(empty + s, ph ^ 1u, abort, a.err)) break;
          mbar_arrive_expect_tx(full + s, bytes);
          load_b<FORM>(maps, t, kb, sa + kTileA, fb);
        }
        load_a<FORM>(maps, t, kb, sa, fb);
      }
      for (uint32_t s = 0; s < kStages && s < it; ++s) {
        const uint32_t last = s + ((it - 1 - s) / kStages) * kStages;
        mbar_wait_bounded(full + s, (last / kStages) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0;
      const uint32_t idesc = idesc_of<FORM>(t);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        if (!role_wait(full + s, ph, abort, a.err)) break;
        tc_fence_after();
        const uint32_t sa = smem_addr(smem + s * kStage);
        mma_block<FORM>(tmem, sa, sa + kTileA, idesc, kb == kb0);
        mma_commit(smem_addr(empty + s));
      }
      mma_commit(smem_addr(done));
    }
    __syncwarp();
  }
  // (the results come after it; lane 0 of warp 0 has waited, the others of its warp and of every other have not)
  if (!a.first) grid_dependency_wait();
  if (!mbar_wait_bounded(done, 0, blocks_ns(kb1 - kb0))) latch_error(a.err, MOE_ETIMEOUT);
  tc_fence_after();
  // Every CTA's MMAs have read their stages: they take the sums from here on.
  cluster_sync_all();
  if (warp >= 2 && some) {
    const int q = warp & 3, half = (warp - 2) >> 2, m = q * 32 + lane;
    for (int i = half; i < kSlices / 2; i += 2) {
      uint32_t r[64];
      if (FORM == kUp)
        tmem_load32x2_wait(tmem + (static_cast<uint32_t>(q * 32) << 16) + 32 * i,
                           tmem + (static_cast<uint32_t>(q * 32) << 16) + 128 + 32 * i, r);
      else
        tmem_load32x2_wait(tmem + (static_cast<uint32_t>(q * 32) << 16) + 64 * i,
                           tmem + (static_cast<uint32_t>(q * 32) << 16) + 64 * i + 32, r);
      if (m >= t.rows) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 2 * i + x;
        const uint32_t to = map_rank(smem_addr(smem + ((j / S) * S + rank) * kSliceBytes + m * 16), j % S);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          // kUp: words 0-3: 16 of g, 4-7: the same of u
          const int o = FORM == kUp ? (v < 4 ? 16 * x + 4 * v : 32 + 16 * x + 4 * (v - 4)) : 32 * x + 4 * v;
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + v * (kBM * 16)),
                       "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3])
                       : "memory");
        }
      }
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kBN);
  }
  // items: half a slice of a row, over as many threads as there are
  const bool f8 = FORM == kUp && a.save == MOE_SAVE_FP8;
  const int own = some && !*abort ? (kSlices - rank + S - 1) / S : 0;
  const int items = 2 * own * t.rows;
  for (int pass = f8 ? 0 : 1; pass < 2; ++pass) {
    for (int item = tid; item < items; item += kThreads) {
      const int row = item % t.rows, rest = item / t.rows, part = rest & 1, local = rest >> 1;
      const int j = local * S + rank;
      float f[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = 0.0f;
      for (int src = 0; src < S; ++src) {
        const uint8_t *from = smem + (local * S + src) * kSliceBytes + row * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // kUp: 8 of g (words 2 part, 2 part + 1) and of u (4 + ..); else 16 columns
          const int word = FORM == kUp ? (i < 2 ? 2 * part + i : 4 + 2 * part + i - 2) : 4 * part + i;
          const float4 x = *reinterpret_cast<const float4 *>(from + word * (kBM * 16));
          f[4 * i] += x.x, f[4 * i + 1] += x.y, f[4 * i + 2] += x.z, f[4 * i + 3] += x.w;
        }
      }
      float g = 0.0f, u = 0.0f;
      if (f8 && pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g = fmaxf(g, fabsf(f[i])), u = fmaxf(u, fabsf(f[8 + i]));
        for (int to = 0; to < S; ++to)
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                           map_rank(smem_addr(tops + (2 * j + part) * kBM + row), to)),
                       "f"(g), "f"(u)
                       : "memory");
        continue;
      }
      if (f8) {
#pragma unroll
        for (int i = 0; i < 2 * kSlices; ++i) {
          const float2 x = tops[i * kBM + row];
          g = fmaxf(g, x.x), u = fmaxf(u, x.y);
        }
      }
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(f[i]);
      finish16<FORM>(a, t, t.row0 + row, FORM == kUp ? 16 * j + 8 * part : 32 * j + 16 * part, v, g, u);
    }
    if (pass == 0) cluster_sync_all();
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Map of a row-major bf16 [z][rows][cols] array (2-D when z = 0), boxes of 64 columns x box_rows rows.
bool ffn_map(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t z, int box_rows,
             CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(z)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * rows * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, z > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

moe_status check_ffn(const moe_ffn_desc *d, FfnSizes *s) {
  if (d == nullptr) return MOE_EINVAL;
  if (d->rows < 0 || d->hidden < 8 || d->hidden % 8 != 0 || d->inter < 8 || d->inter % 8 != 0) return MOE_EINVAL;
  if (d->num_experts < 1 || d->num_experts > MOE_FFN_MAX_EXPERTS || d->num_ranks < 1 || d->num_sms < 0)
    return MOE_EINVAL;
  if (static_cast<int64_t>(d->num_experts) * d->num_ranks > INT32_MAX) return MOE_EINVAL;
  if (d->act != MOE_ACT_SILU && d->act != MOE_ACT_GELU_TANH) return MOE_EINVAL;
  if (d->save != MOE_SAVE_NONE && d->save != MOE_SAVE_BF16 && d->save != MOE_SAVE_FP8) return MOE_EINVAL;
  if (d->save == MOE_SAVE_FP8 && d->inter % kScaleBlock != 0) return MOE_EINVAL;
  // rows, columns and tiles are counted in 32 bits, those of a last tile that are not there among them
  constexpr int32_t most = INT32_MAX - kBN + 1;
  if (d->rows > most || d->hidden > most || d->inter > most) return MOE_EINVAL;
  const int64_t wide = (d->hidden > d->inter ? d->hidden : d->inter) / 64 + 1;
  if ((d->rows / kBM + static_cast<int64_t>(d->num_experts)) * wide > INT32_MAX ||
      3 * d->num_experts * (static_cast<int64_t>(d->hidden) / 64 + 1) * (d->inter / 64 + 1) > INT32_MAX)
    return MOE_EINVAL;
  *s = FfnSizes{d->rows, d->hidden, d->inter, d->num_experts, d->num_ranks, d->act, d->save, d->num_sms};
  return MOE_OK;
}

int group_width(int concurrent, int tile_rows, int tile_cols, int ntiles_n) {
  const int64_t g = std::llround(std::sqrt(static_cast<double>(concurrent) * tile_rows / tile_cols));
  return static_cast<int>(g < 1 ? 1 : (g > ntiles_n ? ntiles_n : g));
}

// Tiles of a launch, at most: an expert with rows has one that is not full.
int64_t most_tiles(const FfnArgs &a) {
  const int64_t experts = a.E < a.rows ? a.E : a.rows;
  return ((a.rows - experts) / kBM + experts) * a.ntiles_n;
}

void cluster_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int S, int smem, cudaStream_t stream) {
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = MOE_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Clusters of S CTAs that run at one time (a cluster stays within a GPC, so fewer than the SMs would hold), asked of
// the device once.
template <int FORM>
int clusters_at_once(int S) {
  static std::atomic<int> known[64][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed);
  if (n != 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, S, kSmemMax, nullptr);
  cfg.gridDim = dim3(S, 1, 1);
  if (!raise_smem_limit(ffn_split_kernel<FORM>, kSmemMax) ||
      cudaOccupancyMaxActiveClusters(&n, ffn_split_kernel<FORM>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();  // an answer, not a failed call
    n = -1;
  }
  known[dev][S].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs that share a tile: as many as leave every cluster its place at once (with 16 tiles in clusters of 8 the last
// two ran after the others, and 64 rows of 7168 -> 2048 took 40 us), with at least four K blocks each.
template <int FORM>
int split_of(const FfnArgs &a, int sms) {
  const int64_t tiles = most_tiles(a);
  int S = static_cast<int>(sms / tiles < kMaxSplit ? sms / tiles : kMaxSplit);
  if (S > a.kblocks / 4) S = a.kblocks / 4;
  while (S > 1 && !(split_fits(S) && tiles <= clusters_at_once<FORM>(S))) --S;
  return S;
}

template <int FORM>
moe_status launch_split(const FfnMaps &maps, const FfnArgs &a, int S, cudaStream_t stream) {
  const int smem = kSmemSplit + 12 * (a.E + 1);
  if (!raise_smem_limit(ffn_split_kernel<FORM>, smem)) return MOE_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, S, smem, stream);
  cfg.gridDim = dim3(static_cast<unsigned>(most_tiles(a) * S), 1, 1);
  if (cudaLaunchKernelEx(&cfg, ffn_split_kernel<FORM>, maps, a, S) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

template <int FORM>
moe_status launch_form(const FfnMaps &maps, FfnArgs a, const FfnSizes &s, cudaStream_t stream) {
  const int all = sm_count();
  const int sms = s.num_sms > 0 && s.num_sms < all ? s.num_sms : all;
  const int smem = FORM == kDw ? kSmemDw : kSmemFixed + 12 * (a.E + 1);
  if (smem > kSmemMax) return MOE_EINVAL;
  int64_t tiles;
  if (FORM == kDw) {
    // narrower tiles where wide ones leave SMs without any (14451 rows of 504 -> 392: 196 us with 24 tiles of 256)
    const int64_t mi = (a.I + kBM - 1) / kBM, mh = (a.H + kBM - 1) / kBM;
    int64_t ni, nh;
    a.out_cols = 2 * kBN;
    do {
      a.out_cols /= 2;
      ni = (a.I + a.out_cols - 1) / a.out_cols, nh = (a.H + a.out_cols - 1) / a.out_cols;
      tiles = a.E * (2 * mi * nh + mh * ni);
    } while (a.out_cols > 64 && tiles < sms);
    a.dw_total = static_cast<int>(tiles);
    a.ntiles_n = 1;
    a.group_n = group_width(sms, kBM, a.out_cols, static_cast<int>(nh > ni ? nh : ni));
  } else {
    a.ntiles_n = (a.n_total + a.out_cols - 1) / a.out_cols;
    a.group_n = group_width(sms, kBM, kBN, a.ntiles_n);
    tiles = most_tiles(a);
  }
  if constexpr (FORM != kDw) {
    const int S = split_of<FORM>(a, sms);
    if (S > 1 && kSmemSplit + 12 * (a.E + 1) <= kSmemMax) return launch_split<FORM>(maps, a, S, stream);
  }
  if (!raise_smem_limit(ffn_gemm_kernel<FORM>, smem)) return MOE_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < sms ? tiles : sms), 1, 1);
  cfg.blockDim = dim3(FORM == kDw ? kThreadsDw : kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<FORM>, maps, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

FfnArgs base_args(const FfnSizes &s, const int32_t *offsets, int32_t *err) {
  FfnArgs a{};
  a.offsets = offsets;
  a.err = err;
  a.rows = s.rows;
  a.E = s.E;
  a.R = s.R;
  a.H = s.H;
  a.I = s.I;
  a.act = s.act;
  a.save = s.save;
  return a;
}

int blocks_of(int k) { return (k + kBK - 1) / kBK; }

// Whether rows of `width` elements of these arrays all begin on 32-byte boundaries (null: not used).
bool wide_rows(int64_t row_bytes, std::initializer_list<const void *> arrays) {
  bool good = row_bytes % 32 == 0;
  for (const void *p : arrays) good = good && aligned32(p);
  return good;
}

bool good16(const void *p) { return p != nullptr && aligned16(p); }
bool good4(const void *p) { return p != nullptr && aligned4(p); }

bool offsets_ok(const FfnSizes &s, const int32_t *offsets) {
  return offsets == nullptr ? s.E == 1 : aligned4(offsets);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_ffn(const moe_ffn_desc *desc, const int32_t *region_offsets, const void *x,
                              const void *w_gate, const void *w_up, const void *w_down, void *h, void *y, void *gate,
                              float *gate_scales, void *up, float *up_scales, int32_t *err, void *stream) {
  FfnSizes s;
  moe_status st = check_ffn(desc, &s);
  if (st != MOE_OK) return st;
  if (!offsets_ok(s, region_offsets) || !good4(err)) return MOE_EINVAL;
  if (s.rows == 0) return MOE_OK;
  if (!good16(x) || !good16(w_gate) || !good16(w_up) || !good16(w_down) || !good16(h) || !good16(y))
    return MOE_EINVAL;
  if (s.save != MOE_SAVE_NONE && (!good16(gate) || !good16(up))) return MOE_EINVAL;
  if (s.save == MOE_SAVE_FP8 && (!good4(gate_scales) || !good4(up_scales))) return MOE_EINVAL;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.rows <= kFewRows && s.save != MOE_SAVE_FP8 && s.num_sms == 0)
    return launch_ffn_few(s, region_offsets, x, w_gate, w_up, w_down, h, y, gate, up, err, cs);
  FfnMaps m{};
  if (!ffn_map(&m.m[0], x, s.H, s.rows, 0, 128) || !ffn_map(&m.m[1], w_gate, s.H, s.I, s.E, 128) ||
      !ffn_map(&m.m[2], w_up, s.H, s.I, s.E, 128))
    return MOE_ECUDA;
  m.m[3] = m.m[4] = m.m[2];
  FfnArgs a = base_args(s, region_offsets, err);
  a.out0 = h;
  a.keep_gate = gate;
  a.keep_up = up;
  a.keep_gate_scales = gate_scales;
  a.keep_up_scales = up_scales;
  a.kblocks = blocks_of(s.H);
  a.n_total = s.I;
  a.out_cols = 128;
  a.wide = wide_rows(INT64_C(2) * s.I, {h, gate, up});
  a.first = 1;
  st = launch_form<kUp>(m, a, s, cs);
  if (st != MOE_OK) return st;
  if (!ffn_map(&m.m[0], h, s.I, s.rows, 0, 128) || !ffn_map(&m.m[1], w_down, s.I, s.H, s.E, 128)) return MOE_ECUDA;
  a = base_args(s, region_offsets, err);
  a.out0 = y;
  a.kblocks = blocks_of(s.I);
  a.n_total = s.H;
  a.out_cols = kBN;
  a.wide = wide_rows(INT64_C(2) * s.H, {y});
  return launch_form<kDown>(m, a, s, cs);
}

extern "C" moe_status moe_ffn_grad(const moe_ffn_desc *desc, const int32_t *region_offsets, const void *x,
                                   const void *gate, const float *gate_scales, const void *up, const float *up_scales,
                                   const void *w_gate, const void *w_up, const void *w_down, const void *grad_y,
                                   void *h, void *grad_gate, void *grad_up, void *grad_x, void *grad_w_gate,
                                   void *grad_w_up, void *grad_w_down, int32_t *err, void *stream) {
  FfnSizes s;
  moe_status st = check_ffn(desc, &s);
  if (st != MOE_OK) return st;
  if (s.save == MOE_SAVE_NONE) return MOE_EINVAL;
  if (!offsets_ok(s, region_offsets) || !good4(err)) return MOE_EINVAL;
  const bool weights = grad_w_gate != nullptr;
  if ((grad_w_up != nullptr) != weights || (grad_w_down != nullptr) != weights) return MOE_EINVAL;
  if (weights && (!aligned16(grad_w_gate) || !aligned16(grad_w_up) || !aligned16(grad_w_down))) return MOE_EINVAL;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.rows == 0) {
    if (!weights) return MOE_OK;
    const size_t n = static_cast<size_t>(s.E) * s.H * s.I * 2;
    if (cudaMemsetAsync(grad_w_gate, 0, n, cs) != cudaSuccess || cudaMemsetAsync(grad_w_up, 0, n, cs) != cudaSuccess ||
        cudaMemsetAsync(grad_w_down, 0, n, cs) != cudaSuccess)
      return MOE_ECUDA;
    return MOE_OK;
  }
  if (!good16(x) || !good16(gate) || !good16(up) || !good16(w_gate) || !good16(w_up) || !good16(w_down) ||
      !good16(grad_y) || !good16(h) || !good16(grad_gate) || !good16(grad_up) || !good16(grad_x))
    return MOE_EINVAL;
  if (s.save == MOE_SAVE_FP8 && (!good4(gate_scales) || !good4(up_scales))) return MOE_EINVAL;

  FfnMaps m{};
  if (!ffn_map(&m.m[0], grad_y, s.H, s.rows, 0, 128) || !ffn_map(&m.m[1], w_down, s.I, s.H, s.E, 64))
    return MOE_ECUDA;
  m.m[2] = m.m[3] = m.m[4] = m.m[1];
  FfnArgs a = base_args(s, region_offsets, err);
  a.out0 = grad_gate;
  a.out1 = grad_up;
  a.out2 = h;
  a.gate = gate;
  a.up = up;
  a.gate_scales = gate_scales;
  a.up_scales = up_scales;
  a.kblocks = blocks_of(s.H);
  a.n_total = s.I;
  a.out_cols = kBN;
  a.wide = wide_rows(INT64_C(2) * s.I, {gate, up, grad_gate, grad_up, h});
  a.first = 1;
  st = launch_form<kDh>(m, a, s, cs);
  if (st != MOE_OK) return st;

  if (!ffn_map(&m.m[0], grad_gate, s.I, s.rows, 0, 128) || !ffn_map(&m.m[1], grad_up, s.I, s.rows, 0, 128) ||
      !ffn_map(&m.m[2], w_gate, s.H, s.I, s.E, 64) || !ffn_map(&m.m[3], w_up, s.H, s.I, s.E, 64))
    return MOE_ECUDA;
  a = base_args(s, region_offsets, err);
  a.out0 = grad_x;
  a.kblocks = 2 * blocks_of(s.I);
  a.n_total = s.H;
  a.out_cols = kBN;
  a.wide = wide_rows(INT64_C(2) * s.H, {grad_x});
  st = launch_form<kDx>(m, a, s, cs);
  if (st != MOE_OK || !weights) return st;

  if (!ffn_map(&m.m[0], grad_gate, s.I, s.rows, 0, 64) || !ffn_map(&m.m[1], grad_up, s.I, s.rows, 0, 64) ||
      !ffn_map(&m.m[2], grad_y, s.H, s.rows, 0, 64) || !ffn_map(&m.m[3], x, s.H, s.rows, 0, 64) ||
      !ffn_map(&m.m[4], h, s.I, s.rows, 0, 64) || !ffn_map(&m.d[0], grad_w_gate, s.H, s.I, s.E, 32) ||
      !ffn_map(&m.d[1], grad_w_up, s.H, s.I, s.E, 32) || !ffn_map(&m.d[2], grad_w_down, s.I, s.H, s.E, 32))
    return MOE_ECUDA;
  for (int i = 0; i < 4; ++i)
    if (!ffn_map(&m.zeros[i], x, s.H, s.rows, 0, 1 << i, CU_TENSOR_MAP_SWIZZLE_NONE)) return MOE_ECUDA;
  a = base_args(s, region_offsets, err);
  return launch_form<kDw>(m, a, s, cs);
}
