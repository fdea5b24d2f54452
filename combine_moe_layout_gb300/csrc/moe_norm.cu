// The norms around a block: what the block put out is normalised (or not), gated
// and scaled, added to the residual stream, and the stream is normalised for the
// next block; with its gradients.
//
//   b = o / rms(o) * w_post  (or o);   r = x + alpha * gate * b;   n = r / rms(r) * w_pre
//   rms(v) = sqrt(mean(v^2) + eps)
//
// Gradients, with q = 1 / rms(r), p = 1 / rms(o) and r as it was kept:
//   dr = grad_r + q (dn w_pre - r q^2 mean(dn w_pre r))          (= grad_x)
//   grad_o = p (t - o p^2 mean(t o)),  t = alpha gate dr w_post   (or alpha gate dr)
//   grad_w_pre = sum_rows dn r q,  s = sum_rows alpha dr o p (row gates inside the sum),
//   grad_w_post = gate s,  grad_gate = w_post s (channels) or alpha sum_k dr b (rows)
// mean(t o) is linear in dr, so that it follows from sums over grad_r, dn w_pre and r
// alone: a row's six sums are taken together and cost one barrier.
//
// Every row is read and written once. 8192 rows of 7168: forward 118 us (fp32
// stream, 88 % of the copy rate), gradients 138 us (bf16, 76 %: a row's chain and
// its instructions). Rows above 8192 columns have four vectors to a thread, and the
// gradient's column sums no longer fit its registers: 2048 rows of 16384 in bf16 take
// 77 us (3.5 TB/s) and 174 us (2.3 TB/s), of 32768 (1024 threads, straight from
// memory) 184 us and 622 us (1.3 TB/s). All arithmetic and sums are in fp32; a
// column's sum over rows is taken by each CTA for its own rows in order, and the CTAs'
// parts are then added in order, so that results do not depend on timing.
#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kNormMaxDim = 32768;
constexpr int kNormThreads = 512;  // threads of a row's CTA, up to four vectors of 8 each; twice that beyond

struct NormArgs {
  const void *x, *o;      // x: of the gradient, the stream r that was kept
  const float *w_post, *gate, *w_pre;
  void *r, *n;
  const void *grad_r, *grad_n;
  void *grad_x, *grad_o;
  float *grad_gate;
  float *parts;           // [2][parts][H]: sums of dn r q and of alpha dr o p
  int32_t *err;
  int rows, H, row_gate, channel_gate, stages;
  float eps, alpha;
};

template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&v)[8]) {
  if constexpr (F32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void vector8(const float *w, int64_t at, float (&v)[8]) { load8<true>(w, at, v); }

// A sum over the block, every thread gets it; `part` is [2][32], its halves taken in turn so that one barrier does.
__device__ __forceinline__ float block_sum(float v, float *part, int &turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  float *mine = part + turn * 32;
  turn ^= 1;
  if (lane == 0) mine[warp] = v;
  __syncthreads();
  v = lane < warps ? mine[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The same for six sums of a row: each step of the butterfly sends half of the values that are left, so that nine
// shuffles do (30 one by one), and eight more behind the barrier. `part` is [2][8][32].
__device__ __forceinline__ void block_sums6(float (&v)[6], float *part, int &turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool b4 = (lane & 16) != 0, b3 = (lane & 8) != 0, b2 = (lane & 4) != 0;
  // values 0-3 stay in the lower lanes, 4-7 (6 and 7: nothing) in the upper ones
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float hi = i < 2 ? v[i + 4] : 0.0f;
    x[i] = (b4 ? hi : v[i]) + __shfl_xor_sync(0xffffffffu, b4 ? v[i] : hi, 16);
  }
  float y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) y[i] = (b3 ? x[i + 2] : x[i]) + __shfl_xor_sync(0xffffffffu, b3 ? x[i] : x[i + 2], 8);
  float z = (b2 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, b2 ? y[0] : y[1], 4);
  z += __shfl_xor_sync(0xffffffffu, z, 2);
  z += __shfl_xor_sync(0xffffffffu, z, 1);
  // lanes 4 i .. 4 i + 3 have value i
  if (warps > 1) {
    float *mine = part + turn * 8 * 32;
    turn ^= 1;
    if ((lane & 3) == 0) mine[(lane >> 2) * 32 + warp] = z;
    __syncthreads();
    z = 0.0f;
    for (int w = lane & 3; w < warps; w += 4) z += mine[(lane >> 2) * 32 + w];
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    z += __shfl_xor_sync(0xffffffffu, z, 1);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, z, 4 * i);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
        "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t at, float2 (&v)[4]) {
  float f[8];
  load8<F32>(base, at, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, const float2 (&v)[4]) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  store8<F32>(base, at, f);
}

// The rows that a CTA takes, t = blockIdx.x, + gridDim.x, ...: up to four row-long arrays each, brought to shared
// memory a few rows ahead by bulk copies of thread 0.
struct RowRing {
  uint64_t *full;       // one barrier for each stage
  uint8_t *data;
  const void *from[4];  // null: not there
  uint32_t bytes[4];    // of a row; 0 where not there
  uint32_t stage_bytes;
  int stages;

  __device__ __forceinline__ void issue(int s, int64_t t) const {
    mbar_arrive_expect_tx(full + s, stage_bytes);
    uint32_t at = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (bytes[i] != 0) {
        bulk_load(data + static_cast<size_t>(s) * stage_bytes + at, static_cast<const uint8_t *>(from[i]) + t * bytes[i],
                  bytes[i], full + s);
        at += bytes[i];
      }
  }
};

// After a copy that did not arrive: the error, and a wait (bounded too) for the copies of the other stages, so that
// none lands in shared memory that is no longer this CTA's.
__device__ __forceinline__ void give_up(const RowRing &r, int stage, uint32_t phase, int32_t *err) {
  latch_error(err, MOE_ETIMEOUT);
  for (int s = 0; s < r.stages; ++s) mbar_wait_bounded(r.full + s, s >= stage ? phase : phase ^ 1u);
}

__device__ __forceinline__ RowRing make_ring(const NormArgs &a, uint8_t *smem, int stages, const void *p0, bool f0,
                                             const void *p1, bool f1, const void *p2, bool f2, const void *p3,
                                             bool f3) {
  RowRing r;
  r.full = reinterpret_cast<uint64_t *>(smem);
  r.data = smem + 64;
  const void *p[4] = {p0, p1, p2, p3};
  const bool f[4] = {f0, f1, f2, f3};
  r.stage_bytes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.from[i] = p[i];
    r.bytes[i] = p[i] == nullptr ? 0u : static_cast<uint32_t>(a.H) * (f[i] ? 4u : 2u);
    r.stage_bytes += r.bytes[i];
  }
  r.stages = stages;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(r.full + s, 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) {
      const int64_t t = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (t < a.rows) r.issue(s, t);
    }
  return r;
}

// RING: the rows come through shared memory; else (rows too long for it) straight from memory.
template <int NV, bool F32, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  extern __shared__ __align__(128) uint8_t smem[];
  RowRing ring;
  if constexpr (RING)
    ring = make_ring(a, smem, a.stages, a.x, F32, a.o, false, nullptr, false, nullptr, false);
  else
    grid_dependency_wait();
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  const int vecs = a.H / 8;
  const float inv = 1.0f / static_cast<float>(a.H);
  // the thread's columns: w_pre and c = w_post gate (of channels), kept where registers allow
  constexpr bool kKeep = NV <= 2;
  float w_kept[kKeep ? NV : 1][8], c_kept[kKeep ? NV : 1][8];
  const bool scaled = a.w_post != nullptr || a.channel_gate;
  auto columns = [&](int v, float (&c)[8]) {
    if (a.w_post != nullptr) {
      vector8(a.w_post, v * 8, c);
      if (a.channel_gate) {
        float g[8];
        vector8(a.gate, v * 8, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] *= g[k];
      }
    } else {
      vector8(a.gate, v * 8, c);
    }
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        vector8(a.w_pre, v * 8, w_kept[i]);
        if (scaled) columns(v, c_kept[i]);
      }
    }
  }
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const void *px, *po;
    if constexpr (RING) {
      if (!mbar_wait_bounded(ring.full + stage, phase)) {
        give_up(ring, stage, phase, a.err);
        return;
      }
      const uint8_t *d = ring.data + static_cast<size_t>(stage) * ring.stage_bytes;
      px = d;
      po = d + ring.bytes[0];
    } else {
      px = static_cast<const uint8_t *>(a.x) + t * a.H * (F32 ? 4 : 2);
      po = static_cast<const uint8_t *>(a.o) + t * a.H * 2;
    }
    float x[NV][8], b[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        load8<F32>(px, v * 8, x[i]);
        if (a.o != nullptr) load8<false>(po, v * 8, b[i]);
      }
    }
    if (a.o != nullptr) {
      float scale = a.alpha;
      if (a.row_gate) scale *= a.gate[t];
      if (a.w_post != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (threadIdx.x + i * blockDim.x < vecs)
#pragma unroll
            for (int k = 0; k < 8; ++k) ss += b[i][k] * b[i][k];
        scale *= 1.0f / sqrtf(block_sum(ss, &part[0][0], turn) * inv + a.eps);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vecs) {
          if (scaled) {
            float c[8];
            if constexpr (!kKeep) columns(v, c);
#pragma unroll
            for (int k = 0; k < 8; ++k) b[i][k] *= kKeep ? c_kept[kKeep ? i : 0][k] : c[k];
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] += scale * b[i][k];
        }
      }
    }
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        if (a.r != nullptr) store8<F32>(a.r, t * a.H + v * 8, x[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += x[i][k] * x[i][k];
      }
    }
    const float total = block_sum(ss, &part[0][0], turn);
    if constexpr (RING) {
      // every thread has read its part of the stage
      const int64_t next = t + static_cast<int64_t>(ring.stages) * gridDim.x;
      if (threadIdx.x == 0 && next < a.rows) ring.issue(stage, next);
      if (++stage == ring.stages) stage = 0, phase ^= 1u;
    }
    const float q = 1.0f / sqrtf(total * inv + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        float w[8];
        if constexpr (!kKeep) vector8(a.w_pre, v * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] *= q * (kKeep ? w_kept[kKeep ? i : 0][k] : w[k]);
        store8<false>(a.n, t * a.H + v * 8, x[i]);
      }
    }
  }
}

template <int NV, bool F32, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormArgs a) {
  __shared__ float part[2][8][32];
  extern __shared__ __align__(128) uint8_t smem[];
  RowRing ring;
  if constexpr (RING)
    ring = make_ring(a, smem, a.stages, a.x, F32, a.grad_n, false, a.grad_r, F32, a.o, false);
  else
    grid_dependency_wait();
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  const int vecs = a.H / 8;
  const float inv = 1.0f / static_cast<float>(a.H);
  // the thread's columns: w_pre, c = w_post gate (of channels), and the sums over rows
  float2 w[NV][4], c[NV][4], acc_n[NV][4], acc_o[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc_n[i][k] = acc_o[i][k] = w[i][k] = both(0.0f);
      c[i][k] = both(1.0f);
    }
    if (v < vecs) {
      load8<true>(a.w_pre, v * 8, w[i]);
      if (a.w_post != nullptr) load8<true>(a.w_post, v * 8, c[i]);
      if (a.channel_gate) {
        float2 g[4];
        load8<true>(a.gate, v * 8, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[i][k] = mul2(c[i][k], g[k]);
      }
    }
  }
  int64_t waiting = -1;  // the row to be asked for into the stage that the last row has left
  int left = 0;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const void *pr, *pn, *pd, *po;
    if constexpr (RING) {
      if (!mbar_wait_bounded(ring.full + stage, phase)) {
        give_up(ring, stage, phase, a.err);
        return;
      }
      const uint8_t *d = ring.data + static_cast<size_t>(stage) * ring.stage_bytes;
      pr = d;
      pn = d + ring.bytes[0];
      pd = d + ring.bytes[0] + ring.bytes[1];
      po = d + ring.bytes[0] + ring.bytes[1] + ring.bytes[2];
    } else {
      pr = static_cast<const uint8_t *>(a.x) + t * a.H * (F32 ? 4 : 2);
      pn = static_cast<const uint8_t *>(a.grad_n) + t * a.H * 2;
      pd = static_cast<const uint8_t *>(a.grad_r) + t * a.H * (F32 ? 4 : 2);
      po = static_cast<const uint8_t *>(a.o) + t * a.H * 2;
    }
    float2 s2[6];  // r^2, dn w r, o^2, and c o with grad_r, dn w, r
#pragma unroll
    for (int i = 0; i < 6; ++i) s2[i] = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        float2 r[4], dn[4];
        load8<F32>(pr, v * 8, r);
        load8<false>(pn, v * 8, dn);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dn[k] = mul2(dn[k], w[i][k]);
          s2[0] = fma2(r[k], r[k], s2[0]);
          s2[1] = fma2(dn[k], r[k], s2[1]);
        }
        if (a.o != nullptr) {
          float2 o[4], dr[4];
          load8<false>(po, v * 8, o);
          if (a.grad_r != nullptr) load8<F32>(pd, v * 8, dr);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 co = mul2(c[i][k], o[k]);
            s2[2] = fma2(o[k], o[k], s2[2]);
            if (a.grad_r != nullptr) s2[3] = fma2(co, dr[k], s2[3]);
            s2[4] = fma2(co, dn[k], s2[4]);
            s2[5] = fma2(co, r[k], s2[5]);
          }
        }
      }
    }
    float s[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = s2[i].x + s2[i].y;
    block_sums6(s, &part[0][0][0], turn);
    if constexpr (RING) {
      // every thread has left the last row's stage
      if (threadIdx.x == 0 && waiting >= 0) ring.issue(left, waiting);
      const int64_t next = t + static_cast<int64_t>(ring.stages) * gridDim.x;
      waiting = next < a.rows ? next : -1;
      left = stage;
      if (++stage == ring.stages) stage = 0, phase ^= 1u;
    }
    const float q = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float m = q * q * s[1] * inv;  // dr = grad_r + q (dn w - m r)
    const float p = a.w_post != nullptr ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    const float dro = s[3] + q * (s[4] - m * s[5]);  // sum dr c o
    float scale = a.alpha * p;
    if (a.row_gate) {
      if (threadIdx.x == 0) a.grad_gate[t] = scale * dro;
      scale *= a.gate[t];
    }
    // grad_o = scale (c dr - f o), f = p^2 mean(dr c o)
    const float f = a.w_post != nullptr ? p * p * dro * inv : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        const int64_t at = t * a.H + v * 8;
        float2 r[4], dn[4], dr[4];
        load8<F32>(pr, v * 8, r);
        load8<false>(pn, v * 8, dn);
        if (a.grad_r != nullptr)
          load8<F32>(pd, v * 8, dr);
        else
#pragma unroll
          for (int k = 0; k < 4; ++k) dr[k] = both(0.0f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc_n[i][k] = fma2(dn[k], mul2(r[k], both(q)), acc_n[i][k]);
          const float2 d = mul2(dn[k], w[i][k]);
          dr[k] = fma2(both(q), fma2(both(-m), r[k], d), dr[k]);
        }
        if (a.o != nullptr) {
          float2 o[4];
          load8<false>(po, v * 8, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 sd = mul2(both(scale), dr[k]);
            acc_o[i][k] = fma2(sd, o[k], acc_o[i][k]);
            o[k] = fma2(c[i][k], sd, mul2(both(-scale * f), o[k]));
          }
          store8<false>(a.grad_o, at, o);
        }
        store8<F32>(a.grad_x, at, dr);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < vecs) {
      store8<true>(a.parts, static_cast<int64_t>(blockIdx.x) * a.H + v * 8, acc_n[i]);
      store8<true>(a.parts, (static_cast<int64_t>(gridDim.x) + blockIdx.x) * a.H + v * 8, acc_o[i]);
    }
  }
}

struct NormSumArgs {
  const float *parts, *w_post, *gate;
  float *grad_w_pre, *grad_w_post, *grad_gate;  // of channels
  int count, H;
};

// Adds the CTAs' parts: blocks of 32 columns, 8 warps that take every eighth part each, added in order.
__global__ void __launch_bounds__(256) norm_sum_kernel(NormSumArgs a) {
  __shared__ float part[8][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int which = blockIdx.y;
  float s = 0.0f;
  if (col < a.H)
    for (int i = warp; i < a.count; i += 8) s += a.parts[(static_cast<int64_t>(which) * a.count + i) * a.H + col];
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= a.H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += part[i][lane];
  if (which == 0) {
    a.grad_w_pre[col] = s;
  } else {
    if (a.grad_w_post != nullptr) a.grad_w_post[col] = s * (a.grad_gate != nullptr ? a.gate[col] : 1.0f);
    if (a.grad_gate != nullptr) a.grad_gate[col] = s * (a.w_post != nullptr ? a.w_post[col] : 1.0f);
  }
}

moe_status check_norm(const moe_norm_desc *d) {
  if (d == nullptr || d->rows < 0 || d->dim < 8 || d->dim % 8 != 0 || d->dim > kNormMaxDim) return MOE_EINVAL;
  if (d->stream_fp32 != 0 && d->stream_fp32 != 1) return MOE_EINVAL;
  if (d->gate != MOE_GATE_NONE && d->gate != MOE_GATE_ROW && d->gate != MOE_GATE_CHANNEL) return MOE_EINVAL;
  if (!(d->eps >= 0.0f) || d->eps > 3.0e38f || !(d->alpha >= -3.0e38f && d->alpha <= 3.0e38f)) return MOE_EINVAL;
  return MOE_OK;
}

bool good16(const void *p) { return p != nullptr && aligned16(p); }

// CTAs on an SM: short rows leave a CTA few warps (4063 rows of 200: forward 5.8 us, 16.5 with two; gradients 15.0 and
// 19.5).
int norm_ctas(int dim) { return dim > 4096 ? 1 : (dim > 1024 ? 2 : (dim > 256 ? 4 : 8)); }

// CTAs of a gradient, each with its part of the sums over rows: by the sizes alone (152 SMs), so that the sums are the
// same on every device.
int norm_parts(const moe_norm_desc *d) {
  const int most = 152 * norm_ctas(d->dim);
  return d->rows < most ? d->rows : most;
}

constexpr int kRingBytes = 200 * 1024;  // for the rows of all CTAs on an SM
constexpr int kRingStages = 4;

struct NormShape {
  int nv, threads, stages, ctas;  // stages: 0: no ring; ctas: on an SM
  int smem;
};

// row_bytes: what a row brings to shared memory.
NormShape norm_shape(int H, int64_t row_bytes, int ctas) {
  NormShape s{};
  const int vecs = H / 8;
  s.nv = 1;
  while (s.nv < 4 && (vecs + s.nv - 1) / s.nv > kNormThreads) s.nv *= 2;
  s.threads = ((vecs + s.nv - 1) / s.nv + 31) & ~31;
  while (ctas > 1 && 2 * row_bytes > kRingBytes / ctas) --ctas;
  s.ctas = ctas;
  const int64_t n = kRingBytes / ctas / row_bytes;
  s.stages = static_cast<int>(n > kRingStages ? kRingStages : n);
  if (s.stages < 2 || s.threads > kNormThreads) s.stages = 0;
  s.smem = s.stages > 0 ? 64 + static_cast<int>(s.stages * row_bytes) : 0;
  return s;
}

template <class K>
moe_status launch_norm(K kernel, int grid, const NormShape &s, NormArgs a, cudaStream_t stream) {
  a.stages = s.stages;
  // (the limit that every kernel has counts its static shared memory too, so the ring asks for more than that)
  constexpr int least = 64 * 1024;
  if (s.smem > 0 && !raise_smem_limit(kernel, s.smem > least ? s.smem : least)) return MOE_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(s.threads), 1, 1);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

template <bool GRAD, bool F32>
moe_status launch_norm_typed(int grid, const NormShape &s, const NormArgs &a, cudaStream_t stream) {
#define MOE_NORM(NV, RING, THREADS)                                                        \
  (GRAD ? launch_norm(norm_grad_kernel<NV, F32, RING, THREADS>, grid, s, a, stream)         \
        : launch_norm(norm_kernel<NV, F32, RING, THREADS>, grid, s, a, stream))
  if (s.stages == 0) return s.threads > kNormThreads ? MOE_NORM(4, false, 1024) : MOE_NORM(4, false, kNormThreads);
  if (s.nv == 1) return MOE_NORM(1, true, kNormThreads);
  if (s.nv == 2) return MOE_NORM(2, true, kNormThreads);
  return MOE_NORM(4, true, kNormThreads);
#undef MOE_NORM
}

template <bool GRAD>
moe_status launch_norm_any(bool fp32, int grid, const NormShape &s, const NormArgs &a, cudaStream_t stream) {
  return fp32 ? launch_norm_typed<GRAD, true>(grid, s, a, stream) : launch_norm_typed<GRAD, false>(grid, s, a, stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_norm(const moe_norm_desc *desc, const void *x, const void *o, const float *w_post,
                               const float *gate, const float *w_pre, void *r, void *n, int32_t *err, void *stream) {
  if (check_norm(desc) != MOE_OK) return MOE_EINVAL;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (desc->rows == 0) return MOE_OK;
  if (o == nullptr && (w_post != nullptr || desc->gate != MOE_GATE_NONE)) return MOE_EINVAL;
  if (!good16(x) || !good16(w_pre) || !good16(n) || (o != nullptr && !good16(r)) || !aligned16(r) || !aligned16(o) ||
      !aligned16(w_post))
    return MOE_EINVAL;
  if (desc->gate != MOE_GATE_NONE && (gate == nullptr || !aligned4(gate))) return MOE_EINVAL;
  if (desc->gate == MOE_GATE_CHANNEL && !aligned16(gate)) return MOE_EINVAL;
  NormArgs a{};
  a.x = x;
  a.o = o;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.r = r;
  a.n = n;
  a.rows = desc->rows;
  a.H = desc->dim;
  a.row_gate = desc->gate == MOE_GATE_ROW;
  a.channel_gate = desc->gate == MOE_GATE_CHANNEL;
  a.eps = desc->eps;
  a.alpha = desc->alpha;
  a.err = err;
  const NormShape s = norm_shape(a.H, static_cast<int64_t>(a.H) * ((desc->stream_fp32 ? 4 : 2) + (o != nullptr ? 2 : 0)),
                                 norm_ctas(a.H));
  const int room = sm_count() * s.ctas;
  return launch_norm_any<false>(desc->stream_fp32 != 0, a.rows < room ? a.rows : room, s, a,
                                static_cast<cudaStream_t>(stream));
}

extern "C" int64_t moe_norm_workspace(const moe_norm_desc *desc) {
  if (check_norm(desc) != MOE_OK) return MOE_EINVAL;
  return static_cast<int64_t>(norm_parts(desc)) * 2 * desc->dim * 4;
}

extern "C" moe_status moe_norm_grad(const moe_norm_desc *desc, const void *r, const void *o, const float *w_post,
                                    const float *gate, const float *w_pre, const void *grad_r, const void *grad_n,
                                    void *grad_x, void *grad_o, float *grad_w_post, float *grad_gate,
                                    float *grad_w_pre, void *workspace, int32_t *err, void *stream) {
  if (check_norm(desc) != MOE_OK) return MOE_EINVAL;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (grad_w_pre == nullptr || !aligned4(grad_w_pre)) return MOE_EINVAL;
  if (w_post != nullptr && (grad_w_post == nullptr || !aligned4(grad_w_post))) return MOE_EINVAL;
  if (desc->gate != MOE_GATE_NONE && !(desc->gate == MOE_GATE_ROW && desc->rows == 0) &&
      (grad_gate == nullptr || !aligned4(grad_gate)))
    return MOE_EINVAL;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (desc->rows == 0) {
    const size_t n = static_cast<size_t>(desc->dim) * 4;
    if (cudaMemsetAsync(grad_w_pre, 0, n, cs) != cudaSuccess) return MOE_ECUDA;
    if (w_post != nullptr && cudaMemsetAsync(grad_w_post, 0, n, cs) != cudaSuccess) return MOE_ECUDA;
    if (desc->gate == MOE_GATE_CHANNEL && cudaMemsetAsync(grad_gate, 0, n, cs) != cudaSuccess) return MOE_ECUDA;
    return MOE_OK;
  }
  if (o == nullptr && (w_post != nullptr || desc->gate != MOE_GATE_NONE)) return MOE_EINVAL;
  if (!good16(r) || !good16(w_pre) || !good16(grad_n) || !good16(grad_x) || !good16(workspace) ||
      (o != nullptr && !good16(grad_o)) || !aligned16(o) || !aligned16(w_post) || !aligned16(grad_r))
    return MOE_EINVAL;
  if (desc->gate != MOE_GATE_NONE && (gate == nullptr || !aligned4(gate))) return MOE_EINVAL;
  if (desc->gate == MOE_GATE_CHANNEL && !aligned16(gate)) return MOE_EINVAL;
  NormArgs a{};
  a.x = r;
  a.o = o;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.grad_r = grad_r;
  a.grad_n = grad_n;
  a.grad_x = grad_x;
  a.grad_o = grad_o;
  a.grad_gate = grad_gate;
  a.parts = static_cast<float *>(workspace);
  a.rows = desc->rows;
  a.H = desc->dim;
  a.row_gate = desc->gate == MOE_GATE_ROW;
  a.channel_gate = desc->gate == MOE_GATE_CHANNEL;
  a.eps = desc->eps;
  a.alpha = desc->alpha;
  a.err = err;
  const int64_t of_stream = desc->stream_fp32 ? 4 : 2;
  const int64_t row_bytes = a.H * (of_stream * (grad_r != nullptr ? 2 : 1) + (o != nullptr ? 4 : 2));
  const int grid = norm_parts(desc);
  const NormShape s = norm_shape(a.H, row_bytes, norm_ctas(a.H));
  const moe_status st = launch_norm_any<true>(desc->stream_fp32 != 0, grid, s, a, cs);
  if (st != MOE_OK) return st;
  NormSumArgs b{a.parts, w_post, gate, grad_w_pre, w_post != nullptr ? grad_w_post : nullptr,
                a.channel_gate ? grad_gate : nullptr, grid, a.H};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.H + 31) / 32), b.grad_w_post != nullptr || a.channel_gate ? 2u : 1u, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = cs;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, norm_sum_kernel, b) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}
