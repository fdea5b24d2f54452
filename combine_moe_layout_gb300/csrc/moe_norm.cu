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
// Both kernels are bound by memory: every row is read and written once. All
// arithmetic and sums are in fp32; a column's sum over rows is taken by each CTA
// for its own rows in order, and the CTAs' parts are then added in order, so that
// results do not depend on timing.
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

// Sums over the block, every thread gets them; `part` is [2][N][32] floats, its halves taken in turn so that one
// barrier does.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float *part, int &turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  float *mine = part + turn * N * 32;
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) mine[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? mine[i * 32 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

template <int NV, bool F32>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a) {
  __shared__ float part[2][32];
  grid_dependency_wait();
  int turn = 0;
  const int vecs = a.H / 8;
  const float inv = 1.0f / static_cast<float>(a.H);
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    float x[NV][8], b[NV][8], sum[1];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        load8<F32>(a.x, t * a.H + v * 8, x[i]);
        if (a.o != nullptr) load8<false>(a.o, t * a.H + v * 8, b[i]);
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
        sum[0] = ss;
        block_sums<1>(sum, &part[0][0], turn);
        scale *= 1.0f / sqrtf(sum[0] * inv + a.eps);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vecs) {
          float w[8];
          if (a.w_post != nullptr) {
            vector8(a.w_post, v * 8, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) b[i][k] *= w[k];
          }
          if (a.channel_gate) {
            vector8(a.gate, v * 8, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) b[i][k] *= w[k];
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
    sum[0] = ss;
    block_sums<1>(sum, &part[0][0], turn);
    const float q = 1.0f / sqrtf(sum[0] * inv + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        float w[8];
        vector8(a.w_pre, v * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] *= q * w[k];
        store8<false>(a.n, t * a.H + v * 8, x[i]);
      }
    }
  }
}

template <int NV, bool F32>
__global__ void __launch_bounds__(1024) norm_grad_kernel(NormArgs a) {
  __shared__ float part[2][6][32];
  grid_dependency_wait();
  int turn = 0;
  const int vecs = a.H / 8;
  const float inv = 1.0f / static_cast<float>(a.H);
  float acc_n[NV][8], acc_o[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc_n[i][k] = acc_o[i][k] = 0.0f;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    float r[NV][8], o[NV][8], dn[NV][8], dr[NV][8];  // dn: then dn w_pre
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};  // r^2, dn w r, o^2, and c o with grad_r, dn w, r
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        const int64_t at = t * a.H + v * 8;
        load8<F32>(a.x, at, r[i]);
        load8<false>(a.grad_n, at, dn[i]);
        if (a.grad_r != nullptr)
          load8<F32>(a.grad_r, at, dr[i]);
        else
#pragma unroll
          for (int k = 0; k < 8; ++k) dr[i][k] = 0.0f;
        if (a.o != nullptr)
          load8<false>(a.o, at, o[i]);
        else
#pragma unroll
          for (int k = 0; k < 8; ++k) o[i][k] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        float w[8], c[8];
        vector8(a.w_pre, v * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = 1.0f;
        if (a.w_post != nullptr) vector8(a.w_post, v * 8, c);
        if (a.channel_gate) {
          float g[8];
          vector8(a.gate, v * 8, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) c[k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = dn[i][k] * w[k], co = c[k] * o[i][k];
          s[0] += r[i][k] * r[i][k];
          s[1] += d * r[i][k];
          s[2] += o[i][k] * o[i][k];
          s[3] += co * dr[i][k];
          s[4] += co * d;
          s[5] += co * r[i][k];
        }
      }
    }
    block_sums<6>(s, &part[0][0][0], turn);
    const float q = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float m = q * q * s[1] * inv;  // dr = grad_r + q (dn w - m r)
    const float p = a.w_post != nullptr ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    const float db = a.alpha * p * (s[3] + q * (s[4] - m * s[5]));  // alpha sum dr c o p
    float scale = a.alpha * p;
    if (a.row_gate) {
      scale *= a.gate[t];
      if (threadIdx.x == 0) a.grad_gate[t] = db;
    }
    // grad_o = scale (c dr - o f), f = p sum(alpha dr c o p) / (alpha H) = p^2 sum(dr c o) / H
    const float f = a.w_post != nullptr ? p * p * (s[3] + q * (s[4] - m * s[5])) * inv : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs) {
        const int64_t at = t * a.H + v * 8;
        float w[8], c[8];
        vector8(a.w_pre, v * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = 1.0f;
        if (a.w_post != nullptr) vector8(a.w_post, v * 8, c);
        if (a.channel_gate) {
          float g[8];
          vector8(a.gate, v * 8, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) c[k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc_n[i][k] += dn[i][k] * (r[i][k] * q);
          dr[i][k] += q * (dn[i][k] * w[k] - m * r[i][k]);
          acc_o[i][k] += scale * dr[i][k] * o[i][k];
          o[i][k] = scale * (c[k] * dr[i][k] - f * o[i][k]);
        }
        store8<F32>(a.grad_x, at, dr[i]);
        if (a.o != nullptr) store8<false>(a.grad_o, at, o[i]);
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

// Rows of a gradient's CTA parts: at most 304 (two CTAs on each of 152 SMs), the same on every device, so that the
// sums are too.
int norm_parts(const moe_norm_desc *d) { return d->rows < 304 ? d->rows : 304; }

struct NormShape {
  int nv, threads;
};

NormShape norm_shape(int H) {
  const int vecs = H / 8;
  int nv = 1;
  while (nv < 4 && (vecs + nv - 1) / nv > kNormThreads) nv *= 2;
  const int t = (vecs + nv - 1) / nv;
  return NormShape{nv, (t + 31) & ~31};
}

template <class K>
moe_status launch_norm(K kernel, int grid, int threads, const NormArgs &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
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
  const NormShape s = norm_shape(a.H);
  const int room = sm_count() * (2048 / s.threads < 32 ? 2048 / s.threads : 32);
  const int grid = a.rows < room ? a.rows : room;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (desc->stream_fp32) {
    if (s.nv == 1) return launch_norm(norm_kernel<1, true>, grid, s.threads, a, cs);
    if (s.nv == 2) return launch_norm(norm_kernel<2, true>, grid, s.threads, a, cs);
    return launch_norm(norm_kernel<4, true>, grid, s.threads, a, cs);
  }
  if (s.nv == 1) return launch_norm(norm_kernel<1, false>, grid, s.threads, a, cs);
  if (s.nv == 2) return launch_norm(norm_kernel<2, false>, grid, s.threads, a, cs);
  return launch_norm(norm_kernel<4, false>, grid, s.threads, a, cs);
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
  const NormShape s = norm_shape(a.H);
  const int grid = norm_parts(desc);
  moe_status st;
  if (desc->stream_fp32)
    st = s.nv == 1   ? launch_norm(norm_grad_kernel<1, true>, grid, s.threads, a, cs)
         : s.nv == 2 ? launch_norm(norm_grad_kernel<2, true>, grid, s.threads, a, cs)
                     : launch_norm(norm_grad_kernel<4, true>, grid, s.threads, a, cs);
  else
    st = s.nv == 1   ? launch_norm(norm_grad_kernel<1, false>, grid, s.threads, a, cs)
         : s.nv == 2 ? launch_norm(norm_grad_kernel<2, false>, grid, s.threads, a, cs)
                     : launch_norm(norm_grad_kernel<4, false>, grid, s.threads, a, cs);
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
