// Shared by the forms of the gated feed-forward block.
#pragma once

#include "moe_common.cuh"

namespace moe {

struct FfnSizes {
  int rows, H, I, E, R, act, save, num_sms;
};

constexpr int kFewRows = 16;  // rows that moe_ffn_few.cu takes

moe_status launch_ffn_few(const FfnSizes &s, const int32_t *offsets, const void *x, const void *w_gate,
                          const void *w_up, const void *w_down, void *h, void *y, void *gate, void *up, int32_t *err,
                          cudaStream_t stream);

namespace {

// act(g) and act'(g), in fp32.
template <bool GRAD>
__device__ __forceinline__ float act_of(float g, int act, float *da) {
  if (act == MOE_ACT_SILU) {
    const float p = 1.0f / (1.0f + expf(-g));
    if constexpr (GRAD) *da = p * (1.0f + g * (1.0f - p));
    return g * p;
  }
  constexpr float k = 0.7978845608028654f, c = 0.044715f;  // sqrt(2 / pi)
  const float t = tanhf(k * (g + c * g * g * g));
  if constexpr (GRAD) *da = 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * k * (1.0f + 3.0f * c * g * g);
  return 0.5f * g * (1.0f + t);
}

}  // namespace
}  // namespace moe
