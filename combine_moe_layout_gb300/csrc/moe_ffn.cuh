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

// 1 / (1 + exp(-v)), to a few units in the last place (2^-20 of it where |v| is below 10): what it goes into is
// rounded to bf16. 0 and 1 at the ends. With expf and a division that rounds, 333 rows of 12 experts take 23.6 us for
// 22.7 and their gradients 46.5 for 45.2, 64 rows of 7168 -> 2048 29.4 for 28.8, 24576 rows 792 for 789.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// act(g) and act'(g), in fp32. The second act, g (1 + tanh(z)) / 2 with z = sqrt(2/pi) (g + 0.044715 g^3), is
// g sigmoid(2 z); so is the derivative: p + g p (1 - p) 2 z'.
template <bool GRAD>
__device__ __forceinline__ float act_of(float g, int act, float *da) {
  float v = g, dv = 1.0f;
  if (act != MOE_ACT_SILU) {
    constexpr float k = 1.5957691216057308f, c = 0.044715f;  // 2 sqrt(2 / pi)
    v = k * (g + c * g * g * g);
    // (p (1 - p) is 0 long before g^2 overflows, and would make the derivative NaN with it)
    if constexpr (GRAD) dv = k * (1.0f + 3.0f * c * fminf(g * g, 1e30f));
  }
  const float p = sigmoid(v);
  if constexpr (GRAD) *da = p + g * p * (1.0f - p) * dv;
  return g * p;
}

}  // namespace
}  // namespace moe
