// Router gate: logits -> the k experts of each token and their weights, and the
// gradient of the weights with respect to the logits.
//
// With l the logits of a token and b the selection bias (0 when absent):
//   s_e = exp(l_e - max l) / sum_i exp(l_i - max l)   (softmax)
//       = 1 / (1 + exp(-l_e))                         (sigmoid)
//   group score = sum of the group's group_top largest s_e + b_e; the
//     keep_groups best groups stay
//   ids = the k largest s_e + b_e of those groups, ties to the lowest index
//   w_j = scale s_{ids j}, divided by the sum of the chosen s when renormalised
// Without a bias the ids are chosen by l itself: s increases with l, so the
// order is the same and two logits whose scores round to the same 32-bit value
// keep it. The same holds for a group score of one member.
//
// Gradient, with g_j = dL/dw_j:
//   softmax, plain:         dl_e = s_e (scale g_e [e chosen] - sum_j scale g_j s_j)
//   softmax, renormalised:  a softmax over the chosen: dl_j = v_j scale (g_j - sum_i g_i v_i),
//                           v the weights at scale 1; 0 elsewhere
//   sigmoid:                dl_j = ds_j s_j (1 - s_j), ds_j = scale g_j, or
//                           scale (g_j - sum_i g_i v_i) / sum s when renormalised
// The bias and the groups only select, so no gradient passes through them.
//
// Both kernels take one warp per token: a lane holds E/32 logits in registers
// (groups of four neighbours, so a row is read with 16-byte (fp32) or 8-byte
// (bf16) loads) and a choice is one warp maximum over integer keys that hold the
// order of a logit and its expert.
//
// Measured, 32768 tokens of 256 fp32 logits, k = 8, renormalised softmax: gate and
// gradient take 27.5 us together, alone 17 (36 MB, 2.1 TB/s) and 12.8. The gate is
// bound by integer instructions: their pipe is busy for 72% of its active cycles,
// and an instruction is issued in 70% of them. So what counts is how few a choice
// takes: with a maximum over all of a lane's values for each choice it took 36 us.
// The gradient (44 MB with the chosen logits' sectors, 3.4 TB/s) waits for its reads
// one after the other (ids, then the chosen logits: 7.4 warps a scheduler), and
// writes 34 MB. 4096 tokens in 8 groups (bf16 logits, sigmoid) take 7.9-8.7 us: issue
// slots are taken in 64% of the active cycles, which are 58% of the kernel's; the
// rest is its start and end. One token: 4.6 us a call, which is its launch.
// Beside them (gate alone, 32768 tokens, four sets of inputs in turn, where the above
// takes 21.7): bf16 logits 16.3; 512 experts 23.0; sigmoid with a selection bias
// 28.7, with 512 experts 50.7 (a division and an exponential for every expert); fp32
// logits that hold bf16 values 24.6, since four rows in ten have two of their best
// agree above the expert's bits and go the exact way.
#include <cuda_bf16.h>

#include <cfloat>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kGateWarps = 8;
constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxGroups = 32;

struct GateArgs {
  const void *logits;
  const float *bias;
  int32_t *idx;        // [N][k]
  float *weights;      // [N][k]
  const float *gw;     // gradient: dL/dweights [N][k]
  void *gl;            // gradient: dL/dlogits [N][E]
  int32_t *err;
  int64_t n;
  int E, k, sigmoid, renorm, groups, keep, top, early;
  int group_size, lanes_per_group;
  uint64_t group_magic;  // ceil(2^32 / group_size): index / group_size = (index * magic) >> 32
  float scale;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The largest of three values, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// +inf counts as the largest finite value in the scores (the limit of both).
__device__ __forceinline__ float finite(float l) { return fminf(l, FLT_MAX); }

// Expert of value i of a lane: four neighbours per lane and pass.
__device__ __forceinline__ int expert_of(int i, int lane) { return ((i >> 2) * 32 + lane) * 4 + (i & 3); }

// A lane's logits of a row. NaN counts as -inf (and is reported).
template <int VPL, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const void *logits, int64_t t, int E, int lane, float (&l)[VPL], bool *nan) {
  const int64_t base = t * E;
  float worst = -INFINITY;
#pragma unroll
  for (int p = 0; p < VPL / 4; ++p) {
    const int e0 = (p * 32 + lane) * 4;
    float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if constexpr (VEC) {
      if (e0 < E) {
        if constexpr (BF16) {
          const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(logits) + base + e0);
          v[0] = __uint_as_float(r.x << 16);
          v[1] = __uint_as_float(r.x & 0xffff0000u);
          v[2] = __uint_as_float(r.y << 16);
          v[3] = __uint_as_float(r.y & 0xffff0000u);
        } else {
          const float4 r = *reinterpret_cast<const float4 *>(static_cast<const float *>(logits) + base + e0);
          v[0] = r.x;
          v[1] = r.y;
          v[2] = r.z;
          v[3] = r.w;
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e0 + c < E) {
          if constexpr (BF16)
            v[c] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(logits)[base + e0 + c]) << 16);
          else
            v[c] = static_cast<const float *>(logits)[base + e0 + c];
        }
    }
    worst = max_nan(max_nan(worst, v[0], v[1]), v[2], v[3]);
#pragma unroll
    for (int c = 0; c < 4; ++c) l[4 * p + c] = v[c];
  }
  *nan = worst != worst;
  if (*nan) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = fmaxf(l[i], -INFINITY);  // -inf for a NaN
  }
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *logits, int64_t i) {
  float v;
  if constexpr (BF16)
    v = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(logits)[i]) << 16);
  else
    v = static_cast<const float *>(logits)[i];
  return fmaxf(v, -INFINITY);
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }  // 1 for +inf

// The sigmoid and, to its own size, what it leaves of one.
__device__ __forceinline__ float sigmoid_and_rest(float l, float *rest) {
  const float z = expf(-l), s = 1.0f / (1.0f + z);
  *rest = fminf(z, FLT_MAX) * s;
  return s;
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }

// Sorts a lane's values, largest first: Batcher's odd-even merge sort.
template <int N, class V>
__device__ __forceinline__ void sort_down(V (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const int first = q % p;
        if (x >= first && (x - first) % (2 * q) < q && x + q < N && x / (2 * p) == (x + q) / (2 * p)) {
          const V hi = larger(v[x], v[x + q]), lo = smaller(v[x], v[x + q]);
          v[x] = hi;
          v[x + q] = lo;
        }
      }
}

// The D largest of a lane's values, largest first: fours are sorted, and two
// sorted lists of four are joined by taking the larger of opposite ends, which
// are the four largest as a bitonic sequence, and sorting that.
template <int N, int D>
__device__ __forceinline__ void largest_of(const uint32_t (&v)[N], uint32_t (&head)[D]) {
  static_assert(D == 4 && N % 4 == 0, "lists of four");
#pragma unroll
  for (int b = 0; b < N; b += 4) {
    uint32_t q[4] = {v[b], v[b + 1], v[b + 2], v[b + 3]};
    sort_down<4>(q);
    if (b == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) head[i] = q[i];
      continue;
    }
    const uint32_t b0 = max(head[0], q[3]), b1 = max(head[1], q[2]), b2 = max(head[2], q[1]), b3 = max(head[3], q[0]);
    const uint32_t a0 = max(b0, b2), a2 = min(b0, b2), a1 = max(b1, b3), a3 = min(b1, b3);
    head[0] = max(a0, a1);
    head[1] = min(a0, a1);
    head[2] = max(a2, a3);
    head[3] = min(a2, a3);
  }
}

// The largest v of the warp.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Place of expert e's value among the warp's values in shared memory: a word
// between the groups keeps equal members of different groups in different banks.
__device__ __forceinline__ int group_of(const GateArgs &a, int e) {
  return static_cast<int>(e * a.group_magic >> 32);
}

// Which groups stay, as a bit per group (the same in every lane). The warp's
// values go through shared memory (gs); lanes_per_group lanes share a group.
__device__ __forceinline__ uint32_t kept_groups(const GateArgs &a, const float *gs, int lane) {
  const int lpg = a.lanes_per_group;
  const int grp = lane / lpg, sub = lane - grp * lpg;
  const bool live = grp < a.groups;
  const float *v = gs + grp * (a.group_size + 1);
  float score = 0.0f;
  int found = 0;
  if (a.top <= 2) {  // the usual sizes in one pass: the two largest, lane by lane and then across the group's lanes
    float b1 = -INFINITY, b2 = -INFINITY;
    if (live) {
#pragma unroll 8
      for (int x = sub; x < a.group_size; x += lpg) {
        const float y = v[x];
        b2 = fmaxf(b2, fminf(b1, y));
        b1 = fmaxf(b1, y);
      }
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    }
    found = b1 > -INFINITY;
    score = a.top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
  } else {  // group_top largest one by one
    uint64_t taken = 0;  // bit i: value sub + i * lpg (fewer than 64 for 1024 experts)
    for (int r = 0; r < a.top; ++r) {
      float best = -INFINITY;
      int bi = a.group_size;
      if (live)
        for (int i = 0, x = sub; x < a.group_size; ++i, x += lpg)
          if (!((taken >> i) & 1ull) && v[x] > best) {
            best = v[x];
            bi = x;
          }
      for (int o = lpg >> 1; o > 0; o >>= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, best, o);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (ob > best || (ob == best && oi < bi)) {
          best = ob;
          bi = oi;
        }
      }
      if (best > -INFINITY) {  // members that are not available add nothing
        score += best;
        ++found;
      }
      const int d = bi - sub;
      if (bi < a.group_size && d >= 0 && d % lpg == 0) taken |= 1ull << (d / lpg);
    }
  }
  if (!live || found == 0) score = -INFINITY;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const float o = __shfl_sync(0xffffffffu, score, g * lpg);
    if (o > score || (o == score && g < grp)) ++rank;
  }
  const uint32_t lanes = __ballot_sync(0xffffffffu, live && found > 0 && rank < a.keep);
  uint32_t kept = 0;
  for (int g = 0; g < a.groups; ++g) kept |= ((lanes >> (g * lpg)) & 1u) << g;
  return kept;
}

template <int VPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(GateArgs a) {
  extern __shared__ float gate_sm[];  // [warps][E + groups], with groups only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  grid_dependency_wait();
  if (a.early) grid_dependents_launch();
  if (t >= a.n) return;

  float l[VPL];
  bool nan = false;
  load_row<VPL, BF16, VEC>(a.logits, t, a.E, lane, l, &nan);

  float mx = -INFINITY, sum = 1.0f;
  if (!a.sigmoid && (!a.renorm || a.bias != nullptr || a.groups > 1)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) mx = fmaxf(mx, finite(l[i]));
    mx = redux_max(mx);
    if (mx == -INFINITY) mx = 0.0f;  // nothing available: every score is 0
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += expf(finite(l[i]) - mx);
    sum = warp_sum(sum);
    if (sum == 0.0f) sum = 1.0f;
  }

  // the values that choose: the logits, or the scores with their bias
  if (a.bias != nullptr || (a.groups > 1 && a.top > 1)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of(i, lane);
      float s = -INFINITY;
      if (e < a.E && l[i] > -INFINITY) {
        s = a.sigmoid ? sigmoid_of(l[i]) : expf(finite(l[i]) - mx) / sum;
        if (a.bias != nullptr) s += __ldg(a.bias + e);
        if (s != s) {
          nan = true;
          s = -INFINITY;
        }
      }
      if (a.groups > 1 && e < a.E) gate_sm[warp * (a.E + a.groups) + e + group_of(a, e)] = s;
      if (a.bias != nullptr) l[i] = s;
    }
  } else if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of(i, lane);
      if (e < a.E) gate_sm[warp * (a.E + a.groups) + e + group_of(a, e)] = l[i];
    }
  }
  if (a.groups > 1) {
    __syncwarp();
    const uint32_t kept = kept_groups(a, gate_sm + warp * (a.E + a.groups), lane);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((kept >> (group_of(a, expert_of(i, lane)) & 31)) & 1u)) l[i] = -INFINITY;
  }
  if (__any_sync(0xffffffffu, nan) && lane == 0) latch_error(a.err, MOE_EINVAL);

  // Most rows: keys that hold a value's order above and, in their last bits, its
  // expert counted down, so that no two are equal. A lane keeps its four largest
  // keys in order, and the largest head of the 32 lists is taken k times: the
  // experts in their order. bf16 values lose nothing to the expert's bits; others
  // may agree in all bits above them (about 1 row in 200 of N(0, 1) logits at 256
  // experts), which shows in neighbours of the chosen and goes the slow way, as
  // does a row with four of its chosen experts in one lane that holds more.
  constexpr uint32_t kExperts = VPL * 32 - 1;  // the expert's bits
  constexpr uint32_t kNone = 0x007fffffu;      // the largest key of -inf
  int my_e = -1, place = lane;
  float my_l = -INFINITY;
  bool slow = false;
  {
    uint32_t keys[VPL], head[4];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t u = __float_as_uint(l[i] + 0.0f);  // -0 as +0
      const uint32_t order = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
      keys[i] = (order & ~kExperts) | (kExperts - expert_of(i, lane));
    }
    largest_of(keys, head);
    uint32_t key = 0, last = 0;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      last = __reduce_max_sync(0xffffffffu, head[0]);
      if (lane == j) key = last;
      if (head[0] == last) {
        head[0] = head[1];
        head[1] = head[2];
        head[2] = head[3];
        head[3] = 0;
      }
    }
    if (key > kNone) my_e = static_cast<int>(kExperts - (key & kExperts));
    // a chosen value too near to the one before it or to the best of those left, or a lane that ran out
    if (!BF16 || a.bias != nullptr) {
      const uint32_t before = __shfl_up_sync(0xffffffffu, key, 1);
      slow = (lane > 0 && key > kNone && (key ^ before) <= kExperts) ||
             (head[0] > kNone && (head[0] ^ last) <= kExperts);
    }
    if (VPL > 4) slow |= head[0] == 0;
    slow = __any_sync(0xffffffffu, slow);
  }
  if (!slow) {
    if (my_e >= 0) my_l = load_logit<BF16>(a.logits, t * a.E + my_e);
  } else {
    // the score of a logit as the choice sees it
    const auto choosing = [&](float logit, int e) {
      if (a.bias == nullptr) return logit;
      return (a.sigmoid ? sigmoid_of(logit) : expf(finite(logit) - mx) / sum) + __ldg(a.bias + e);
    };
    __shared__ int chosen[kGateWarps][kMaxTopk];
    float head[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) head[i] = l[i];
    sort_down<VPL>(head);
    my_e = -1;
    // any values: T with its equals counted, the lowest experts among them, and the order by comparing
    int over = 0, count = 0;  // values > T, and values taken
    float T = INFINITY;
    while (count < a.k) {
      const float top = redux_max(head[0]);
      if (top == -INFINITY) break;
      if (top < T) over = count;  // (a lane may hold equals of T one after the other)
      T = top;
      const bool from = head[0] == top;
      count += __popc(__ballot_sync(0xffffffffu, from));
      if (from) {
#pragma unroll
        for (int i = 0; i + 1 < VPL; ++i) head[i] = head[i + 1];
        head[VPL - 1] = -INFINITY;
      }
    }
    uint32_t pick = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (l[i] >= T) pick |= 1u << i;
      if (l[i] == T) equal |= 1u << i;
    }
    count = __reduce_add_sync(0xffffffffu, __popc(pick));  // (a lane's equals of T behind its head were not counted)
    if (count > a.k) {
      pick &= ~equal;
      for (int r = over; r < a.k; ++r) {
        const int e = equal != 0 ? expert_of(__ffs(equal) - 1, lane) : 0x7fffffff;
        if (__reduce_min_sync(0xffffffffu, e) == e && equal != 0) {
          pick |= equal & (0u - equal);
          equal &= equal - 1;
        }
      }
      count = a.k;
    }
    for (int base = 0; base < count;) {
      const unsigned have = __ballot_sync(0xffffffffu, pick != 0);
      if (have == 0) break;
      if (pick != 0) {
        const int at = base + __popc(have & ((1u << lane) - 1u));
        if (at < kMaxTopk) chosen[warp][at] = expert_of(__ffs(pick) - 1, lane);
        pick &= pick - 1;
      }
      base += __popc(have);
    }
    __syncwarp();
    float my_v = -INFINITY;
    if (lane < count) {
      my_e = chosen[warp][lane];
      my_l = load_logit<BF16>(a.logits, t * a.E + my_e);
      my_v = choosing(my_l, my_e);
      place = 0;
    }
    for (int j = 0; j < count; ++j) {
      const float v = __shfl_sync(0xffffffffu, my_v, j);
      const int e = __shfl_sync(0xffffffffu, my_e, j);
      if (lane < count && (v > my_v || (v == my_v && e < my_e))) ++place;
    }
  }
  my_l = finite(my_l);

  float w = 0.0f;
  if (a.sigmoid) {
    if (my_e >= 0) w = sigmoid_of(my_l);
    if (a.renorm) {
      const float s = warp_sum(w);
      w = s > 0.0f ? w / s : 0.0f;
    }
  } else if (a.renorm) {
    const float m = redux_max(my_l);
    if (my_e >= 0) w = expf(my_l - m);
    const float s = warp_sum(w);
    w = s > 0.0f ? w / s : 0.0f;
  } else if (my_e >= 0) {
    w = expf(my_l - mx) / sum;
  }
  if (lane < a.k) {
    a.idx[t * a.k + place] = my_e;
    a.weights[t * a.k + place] = w * a.scale;
  }
}

// x of this lane, or the sum of x over all lanes that name the same expert, in their order.
__device__ __forceinline__ float over_entries(float x, int my_e, int k) {
  float sum = 0.0f;
  for (int j = 0; j < k; ++j) {
    const float v = __shfl_sync(0xffffffffu, x, j);
    if (__shfl_sync(0xffffffffu, my_e, j) == my_e) sum += v;
  }
  return sum;
}

// The gradient's row is zero (renormalised softmax and sigmoid) or -s_e times
// one number (plain softmax), but for the k chosen. A renormalised row needs the
// chosen logits only, so the other E - k are not read.
//
// A score near one leaves 1 - s small, and it is lost when it is taken from the
// rounded s (a logit of 17 gave a sigmoid's gradient of zero). The sigmoid's is
// exp(-l) s. A softmax' differences g_j - sum_i g_i s_i are taken as
//   s_t (g_j - g_t) + g_j r - sum_{i != t} g_i s_i
// with t the largest score and r = sum_{i != t} s_i, the rest, added up without it:
// nothing there is the small difference of two large numbers. 32768 tokens of 256
// fp32 logits, k = 8, with the gate: 27.5 us (renormalised softmax, as with the
// plain differences), 32.4 (softmax; 31.1 with them), 28.9 (renormalised sigmoid;
// 27.8).
template <int VPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_grad_kernel(GateArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  grid_dependency_wait();
  if (a.early) grid_dependents_launch();
  if (t >= a.n) return;

  int my_e = -1;
  float g = 0.0f, my_l = -INFINITY;
  if (lane < a.k) {
    my_e = a.idx[t * a.k + lane];
    if (my_e < 0 || my_e >= a.E) {
      if (my_e != kMaskedExpert) latch_error(a.err, MOE_EINVAL);
      my_e = -1;
    } else {
      g = a.gw[t * a.k + lane];
      my_l = finite(load_logit<BF16>(a.logits, t * a.E + my_e));
    }
  }
  // The choices' elements go through the warp's row in shared memory (comparing every value with every choice cost as
  // much as the rest of the kernel). What no choice wrote stays kUnset, a NaN that no arithmetic gives. An expert
  // named by two entries shows in the marks: its terms are added up, in order, in both.
  constexpr uint32_t kUnset = 0xffffffffu;
  __shared__ __align__(16) uint32_t rows[kGateWarps][VPL * 32];
  uint32_t *row = rows[warp];
#pragma unroll
  for (int p = 0; p < VPL / 4; ++p)
    *reinterpret_cast<uint4 *>(row + (p * 32 + lane) * 4) = make_uint4(kUnset, kUnset, kUnset, kUnset);
  __syncwarp();
  if (my_e >= 0) row[my_e] = lane;
  __syncwarp();
  const bool any_twice = __any_sync(0xffffffffu, my_e >= 0 && row[my_e] != static_cast<uint32_t>(lane));
  __syncwarp();

  float out[VPL];
  float d = 0.0f;  // dL/dl of this lane's choice
#pragma unroll
  for (int i = 0; i < VPL; ++i) out[i] = 0.0f;
  if (a.renorm) {
    float p = 0.0f, most = 1.0f, rest_p = 1.0f;  // the score; of a softmax relative to the largest
    if (a.sigmoid) {
      if (my_e >= 0) p = sigmoid_and_rest(my_l, &rest_p);
      most = redux_max(p);
    } else {
      const float m = redux_max(my_l);
      if (my_l > -INFINITY) p = expf(my_l - m);
      most = m > -INFINITY ? 1.0f : 0.0f;
    }
    if (most > 0.0f) {  // (the whole warp)
      const int top = __ffs(__ballot_sync(0xffffffffu, p == most)) - 1;
      const float rest = warp_sum(lane == top ? 0.0f : p), total = most + rest;
      const float v = p / total;
      const float others = warp_sum(lane == top ? 0.0f : g * v);
      d = most / total * (g - __shfl_sync(0xffffffffu, g, top)) + (g * (rest / total) - others);
      d *= a.sigmoid ? p * rest_p / total : v;
    }
    d *= a.scale;
    if (any_twice) d = over_entries(d, my_e, a.k);
  } else if (a.sigmoid) {
    float rest = 0.0f;
    const float s = sigmoid_and_rest(my_l, &rest);
    if (my_e >= 0) d = a.scale * g * (s * rest);
    if (any_twice) d = over_entries(d, my_e, a.k);
  } else {
    float l[VPL];
    bool nan = false;
    load_row<VPL, BF16, VEC>(a.logits, t, a.E, lane, l, &nan);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) mx = fmaxf(mx, l[i] = finite(l[i]));
    mx = redux_max(mx);
    const bool some = mx > -INFINITY;
    if (!some) mx = 0.0f;
    // exp(0) = 1 is the largest; the rest is what is below one and all but one of the ones
    float rest = 0.0f, ones = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - mx);
      (l[i] < 1.0f ? rest : ones) += l[i];
    }
    const unsigned with = __ballot_sync(0xffffffffu, ones > 0.0f);
    if (lane == __ffs(with) - 1) ones -= 1.0f;
    rest = warp_sum(rest + ones);
    const float inv = some ? 1.0f / (1.0f + rest) : 0.0f;  // also the largest score
    // the largest among the chosen, if it is one (of several equal ones any is as good as another)
    const float p = my_l > -INFINITY ? expf(my_l - mx) : 0.0f, s = p * inv;
    const int from = __ffs(__ballot_sync(0xffffffffu, p == 1.0f)) - 1;
    const int top_e = __shfl_sync(0xffffffffu, my_e, from & 31);
    const float others = warp_sum(from >= 0 && my_e == top_e ? 0.0f : g * s);
    if (any_twice) g = over_entries(g, my_e, a.k);
    const float g_top = __shfl_sync(0xffffffffu, g, from & 31), at_top = from >= 0 ? g_top : 0.0f;
    const float sum = a.scale * (at_top * inv + others);
    d = a.scale * (s * (inv * (g - at_top) + (g * (rest * inv) - others)));
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] = -sum * (l[i] * inv);
  }
  if (my_e >= 0) row[my_e] = __float_as_uint(d);
  __syncwarp();
#pragma unroll
  for (int p = 0; p < VPL / 4; ++p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(row + (p * 32 + lane) * 4);
    if (v.x != kUnset) out[4 * p] = __uint_as_float(v.x);
    if (v.y != kUnset) out[4 * p + 1] = __uint_as_float(v.y);
    if (v.z != kUnset) out[4 * p + 2] = __uint_as_float(v.z);
    if (v.w != kUnset) out[4 * p + 3] = __uint_as_float(v.w);
  }
  const int64_t base = t * a.E;
#pragma unroll
  for (int p = 0; p < VPL / 4; ++p) {
    const int e0 = (p * 32 + lane) * 4;
    if constexpr (VEC) {
      if (e0 >= a.E) continue;
      if constexpr (BF16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(out[4 * p], out[4 * p + 1]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(out[4 * p + 2], out[4 * p + 3]);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.gl) + base + e0) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.gl) + base + e0) =
            make_float4(out[4 * p], out[4 * p + 1], out[4 * p + 2], out[4 * p + 3]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e0 + c < a.E) {
          if constexpr (BF16)
            static_cast<__nv_bfloat16 *>(a.gl)[base + e0 + c] = __float2bfloat16_rn(out[4 * p + c]);
          else
            static_cast<float *>(a.gl)[base + e0 + c] = out[4 * p + c];
        }
    }
  }
}

template <int VPL>
moe_status launch_gate_v(const GateArgs &a, bool bf16, bool vec, bool grad, cudaStream_t stream) {
  void (*fn)(GateArgs) =
      grad ? (bf16 ? (vec ? gate_grad_kernel<VPL, true, true> : gate_grad_kernel<VPL, true, false>)
                   : (vec ? gate_grad_kernel<VPL, false, true> : gate_grad_kernel<VPL, false, false>))
           : (bf16 ? (vec ? gate_kernel<VPL, true, true> : gate_kernel<VPL, true, false>)
                   : (vec ? gate_kernel<VPL, false, true> : gate_kernel<VPL, false, false>));
  cudaLaunchConfig_t cfg = {};
  const int64_t blocks = (a.n + kGateWarps - 1) / kGateWarps;
  if (blocks > 0x7fffffffll) return MOE_EINVAL;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kGateWarps * 32, 1, 1);
  // at most 8 warps x (1024 experts + 32 groups) x 4 bytes = 33 KB
  cfg.dynamicSmemBytes = !grad && a.groups > 1 ? static_cast<size_t>(kGateWarps) * (a.E + a.groups) * sizeof(float) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  use_pdl(cfg, attr);
  if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) return MOE_ECUDA;
  return launch_status();
}

moe_status launch_gate(const GateArgs &a, bool bf16, bool grad, cudaStream_t stream) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | (grad ? reinterpret_cast<uintptr_t>(a.gl) : 0);
  const bool vec = a.E % 4 == 0 && (at & (bf16 ? 7u : 15u)) == 0;
  if (a.E <= 128) return launch_gate_v<4>(a, bf16, vec, grad, stream);
  if (a.E <= 256) return launch_gate_v<8>(a, bf16, vec, grad, stream);
  if (a.E <= 512) return launch_gate_v<16>(a, bf16, vec, grad, stream);
  return launch_gate_v<32>(a, bf16, vec, grad, stream);
}

moe_status gate_args(const moe_desc *desc, const moe_gate_opts *o, GateArgs *a) {
  Sizes s;
  const moe_status st = check_desc(desc, &s);
  if (st != MOE_OK) return st;
  if (o == nullptr || s.E > kGateMaxExperts) return MOE_EINVAL;
  if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if ((o->renormalize | o->logits_bf16) & ~1) return MOE_EINVAL;
  if (!(o->scale - o->scale == 0.0f)) return MOE_EINVAL;  // not finite
  const int g = o->num_groups;
  if (g < 0 || g > kGateMaxGroups) return MOE_EINVAL;
  *a = GateArgs{};
  a->n = s.ntok;
  a->E = s.E;
  a->k = s.k;
  a->sigmoid = o->score == MOE_SCORE_SIGMOID;
  a->renorm = o->renormalize;
  a->scale = o->scale;
  a->early = early_trigger(s.ntok);
  a->groups = 1;
  if (g > 1) {
    if (s.E % g != 0) return MOE_EINVAL;
    const int size = s.E / g;
    if (o->keep_groups < 1 || o->keep_groups > g || o->group_top < 1 || o->group_top > size ||
        static_cast<int64_t>(o->keep_groups) * size < s.k)
      return MOE_EINVAL;
    a->groups = g;
    a->keep = o->keep_groups;
    a->top = o->group_top;
    a->group_size = size;
    a->group_magic = ((1ull << 32) + size - 1) / size;
    int lpg = 32;
    while (lpg * g > 32) lpg >>= 1;
    a->lanes_per_group = lpg;
  }
  return MOE_OK;
}

bool aligned_elem(const void *p, bool bf16) { return (reinterpret_cast<uintptr_t>(p) & (bf16 ? 1u : 3u)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_gate(const moe_desc *desc, const moe_gate_opts *opts, const void *logits, const float *bias,
                               int32_t *topk_idx, float *topk_weights, int32_t *err, void *stream) {
  GateArgs a;
  const moe_status st = gate_args(desc, opts, &a);
  if (st != MOE_OK) return st;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (a.n == 0) return MOE_OK;
  const bool bf16 = opts->logits_bf16 != 0;
  if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr) return MOE_EINVAL;
  if (!aligned_elem(logits, bf16) || !aligned4(bias) || !aligned4(topk_idx) || !aligned4(topk_weights))
    return MOE_EINVAL;
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.weights = topk_weights;
  a.err = err;
  return launch_gate(a, bf16, false, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_gate_grad(const moe_desc *desc, const moe_gate_opts *opts, const void *logits,
                                    const int32_t *topk_idx, const float *grad_weights, void *grad_logits,
                                    int32_t *err, void *stream) {
  GateArgs a;
  const moe_status st = gate_args(desc, opts, &a);
  if (st != MOE_OK) return st;
  if (err == nullptr || !aligned4(err)) return MOE_EINVAL;
  if (a.n == 0) return MOE_OK;
  const bool bf16 = opts->logits_bf16 != 0;
  if (logits == nullptr || topk_idx == nullptr || grad_weights == nullptr || grad_logits == nullptr)
    return MOE_EINVAL;
  if (!aligned_elem(logits, bf16) || !aligned_elem(grad_logits, bf16) || !aligned4(topk_idx) ||
      !aligned4(grad_weights))
    return MOE_EINVAL;
  a.logits = logits;
  a.idx = const_cast<int32_t *>(topk_idx);
  a.gw = grad_weights;
  a.gl = grad_logits;
  a.err = err;
  return launch_gate(a, bf16, true, static_cast<cudaStream_t>(stream));
}
