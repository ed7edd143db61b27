// The router's choice: the top_k experts of every token from its E logits, and
// their weights.
//
//   key_e = logit_e, or (with a selection bias or expert groups)
//           sigmoid(logit_e) + bias_e in 64 bits
//   with groups: a group's score is the sum of its two largest keys; only the
//           experts of the topk_group best groups are eligible
//   ids   = the top_k eligible experts by key, largest first; equal keys and
//           equal group scores go to the lower index
//   w     = softmax (over all experts) or sigmoid of the chosen logits, in
//           fp32; optionally divided by their sum + 1e-20; times `scale`
//
// Experts whose logit or bias is -inf or NaN are never chosen; a token with fewer than
// top_k eligible experts gets ids of -1 with weight 0 behind the others.
// Biased scores are ordered in 64 bits because a choice between two close
// scores must not depend on how a 32-bit sigmoid is rounded.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace fp8bs {

namespace {

constexpr int kWarps = 4;   // rows per block, one warp each

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t M;
  int E, top_k, n_group, topk_group;
  int bf16, sigmoid, renorm;
  float scale;
};

// An order-preserving map of floating-point values onto unsigned integers.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 becomes +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | (1ull << 63));
}

// Largest key of the warp; every lane gets it.
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32);
  const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(top) << 32) | lo;
}

__device__ __forceinline__ float sigmoid32(float x) { return 1.0f / (1.0f + expf(-x)); }

// Lane l of a row's warp holds the experts l, l + 32, ... (kPer of them). A
// key of 0 stands for "not eligible": every ordered finite value is above it.
template <int kPer, bool kScore>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteArgs a) {
  using Key = typename std::conditional<kScore, uint64_t, uint32_t>::type;
  extern __shared__ double group_keys[];   // [kWarps][E], with groups only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  grid_dependency_wait();
  grid_launch_dependents();
  if (m >= a.M) return;
  const float ninf = __uint_as_float(0xFF800000u);
  float x[kPer];
  Key key[kPer];
  double* gk = group_keys + static_cast<int64_t>(warp) * a.E;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    x[i] = ninf;
    if (e < a.E)
      x[i] = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[m * a.E + e])
                    : static_cast<const float*>(a.logits)[m * a.E + e];
    const bool live = x[i] > ninf;   // false for NaN too
    if (!live) x[i] = ninf;
    if constexpr (kScore) {
      double k = 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
      if (a.bias != nullptr && e < a.E) k += static_cast<double>(a.bias[e]);
      key[i] = live && k > -HUGE_VAL ? ordered(k) : 0u;
      if (a.n_group > 1 && e < a.E) gk[e] = key[i] ? k : -HUGE_VAL;
    } else {
      key[i] = live ? ordered(x[i]) : 0u;
    }
  }
  if constexpr (kScore) {
    if (a.n_group > 1) {
      __syncwarp();
      // lane g scores group g (n_group <= 32)
      const int per = a.E / a.n_group;
      double first = -HUGE_VAL, second = -HUGE_VAL;
      if (lane < a.n_group) {
        for (int j = 0; j < per; ++j) {
          const double k = gk[lane * per + j];
          if (k > first) {
            second = first;
            first = k;
          } else if (k > second) {
            second = k;
          }
        }
      }
      const double total = second > -HUGE_VAL ? first + second : first;
      int ahead = 0;   // groups before this one in the order of the scores
      for (int g = 0; g < a.n_group; ++g) {
        const double other = __shfl_sync(0xffffffffu, total, g);
        ahead += (other > total || (other == total && g < lane)) ? 1 : 0;
      }
      const uint32_t open =
          __ballot_sync(0xffffffffu, lane < a.n_group && ahead < a.topk_group);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && !((open >> (e / per)) & 1u)) key[i] = 0u;
      }
    }
  }
  // softmax over all experts
  float top = ninf, sum = 0.0f;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = fmaxf(top, x[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (top > ninf) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += expf(x[i] - top);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  // top_k times the largest key left; lane j keeps choice j (top_k <= 32)
  int my_id = -1;
  float my_w = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    Key best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    }
    const Key all = warp_max(best);
    if (all == 0u) break;
    const uint32_t e = best == all ? static_cast<uint32_t>(lane + 32 * at) : 0xFFFFFFFFu;
    const uint32_t id = __reduce_min_sync(0xffffffffu, e);
    float xv = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (static_cast<uint32_t>(lane + 32 * i) == id) {
        key[i] = 0u;
        xv = x[i];
      }
    }
    xv = __shfl_sync(0xffffffffu, xv, static_cast<int>(id & 31u));
    if (lane == j) {
      my_id = static_cast<int>(id);
      my_w = a.sigmoid ? sigmoid32(xv) : expf(xv - top) / sum;
    }
  }
  if (a.renorm) {
    float total = my_w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    my_w = my_w / (total + 1e-20f);
  }
  if (lane < a.top_k) {
    a.ids[m * a.top_k + lane] = my_id;
    a.weights[m * a.top_k + lane] = my_w * a.scale;
  }
}

template <int kPer>
cudaError_t launch_route(const RouteArgs& a, bool score, cudaStream_t stream) {
  const int64_t blocks = (a.M + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  // at most 4 x 1024 x 8 bytes
  cfg.dynamicSmemBytes = a.n_group > 1 ? sizeof(double) * kWarps * static_cast<size_t>(a.E) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return score ? cudaLaunchKernelEx(&cfg, route_kernel<kPer, true>, a)
               : cudaLaunchKernelEx(&cfg, route_kernel<kPer, false>, a);
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, bool bf16, const float* bias, bool sigmoid,
                             int64_t M, int64_t E, int64_t top_k, int64_t n_group,
                             int64_t topk_group, bool renorm, float scale, int32_t* ids,
                             float* weights, cudaStream_t stream) {
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.M = M;
  a.E = static_cast<int>(E);
  a.top_k = static_cast<int>(top_k);
  a.n_group = static_cast<int>(n_group);
  a.topk_group = static_cast<int>(topk_group);
  a.bf16 = bf16;
  a.sigmoid = sigmoid;
  a.renorm = renorm;
  a.scale = scale;
  const bool score = bias != nullptr || n_group > 1;
  if (E <= 32) return launch_route<1>(a, score, stream);
  if (E <= 64) return launch_route<2>(a, score, stream);
  if (E <= 128) return launch_route<4>(a, score, stream);
  if (E <= 256) return launch_route<8>(a, score, stream);
  if (E <= 512) return launch_route<16>(a, score, stream);
  return launch_route<32>(a, score, stream);
}

}  // namespace fp8bs
