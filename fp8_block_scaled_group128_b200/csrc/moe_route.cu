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

constexpr int kWarps = 4;   // warps of a block where there are many rows

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t M;
  int E, top_k, n_group, topk_group;
  int bf16, sigmoid, renorm;
  int lg_lanes;   // log2 of the lanes that scan a group
  int per_inv;    // ceil(2^20 / experts of a group)
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

__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
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

// sigmoid(x) in double precision for -60 <= x <= 60 without a branch, so that
// the experts of a lane overlap (above 60 it is 1 to 2^-86): e^-x = 2^n e^r with
// r = -x - n ln 2 (ln 2 in two parts, Cody and Waite), e^r by its Taylor series
// to r^13 (|r| <= ln 2 / 2: the rest is below 2^-57), and 1 / (1 + e^-x) by two
// Newton steps from an fp32 reciprocal.
__device__ __forceinline__ double sigmoid64(double x) {
  const double magic = 6755399441055744.0;             // 1.5 * 2^52: rounds to an integer
  const double t = fma(-x, 1.4426950408889634, magic);
  const double n = t - magic;
  double r = fma(n, -6.93147180369123816490e-01, -x);
  r = fma(n, -1.90821492927058770002e-10, r);
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  const double e = __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
  const double d = 1.0 + e;
  double q = static_cast<double>(__frcp_rn(static_cast<float>(d)));
  q = fma(q, fma(-d, q, 1.0), q);
  return fma(q, fma(-d, q, 1.0), q);
}

// The same for x < -60: e^x (1 + e^x is 1 there, to 2^-86).
__device__ __noinline__ double sigmoid64_low(double x) { return exp(x); }

// A row belongs to blockDim.x threads, which leave the experts' keys in shared
// memory; the first of their warps chooses. Lane l of it answers for the experts
// l, l + 32, ... and keeps the best of them. A key of 0 stands for "not
// eligible": every ordered finite value is above it. The loops stay rolled: one
// row's time goes mostly into fetching code.
template <bool kScore>
__global__ void __launch_bounds__(1024) route_kernel(const RouteArgs a) {
  using Key = typename std::conditional<kScore, uint64_t, uint32_t>::type;
  extern __shared__ uint64_t smem[];   // [blockDim.y][E] keys
  const int lane = threadIdx.x & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  grid_dependency_wait();
  grid_launch_dependents();
  const bool live = m < a.M;
  const float ninf = __uint_as_float(0xFF800000u);
  const int E = a.E;
  Key* keys = reinterpret_cast<Key*>(smem) + threadIdx.y * E;
  const int64_t row = m * E;
  auto logit = [&](int e) {
    return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[row + e])
                  : static_cast<const float*>(a.logits)[row + e];
  };
  if (live) {
#pragma unroll 2
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      const float x = logit(e);
      const bool there = x > ninf;   // false for NaN too
      if constexpr (kScore) {
        double k = -HUGE_VAL;
        if (there) k = x >= -60.0f ? sigmoid64(fminf(x, 60.0f)) : sigmoid64_low(x);
        if (a.bias != nullptr) k += static_cast<double>(a.bias[e]);
        reinterpret_cast<double*>(keys)[e] = there && k > -HUGE_VAL ? k : -HUGE_VAL;
      } else {
        keys[e] = there ? ordered(x) : 0u;
      }
    }
  }
  if (blockDim.x > 32) {
    __syncthreads();
  } else {
    __syncwarp();
  }
  if (!live || threadIdx.x >= 32) return;
  uint32_t open = 0xffffffffu;   // a bit for each group
  if constexpr (kScore) {
    if (a.n_group > 1) {
      // a group's two largest keys: L lanes each scan a part of it, then join
      const double* gk = reinterpret_cast<const double*>(keys);
      const int per = E / a.n_group, L = 1 << a.lg_lanes;
      const int g = lane >> a.lg_lanes, part = lane & (L - 1);
      double first = -HUGE_VAL, second = -HUGE_VAL;
      if (g < a.n_group) {
#pragma unroll 2
        for (int j = part; j < per; j += L) {
          const double v = gk[g * per + j];
          const double low = v > first ? first : v;
          first = v > first ? v : first;
          second = low > second ? low : second;
        }
      }
#pragma unroll 1
      for (int off = 1; off < L; off <<= 1) {
        const double f = __shfl_xor_sync(0xffffffffu, first, off);
        const double s = __shfl_xor_sync(0xffffffffu, second, off);
        const double low = f > first ? first : f;
        first = f > first ? f : first;
        second = s > second ? s : second;
        second = low > second ? low : second;
      }
      const double total = second > -HUGE_VAL ? first + second : first;
      int ahead = 0;   // groups before this one in the order of the scores
#pragma unroll 2
      for (int o = 0; o < a.n_group; ++o) {
        const double other = __shfl_sync(0xffffffffu, total, o << a.lg_lanes);
        ahead += (other > total || (other == total && o < g)) ? 1 : 0;
      }
      // lane l answers for group l from here on
      const int ahead_l = __shfl_sync(0xffffffffu, ahead, (lane << a.lg_lanes) & 31);
      open = __ballot_sync(0xffffffffu, lane < a.n_group && ahead_l < a.topk_group);
    }
  }
  Key best = 0u;
  int best_e = 0;
#pragma unroll 2
  for (int e = lane; e < E; e += 32) {
    Key key;
    if constexpr (kScore) {
      const double k = reinterpret_cast<const double*>(keys)[e];
      const bool in = (open >> ((e * a.per_inv) >> 20)) & 1u;   // group e / (E / n_group)
      key = in && k > -HUGE_VAL ? ordered(k) : 0u;
      keys[e] = key;
    } else {
      key = keys[e];
    }
    if (key > best) {
      best = key;
      best_e = e;
    }
  }
  __syncwarp();
  // softmax over all experts (never with scores: the keys are the logits)
  float top = ninf, sum = 0.0f;
  if constexpr (!kScore) {
    if (!a.sigmoid) {
      const uint32_t t = __reduce_max_sync(0xffffffffu, best);
      top = t == 0u ? ninf : unordered(t);
#pragma unroll 2
      for (int e = lane; e < E; e += 32)
        if (keys[e] != 0u) sum += expf(unordered(keys[e]) - top);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
  }
  // top_k times the largest key left; lane j keeps choice j (top_k <= 32). The
  // whole warp looks for the next best key of the lane that lost one.
  int my_id = -1;
#pragma unroll 1
  for (int j = 0; j < a.top_k; ++j) {
    const Key all = warp_max(best);
    if (all == 0u) break;
    const int id = __reduce_min_sync(0xffffffffu, best == all ? best_e : 0x7FFFFFFF);
    if (lane == j) my_id = id;
    if (j == a.top_k - 1) break;
    const int e = (id & 31) + 32 * lane;
    const Key left = e != id && e < E ? keys[e] : 0u;
    if (e == id) keys[id] = 0u;   // only this lane reads it
    const Key next = warp_max(left);
    const int next_e = __reduce_min_sync(0xffffffffu, left == next ? e : 0x7FFFFFFF);
    if (lane == (id & 31)) {
      best = next;
      best_e = next_e;
    }
  }
  float my_w = 0.0f;
  if (my_id >= 0) {
    const float x = logit(my_id);
    my_w = a.sigmoid ? sigmoid32(x) : expf(x - top) / sum;
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

template <bool kScore>
cudaError_t launch_route(const RouteArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  // up to four rows an SM: a thread for each expert (one row of 256: 4.1 us, with a warp 6.9);
  // many: one or two warps for a row (4096 rows of 256: 11.1 us with two, 12.2 with
  // one, 13.5 with eight)
  const bool few = a.M <= 4 * dev.sm_count;
  const int T = few ? (a.E + 31) / 32 * 32 : a.E > 64 ? 64 : 32;
  const int R = few ? 1 : 32 * kWarps / T;
  const int64_t blocks = (a.M + R - 1) / R;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>(R), 1);
  // at most 2 x 1024 x 8 bytes (four rows have no more than 64 experts)
  cfg.dynamicSmemBytes = (kScore ? 8 : 4) * R * static_cast<size_t>(a.E);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_kernel<kScore>, a);
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, bool bf16, const float* bias, bool sigmoid,
                             int64_t M, int64_t E, int64_t top_k, int64_t n_group,
                             int64_t topk_group, bool renorm, float scale, int32_t* ids,
                             float* weights, const DeviceInfo& dev, cudaStream_t stream) {
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
  a.lg_lanes = 0;
  while ((2 << a.lg_lanes) * n_group <= 32) ++a.lg_lanes;
  const int per = static_cast<int>(E / n_group);
  a.per_inv = ((1 << 20) + per - 1) / per;   // exact quotients for e < 1024
  return bias != nullptr || n_group > 1 ? launch_route<true>(a, dev, stream)
                                        : launch_route<false>(a, dev, stream);
}

}  // namespace fp8bs
