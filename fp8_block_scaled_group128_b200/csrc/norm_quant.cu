// Residual addition, root-mean-square norm and 1x128 quantization in one pass
// over the rows: the input of a fine-grained FP8 linear (or of a mixture of
// experts) from the residual stream.
//
//   r[m][k] = bf16_rn(x[m][k] + res[m][k])         (x itself without a residual)
//   n[m][k] = r[m][k] * rstd[m] * w[k],  rstd[m] = 1 / sqrt(mean_k r[m][k]^2 + eps)
//   s[m][g] = max_{k in group g} |n[m][k]| / 448    (or its UE8M0 form)
//   q[m][k] = e4m3(n[m][k] / s[m][g]),  y[m][k] = bf16_rn(n[m][k])
//
// The norm is taken of the rounded r, the value that the residual stream
// keeps and later layers read. n stays in fp32: the codes are rounded once,
// from n, and not from the bf16 y.
//
// Bound: HBM. A row is read once and held in registers as bf16 between the sum
// of squares and the codes.
#include "common.cuh"
#include "e4m3_codec.cuh"
#include "kernels.h"

namespace fp8bs {

namespace {

struct NormArgs {
  const uint4* x;
  const uint4* res;      // null: no residual
  const uint4* w;        // null: ones
  uint4* res_out;        // may be null, or equal to x or res
  uint4* y;              // may be null
  uint2* q;
  void* s;               // fp32, or UE8M0 codes
  int64_t M;
  int chunks;            // K / 8
  float inv_k;           // 1 / K
  float eps;
};

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return bf16x2_of(__uint_as_float(a << 16) + __uint_as_float(b << 16),
                   __uint_as_float(a & 0xFFFF0000u) + __uint_as_float(b & 0xFFFF0000u));
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// A row belongs to blockDim.x threads (a multiple of 32); thread t holds the
// 16-byte chunks t, t + blockDim.x, ... (kV of them). 16 neighbouring threads
// hold one group of 128. A block has blockDim.y rows.
template <int kV, bool kE8>
__global__ void __launch_bounds__(1024) norm_quant_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int T = blockDim.x, t = threadIdx.x;
  const int lane = t & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = m < a.M;
  const int64_t base = m * a.chunks;
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 r[kV];
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * T + t;
    r[v] = make_uint4(0u, 0u, 0u, 0u);
    if (live && c < a.chunks) {
      r[v] = a.x[base + c];
      if (a.res != nullptr) {
        const uint4 b = a.res[base + c];
        r[v] = make_uint4(add_bf16x2(r[v].x, b.x), add_bf16x2(r[v].y, b.y),
                          add_bf16x2(r[v].z, b.z), add_bf16x2(r[v].w, b.w));
      }
      if (a.res_out != nullptr) a.res_out[base + c] = r[v];
    }
    float f[8];
    unpack8(r[v], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (T > 32) {
    const int warps = T >> 5;
    float* mine = red + threadIdx.y * warps;   // blockDim.x * blockDim.y <= 1024
    if (lane == 0) mine[t >> 5] = sum;
    __syncthreads();
    sum = lane < warps ? mine[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  const float rstd = __frsqrt_rn(fmaf(sum, a.inv_k, a.eps));
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * T + t;
    const bool on = live && c < a.chunks;
    float n[8], w[8];
    unpack8(r[v], n);
    if (a.w != nullptr && on) {
      unpack8(__ldg(a.w + c), w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    }
    // the magnitudes are compared as integers, so that a NaN is the largest
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = (n[i] * rstd) * w[i];
      mx = max(mx, __float_as_uint(n[i]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float amax = __uint_as_float(mx);
    uint2 q;
    if constexpr (kE8) {
      const uint32_t code = ue8m0_code_of_amax(amax);
      q = encode8f_pow2(n, ue8m0_inv_scale(code));
      if (on && (t & 15) == 0)
        static_cast<uint8_t*>(a.s)[(base + c) >> 4] = static_cast<uint8_t>(code);
    } else {
      const float sc = scale_of_amax(amax);
      q = encode8f(n, ScaleDivider(sc));
      if (on && (t & 15) == 0) static_cast<float*>(a.s)[(base + c) >> 4] = sc;
    }
    if (on) {
      a.q[base + c] = q;
      if (a.y != nullptr)
        a.y[base + c] = make_uint4(bf16x2_of(n[0], n[1]), bf16x2_of(n[2], n[3]),
                                   bf16x2_of(n[4], n[5]), bf16x2_of(n[6], n[7]));
    }
  }
}

template <bool kE8>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  // threads per row: one chunk each up to 1024 threads, then 2, 4 or 8 chunks
  int V = 1;
  while (V * 1024 < a.chunks) V *= 2;
  const int T = ((a.chunks + V - 1) / V + 31) / 32 * 32;
  const int R = T <= 128 ? 256 / T : 1;
  const int64_t blocks = (a.M + R - 1) / R;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>(R), 1);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  switch (V) {
    case 1: return cudaLaunchKernelEx(&cfg, norm_quant_kernel<1, kE8>, a);
    case 2: return cudaLaunchKernelEx(&cfg, norm_quant_kernel<2, kE8>, a);
    case 4: return cudaLaunchKernelEx(&cfg, norm_quant_kernel<4, kE8>, a);
    default: return cudaLaunchKernelEx(&cfg, norm_quant_kernel<8, kE8>, a);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm_quant(const void* x, const void* res, const void* w, float eps,
                                     int64_t M, int64_t K, void* res_out, void* y, void* q,
                                     void* s, bool ue8m0, cudaStream_t stream) {
  NormArgs a;
  a.x = static_cast<const uint4*>(x);
  a.res = static_cast<const uint4*>(res);
  a.w = static_cast<const uint4*>(w);
  a.res_out = static_cast<uint4*>(res_out);
  a.y = static_cast<uint4*>(y);
  a.q = static_cast<uint2*>(q);
  a.s = s;
  a.M = M;
  a.chunks = static_cast<int>(K / 8);
  a.inv_k = 1.0f / static_cast<float>(K);
  a.eps = eps;
  return ue8m0 ? launch_norm<true>(a, stream) : launch_norm<false>(a, stream);
}

}  // namespace fp8bs
