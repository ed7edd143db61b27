// The expert MLP of a mixture-of-experts layer for a few tokens.
//
//   for every token m and choice j with expert e = ids[m][j] - first_expert in
//   [0, E):
//     g, u = the block-scaled products of qa[m] with the gate rows [0, I) and
//            the up rows [I, 2I) of expert e (fp32)
//     h    = silu(g) * u, quantized in 1x128 groups (fp32 h, rounded once)
//     d_j  = the block-scaled product of h's codes with expert e's down rows
//   y[m] = bf16_rn(sum_j weights[m][j] * d_j)
#include "common.cuh"
#include "e4m3_codec.cuh"
#include "kernels.h"

namespace fp8bs {

namespace {

__device__ __forceinline__ float scale_at(const void* s, int64_t i, bool e8) {
  if (!e8) return static_cast<const float*>(s)[i];
  const uint32_t c = static_cast<const uint8_t*>(s)[i];
  return c == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(c << 23);
}

__device__ __forceinline__ float dot4(uint32_t a, uint32_t b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_fp8_e4m3 x, y;
    x.__x = static_cast<uint8_t>(a >> (8 * i));
    y.__x = static_cast<uint8_t>(b >> (8 * i));
    s = fmaf(static_cast<float>(x), static_cast<float>(y), s);
  }
  return s;
}

// One warp's block-scaled dot product of a row of codes with a weight row.
__device__ float row_dot(const uint8_t* a, const void* sa, int64_t sa0, const uint8_t* w,
                         const void* sw, int64_t sw0, int KB, bool e8) {
  const int lane = threadIdx.x & 31;
  float acc = 0.0f;
  for (int kb = 0; kb < KB; ++kb) {
    const float s = scale_at(sa, sa0 + kb, e8) * scale_at(sw, sw0 + kb, e8);
    acc = fmaf(s,
               dot4(reinterpret_cast<const uint32_t*>(a)[kb * 32 + lane],
                    reinterpret_cast<const uint32_t*>(w)[kb * 32 + lane]),
               acc);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  return acc;
}

// Block (group of 128 intermediate columns, pair): h's codes and scale.
__global__ void __launch_bounds__(256) moe_gate_up_kernel(MoeArgs a, uint8_t* qh, void* sh,
                                                          bool e8) {
  __shared__ float hs[128];
  const int pair = blockIdx.y, m = pair / a.top_k, grp = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int e = a.ids[pair] - a.first_expert;
  if (e < 0 || e >= a.E) return;
  const int KB = a.K / 128, IB = a.I / 128;
  const uint8_t* row = a.qa + static_cast<int64_t>(m) * a.K;
  for (int c = warp; c < 128; c += 8) {
    const int64_t n = static_cast<int64_t>(e) * 2 * a.I + grp * 128 + c;
    const int64_t s0 = (static_cast<int64_t>(e) * 2 * IB + grp) * KB;
    const float g = row_dot(row, a.sa, static_cast<int64_t>(m) * KB, a.qg + n * a.K, a.sg, s0, KB, e8);
    const float u = row_dot(row, a.sa, static_cast<int64_t>(m) * KB, a.qg + (n + a.I) * a.K, a.sg,
                            s0 + static_cast<int64_t>(IB) * KB, KB, e8);
    if (lane == 0) hs[c] = silu_f32(g) * u;
  }
  __syncthreads();
  if (warp != 0) return;
  uint32_t mx = 0u;
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = hs[4 * lane + i];
    mx = max(mx, __float_as_uint(h[i]) & 0x7FFFFFFFu);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  const float amax = __uint_as_float(mx);
  const int64_t at = static_cast<int64_t>(pair) * IB + grp;
  uint32_t q;
  if (e8) {
    const uint32_t code = ue8m0_code_of_amax(amax);
    q = codes4f_pow2(h[0], h[1], h[2], h[3], ue8m0_inv_scale(code));
    if (lane == 0) static_cast<uint8_t*>(sh)[at] = static_cast<uint8_t>(code);
  } else {
    const float sc = scale_of_amax(amax);
    q = codes4f(h[0], h[1], h[2], h[3], ScaleDivider(sc));
    if (lane == 0) static_cast<float*>(sh)[at] = sc;
  }
  reinterpret_cast<uint32_t*>(qh)[at * 32 + lane] = q;
}

// Block (128 output columns, token): the weighted sum of the down products.
__global__ void __launch_bounds__(256) moe_down_kernel(MoeArgs a, const uint8_t* qh,
                                                       const void* sh, bool e8) {
  const int m = blockIdx.y, nb = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int KB = a.K / 128, IB = a.I / 128;
  for (int c = warp; c < 128; c += 8) {
    float y = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t pair = static_cast<int64_t>(m) * a.top_k + j;
      const int e = a.ids[pair] - a.first_expert;
      if (e < 0 || e >= a.E) continue;
      const int64_t n = static_cast<int64_t>(e) * a.K + nb * 128 + c;
      const float d = row_dot(qh + pair * a.I, sh, pair * IB, a.qd + n * a.I, a.sd,
                              (static_cast<int64_t>(e) * KB + nb) * IB, IB, e8);
      y = fmaf(a.weights[pair], d, y);
    }
    if (lane == 0) a.y[static_cast<int64_t>(m) * a.K + nb * 128 + c] = __float2bfloat16_rn(y);
  }
}

}  // namespace

size_t moe_workspace_bytes(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  (void)K;
  (void)E;
  const size_t pairs = static_cast<size_t>(M) * static_cast<size_t>(top_k);
  return (pairs * I + 255) / 256 * 256 + pairs * (I / 128) * 4;
}

int launch_moe_mlp(const MoeArgs& a, bool ue8m0, cudaStream_t stream) {
  uint8_t* qh = static_cast<uint8_t*>(a.workspace);
  const size_t pairs = static_cast<size_t>(a.M) * a.top_k;
  void* sh = qh + (pairs * a.I + 255) / 256 * 256;
  moe_gate_up_kernel<<<dim3(a.I / 128, static_cast<unsigned>(pairs)), 256, 0, stream>>>(a, qh, sh,
                                                                                       ue8m0);
  moe_down_kernel<<<dim3(a.K / 128, a.M), 256, 0, stream>>>(a, qh, sh, ue8m0);
  return cudaGetLastError() == cudaSuccess ? FP8BS_OK : FP8BS_ERR_CUDA;
}

}  // namespace fp8bs
