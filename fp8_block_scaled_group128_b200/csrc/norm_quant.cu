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
// Bound: HBM; a row is read once. Few rows are held in registers (as bf16)
// between the sum of squares and the codes, with as many threads as a row has
// chunks: one row of 4096 2.1 us, 64 rows of 7168 3.3 us (in a graph). Rows above
// 32768 keep eight chunks a thread and spill some (16 rows of 65536 16.7 us). Many
// rows go through shared memory (norm_row_kernel).
#include <mutex>

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

// The same in one instruction: rounding the sum at once gives the same value
// (two bf16 values' sum is exact in fp32 unless the smaller one is too small to
// move the larger).
__device__ __forceinline__ uint32_t hadd_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest magnitude, NaN if one is.
__device__ __forceinline__ float absmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float absmax_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes of eight values for a scale: x * (1 / s). The hardware's reciprocal r0 =
// (1 + d) / s has |d| <= 2^-23 (one ulp); a Newton step leaves d^2 and one
// rounding, together below 2^-23.99 relative. A quotient of mantissa m < 2 is then
// off by m / 2 ulps from 1 / s and half an ulp from the product, below 1.6 in all
// (without the step m + 1/2, up to 2.5; it costs nothing measurable). For scales
// whose reciprocal is not a normal number, zero and NaN the IEEE quotients.
__device__ __forceinline__ uint2 encode8_by_reciprocal(const float (&x)[8], float s) {
  if (!(s >= 7.88860905e-31f)) return encode8f(x, ScaleDivider(s));   // 2^-100
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = fmaf(inv, fmaf(-s, inv, 1.0f), inv);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) mul2(q[i], q[i + 1], x[i], x[i + 1], inv, inv);
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(q[4], q[5]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t d = __nv_cvt_float2_to_fp8x2(make_float2(q[6], q[7]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(prmt(a, b, 0x5410u), prmt(c, d, 0x5410u));
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// rstd is taken from the fp32 sum of squares where the mean + eps is in this
// range: then no sum can have overflowed, and squares too small for fp32 are
// below 2^-48 of the mean.
constexpr float kMeanLow = 7.88860905e-31f;   // 2^-100
constexpr float kMeanHigh = 3.402823466e38f;
constexpr float kSmallScale = 1.2089258196146292e+24f;   // 2^80

// Elsewhere (NaN too) every warp of the row takes the sum again from global
// memory, in double precision, in which bf16 squares are exact and cannot leave
// the range. rstd of a row of bf16 subnormals is beyond fp32: with `small` it is
// that of the row times 2^80, by which each thread then multiplies its values
// (exactly, in bf16 too). A mean above 2^252 gives an rstd with two bits less.
// The two comparisons cost ordinary calls 0.07 us (one row of 4096: 2.24 us in a
// graph) and up to 2.5% (1037 rows of 14336, UE8M0: 14.9 us).
__device__ __forceinline__ float rstd_of_extreme_row(const NormArgs& a, int64_t base, int chunks,
                                                     bool& small) {
  const bool kept = a.res_out != nullptr;   // x and res may have been overwritten with it
  const uint4* r = (kept ? a.res_out : a.x) + base;
  __syncwarp();
  double sum = 0.0;
#pragma unroll 1
  for (int c = threadIdx.x & 31; c < chunks; c += 32) {
    uint4 v = r[c];
    if (!kept && a.res != nullptr) {
      const uint4 b = a.res[base + c];
      v = make_uint4(add_bf16x2(v.x, b.x), add_bf16x2(v.y, b.y), add_bf16x2(v.z, b.z),
                     add_bf16x2(v.w, b.w));
    }
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = f[i];
      sum = fma(d, d, sum);
    }
  }
#pragma unroll 1
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const double mean = fma(sum, static_cast<double>(a.inv_k), static_cast<double>(a.eps));
  small = mean < 1.0;
  const double square = small ? 1.461501637330903e+48 : 6.842277657836021e-49;   // 2^160, 2^-160
  const float rstd = __frsqrt_rn(static_cast<float>(mean * square));
  return small ? rstd : rstd * 8.271806125530277e-25f;   // 2^-80
}

__device__ __forceinline__ uint4 scaled8(const uint4 v) {
  float f[8];
  unpack8(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= kSmallScale;
  return make_uint4(bf16x2_of(f[0], f[1]), bf16x2_of(f[2], f[3]), bf16x2_of(f[4], f[5]),
                    bf16x2_of(f[6], f[7]));
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
  const float mean = fmaf(sum, a.inv_k, a.eps);
  float rstd = __frsqrt_rn(mean);
  bool small = false;
  if (!(mean >= kMeanLow && mean <= kMeanHigh))   // the same in all threads of a row
    rstd = rstd_of_extreme_row(a, base, live ? a.chunks : 0, small);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * T + t;
    const bool on = live && c < a.chunks;
    float n[8], w[8];
    unpack8(r[v], n);
    if (small) {
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] *= kSmallScale;
    }
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
      const uint32_t code = ue8m0_code_or_nan(amax);
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

// ------------------------------------------------------------- many rows --
// A block per row (or several short ones), the row in shared memory: one bulk
// copy brings it, the first pass adds the residual and the squares, the second
// makes the codes. A thread's registers hold one 16-byte chunk at a time, so
// that enough blocks are resident to keep HBM busy while others compute.
//
// 8192 rows of 4096 with residual and y: 49.3 to 50.6 us, 92 to 93% of the copy
// bandwidth (in registers: 53.7), 47.2 in a graph (UE8M0 47.4); 1037 rows of
// 14336, codes only: 15.4 us (in registers: 24.2; UE8M0 14.8), bound by
// instructions there, 22 for an element; 2048 rows of 7168: 24.5 in a graph. A
// persistent kernel whose teams of warps held their rows in registers behind a
// ring of bulk copies took 59, 19.5 and 27 us.
constexpr int kRowSmem = 100 * 1024;   // at least two blocks per SM
constexpr int kRowThreads = 512;

struct RowArgs {
  NormArgs n;
  long long wait_limit;
  int* err;
};

template <bool kE8, bool kRes>
__global__ void __launch_bounds__(kRowThreads) norm_row_kernel(const RowArgs a) {
  extern __shared__ __align__(128) uint8_t rows_smem[];
  __shared__ uint64_t full;
  __shared__ float red[32];
  const int T = blockDim.x, t = threadIdx.x, lane = t & 31;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * blockDim.y;
  const int rows = static_cast<int>(min(static_cast<int64_t>(blockDim.y), a.n.M - m0));
  const bool first = t == 0 && threadIdx.y == 0;
  if (first) {
    mbar_init(&full, 1);
    fence_mbarrier_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (first) {
    const uint32_t bytes = static_cast<uint32_t>(rows * a.n.chunks * 16);
    mbar_arrive_expect_tx(&full, kRes ? 2 * bytes : bytes);
    bulk_load(rows_smem, a.n.x + m0 * a.n.chunks, bytes, &full);
    if constexpr (kRes)
      bulk_load(rows_smem + blockDim.y * a.n.chunks * 16, a.n.res + m0 * a.n.chunks, bytes, &full);
  }
  // one warp polls for all: the others' polls would take half of the issue slots
  const bool polls = t < 32 && threadIdx.y == 0;
  __syncwarp();
  if (!__syncthreads_and(!polls || mbar_wait(&full, 0, a.wait_limit))) {
    if (first) {
      record_device_error(a.err, FP8BS_ERR_DEVICE_TIMEOUT);
      mbar_wait(&full, 0, kDefaultWaitCycles);   // the copy must have landed before the exit
    }
    return;
  }
  const int y = threadIdx.y;
  const bool live = y < rows;
  const int chunks = live ? a.n.chunks : 0;
  const int64_t base = (m0 + y) * a.n.chunks;
  uint4* row = reinterpret_cast<uint4*>(rows_smem) + y * a.n.chunks;
  const uint4* res = row + blockDim.y * a.n.chunks;
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
  for (int c = t; c < chunks; c += T) {
    uint4 r = row[c];
    if constexpr (kRes) {
      const uint4 b = res[c];
      r = make_uint4(hadd_bf16x2(r.x, b.x), hadd_bf16x2(r.y, b.y), hadd_bf16x2(r.z, b.z),
                     hadd_bf16x2(r.w, b.w));
      row[c] = r;
    }
    if (a.n.res_out != nullptr) a.n.res_out[base + c] = r;
    float f[8];
    unpack8(r, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) fma2(s0, s1, f[i], f[i + 1], f[i], f[i + 1]);
  }
  float sum = s0 + s1;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (T > 32) {
    const int warps = T >> 5;
    float* mine = red + y * warps;
    if (lane == 0) mine[t >> 5] = sum;
    __syncthreads();
    sum = lane < warps ? mine[lane] : 0.0f;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    sum = __shfl_sync(0xffffffffu, sum, 0);
  }
  const float mean = fmaf(sum, a.n.inv_k, a.n.eps);
  float rstd = __frsqrt_rn(mean);
  if (!(mean >= kMeanLow && mean <= kMeanHigh)) {   // the same in all threads of a row
    bool small;
    rstd = rstd_of_extreme_row(a.n, base, chunks, small);
    if (small) {
#pragma unroll 1
      for (int c = t; c < chunks; c += T) row[c] = scaled8(row[c]);
    }
  }
  // a thread reads the chunks that it wrote; T is a multiple of 16, so that 16
  // neighbouring threads have a group of 128 (all or none of them)
#pragma unroll 1
  for (int c = t; c < (chunks + 31) / 32 * 32; c += T) {
    const bool on = c < chunks;
    float n[8], w[8];
    unpack8(on ? row[c] : make_uint4(0u, 0u, 0u, 0u), n);
    uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (a.n.w != nullptr && on) wv = __ldg(a.n.w + c);
    unpack8(wv, w);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      mul2(n[i], n[i + 1], n[i], n[i + 1], rstd, rstd);
      mul2(n[i], n[i + 1], n[i], n[i + 1], w[i], w[i + 1]);
    }
    if (on && a.n.y != nullptr)
      a.n.y[base + c] = make_uint4(bf16x2_of(n[0], n[1]), bf16x2_of(n[2], n[3]),
                                   bf16x2_of(n[4], n[5]), bf16x2_of(n[6], n[7]));
    float mx = absmax_nan(absmax_nan(n[0], n[1], n[2]), absmax_nan(n[3], n[4], n[5]),
                          absmax_nan(n[6], n[7]));
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1)
      mx = absmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    uint2 q;
    if constexpr (kE8) {
      const uint32_t code = ue8m0_code_or_nan(mx);
      q = encode8f_pow2(n, ue8m0_inv_scale(code));
      if (on && (t & 15) == 0)
        static_cast<uint8_t*>(a.n.s)[(base + c) >> 4] = static_cast<uint8_t>(code);
    } else {
      const float sc = scale_of_amax(mx);
      q = encode8_by_reciprocal(n, sc);
      if (on && (t & 15) == 0) static_cast<float*>(a.n.s)[(base + c) >> 4] = sc;
    }
    if (on) a.n.q[base + c] = q;
  }
}

template <bool kE8, bool kRes>
cudaError_t launch_rows(const RowArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = norm_row_kernel<kE8, kRes>;
  static std::once_flag flags[64];
  cudaError_t attr_err = cudaSuccess;
  std::call_once(flags[dev.device], [&] {
    attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
  });
  if (attr_err != cudaSuccess) return attr_err;
  // two chunks for a thread (8192 rows of 4096: 49.3 us, with four 51.1)
  int T = ((a.n.chunks + 1) / 2 + 31) / 32 * 32;
  if (T > kRowThreads) T = kRowThreads;
  const int R = T >= 128 ? 1 : 128 / T;
  const int64_t blocks = (a.n.M + R - 1) / R;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>(R), 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(R) * a.n.chunks * (kRes ? 32 : 16);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
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
                                     void* s, bool ue8m0, const DeviceInfo& dev,
                                     long long wait_limit, int* err, cudaStream_t stream) {
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
  // more rows than SMs: the rows' latency no longer decides (150 rows of 7168: 4.6 us
  // either way)
  const bool many = K * (res != nullptr ? 4 : 2) <= kRowSmem && M > dev.sm_count;
  if (many) {
    const RowArgs rows{a, wait_limit, err};
    if (res != nullptr)
      return ue8m0 ? launch_rows<true, true>(rows, dev, stream)
                   : launch_rows<false, true>(rows, dev, stream);
    return ue8m0 ? launch_rows<true, false>(rows, dev, stream)
                 : launch_rows<false, false>(rows, dev, stream);
  }
  return ue8m0 ? launch_norm<true>(a, stream) : launch_norm<false>(a, stream);
}

}  // namespace fp8bs
