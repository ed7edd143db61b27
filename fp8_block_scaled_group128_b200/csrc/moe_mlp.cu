// The expert MLP of a mixture-of-experts layer for a few tokens.
//
//   for every token m and choice j with expert e = ids[m][j] - first_expert in
//   [0, E):
//     g, u = the block-scaled products of qa[m] with the gate rows [0, I) and
//            the up rows [I, 2I) of expert e (fp32)
//     h    = silu(g) * u, quantized in 1x128 groups (fp32 h, rounded once)
//     d_j  = the block-scaled product of h's codes with expert e's down rows
//   y[m] = bf16_rn(sum_j weights[m][j] * d_j)
//
// Bound: HBM. Every chosen expert's 3 I K weight bytes are read once, whatever
// the number of its tokens; at the copy bandwidth an SM gets a 128 x 128 tile
// (16 KB) every ~700 cycles, and both the MMAs and the promotion of a tile
// take less than that for up to 128 tokens.
//
// Three launches, chained by programmatic dependent launch:
//
//   moe_plan_kernel     one block: the chosen experts in order, each with its
//                       list of tokens ("rows"), and the join counters zeroed
//   moe_gemm_kernel<gate+up>  h's codes and scales, per row
//   moe_gemm_kernel<down>     y
//
// Both GEMMs put 128 weight rows on the MMA's M side and an expert's tokens on
// its N side (16 to 128, the expert's own count rounded up to 16). Their work
// is a list of units, one 128-deep K-block of a tile each (gate and up of 128
// intermediate columns; 128 output columns of one expert), in an order that
// puts the units of a result next to each other. The list is cut into equal
// contiguous ranges, one per CTA, so that every SM reads the same number of
// weight bytes however many experts were chosen; a result whose units fall
// into several CTAs is joined by the last of them to finish, which adds the
// fp32 partial results in the order of the CTAs (the same bytes every call; no
// CTA waits for another).
//
//   warp 0        TMA producer: weight tiles and the tokens' K-block
//   warp 1        MMA issuer: 4 (x 2) tcgen05.mma of K = 32 per unit into one
//                 of the TMEM buffers
//   warp 2        scale products sA * sW of 8 units at a time, into shared
//                 memory
//   warps 4..11   two promotion warpgroups, each half of the token columns:
//                 TMEM -> registers times the scale products; at the end of a
//                 tile SwiGLU and quantization, or the weighted sum over the
//                 experts in shared memory
//
// Every wait is bounded as in gemm_kernel.cuh.
#include <mutex>

#include "common.cuh"
#include "e4m3_codec.cuh"
#include "kernels.h"

namespace fp8bs {

namespace {

constexpr int kMaxCtas = 160;      // grid bound behind the workspace size
constexpr int kPlanThreads = 1024;
constexpr int kBatch = 8;          // units per batch of scale products
constexpr int kThreads = 384;
constexpr int kPromo = 256;        // promotion threads

// What the plan kernel leaves for the GEMMs.
struct Plan {
  int* n_act;        // number of chosen experts
  int2* act;         // [n_act + 1]: (expert, its first row); the last entry ends the rows
  int* row_tok;      // [rows] token of a row
  float* row_w;      // [rows] weight of the row's token for its expert
  int* count_gu;     // [n_act * I / 128] join counters of the gate+up tiles
  int* count_down;   // [K / 128] join counters of the down tiles
};

struct Workspace {
  Plan plan;
  uint8_t* qh;       // [rows][I]
  void* sh;          // [rows][I / 128]
  float* partial;    // [2 kMaxCtas][M][256] (gate+up) or [2 kMaxCtas][M][128] (down)
  size_t bytes;
};

Workspace carve(void* base, int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  const size_t rows = static_cast<size_t>(M * top_k);
  const size_t act = static_cast<size_t>(E < M * top_k ? E : M * top_k);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  Workspace w;
  w.plan.n_act = reinterpret_cast<int*>(take(4));
  w.plan.act = reinterpret_cast<int2*>(take((act + 1) * 8));
  w.plan.row_tok = reinterpret_cast<int*>(take(rows * 4));
  w.plan.row_w = reinterpret_cast<float*>(take(rows * 4));
  w.plan.count_gu = reinterpret_cast<int*>(take(act * (I / 128) * 4));
  w.plan.count_down = reinterpret_cast<int*>(take(K / 128 * 4));
  w.qh = take(rows * I);
  w.sh = take(rows * (I / 128) * 4);
  w.partial = reinterpret_cast<float*>(take(static_cast<size_t>(2 * kMaxCtas) * M * 256 * 4));
  w.bytes = at;
  return w;
}

// -------------------------------------------------------------------- plan --
// A choice counts once per token and expert: of a token's choices of the same
// expert the first one makes the row and carries the sum of their weights (in
// the order of the choices). The order of an expert's rows comes from atomics
// and may differ from call to call; nothing computed depends on it.
__global__ void __launch_bounds__(kPlanThreads)
    moe_plan_kernel(const int32_t* __restrict__ ids, const float* __restrict__ weights, int pairs,
                    int top_k, int E, int first_expert, int n_gu, int n_down, Plan plan) {
  __shared__ int expert[kMoeMaxM * kMoeMaxTopK];   // local expert of a choice, -1: none
  __shared__ int fill[kMoeMaxE];                   // next row of an expert
  __shared__ uint32_t warp_sum[kPlanThreads / 32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  fill[t] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = t; i < pairs; i += kPlanThreads) {
    const int64_t e = static_cast<int64_t>(ids[i]) - first_expert;
    expert[i] = e >= 0 && e < E ? static_cast<int>(e) : -1;
  }
  for (int i = t; i < n_gu; i += kPlanThreads) plan.count_gu[i] = 0;
  for (int i = t; i < n_down; i += kPlanThreads) plan.count_down[i] = 0;
  __syncthreads();
  auto is_row = [&](int i) {   // the token's first choice of this expert
    if (expert[i] < 0) return false;
    for (int j = i / top_k * top_k; j < i; ++j)
      if (expert[j] == expert[i]) return false;
    return true;
  };
  for (int i = t; i < pairs; i += kPlanThreads)
    if (is_row(i)) atomicAdd(&fill[expert[i]], 1);
  __syncthreads();
  // exclusive prefix over the experts of (chosen experts << 16 | rows): at
  // most 1024 experts and 4096 rows
  const uint32_t mine = fill[t] > 0 ? (1u << 16) | static_cast<uint32_t>(fill[t]) : 0u;
  uint32_t scan = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += o;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  uint32_t before = 0u, total = 0u;
  {
    const uint32_t s = warp_sum[lane];
    total = __reduce_add_sync(0xffffffffu, s);
    before = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u);
  }
  const uint32_t excl = before + scan - mine;
  if (mine != 0u) plan.act[excl >> 16] = make_int2(t, static_cast<int>(excl & 0xFFFFu));
  fill[t] = static_cast<int>(excl & 0xFFFFu);
  if (t == 0) {
    *plan.n_act = static_cast<int>(total >> 16);
    plan.act[total >> 16] = make_int2(-1, static_cast<int>(total & 0xFFFFu));
  }
  __syncthreads();
  for (int i = t; i < pairs; i += kPlanThreads) {
    if (!is_row(i)) continue;
    const int end = i / top_k * top_k + top_k;
    float w = weights[i];
    for (int j = i + 1; j < end; ++j)
      if (expert[j] == expert[i]) w += weights[j];
    const int row = atomicAdd(&fill[expert[i]], 1);
    plan.row_tok[row] = i / top_k;
    plan.row_w[row] = w;
  }
}

// ------------------------------------------------------------------- GEMMs --
struct GemmMoeArgs {
  Plan plan;
  const void* sx;    // scales of the token operand: sa [M][K/128], or sh [rows][I/128]
  const void* sw;    // weight scales: [E][2I/128][K/128], or [E][K/128][I/128]
  uint8_t* qh;       // gate+up: the codes of h [rows][I]
  void* sh;          // gate+up: their scales [rows][I/128]
  __nv_bfloat16* y;  // down: [M][K]
  float* partial;
  int M, K, I;
  long long wait_limit;
  int* err;
};

__device__ __forceinline__ float scale_value(const void* s, int64_t i, bool e8) {
  if (!e8) return static_cast<const float*>(s)[i];
  const uint32_t c = static_cast<const uint8_t*>(s)[i];
  return c == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(c << 23);
}

template <int kN, bool kDown>
struct MoeCfg {
  static_assert(kN == 16 || kN == 32 || kN == 64 || kN == 128, "token columns");
  static constexpr int kParts = kDown ? 1 : 2;             // weight tiles per unit
  static constexpr int kWBytes = kParts * 128 * 128;
  static constexpr int kXBytes = kN * 128;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kBufCols = kParts * kN;             // TMEM columns of a unit
  static constexpr int kBufs = 512 / kBufCols < 8 ? 512 / kBufCols : 8;
  static constexpr int kTmemCols =
      kBufs * kBufCols <= 128 ? 128 : kBufs * kBufCols <= 256 ? 256 : 512;
  // scale products: [2 batches][kBatch][kParts][kN], a unit's row padded
  static constexpr int kRow = kParts * kN + 4;
  static constexpr int kTabBytes = 2 * kBatch * kRow * 4;
  // end of a tile: gate+up: codes [kN][128] and warp maxima [kN][4];
  // down: the fp32 sums [kN tokens][128]
  static constexpr int kEndBytes = kDown ? kN * 128 * 4 : kN * 128 + kN * 16;
  static constexpr int kActBytes = (static_cast<int>(kMoeMaxE) + 1) * 8;
  static constexpr int kFixed = kTabBytes + kEndBytes + kActBytes + 1024 /* barriers */ + 1024;
  static constexpr int kFit = (227 * 1024 - kFixed) / kStageBytes;
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static_assert(kStages >= 3, "at least three stages");
  static constexpr int kOffX = kStages * kWBytes;
  static constexpr int kOffTab = kOffX + kStages * kXBytes;
  static constexpr int kOffEnd = kOffTab + kTabBytes;
  static constexpr int kOffAct = kOffEnd + kEndBytes;
  static constexpr int kOffBar = kOffAct + (kActBytes + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 4 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr int kHalf = kN / 2;                     // columns of a promotion thread, at most
};

// The unit list of one launch and this CTA's range of it. A tile is one result
// (gate+up: expert and group of 128 intermediate columns; down: 128 output
// columns, over all experts); a segment is the part of it that is walked with
// one set of token rows.
struct Range {
  int64_t begin, end, units;
  int ctas;   // CTAs that have work: each has at least one unit
  __device__ __forceinline__ Range(int64_t u, int grid, int cta) : units(u) {
    ctas = u < grid ? static_cast<int>(u) : grid;
    begin = cta < ctas ? u * cta / ctas : u;
    end = cta < ctas ? u * (cta + 1) / ctas : u;
  }
  __device__ __forceinline__ int owner(int64_t unit) const {
    return static_cast<int>(((unit + 1) * ctas - 1) / units);
  }
  __device__ __forceinline__ int64_t begin_of(int cta) const { return units * cta / ctas; }
};

template <int kN, bool kDown, bool kE8>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w,
                    const __grid_constant__ CUtensorMap tmap_x, const GemmMoeArgs args) {
  using C = MoeCfg<kN, kDown>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sm_w = smem;
  uint8_t* sm_x = smem + C::kOffX;
  float* tab = reinterpret_cast<float*>(smem + C::kOffTab);
  int2* act = reinterpret_cast<int2*>(smem + C::kOffAct);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kBufs;
  uint64_t* sfull = tempty + C::kBufs;
  uint64_t* sempty = sfull + 2;
  uint64_t* mma_done = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = args.wait_limit;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kPromo / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], kPromo / 32);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int n_act = __ldcg(args.plan.n_act);
  for (int i = threadIdx.x; i <= n_act; i += kThreads) act[i] = __ldcg(args.plan.act + i);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int IB = args.I / 128, KB = args.K / 128;
  const int depth = kDown ? IB : KB;                   // units of a segment
  const int tile_units = kDown ? n_act * IB : KB;      // units of a tile
  const Range range(static_cast<int64_t>(kDown ? KB : IB) * n_act * depth,
                    static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x));
  // segment s: expert index and tile coordinate
  auto seg_act = [&](int64_t s) { return static_cast<int>(kDown ? s % n_act : s / IB); };
  auto seg_tile = [&](int64_t s) { return static_cast<int>(kDown ? s / n_act : s % IB); };

  auto stopped = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer --
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (int64_t u = range.begin; u < range.end && !stopped();) {
      const int64_t s = u / depth;
      const int k0 = static_cast<int>(u - s * depth);
      const int k1 = static_cast<int>(min(static_cast<int64_t>(depth), k0 + range.end - u));
      const int a = seg_act(s), tile = seg_tile(s);
      const int e = act[a].x, row0 = act[a].y, n = act[a + 1].y - row0;
      const int wrow = kDown ? e * args.K + tile * 128 : e * 2 * args.I + tile * 128;
      int tok[4] = {0, 0, 0, 0};
      const int n4 = (n + 3) / 4, n16 = (n + 15) / 16;
      if (!kDown && lane < n4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tok[q] = args.plan.row_tok[row0 + min(4 * lane + q, n - 1)];
      }
      const uint32_t bytes = C::kWBytes + (kDown ? n16 * 2048 : n4 * 512);
      for (int k = k0; k < k1; ++k) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, limit)) {
          if (lane == 0) record_device_error(args.err, FP8BS_ERR_DEVICE_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        uint8_t* w = sm_w + stage * C::kWBytes;
        uint8_t* x = sm_x + stage * C::kXBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], bytes);
          tma_load_2d(w, &tmap_w, &full[stage], k * 128, wrow);
          if constexpr (!kDown) tma_load_2d(w + 16384, &tmap_w, &full[stage], k * 128, wrow + args.I);
          if constexpr (kDown) {
            for (int i = 0; i < n16; ++i)
              tma_load_2d(x + i * 2048, &tmap_x, &full[stage], k * 128, row0 + i * 16);
          }
        }
        __syncwarp();
        if (!kDown && lane < n4)
          tma_gather4_2d(x + lane * 512, &tmap_x, &full[stage], k * 128, tok[0], tok[1], tok[2],
                         tok[3]);
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      u += k1 - k0;
    }
    // every copy issued must have landed before the CTA exits
    const int pending = issued < C::kStages ? issued : C::kStages;
    for (int i = 0; i < pending; ++i) {
      int st = stage - 1 - i;
      uint32_t ph = phase;
      if (st < 0) {
        st += C::kStages;
        ph ^= 1u;
      }
      mbar_wait(&full[st], ph, kDefaultWaitCycles);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    int stage = 0, tb = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    const uint64_t dw0 = sw128_kmajor_desc(smem_u32(sm_w));
    const uint64_t dx0 = sw128_kmajor_desc(smem_u32(sm_x));
    for (int64_t u = range.begin; ok && u < range.end && !stopped();) {
      const int64_t s = u / depth;
      const int k0 = static_cast<int>(u - s * depth);
      const int k1 = static_cast<int>(min(static_cast<int64_t>(depth), k0 + range.end - u));
      const int a = seg_act(s);
      const int n = act[a + 1].y - act[a].y;
      const uint32_t idesc = idesc_e4m3_f32(128, (n + 15) / 16 * 16);
      for (int k = k0; ok && k < k1; ++k) {
        if (!mbar_wait_warp(&full[stage], phase, limit) ||
            !mbar_wait_warp(&tempty[tb], tphase ^ 1u, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dw = dw0 + static_cast<uint32_t>((stage * C::kWBytes) >> 4);
        const uint64_t dx = dx0 + static_cast<uint32_t>((stage * C::kXBytes) >> 4);
        const uint32_t d = tmem_base + static_cast<uint32_t>(tb * C::kBufCols);
        if (elect_one()) {
#pragma unroll
          for (int p = 0; p < C::kParts; ++p) {
            const uint64_t dp = dw + static_cast<uint32_t>((p * 16384) >> 4);
            const uint32_t dd = d + static_cast<uint32_t>(p * kN);
            mma_f8f6f4_c<false>(dd, dp, dx, idesc);
            mma_f8f6f4_c<true>(dd, dp + (32 >> 4), dx + (32 >> 4), idesc);
            mma_f8f6f4_c<true>(dd, dp + (64 >> 4), dx + (64 >> 4), idesc);
            mma_f8f6f4_c<true>(dd, dp + (96 >> 4), dx + (96 >> 4), idesc);
          }
          mma_commit(&tfull[tb]);
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++tb == C::kBufs) {
          tb = 0;
          tphase ^= 1u;
        }
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      u += k1 - k0;
    }
    if (!ok) {
      if (lane == 0) record_device_error(args.err, FP8BS_ERR_DEVICE_TIMEOUT);
      *abort_flag = 1;
    }
    if (elect_one()) mma_commit(mma_done);
    __syncwarp();
    mbar_wait(mma_done, 0, kDefaultWaitCycles);
  } else if (warp == 2) {
    // -------------------------------------------------------- scale products --
    // A batch is up to 8 consecutive units of a segment; lane: unit j = lane % 8
    // and columns lane / 8, + 4, + 8, ... (a column's 8 scales lie next to each
    // other in memory).
    const int j = lane & 7;
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t u = range.begin; ok && u < range.end && !stopped();) {
      const int64_t s = u / depth;
      const int k0 = static_cast<int>(u - s * depth);
      const int k1 = static_cast<int>(min(static_cast<int64_t>(depth), k0 + range.end - u));
      const int a = seg_act(s), tile = seg_tile(s);
      const int e = act[a].x, row0 = act[a].y, n = act[a + 1].y - row0;
      const int64_t w0 = kDown ? (static_cast<int64_t>(e) * KB + tile) * IB
                               : (static_cast<int64_t>(e) * 2 * IB + tile) * KB;
      const int64_t w1 = w0 + static_cast<int64_t>(IB) * KB;   // the up block's scales
      for (int k = k0; ok && k < k1; k += kBatch) {
        const bool on = k + j < k1;
        float sw0 = 0.0f, sw1 = 0.0f;
        if (on) {
          sw0 = scale_value(args.sw, w0 + k + j, kE8);
          if constexpr (!kDown) sw1 = scale_value(args.sw, w1 + k + j, kE8);
        }
        if (!mbar_wait_warp(&sempty[buf], phase ^ 1u, limit)) {
          ok = false;
          break;
        }
        float* out = tab + (buf * kBatch + j) * C::kRow;
        for (int c = lane >> 3; c < n; c += 16) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int cc = c + 4 * i;
            v[i] = 0.0f;
            if (on && cc < n) {
              const int row = kDown ? row0 + cc : args.plan.row_tok[row0 + cc];
              v[i] = scale_value(args.sx, static_cast<int64_t>(row) * depth + k + j, kE8);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (c + 4 * i < n) {
              out[c + 4 * i] = v[i] * sw0;
              if constexpr (!kDown) out[kN + c + 4 * i] = v[i] * sw1;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[buf]);
        if (++buf == 2) {
          buf = 0;
          phase ^= 1u;
        }
      }
      u += k1 - k0;
    }
    if (!ok) {
      if (lane == 0) record_device_error(args.err, FP8BS_ERR_DEVICE_TIMEOUT);
      *abort_flag = 1;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ promotion --
    const int wg = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;                  // weight row of the tile
    const int pt = static_cast<int>(threadIdx.x) - 128;   // 0 .. 255
    const uint32_t tlane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* codes = smem + C::kOffEnd;                                  // gate+up: [kN][128]
    uint32_t* maxima = reinterpret_cast<uint32_t*>(smem + C::kOffEnd + kN * 128);   // [kN][4]
    float* sums = reinterpret_cast<float*>(smem + C::kOffEnd);           // down: [kN][128]
    int tb = 0, buf = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    float acc[C::kParts][C::kHalf];

    // Hands one result's partial values (already in this CTA's slot) to the
    // other CTAs that have parts of it; true in the last one, which adds them.
    auto join = [&](int* counter, int parts) {
      __threadfence();
      named_bar_sync(1, kPromo);
      if (pt == 0) {
        const int before = ok ? atomicAdd(counter, 1) : -1;
        __threadfence();
        *last_flag = before == parts - 1 ? 1 : 0;
      }
      named_bar_sync(1, kPromo);
      __threadfence();
      return *last_flag != 0;
    };
    // slot of a CTA's part of the tile that begins at unit t0: 0 if the CTA's
    // range begins in the tile, else 1 (the tile is its last)
    auto slot_of = [&](int cta, int64_t t0) {
      return 2 * cta + (range.begin_of(cta) >= t0 ? 0 : 1);
    };
    if constexpr (kDown) {
      for (int i = pt; i < args.M * 128; i += kPromo) sums[i] = 0.0f;
      named_bar_sync(1, kPromo);
    }

    for (int64_t u = range.begin; u < range.end;) {
      const int64_t s = u / depth;
      const int k0 = static_cast<int>(u - s * depth);
      const int k1 = static_cast<int>(min(static_cast<int64_t>(depth), k0 + range.end - u));
      const int a = seg_act(s), tile = seg_tile(s);
      const int row0 = act[a].y, n = act[a + 1].y - row0;
      const int half = (n + 15) / 16 * 8;     // columns of each warpgroup
      const int col0 = wg * half;
#pragma unroll
      for (int p = 0; p < C::kParts; ++p)
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) acc[p][c] = 0.0f;

      for (int k = k0; k < k1; ++k) {
        const int j = (k - k0) % kBatch;
        if (ok && j == 0) ok = mbar_wait(&sfull[buf], sphase, limit);
        if (ok) ok = mbar_wait(&tfull[tb], tphase, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc_fence_after();
          const float* sc = tab + (buf * kBatch + j) * C::kRow + col0;
          const uint32_t ta = tlane + static_cast<uint32_t>(tb * C::kBufCols + col0);
#pragma unroll
          for (int c = 0; c < C::kHalf; c += 8) {
            if (c < half) {
              float v[C::kParts][8];
#pragma unroll
              for (int p = 0; p < C::kParts; ++p) tmem_ld8(ta + p * kN + c, v[p]);
              tmem_wait_ld();
#pragma unroll
              for (int p = 0; p < C::kParts; ++p) {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                  const float4 q = *reinterpret_cast<const float4*>(sc + p * kN + c + i);
                  fma2(acc[p][c + i], acc[p][c + i + 1], v[p][i], v[p][i + 1], q.x, q.y);
                  fma2(acc[p][c + i + 2], acc[p][c + i + 3], v[p][i + 2], v[p][i + 3], q.z, q.w);
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[tb]);
          if (lane == 0 && (j == kBatch - 1 || k == k1 - 1)) mbar_arrive(&sempty[buf]);
        }
        if (j == kBatch - 1 || k == k1 - 1) {
          if (++buf == 2) {
            buf = 0;
            sphase ^= 1u;
          }
        }
        if (++tb == C::kBufs) {
          tb = 0;
          tphase ^= 1u;
        }
      }
      u += k1 - k0;

      if constexpr (!kDown) {
        const int64_t t0 = s * depth;
        bool mine = true;
        if (k1 - k0 < depth) {   // the tile's K range is shared with other CTAs
          float* part = args.partial +
                        static_cast<int64_t>(slot_of(blockIdx.x, t0)) * args.M * 256 + row;
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c) {
            if (c < half && col0 + c < n) {
              __stcg(part + (col0 + c) * 256, acc[0][c]);
              __stcg(part + (col0 + c) * 256 + 128, acc[1][c]);
            }
          }
          const int c0 = range.owner(t0), c1 = range.owner(t0 + depth - 1);
          mine = join(args.plan.count_gu + s, c1 - c0 + 1);
          if (mine) {
#pragma unroll
            for (int p = 0; p < C::kParts; ++p)
#pragma unroll
              for (int c = 0; c < C::kHalf; ++c) acc[p][c] = 0.0f;
            for (int q = c0; q <= c1; ++q) {
              const float* from =
                  args.partial + static_cast<int64_t>(slot_of(q, t0)) * args.M * 256 + row;
#pragma unroll
              for (int c = 0; c < C::kHalf; ++c) {
                if (c < half && col0 + c < n) {
                  acc[0][c] += __ldcg(from + (col0 + c) * 256);
                  acc[1][c] += __ldcg(from + (col0 + c) * 256 + 128);
                }
              }
            }
          }
        }
        if (mine) {   // the same in all promotion warps, unlike ok: barriers follow
          // h = silu(g) * u of this thread's intermediate column; a token's
          // group of 128 lies across the warpgroup's threads
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c) {
            if (c < half) {
              acc[0][c] = silu_f32(acc[0][c]) * acc[1][c];
              const uint32_t m =
                  __reduce_max_sync(0xffffffffu, __float_as_uint(acc[0][c]) & 0x7FFFFFFFu);
              if (lane == 0) maxima[(col0 + c) * 4 + quarter] = m;
            }
          }
          named_bar_sync(2 + wg, 128);
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c) {
            if (c < half && col0 + c < n) {
              const uint4 m4 = *reinterpret_cast<const uint4*>(maxima + (col0 + c) * 4);
              const float amax = __uint_as_float(max(max(m4.x, m4.y), max(m4.z, m4.w)));
              const int64_t at = static_cast<int64_t>(row0 + col0 + c) * IB + tile;
              uint32_t q;
              if constexpr (kE8) {
                const uint32_t code = ue8m0_code_of_amax(amax);
                q = __nv_cvt_float_to_fp8(acc[0][c] * ue8m0_inv_scale(code), __NV_SATFINITE,
                                          __NV_E4M3);
                if (row == 0) static_cast<uint8_t*>(args.sh)[at] = static_cast<uint8_t>(code);
              } else {
                const float sc = scale_of_amax(amax);
                q = code1f(acc[0][c], ScaleDivider(sc));
                if (row == 0) static_cast<float*>(args.sh)[at] = sc;
              }
              codes[(col0 + c) * 128 + row] = static_cast<uint8_t>(q);
            }
          }
          named_bar_sync(2 + wg, 128);
          for (int i = row; i < half * 8; i += 128) {   // 16-byte chunks
            const int c = col0 + (i >> 3);
            if (ok && c < n)
              *reinterpret_cast<uint4*>(args.qh + static_cast<int64_t>(row0 + c) * args.I +
                                        tile * 128 + (i & 7) * 16) =
                  *reinterpret_cast<const uint4*>(codes + c * 128 + (i & 7) * 16);
          }
        }
      } else {
        // this expert's share of the tokens' sums
        const int* toks = args.plan.row_tok + row0;
        const float* ws = args.plan.row_w + row0;
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) {
          if (c < half && col0 + c < n) {
            float* at = sums + toks[col0 + c] * 128 + row;
            *at = fmaf(ws[col0 + c], acc[0][c], *at);
          }
        }
        const int64_t t0 = static_cast<int64_t>(tile) * tile_units;
        // between two segments too: the next expert's columns may put a token
        // into the other warpgroup
        named_bar_sync(1, kPromo);
        if (u == range.end || u == t0 + tile_units) {
          // the end of this CTA's part of the tile; a warp takes every eighth
          // token, a lane four of its 128 columns
          const bool whole = range.begin <= t0 && u == t0 + tile_units;
          const int pw = pt >> 5;
          const int c0 = range.owner(t0), c1 = range.owner(t0 + tile_units - 1);
          bool mine = true;
          if (!whole) {
            float4* part = reinterpret_cast<float4*>(
                args.partial + static_cast<int64_t>(slot_of(blockIdx.x, t0)) * args.M * 128);
            for (int m = pw; m < args.M; m += kPromo / 32)
              __stcg(part + m * 32 + lane, reinterpret_cast<const float4*>(sums)[m * 32 + lane]);
            mine = join(args.plan.count_down + tile, c1 - c0 + 1);
          }
          if (mine && ok) {
            for (int m = pw; m < args.M; m += kPromo / 32) {
              float4 v = reinterpret_cast<const float4*>(sums)[m * 32 + lane];
              if (!whole) {
                v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int q = c0; q <= c1; ++q) {
                  const float4 o = __ldcg(
                      reinterpret_cast<const float4*>(
                          args.partial + static_cast<int64_t>(slot_of(q, t0)) * args.M * 128) +
                      m * 32 + lane);
                  v.x += o.x;
                  v.y += o.y;
                  v.z += o.z;
                  v.w += o.w;
                }
              }
              const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y);
              const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z, v.w);
              *reinterpret_cast<uint2*>(args.y + static_cast<int64_t>(m) * args.K + tile * 128 +
                                        lane * 4) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                             *reinterpret_cast<const uint32_t*>(&hi));
            }
          }
          named_bar_sync(1, kPromo);
          for (int i = pt; i < args.M * 128; i += kPromo) sums[i] = 0.0f;
          named_bar_sync(1, kPromo);
        }
      }
    }
    if (!ok) {
      if (lane == 0) record_device_error(args.err, FP8BS_ERR_DEVICE_TIMEOUT);
      *abort_flag = 1;
    }
    if constexpr (kDown) {
      if (n_act == 0) {   // no token has a choice here
        const int64_t total = static_cast<int64_t>(args.M) * args.K / 8;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPromo + pt; i < total;
             i += static_cast<int64_t>(gridDim.x) * kPromo)
          reinterpret_cast<uint4*>(args.y)[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int kN, bool kDown, bool kE8>
int launch_gemm(const CUtensorMap& tw, const CUtensorMap& tx, const GemmMoeArgs& args, int grid,
                int device, cudaStream_t stream) {
  using C = MoeCfg<kN, kDown>;
  auto kern = moe_gemm_kernel<kN, kDown, kE8>;
  static std::once_flag flags[64];
  cudaError_t attr_err = cudaSuccess;
  std::call_once(flags[device], [&] {
    attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (attr_err != cudaSuccess) return FP8BS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, args) == cudaSuccess ? FP8BS_OK : FP8BS_ERR_CUDA;
}

template <bool kDown, bool kE8>
int launch_gemm_n(const CUtensorMap& tw, const CUtensorMap& tx, const GemmMoeArgs& args, int grid,
                  int device, cudaStream_t stream) {
  if (args.M <= 16) return launch_gemm<16, kDown, kE8>(tw, tx, args, grid, device, stream);
  if (args.M <= 32) return launch_gemm<32, kDown, kE8>(tw, tx, args, grid, device, stream);
  if (args.M <= 64) return launch_gemm<64, kDown, kE8>(tw, tx, args, grid, device, stream);
  return launch_gemm<128, kDown, kE8>(tw, tx, args, grid, device, stream);
}

}  // namespace

size_t moe_workspace_bytes(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  return carve(nullptr, M, K, I, E, top_k).bytes;
}

int launch_moe_mlp(const MoeArgs& a, bool ue8m0, cudaStream_t stream) {
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  const int64_t pairs = static_cast<int64_t>(a.M) * a.top_k;
  const int64_t act = a.E < pairs ? a.E : pairs;
  const Workspace w = carve(a.workspace, a.M, a.K, a.I, a.E, a.top_k);
  alignas(64) CUtensorMap twg, twd, txa, txh;
  if (int st = encode_tmap_2d_u8(&twg, a.qg, a.K, static_cast<uint64_t>(a.E) * 2 * a.I, a.K, 128,
                                 128, kSwizzle128B))
    return st;
  if (int st = encode_tmap_2d_u8(&twd, a.qd, a.I, static_cast<uint64_t>(a.E) * a.K, a.I, 128, 128,
                                 kSwizzle128B))
    return st;
  if (int st = encode_tmap_2d_u8(&txa, a.qa, a.K, a.M, a.K, 128, 1, kSwizzle128B)) return st;
  if (int st = encode_tmap_2d_u8(&txh, w.qh, a.I, pairs, a.I, 128, 16, kSwizzle128B)) return st;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, moe_plan_kernel, a.ids, a.weights, static_cast<int>(pairs), a.top_k,
                         a.E, a.first_expert, static_cast<int>(act * (a.I / 128)), a.K / 128,
                         w.plan) != cudaSuccess)
    return FP8BS_ERR_CUDA;

  GemmMoeArgs g{};
  g.plan = w.plan;
  g.qh = w.qh;
  g.sh = w.sh;
  g.y = a.y;
  g.partial = w.partial;
  g.M = a.M;
  g.K = a.K;
  g.I = a.I;
  g.wait_limit = a.wait_limit;
  g.err = a.err;
  const int grid = dev.sm_count < kMaxCtas ? dev.sm_count : kMaxCtas;
  g.sx = a.sa;
  g.sw = a.sg;
  if (int st = ue8m0 ? launch_gemm_n<false, true>(twg, txa, g, grid, dev.device, stream)
                     : launch_gemm_n<false, false>(twg, txa, g, grid, dev.device, stream))
    return st;
  g.sx = w.sh;
  g.sw = a.sd;
  return ue8m0 ? launch_gemm_n<true, true>(twd, txh, g, grid, dev.device, stream)
               : launch_gemm_n<true, false>(twd, txh, g, grid, dev.device, stream);
}

}  // namespace fp8bs
