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
// Bound: HBM, where the experts are wide and not crowded. Every chosen expert's
// 3 I K weight bytes are read once for up to 64 of its tokens; at the copy bandwidth an SM gets a 128 x 128 tile
// (16 KB) every ~700 cycles, and both the MMAs and the promotion of a tile
// take less than that. Measured, the weights' bytes over the time, of the copy
// bandwidth: 64 tokens on 32 of 256 experts of 7168 x 2048 186 to 206 us (91 to
// 100%), one token through 2 of 8 experts of 4096 x 14336 62.7 us (86%), 13 tokens
// on 27 experts of 2432 x 1408 53 us (76%), 128 tokens over 8 experts of 7168 x
// 2048 79 us (68%). The weights stream at the copy bandwidth in between; the
// rest is the way to the first tile (5 us: the plan, a ticket, the first loads)
// and from the last one to y (8 us: the chunks in flight, their count, the sums),
// and in calls below 40 us the way from gate+up over h to down (6 to 10 us).
// The smallest call takes 12.9 us.
//
// Far from that bound: narrow experts, whose down results are one or two units
// deep, so that a ticket, the hand-over to six readers, the partial sums and a
// count go with every 16 to 64 KB (16 tokens on 64 experts of 7168 x 128 58 us of
// 21.4; 64 on 32 of 4096 x 256 44 of 15.4; 8 on 64 of 2048 x 256 30 of 9.6); and few
// crowded experts, whose lists have less than three chunks for an SM or leave some
// without any (128 tokens on 2 experts of 4096 x 1536 31 us of 5.8, 64 on 4 of
// 3584 x 2560 42 of 16.8).
//
// Two launches, chained by programmatic dependent launch:
//
//   moe_plan_kernel  one block: the chosen experts in order, each with its
//                    tokens ("rows"), how the work is cut, the counters zeroed
//   moe_mlp_kernel   one CTA per SM: gate+up and down
//
// Both products put 128 weight rows on the MMA's M side and tokens on its N
// side: the rows of one expert, in blocks of at most 64. An expert with more is
// walked twice, all of one product's weights for the first block before the second:
// the second time they come from L2 where they fit (128 tokens on one expert of
// 7168 x 2048: 45.1 MB from HBM for 44.0 MB of weights), else from HBM again (of
// 7168 x 9216: 372 for 198 MB). The work is a list of chunks: some K-blocks of one result (gate+up: expert and 128
// intermediate columns; down: expert and 128 output columns). A CTA claims the
// next chunk from a counter, streams its weights, writes the chunk's fp32
// partial sums to the workspace and goes on; nothing in that stream waits for
// another CTA. (Joining the parts inside the stream cost 4 us each time, most
// of it the round trips of a fence and an atomic behind the weights in flight.)
//
// Finisher warps, of all CTAs, claim the results in the same order, wait for
// their chunks and add the parts up in a fixed order, so that the bytes are
// the same every call:
//
//   h   one to four rows x 128 intermediate columns: SwiGLU, codes and scales
//   y   32 output columns of some tokens: the weighted sum over a token's experts
//
// Down's chunks follow gate+up's in the list, K-blocks first, then output
// columns; y follows h. A down chunk waits until h of its K-blocks is complete.
// Both lists are claimed in order, by CTAs that are running; gate+up's chunks
// wait for no one, h for those only, down's chunks for h, y for all: every wait
// ends however few of the CTAs are resident.
//
//   warp 0        claims chunks; TMA producer of the weight tiles
//   warp 1        MMA issuer: 8 tcgen05.mma of K = 32 per unit (two tiles) into
//                 one of the TMEM buffers
//   warps 2, 4    scale products sA * sW of up to 8 units at a time, in turn,
//                 into shared memory
//   warp 3        TMA producer of the tokens' K-blocks
//   warp 5        counts the chunks whose partial sums are written
//   warps 6 ..    finishers (kFin)
//   the last      promotion warpgroups, each a share of the token columns:
//                 TMEM -> registers times the scale products -> workspace;
//                 finishers when the chunks are used up
//
// The weights of a call can evict the kernel's code from L2, and then the first
// pass through each piece of code waits for HBM behind them (5 us for the scale
// products when they were unrolled): what runs before the first tile is kept
// short, a chunk is decoded once and handed on, both products share their loops,
// and the weights are loaded evict-first.
//
// Every wait is bounded as in gemm_kernel.cuh.
#include <mutex>

#include "common.cuh"
#include "e4m3_codec.cuh"
#include "kernels.h"

namespace fp8bs {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBlockRows = 64;     // tokens of one expert that are walked together
constexpr int kFin = 2;            // finisher warps (more take registers from the sums)
constexpr int kBatch = 8;          // units per batch of scale products
constexpr int kTabs = 4;           // buffers of scale products
constexpr int64_t kPartFloats = 8 << 20;   // partial sums of a product, but for large problems

constexpr int kSmemBytes = 227 * 1024;
constexpr int kTileBytes = 128 * 128;
constexpr int kUnitBytes = 2 * kTileBytes;
constexpr int kMaxStages = 5;      // units in flight, at most
constexpr int kMaxBufs = 16;       // TMEM buffers, at most
constexpr int kMail = 8;           // chunks between claim and count, at most

// How the work of a call is cut. A unit is 256 weight rows x 128 (gate+up: 128
// gate rows and the 128 up rows of the same intermediate columns) or 128 x 256
// (down: two K-blocks of 128 output columns; one at the end of an odd number).
struct alignas(16) Head {
  int blocks, rows;     // expert blocks; rows of all
  int ncol, xbytes;     // TMEM columns of a product; bytes of a K-block of tokens
  int stages, bufs;     // units in shared memory; TMEM buffers
  int q_gu, cpt;        // units of a gate+up chunk; chunks of a result
  int q_down, cps;      // units of a down chunk; chunks of a block's part of a result
  int n_gu, total;      // chunks of gate+up; of both
  int fin_rows, groups; // rows of an h task; h tasks of a gate+up result
  int n_h, n_tasks;     // h tasks; of both kinds
  int top;              // rows of a token, at most
  int pad[3];
};

// What is known before the plan.
struct Shape {
  int M, K, I, top_k;
  int sms;
  int room;             // shared memory for units
  int cap_gu, cap_down; // rows of partial sums that the workspace holds
  int y_items;          // (token, 32 columns) of a y task
  int y_tasks;          // y tasks of 128 output columns
};

// A chunk is about a twelfth of an SM's share, so that the SMs finish together
// (they do not get equal bandwidth), but not below 8 units (one token through 2
// experts of 4096 x 14336: 76 us with 4, 70 with 8, 72 with 16), nor below an
// eighth of its tokens, where the partial sums weigh more than a quarter of the
// weights.
struct Cut {
  int q, n;   // units of a chunk; chunks of `depth` units
};
__host__ __device__ inline Cut cut_list(int units, int depth, int sms, int most, int cap) {
  const int each = (units + sms - 1) / sms;
  // (with less than 8 units for an SM at most 8 chunks, which the finishers
  // load together)
  const int few = (depth + 7) / 8;
  int q = each < 8 ? (each > few ? each : few) : each < 96 ? 8 : each / 12;
  const int least = most < 8 ? 1 : (most + 7) / 8;
  if (q < least) q = least;
  int n = (depth + q / 2) / q;
  if (n > cap) n = cap;
  if (n < 1) n = 1;
  Cut c;
  c.q = (depth + n - 1) / n;
  c.n = (depth + c.q - 1) / c.q;
  return c;
}

// The cut of gate+up (list 0) or down (list 1).
__host__ __device__ inline Cut cut_of(int list, int blocks, int rows, int most, const Shape& s) {
  const int KB = s.K / 128, IB = s.I / 128, DU = (IB + 1) / 2;
  return cut_list(blocks * KB * (list ? DU : IB), list ? DU : KB, s.sms, most,
                  (list ? s.cap_down : s.cap_gu) / (rows < 1 ? 1 : rows));
}

__host__ __device__ inline Head head_of(int blocks, int rows, int most, int top, Cut gu, Cut down,
                                        const Shape& s) {
  const int KB = s.K / 128, IB = s.I / 128;
  Head h;
  h.blocks = blocks;
  h.rows = rows;
  h.ncol = most <= 16 ? 16 : most <= 32 ? 32 : 64;
  h.xbytes = (most + 15) / 16 * 2048;
  h.stages = s.room / (kUnitBytes + 2 * h.xbytes);
  if (h.stages > kMaxStages) h.stages = kMaxStages;
  h.bufs = 256 / h.ncol;
  h.q_gu = gu.q;
  h.cpt = gu.n;
  h.q_down = down.q;
  h.cps = down.n;
  h.n_gu = blocks * IB * h.cpt;
  h.total = h.n_gu + blocks * h.cps * KB;
  // an h task has one row where that is at most three tasks for a finisher warp,
  // else two or four
  h.fin_rows = 1;
  while (h.fin_rows < 4 &&
         blocks * IB * ((most + h.fin_rows - 1) / h.fin_rows) > 3 * kFin * s.sms)
    h.fin_rows *= 2;
  h.groups = (most + h.fin_rows - 1) / h.fin_rows;
  h.n_h = blocks * IB * h.groups;
  h.n_tasks = h.n_h + KB * s.y_tasks;
  h.top = top;
  return h;
}

// A chunk, as the producer of the weights hands it on.
struct alignas(16) Chunk {
  int kind;        // 0: gate+up, 1: down, -1: the end
  int expert;
  int row0, n;     // rows of the block
  int tile;        // 128 intermediate, or output, columns
  int c;           // chunk of the result (gate+up), of the block's part of it (down)
  int k0, k1;      // units
  int count;       // its counter
  int ready;       // down: counter of the h tasks that it needs ...
  int needs;       // ... and their number
  int pad;
};

__host__ __device__ inline Chunk chunk_at(const Head& h, int t, int KB, int IB) {
  Chunk ch;
  int a, q, depth;
  if (t >= h.n_gu) {
    t -= h.n_gu;
    const int s = t / KB;
    ch.kind = 1;
    ch.tile = t - s * KB;
    a = s / h.cps;
    ch.c = s - a * h.cps;
    q = h.q_down;
    depth = (IB + 1) / 2;
    ch.count = ch.tile;
  } else {
    const int s = t / h.cpt;
    ch.kind = 0;
    ch.c = t - s * h.cpt;
    a = s / IB;
    ch.tile = s - a * IB;
    q = h.q_gu;
    depth = KB;
    ch.count = s;
  }
  ch.expert = a;   // the block; its expert and rows are looked up
  ch.row0 = ch.n = 0;
  ch.k0 = ch.c * q;
  ch.k1 = ch.k0 + q < depth ? ch.k0 + q : depth;
  ch.ready = a * h.cps + ch.c;
  ch.needs = ((2 * ch.k1 < IB ? 2 * ch.k1 : IB) - 2 * ch.k0) * h.groups;
  ch.pad = 0;
  return ch;
}

struct Barriers {
  uint64_t fullw[kMaxStages], fullx[kMaxStages], empty[kMaxStages];
  uint64_t tfull[kMaxBufs], tempty[kMaxBufs];
  uint64_t sfull[kTabs], sempty[kTabs];
  uint64_t mfull[kMail], mempty[kMail], dumped[kMail];
  uint64_t mma_done, pairs;
  static constexpr int kCount = 3 * kMaxStages + 2 * kMaxBufs + 2 * kTabs + 3 * kMail + 2;
};

struct alignas(16) Shared {
  Chunk mail[kMail];
  Barriers bar;
  uint32_t tmem_slot;
  int abort_flag;
};

// Shared memory of a CTA: Shared, the rows and weights of the choices [pairs],
// the scale products, the units' weight tiles, their token blocks.
struct Layout {
  int off_row, off_w, off_tab, off_tiles;
  __host__ Layout(int pairs, int ncol_max) {
    off_row = static_cast<int>(sizeof(Shared));
    off_w = off_row + (pairs * 2 + 15) / 16 * 16;
    off_tab = off_w + (pairs * 4 + 15) / 16 * 16;
    off_tiles = (off_tab + kTabs * kBatch * (2 * ncol_max + 4) * 4 + 1023) / 1024 * 1024;
  }
  __host__ int room() const { return kSmemBytes - 1024 - off_tiles; }
};

// What the plan kernel leaves for the MLP kernel.
struct Plan {
  Head* head;
  int* ticket;       // [4]: chunks claimed; tasks claimed; h tasks complete; -
  int2* act;         // [blocks + 1]: (expert, its first row); the last entry ends the rows
  int* row_tok;      // [rows] token of a row
  int* pair_row;     // [M][top_k] a token's rows in the order of its choices, then -1
  float* pair_w;     // [M][top_k] their weights
  int* counters;     // zeroed:
  int* count_gu;     //   [blocks * I / 128] chunks written of a gate+up result
  int* count_down;   //   [K / 128] chunks written of a down result
  int* ready;        //   [blocks * units of I] h tasks complete of a down K-range
  int n_counters;
};

struct Workspace {
  Plan plan;
  uint8_t* qh;         // [rows][I]
  void* sh;            // [rows][I / 128]
  float* part_gu;      // [chunks of a result][rows][I / 128][256]
  float* part_down;    // [chunks of a block's part of a result][rows][K]
  int cap_gu, cap_down;   // rows that they hold
  size_t bytes;
};

Workspace carve(void* base, int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  const int64_t rows = M * top_k;
  const int64_t act = (E < rows ? E : rows) + rows / (kBlockRows + 1);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  // what kPartFloats hold, from 1 to 64 parts where all choices are here (never
  // less for more tokens: a workspace serves every smaller call)
  auto part_rows = [&](int64_t width) {
    const int64_t one = rows * width, most = 64 * one < kPartFloats ? 64 * one : kPartFloats;
    return static_cast<int>((one > most ? one : most) / width);
  };
  Workspace w;
  w.plan.head = reinterpret_cast<Head*>(take(sizeof(Head)));
  w.plan.ticket = reinterpret_cast<int*>(take(16));
  w.plan.act = reinterpret_cast<int2*>(take((act + 1) * 8));
  w.plan.row_tok = reinterpret_cast<int*>(take(rows * 4));
  w.plan.pair_row = reinterpret_cast<int*>(take(rows * 4));
  w.plan.pair_w = reinterpret_cast<float*>(take(rows * 4));
  const int64_t n_gu = act * (I / 128), n_down = K / 128, n_ready = act * ((I / 128 + 1) / 2);
  w.plan.counters = reinterpret_cast<int*>(take((n_gu + n_down + n_ready) * 4));
  w.plan.count_gu = w.plan.counters;
  w.plan.count_down = w.plan.count_gu + n_gu;
  w.plan.ready = w.plan.count_down + n_down;
  w.plan.n_counters = static_cast<int>(n_gu + n_down + n_ready);
  w.qh = take(rows * I);
  w.sh = take(rows * (I / 128) * 4);
  w.cap_gu = part_rows(2 * I);
  w.cap_down = part_rows(K);
  w.part_gu = reinterpret_cast<float*>(take(static_cast<size_t>(w.cap_gu) * 2 * I * 4));
  w.part_down = reinterpret_cast<float*>(take(static_cast<size_t>(w.cap_down) * K * 4));
  w.bytes = at;
  return w;
}

// -------------------------------------------------------------------- plan --
// A choice counts once per token and expert: of a token's choices of the same
// expert the first one makes the row and carries the sum of their weights (in
// the order of the choices).

// Up to 32 choices: one warp, a lane for each choice, without a barrier. The
// blocks come in the order of the experts' first choices.
__device__ __forceinline__ void plan_few(const int32_t* ids, const float* weights, int pairs, int E,
                                         int first_expert, const Plan& plan, const Shape& shape) {
  const int lane = threadIdx.x, top_k = shape.top_k;
  int e = -1 - lane;   // no expert: like no other lane's
  float w = 0.0f;
  if (lane < pairs) {
    const int64_t local = static_cast<int64_t>(ids[lane]) - first_expert;
    w = weights[lane];
    if (local >= 0 && local < E) e = static_cast<int>(local);
  }
  const uint32_t all = 0xffffffffu, before = (1u << lane) - 1u;
  const int tok = lane / top_k, first = tok * top_k;
  const uint32_t token = (top_k == 32 ? all : (1u << top_k) - 1u) << (first & 31);
  const uint32_t same = __match_any_sync(all, e);
  const bool row = e >= 0 && (same & token & before) == 0u;
  for (int j = 0; j < top_k; ++j) {
    const int from = (first + j) & 31;
    const float other = __shfl_sync(all, w, from);
    if (from > lane && ((same & token) >> from & 1u)) w += other;
  }
  const uint32_t rows = __ballot_sync(all, row);
  const uint32_t mine = same & rows;                       // the expert's rows
  const bool leads = row && (mine & before) == 0u;
  const uint32_t leaders = __ballot_sync(all, leads);
  const int n = row ? __popc(mine) : 0;
  int scan = leads ? n : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(all, scan, off);
    if (lane >= off) scan += o;
  }
  const int row0 = __shfl_sync(all, scan - n, mine ? __ffs(static_cast<int>(mine)) - 1 : 0);
  const int most = __reduce_max_sync(all, n);
  const int of_token = lane < pairs ? __popc(rows & token) : 0;
  const int top = __reduce_max_sync(all, of_token);
  const int blocks = __popc(leaders), n_rows = __popc(rows);
  // (lanes 0 and 1 are what counts)
  const Cut c = cut_of(lane & 1, blocks, n_rows, most, shape);
  Cut down;
  down.q = __shfl_sync(all, c.q, 1);
  down.n = __shfl_sync(all, c.n, 1);
  if (lane == 0) {
    *plan.head = head_of(blocks, n_rows, most, top, c, down, shape);
    plan.act[blocks] = make_int2(-1, n_rows);
  }
  if (leads) plan.act[__popc(leaders & before)] = make_int2(e, row0);
  if (row) {
    const int r = row0 + __popc(mine & before), place = first + __popc(rows & token & before);
    plan.row_tok[r] = tok;
    plan.pair_row[place] = r;
    plan.pair_w[place] = w;
  }
  if (lane < pairs && lane - first >= of_token) plan.pair_row[lane] = -1;
}

// The order of an expert's rows comes from atomics here and may differ from
// call to call; nothing computed depends on it. The block has a thread for every
// expert at least, and two warps at least.
__global__ void __launch_bounds__(kPlanThreads, 1)
    moe_plan_kernel(const int32_t* __restrict__ ids, const float* __restrict__ weights, int pairs,
                    int E, int first_expert, const Plan plan, const Shape shape) {
  __shared__ int expert[kMoeMaxM * kMoeMaxTopK];   // local expert of a choice, -1: none
  __shared__ float share[kMoeMaxM * kMoeMaxTopK];  // weight of a choice
  __shared__ int fill[kPlanThreads];               // next row of an expert
  __shared__ uint8_t is_row[kMoeMaxM * kMoeMaxTopK];   // the token's first choice of this expert
  __shared__ uint32_t warp_sum[kPlanThreads / 32];
  __shared__ int token_rows[kMoeMaxM];
  __shared__ int most, most_of_token;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, T = blockDim.x;
  const int top_k = shape.top_k;
  if (pairs <= 32) {
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
      plan_few(ids, weights, pairs, E, first_expert, plan, shape);
    } else {
      if (t < 36) plan.ticket[t - 32] = 0;
#pragma unroll 1
      for (int i = t - 32; i < plan.n_counters; i += T - 32) plan.counters[i] = 0;
    }
    return;
  }
  fill[t] = 0;
  if (t < kPlanThreads / 32) warp_sum[t] = 0u;
  if (t < kMoeMaxM) token_rows[t] = 0;
  if (t == 0) most = most_of_token = 0;
  grid_dependency_wait();
  grid_launch_dependents();
#pragma unroll 1
  for (int i = t; i < pairs; i += T) {
    const int64_t e = static_cast<int64_t>(ids[i]) - first_expert;
    share[i] = weights[i];
    expert[i] = e >= 0 && e < E ? static_cast<int>(e) : -1;
  }
#pragma unroll 1
  for (int i = t; i < plan.n_counters; i += T) plan.counters[i] = 0;
  if (t < 4) plan.ticket[t] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = t; i < pairs; i += T) {
    const int e = expert[i];
    bool row = e >= 0;
    for (int j = i / top_k * top_k; j < i; ++j) row &= expert[j] != e;
    is_row[i] = row;
    if (row) {
      atomicAdd(&fill[e], 1);
      atomicAdd(&token_rows[i / top_k], 1);
    }
  }
  __syncthreads();
  // exclusive prefix over the experts of (blocks << 16 | rows): at most 4096
  // rows, in at most 1024 + 63 blocks
  const int n = fill[t];
  const int blocks = (n + kBlockRows - 1) / kBlockRows;
  const uint32_t mine = (static_cast<uint32_t>(blocks) << 16) | static_cast<uint32_t>(n);
  uint32_t scan = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += o;
  }
  if (lane == 31) warp_sum[warp] = scan;
  // rows of the largest block (a block count of 1 or 2)
  const int top = __reduce_max_sync(0xffffffffu, blocks > 1 ? (n + 1) / 2 : n);
  if (lane == 0 && top > 0) atomicMax(&most, top);
  if (t < shape.M) atomicMax(&most_of_token, token_rows[t]);
  __syncthreads();
  const uint32_t sums = warp_sum[lane];
  const uint32_t total = __reduce_add_sync(0xffffffffu, sums);
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u);
  const uint32_t excl = before + scan - mine;
  const int row0 = static_cast<int>(excl & 0xFFFFu);
  if (blocks > 0) plan.act[excl >> 16] = make_int2(t, row0);
  if (blocks > 1) plan.act[(excl >> 16) + 1] = make_int2(t, row0 + n / 2);
  fill[t] = row0;
  __syncthreads();
  if (warp == (T >> 5) - 1) {
    const int rows = static_cast<int>(total & 0xFFFFu), n_blocks = static_cast<int>(total >> 16);
    const Cut c = cut_of(lane & 1, n_blocks, rows, most, shape);
    Cut down;
    down.q = __shfl_sync(0xffffffffu, c.q, 1);
    down.n = __shfl_sync(0xffffffffu, c.n, 1);
    if (lane == 0) {
      plan.act[n_blocks] = make_int2(-1, rows);
      *plan.head = head_of(n_blocks, rows, most, most_of_token, c, down, shape);
    }
  }
#pragma unroll 1
  for (int i = t; i < pairs; i += T) {
    const int first = i / top_k * top_k, end = first + top_k;
    const int rows = token_rows[i / top_k];
    int place = 0;   // rows of the token before this one
    float w = share[i];
#pragma unroll 2
    for (int j = first; j < end; ++j) {
      place += j < i && is_row[j];
      if (j > i && expert[j] == expert[i]) w += share[j];
    }
    if (is_row[i]) {
      const int row = atomicAdd(&fill[expert[i]], 1);
      plan.row_tok[row] = i / top_k;
      plan.pair_row[first + place] = row;
      plan.pair_w[first + place] = w;
    }
    if (i - first >= rows) plan.pair_row[i] = -1;
  }
}

// --------------------------------------------------------------------- MLP --
struct MlpArgs {
  Plan plan;
  Shape shape;
  const void* sa;    // [M][K/128]
  const void* sg;    // [E][2I/128][K/128]
  const void* sd;    // [E][K/128][I/128]
  uint8_t* qh;       // [rows][I]
  void* sh;          // [rows][I/128]
  __nv_bfloat16* y;  // [M][K]
  float* part_gu;
  float* part_down;
  int off_row, off_w, off_tab, off_tiles;
  long long wait_limit;
  int* err;
};

// A UE8M0 code c stands for 2^(c - 127), and 255 for NaN.
__device__ __forceinline__ float scale_value(const void* s, int64_t i, bool e8) {
  if (!e8) return __ldcg(static_cast<const float*>(s) + i);
  const uint32_t c = __ldcg(static_cast<const uint8_t*>(s) + i);
  const uint32_t odd = c == 0u ? 0x00400000u : 0x7FFFFFFFu;
  return __uint_as_float(c - 1u < 254u ? c << 23 : odd);
}

__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Orders this thread's generic-proxy accesses before later async-proxy (TMA)
// accesses, in global memory too.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// Waits until *p >= target, for at most `limit` cycles; the whole warp.
__device__ __forceinline__ bool wait_count_warp(const int* p, int target, long long limit) {
  const long long t0 = clock64();
  bool ok = true;
  while (load_acquire(p) < target) {
    if (clock64() - t0 > limit) {
      ok = false;
      break;
    }
    __nanosleep(100);
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ Head load_head(const Head* p) {
  Head h;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(Head)) / 16; ++i)
    reinterpret_cast<int4*>(&h)[i] = __ldcg(reinterpret_cast<const int4*>(p) + i);
  return h;
}

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}

__device__ __forceinline__ float4 shfl_xor4(const float4& a, int off) {
  return make_float4(__shfl_xor_sync(0xffffffffu, a.x, off), __shfl_xor_sync(0xffffffffu, a.y, off),
                     __shfl_xor_sync(0xffffffffu, a.z, off), __shfl_xor_sync(0xffffffffu, a.w, off));
}

struct Ring {   // position in a ring of n barriers
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// kN: most token columns; kWgs: promotion warpgroups.
template <int kN, int kWgs, bool kE8>
__global__ void __launch_bounds__(32 * (6 + kFin) + 128 * kWgs, 1)
    moe_mlp_kernel(const __grid_constant__ CUtensorMap tmap_g,
                   const __grid_constant__ CUtensorMap tmap_d,
                   const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ CUtensorMap tmap_h,
                   const __grid_constant__ MlpArgs args) {
  constexpr int kPromo0 = 6 + kFin;    // first promotion warp
  constexpr int kPer = kN / kWgs;      // columns of a promotion thread, at most
  static_assert(kPer % 8 == 0, "promotion works on eight columns at a time");
  static_assert(kPromo0 % 4 == 0, "a promotion warp's TMEM lanes go by its number");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  Barriers& bar = sh.bar;
  volatile int* abort_flag = &sh.abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = args.wait_limit;
  if (threadIdx.x < Barriers::kCount) {
    // arrivals: one, but for those of the promotion warps, of a chunk's readers
    // (its place in the ring: warps 1 to 5 and promotion) and of the finishers
    uint64_t* b = reinterpret_cast<uint64_t*>(&bar) + threadIdx.x;
    uint32_t count = 1;
    if ((b >= bar.tempty && b < bar.tempty + kMaxBufs) ||
        (b >= bar.sempty && b < bar.sempty + kTabs) || (b >= bar.dumped && b < bar.dumped + kMail))
      count = 4 * kWgs;
    if (b >= bar.mempty && b < bar.mempty + kMail) count = 5 + 4 * kWgs;
    if (b == &bar.pairs) count = kFin;
    mbar_init(b, count);
    fence_mbarrier_init();
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    tma_prefetch_desc(&tmap_g);
    tma_prefetch_desc(&tmap_d);
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_h);
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sh.tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();
  int ticket = 0;
  if (threadIdx.x == 0) ticket = atomicAdd(args.plan.ticket, 1);
  const Head head = load_head(args.plan.head);
  const int KB = args.shape.K / 128, IB = args.shape.I / 128;
  float* tab = reinterpret_cast<float*>(smem + args.off_tab);
  uint8_t* tiles = smem + args.off_tiles;
  uint8_t* xtiles = tiles + head.stages * kUnitBytes;
  const int tab_row = 2 * head.ncol + 4;   // floats of a unit's scale products, padded
  const int2* act = args.plan.act;
  const int* row_tok = args.plan.row_tok;
  int* h_done = args.plan.ticket + 2;

  auto stopped = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };
  auto give_up = [&]() {
    if (lane == 0) record_device_error(args.err, FP8BS_ERR_DEVICE_TIMEOUT);
    *abort_flag = 1;
  };
  // The next chunk for a reader of the ring; false at the end. `keep` leaves
  // its place in the ring occupied.
  Ring mr;
  auto next_chunk = [&](Chunk& ch, bool keep) {
    bool ok = !stopped();
    if (ok) {
      ok = mbar_wait_warp(&bar.mfull[mr.i], mr.phase, limit);
      if (!ok) give_up();
    }
    if (!ok) return false;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      reinterpret_cast<int4*>(&ch)[i] = reinterpret_cast<const int4*>(&sh.mail[mr.i])[i];
    if (ch.kind < 0) return false;
    __syncwarp();
    if (!keep) {
      if (lane == 0) mbar_arrive(&bar.mempty[mr.i]);
      mr.next(kMail);
    }
    return true;
  };
  // h of a down chunk's K-blocks is complete
  bool all_ready = false;
  auto wait_h = [&](const Chunk& ch) {
    if (all_ready) return true;
    if (!__all_sync(0xffffffffu, load_acquire(args.plan.ready + ch.ready) >= ch.needs))
      return wait_count_warp(args.plan.ready + ch.ready, ch.needs, limit);
    all_ready = __all_sync(0xffffffffu, load_acquire(h_done) >= head.n_h);
    return true;
  };

  if (warp == 0) {
    // -------------------------------------------- chunks and weight tiles --
    Ring r;
    int issued = 0;
    bool ok = true;
    // read once: the partial sums and the kernel's code should stay in L2
    // instead (231 -> 223 us for 64 tokens on 32 experts of 7168 x 2048)
    const uint64_t policy = policy_evict_first();
    ticket = __shfl_sync(0xffffffffu, ticket, 0);
    while (!stopped()) {
      const bool end = ticket >= head.total;
      Chunk ch = chunk_at(head, ticket, KB, IB);
      if (end) {
        ch.kind = -1;
      } else {
        const int2 b = act[ch.expert];
        const int2 b1 = act[ch.expert + 1];
        ch.n = b1.y - b.y;
        ch.expert = b.x;
        ch.row0 = b.y;
      }
      ok = mbar_wait_warp(&bar.mempty[mr.i], mr.phase ^ 1u, limit);
      if (!ok) break;
      int next = 0;
      if (lane == 0) {
        sh.mail[mr.i] = ch;
        mbar_arrive(&bar.mfull[mr.i]);
        // the answer comes while this chunk's loads are issued
        if (!end) next = atomicAdd(args.plan.ticket, 1);
      }
      __syncwarp();
      mr.next(kMail);
      if (end) break;
      // a unit's tiles: gate+up (k, y) and (k, y + I); down (2k, y) and (2k + 1, y)
      const bool down = ch.kind != 0;
      const CUtensorMap* map = down ? &tmap_d : &tmap_g;
      const int y = ch.expert * (down ? args.shape.K : 2 * args.shape.I) + ch.tile * 128;
      const int y2 = down ? y : y + args.shape.I;
      const int step = down ? 256 : 128, dx = down ? 128 : 0;
#pragma unroll 1
      for (int k = ch.k0; k < ch.k1; ++k) {
        ok = mbar_wait_warp(&bar.empty[r.i], r.phase ^ 1u, limit);
        if (!ok) break;
        const bool two = !down || 2 * k + 1 < IB;
        if (elect_one()) {
          uint8_t* to = tiles + r.i * kUnitBytes;
          mbar_arrive_expect_tx(&bar.fullw[r.i], two ? kUnitBytes : kTileBytes);
          tma_load_2d_hint(to, map, &bar.fullw[r.i], k * step, y, policy);
          if (two)
            tma_load_2d_hint(to + kTileBytes, map, &bar.fullw[r.i], k * step + dx, y2, policy);
        }
        __syncwarp();
        ++issued;
        r.next(head.stages);
      }
      if (!ok) break;
      ticket = __shfl_sync(0xffffffffu, next, 0);
    }
    if (!ok) give_up();
    // every copy issued must have landed before the CTA exits
    const int pending = issued < head.stages ? issued : head.stages;
#pragma unroll 1
    for (int i = 0; i < pending; ++i) {
      int st = r.i - 1 - i;
      uint32_t ph = r.phase;
      if (st < 0) {
        st += head.stages;
        ph ^= 1u;
      }
      mbar_wait(&bar.fullw[st], ph, kDefaultWaitCycles);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    Ring r, b;
    bool ok = true;
    const uint64_t dw0 = sw128_kmajor_desc(smem_u32(tiles));
    const uint64_t dx0 = sw128_kmajor_desc(smem_u32(xtiles));
    Chunk ch;
    while (ok && next_chunk(ch, false)) {
      const uint32_t idesc = idesc_e4m3_f32(128, (ch.n + 15) / 16 * 16);
#pragma unroll 1
      for (int k = ch.k0; k < ch.k1; ++k) {
        ok = mbar_wait_warp(&bar.tempty[b.i], b.phase ^ 1u, limit) &&
             mbar_wait_warp(&bar.fullx[r.i], r.phase, limit) &&
             mbar_wait_warp(&bar.fullw[r.i], r.phase, limit);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dw = dw0 + static_cast<uint32_t>((r.i * kUnitBytes) >> 4);
        const uint64_t dx = dx0 + static_cast<uint32_t>((r.i * 2 * head.xbytes) >> 4);
        const uint32_t d = tmem_base + static_cast<uint32_t>(b.i * 2 * head.ncol);
        // the second product: of gate+up's other tile with the same tokens, of
        // down's next K-block; the first again (times 0 later) where that is missing
        const bool two = ch.kind == 0 || 2 * k + 1 < IB;
        const uint64_t ew = dw + (two ? kTileBytes >> 4 : 0);
        const uint64_t ex = dx + static_cast<uint32_t>(two && ch.kind != 0 ? head.xbytes >> 4 : 0);
        const uint32_t e = d + static_cast<uint32_t>(head.ncol);
        if (elect_one()) {
          mma_f8f6f4_c<false>(d, dw, dx, idesc);
          mma_f8f6f4_c<true>(d, dw + (32 >> 4), dx + (32 >> 4), idesc);
          mma_f8f6f4_c<true>(d, dw + (64 >> 4), dx + (64 >> 4), idesc);
          mma_f8f6f4_c<true>(d, dw + (96 >> 4), dx + (96 >> 4), idesc);
          mma_f8f6f4_c<false>(e, ew, ex, idesc);
          mma_f8f6f4_c<true>(e, ew + (32 >> 4), ex + (32 >> 4), idesc);
          mma_f8f6f4_c<true>(e, ew + (64 >> 4), ex + (64 >> 4), idesc);
          mma_f8f6f4_c<true>(e, ew + (96 >> 4), ex + (96 >> 4), idesc);
          mma_commit(&bar.tfull[b.i]);
          mma_commit(&bar.empty[r.i]);
        }
        __syncwarp();
        r.next(head.stages);
        b.next(head.bufs);
      }
    }
    if (!ok) give_up();
    if (elect_one()) mma_commit(&bar.mma_done);
    __syncwarp();
    mbar_wait(&bar.mma_done, 0, kDefaultWaitCycles);
  } else if (warp == 2 || warp == 4) {
    // -------------------------------------------------------- scale products --
    // A batch is up to 8 consecutive units of a chunk; the two warps take them
    // in turn. Lane: unit j = lane % 8 and columns lane / 8, + 4, + 8, ... (a
    // column's 8 scales lie next to each other in memory). The loads of a batch
    // (of its first columns) are under way before the buffer is waited for.
    const int j = lane & 7;
    constexpr int kLoads = kN < 32 ? 4 : 8;
    Ring b;
    bool ok = true;
    Chunk ch;
    while (ok && next_chunk(ch, false)) {
      const bool down = ch.kind != 0;
      const void* sw = down ? args.sd : args.sg;
      const void* sx = down ? args.sh : args.sa;
      const int kbs = down ? IB : KB;   // scales of a row
      const int64_t w0 =
          (static_cast<int64_t>(ch.expert) * (down ? KB : 2 * IB) + ch.tile) * kbs;
      const int64_t w1 = down ? 1 : static_cast<int64_t>(IB) * kbs;   // to the second tile's
      bool waited = !down;
#pragma unroll 1
      for (int k = ch.k0; k < ch.k1; k += kBatch, b.next(kTabs)) {
        if ((b.i & 1) != (warp == 4)) continue;
        // the unit's (first) K-block and its second one; what is behind the last
        // unit or column is loaded from the last, so that no load has to wait for
        // a branch
        const int kb = min(down ? 2 * (k + j) : k + j, kbs - 1);
        const bool two = !down || kb + 1 < kbs;
        const float s0 = scale_value(sw, w0 + kb, kE8);
        const float s1 = scale_value(sw, w0 + kb + (two ? w1 : 0), kE8);
        if (!waited) {
          ok = wait_h(ch);
          if (!ok) break;
          waited = true;
        }
        float* out = tab + (b.i * kBatch + j) * tab_row;
#pragma unroll 1
        for (int c0 = 0; c0 < ch.n; c0 += 4 * kLoads) {
          int64_t at[kLoads];
          float v[kLoads], z[kLoads];
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = ch.row0 + min(c0 + (lane >> 3) + 4 * i, ch.n - 1);
            at[i] = static_cast<int64_t>(down ? r : row_tok[r]) * kbs + kb;
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            v[i] = scale_value(sx, at[i], kE8);
            z[i] = scale_value(sx, at[i] + (down && two ? 1 : 0), kE8);
          }
          if (c0 == 0) {
            ok = mbar_wait_warp(&bar.sempty[b.i], b.phase ^ 1u, limit);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int c = c0 + (lane >> 3) + 4 * i;
            if (c < ch.n) {
              out[c] = v[i] * s0;
              out[head.ncol + c] = two ? z[i] * s1 : 0.0f;
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sfull[b.i]);
      }
    }
    if (!ok) give_up();
  } else if (warp == 3) {
    // -------------------------------------------------------- token blocks --
    Ring r;
    int issued = 0;
    bool ok = true;
    Chunk ch;
    while (ok && next_chunk(ch, false)) {
      const bool down = ch.kind != 0;
      const int n4 = (ch.n + 3) / 4, n16 = (ch.n + 15) / 16;
      int tok[4] = {0, 0, 0, 0};
      if (down) {
        const bool fenced = all_ready;
        ok = wait_h(ch);
        if (!fenced) fence_proxy_async_all();   // h's codes were written through the generic proxy
      } else if (lane < n4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tok[q] = row_tok[ch.row0 + min(4 * lane + q, ch.n - 1)];
      }
#pragma unroll 1
      for (int k = ch.k0; ok && k < ch.k1; ++k) {
        ok = mbar_wait_warp(&bar.empty[r.i], r.phase ^ 1u, limit);
        if (!ok) break;
        uint8_t* to = xtiles + r.i * 2 * head.xbytes;
        const bool two = down && 2 * k + 1 < IB;
        if (elect_one())
          mbar_arrive_expect_tx(&bar.fullx[r.i], down ? n16 * (two ? 4096 : 2048) : n4 * 512);
        __syncwarp();
        if (!down) {
          if (lane < n4)
            tma_gather4_2d(to + lane * 512, &tmap_a, &bar.fullx[r.i], k * 128, tok[0], tok[1],
                           tok[2], tok[3]);
        } else if (lane < 2 * n16 && (two || !(lane & 1))) {
          tma_load_2d(to + (lane & 1) * head.xbytes + (lane >> 1) * 2048, &tmap_h,
                      &bar.fullx[r.i], k * 256 + (lane & 1) * 128, ch.row0 + (lane >> 1) * 16);
        }
        __syncwarp();
        ++issued;
        r.next(head.stages);
      }
    }
    if (!ok) give_up();
    const int pending = issued < head.stages ? issued : head.stages;
#pragma unroll 1
    for (int i = 0; i < pending; ++i) {
      int st = r.i - 1 - i;
      uint32_t ph = r.phase;
      if (st < 0) {
        st += head.stages;
        ph ^= 1u;
      }
      mbar_wait(&bar.fullx[st], ph, kDefaultWaitCycles);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------ counts chunks --
    // A chunk's place in the ring is given back only here and after its count,
    // which keeps `dumped` within one phase.
    Chunk ch;
    bool ok = true;
    while (ok && next_chunk(ch, true)) {
      ok = mbar_wait_warp(&bar.dumped[mr.i], mr.phase, limit);
      if (ok && lane == 0) {
        __threadfence();   // the partial sums of all promotion warps before the count
        atomicAdd((ch.kind != 0 ? args.plan.count_down : args.plan.count_gu) + ch.count, 1);
        mbar_arrive(&bar.mempty[mr.i]);
      }
      __syncwarp();
      mr.next(kMail);
    }
    if (!ok) give_up();
  } else if (warp >= kPromo0) {
    // ------------------------------------------------------------ promotion --
    const int wg = (warp - kPromo0) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;                  // weight row of the tile
    const uint32_t tlane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const int ncol = head.ncol;
    Ring tb, sb;
    bool ok = true;
    for (;;) {
      int col0, cols, k, k1;
      {
        Chunk ch;
        if (!next_chunk(ch, true)) break;
        // this warpgroup's columns: [col0, col0 + cols)
        const int per = (ch.n + 8 * kWgs - 1) / (8 * kWgs) * 8;
        col0 = wg * per;
        cols = max(0, min(per, (ch.n + 7) / 8 * 8 - col0));
        k = 0;
        k1 = ch.k1 - ch.k0;
      }
      // the two products of the chunk's units times their scale products
      float acc[2][kPer];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[p][c] = 0.0f;
#pragma unroll 1
      for (; k < k1; ++k) {
        const int j = k % kBatch;
        const bool batch_end = j == kBatch - 1 || k == k1 - 1;
        if (j == 0) ok = mbar_wait_warp(&bar.sfull[sb.i], sb.phase, limit);
        ok = ok && mbar_wait_warp(&bar.tfull[tb.i], tb.phase, limit);
        if (!ok) break;
        tc_fence_after();
        const float* sc = tab + (sb.i * kBatch + j) * tab_row + col0;
        const uint32_t ta = tlane + static_cast<uint32_t>(tb.i * 2 * ncol + col0);
#pragma unroll
        for (int c = 0; c < kPer; c += 8) {
          if (c < cols) {
            float v[2][8];
#pragma unroll
            for (int p = 0; p < 2; ++p) tmem_ld8(ta + p * ncol + c, v[p]);
            tmem_wait_ld();
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
              for (int i = 0; i < 8; i += 4) {
                const float4 q = *reinterpret_cast<const float4*>(sc + p * ncol + c + i);
                fma2(acc[p][c + i], acc[p][c + i + 1], v[p][i], v[p][i + 1], q.x, q.y);
                fma2(acc[p][c + i + 2], acc[p][c + i + 3], v[p][i + 2], v[p][i + 3], q.z, q.w);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.tempty[tb.i]);
          if (batch_end) mbar_arrive(&bar.sempty[sb.i]);
        }
        if (batch_end) sb.next(kTabs);
        tb.next(head.bufs);
      }
      if (!ok) break;
      // gate+up: both values; down: their sum. (The chunk is read again: the sums
      // leave no registers to keep it.)
      const Chunk& ch = sh.mail[mr.i];
      const bool down = ch.kind != 0;
      const int64_t step = down ? args.shape.K : IB * 256;
      float* to = (down ? args.part_down + ch.tile * 128 : args.part_gu + ch.tile * 256) +
                  (static_cast<int64_t>(ch.c) * head.rows + ch.row0 + col0) * step + row;
      const int mine = min(cols, ch.n - col0);
#pragma unroll
      for (int c = 0; c < kPer; ++c, to += step) {
        if (c < mine) {
          __stcg(to, down ? acc[0][c] + acc[1][c] : acc[0][c]);
          if (!down) __stcg(to + 128, acc[1][c]);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.dumped[mr.i]);
        mbar_arrive(&bar.mempty[mr.i]);
      }
      mr.next(kMail);
    }
    if (!ok) give_up();
    tc_fence_before();
  }
  if (warp >= 6) {
    // ------------------------------------------------------------ finishers --
    // read again: the promotion warps have no registers to carry it
    const Head head = load_head(args.plan.head);
    bool ok = true;
    int16_t* pair_row = reinterpret_cast<int16_t*>(smem + args.off_row);
    float* pair_w = reinterpret_cast<float*>(smem + args.off_w);
    if (warp < kPromo0) {   // for the promotion warps too: y is long after
#pragma unroll 1
      for (int i = threadIdx.x - 192; i < args.shape.M * args.shape.top_k; i += 32 * kFin) {
        pair_row[i] = static_cast<int16_t>(__ldcg(args.plan.pair_row + i));
        pair_w[i] = __ldcg(args.plan.pair_w + i);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.pairs);
    }
    bool pairs_there = false;
    const int64_t gu_row = static_cast<int64_t>(IB) * 256;   // floats of a row of part_gu
    while (!stopped()) {
      int task = 0;
      if (lane == 0) task = atomicAdd(args.plan.ticket + 1, 1);
      task = __shfl_sync(0xffffffffu, task, 0);
      if (task >= head.n_tasks) break;
      if (task < head.n_h) {
        // h = silu(g) * u of some rows: the warp has a row's 128 columns, a lane
        // four of them
        const int s = task / head.groups;
        const int a = s / IB, tile = s - a * IB;
        const int row0 = act[a].y + (task - s * head.groups) * head.fin_rows;
        const int row1 = min(row0 + head.fin_rows, act[a + 1].y);
        if (row0 < row1) ok = wait_count_warp(args.plan.count_gu + s, head.cpt, limit);
        if (!ok) break;
        // eight parts are loaded together: of two rows where a row has at most four
        const bool pair = head.cpt <= 4;
        const int64_t part = head.rows * gu_row / 4;
#pragma unroll 1
        for (int row = row0; row < row1; row += pair ? 2 : 1) {
          const float4* from =
              reinterpret_cast<const float4*>(args.part_gu + row * gu_row + tile * 256) + lane;
          float4 g[2], u[2];
          g[0] = u[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
          for (int q = 0; q < head.cpt; q += 8) {
            float4 x[8], z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = pair ? i >> 2 : 0, p = pair ? i & 3 : q + i;
              x[i] = z[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (p < head.cpt && row + r < row1) {
                x[i] = __ldcg(from + r * (gu_row / 4) + p * part);
                z[i] = __ldcg(from + r * (gu_row / 4) + p * part + 32);
              }
            }
            g[1] = x[4];
            u[1] = z[4];
            add4(g[0], x[0]);
            add4(u[0], z[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              add4(g[0], x[i]);
              add4(u[0], z[i]);
              add4(g[1], x[4 + i]);
              add4(u[1], z[4 + i]);
            }
            if (!pair) {
              add4(g[0], g[1]);
              add4(u[0], u[1]);
            }
          }
#pragma unroll 1
          for (int r = 0; r < (pair ? 2 : 1) && row + r < row1; ++r) {
            const float4 gr = r == 0 ? g[0] : g[1], ur = r == 0 ? u[0] : u[1];
            const float h[4] = {silu_f32(gr.x) * ur.x, silu_f32(gr.y) * ur.y,
                                silu_f32(gr.z) * ur.z, silu_f32(gr.w) * ur.w};
            // magnitudes are compared as integers, so that a NaN is the largest
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(h[i]) & 0x7FFFFFFFu);
            const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, m));
            const int64_t at = static_cast<int64_t>(row + r) * IB + tile;
            uint32_t q;
            if constexpr (kE8) {
              const uint32_t code = ue8m0_code_or_nan(amax);
              q = codes4f_pow2(h[0], h[1], h[2], h[3], ue8m0_inv_scale(code));
              if (lane == 0) static_cast<uint8_t*>(args.sh)[at] = static_cast<uint8_t>(code);
            } else {
              const float sc = scale_of_amax(amax);
              q = codes4f(h[0], h[1], h[2], h[3], ScaleDivider(sc));
              if (lane == 0) static_cast<float*>(args.sh)[at] = sc;
            }
            *reinterpret_cast<uint32_t*>(args.qh + at * 128 + lane * 4) = q;
          }
        }
        fence_proxy_async_all();   // TMA reads the codes
        __syncwarp();
        if (lane == 0) {
          __threadfence();
          atomicAdd(args.plan.ready + a * head.cps + tile / 2 / head.q_down, 1);
          atomicAdd(h_done, 1);
        }
      } else {
        // y of some (token, quarter of the 128 columns). Eight lanes have an
        // item's 32 columns; the warp's 16 slots (four groups of lanes, four
        // registers) are the parts of one item or, where it has fewer, of several
        const int s = task - head.n_h;
        const int tile = s / args.shape.y_tasks;
        const int item0 = (s - tile * args.shape.y_tasks) * args.shape.y_items;
        const int item1 = min(item0 + args.shape.y_items, 4 * args.shape.M);
        ok = wait_count_warp(args.plan.count_down + tile, head.blocks * head.cps, limit);
        if (!ok) break;
        if (!pairs_there) ok = mbar_wait_warp(&bar.pairs, 0, limit);
        if (!ok) break;
        pairs_there = true;
        // part p: chunk p % cps of the token's row p / cps
        const int parts = head.top * head.cps;
        const int lg = parts > 8 ? 4 : parts > 4 ? 3 : parts > 2 ? 2 : parts > 1 ? 1 : 0;   // slots of an item
        const int grp = lane >> 3;
#pragma unroll 1
        for (int it = item0; it < item1; it += 16 >> lg) {
          float4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
          for (int p0 = 0; p0 < parts; p0 += 1 << lg) {
            float4 x[4];
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int slot = 4 * i + grp;
              const int item = it + (slot >> lg), p = p0 + (slot & ((1 << lg) - 1));
              const int j = head.cps == 1 ? p : p / head.cps;
              const bool there = item < item1 && p < parts;
              const int pair = there ? (item >> 2) * args.shape.top_k + j : 0;
              const int r = there ? pair_row[pair] : -1;
              w[i] = r >= 0 ? pair_w[pair] : 0.0f;
              const float* from = args.part_down +
                                  (static_cast<int64_t>(p - j * head.cps) * head.rows + r) *
                                      args.shape.K +
                                  tile * 128 + (item & 3) * 32;
              x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (r >= 0) x[i] = __ldcg(reinterpret_cast<const float4*>(from) + (lane & 7));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i].x = fmaf(w[i], x[i].x, v[i].x);
              v[i].y = fmaf(w[i], x[i].y, v[i].y);
              v[i].z = fmaf(w[i], x[i].z, v[i].z);
              v[i].w = fmaf(w[i], x[i].w, v[i].w);
            }
          }
          // an item's slots: registers first, then groups of lanes
          if (lg >= 3) {
            add4(v[0], v[1]);
            add4(v[2], v[3]);
          }
          if (lg == 4) add4(v[0], v[2]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int slot = 4 * i;
            if ((slot & ((1 << lg) - 1)) != 0) continue;   // the same in all lanes
            if (lg >= 1) add4(v[i], shfl_xor4(v[i], 8));
            if (lg >= 2) add4(v[i], shfl_xor4(v[i], 16));
            const int item = it + ((slot + grp) >> lg);
            if (item < item1 && (grp & ((1 << lg) - 1)) == 0) {
              const __nv_bfloat162 lo = __floats2bfloat162_rn(v[i].x, v[i].y);
              const __nv_bfloat162 hi = __floats2bfloat162_rn(v[i].z, v[i].w);
              *reinterpret_cast<uint2*>(args.y + static_cast<int64_t>(item >> 2) * args.shape.K +
                                        tile * 128 + (item & 3) * 32 + (lane & 7) * 4) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                             *reinterpret_cast<const uint32_t*>(&hi));
            }
          }
        }
      }
    }
    if (!ok) give_up();
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int kN, int kWgs, bool kE8>
int launch_mlp(const CUtensorMap (&maps)[4], const MlpArgs& args, int grid, int device,
               cudaStream_t stream) {
  auto kern = moe_mlp_kernel<kN, kWgs, kE8>;
  static std::once_flag flags[64];
  cudaError_t attr_err = cudaSuccess;
  std::call_once(flags[device], [&] {
    attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (attr_err != cudaSuccess) return FP8BS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(32 * (6 + kFin) + 128 * kWgs, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], args) == cudaSuccess
             ? FP8BS_OK
             : FP8BS_ERR_CUDA;
}

template <bool kE8>
int launch_mlp_n(const CUtensorMap (&maps)[4], const MlpArgs& args, int device,
                 cudaStream_t stream) {
  if (args.shape.M <= 16) return launch_mlp<16, 2, kE8>(maps, args, args.shape.sms, device, stream);
  if (args.shape.M <= 32) return launch_mlp<32, 2, kE8>(maps, args, args.shape.sms, device, stream);
  return launch_mlp<64, 2, kE8>(maps, args, args.shape.sms, device, stream);
}

}  // namespace

size_t moe_workspace_bytes(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  return carve(nullptr, M, K, I, E, top_k).bytes;
}

int launch_moe_mlp(const MoeArgs& a, bool ue8m0, cudaStream_t stream) {
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  const int pairs = a.M * a.top_k;
  const Workspace w = carve(a.workspace, a.M, a.K, a.I, a.E, a.top_k);
  alignas(64) CUtensorMap maps[4];   // gate+up, down, tokens, h
  if (int st = encode_tmap_2d_u8(&maps[0], a.qg, a.K, static_cast<uint64_t>(a.E) * 2 * a.I, a.K,
                                 128, 128, kSwizzle128B))
    return st;
  if (int st = encode_tmap_2d_u8(&maps[1], a.qd, a.I, static_cast<uint64_t>(a.E) * a.K, a.I, 128,
                                 128, kSwizzle128B))
    return st;
  if (int st = encode_tmap_2d_u8(&maps[2], a.qa, a.K, a.M, a.K, 128, 1, kSwizzle128B)) return st;
  if (int st = encode_tmap_2d_u8(&maps[3], w.qh, a.I, pairs, a.I, 128, 16, kSwizzle128B))
    return st;

  const Layout lay(pairs, a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64);
  MlpArgs g{};
  g.plan = w.plan;
  g.shape.M = a.M;
  g.shape.K = a.K;
  g.shape.I = a.I;
  g.shape.top_k = a.top_k;
  g.shape.sms = dev.sm_count;
  g.shape.room = lay.room();
  g.shape.cap_gu = w.cap_gu;
  g.shape.cap_down = w.cap_down;
  // one y task for each warp that can take one (promotion's too, by then)
  const int y_all = 4 * a.M * (a.K / 128);
  g.shape.y_items = (y_all + 10 * dev.sm_count - 1) / (10 * dev.sm_count);
  g.shape.y_tasks = (4 * a.M + g.shape.y_items - 1) / g.shape.y_items;
  g.sa = a.sa;
  g.sg = a.sg;
  g.sd = a.sd;
  g.qh = w.qh;
  g.sh = w.sh;
  g.y = a.y;
  g.part_gu = w.part_gu;
  g.part_down = w.part_down;
  g.off_row = lay.off_row;
  g.off_w = lay.off_w;
  g.off_tab = lay.off_tab;
  g.off_tiles = lay.off_tiles;
  g.wait_limit = a.wait_limit;
  g.err = a.err;

  // a thread for each expert; more where there are more choices
  const int want = a.E > pairs ? a.E : pairs;
  const int threads = want < 256 ? 256 : want < kPlanThreads ? (want + 31) / 32 * 32 : kPlanThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, moe_plan_kernel, a.ids, a.weights, pairs, a.E, a.first_expert,
                         g.plan, g.shape) != cudaSuccess)
    return FP8BS_ERR_CUDA;
  return ue8m0 ? launch_mlp_n<true>(maps, g, dev.device, stream)
               : launch_mlp_n<false>(maps, g, dev.device, stream);
}

}  // namespace fp8bs
