/*
 * fp8bs.h - C ABI of the fine-grained (block-scaled, group-128) FP8 linear
 * layer for NVIDIA B200 (sm_100a).
 *
 * The layer computes Y = X . W^T for bf16 X [M, K] and W [N, K] through 8-bit
 * floating point:
 *
 *   - activations are quantised per token in groups of 128 input channels,
 *     one fp32 scale per group, computed at run time ("FP8 à granularité
 *     fine", Hugging Face transformers docs, opening bullets and section
 *     "Chemin rapide de DeepGEMM": activation_scheme="dynamic");
 *   - weights are quantised per 128x128 block, one fp32 scale per block (same
 *     page, opening bullets: weight_block_size=(128, 128); section "Format
 *     d'échelle UE8M0": scales kept as plain float32, scale_fmt="float");
 *   - Y[m,n] = sum_kb sA[m,kb] * sW[n/128,kb] * sum_{k in kb} qA[m,k] qW[n,k],
 *     accumulated in fp32 and rounded to bf16;
 *   - a 2:4 variant keeps the two largest |w| of every 4 contiguous weights
 *     along K ("Déployer la parcimonie 2:4 avec FP8 sur Hopper", steps 2, 4,
 *     6 and "Exemples pratiques 1"; "Combiner élagage et quantification ...",
 *     section "La clé : la sparsité structurée 2:4") and multiplies the
 *     compressed weights.
 *
 * Number format: OCP FP8 E4M3 ("fn": bias 7, no infinities, max 448).
 * Scale of a group or block: s = amax / 448 (fp32 IEEE division). Element
 * code: e4m3(x / s) with one fp32 IEEE division, round-to-nearest-even,
 * saturating to +-448. A group or block whose amax is 0 has s = 0 and every
 * element encodes as a zero carrying the element's sign (0x00 or 0x80).
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller. The library
 *     never allocates, frees or synchronises; every call is asynchronous on
 *     `stream` (a cudaStream_t; NULL means the legacy default stream).
 *   - All matrices are dense row-major, with no leading-dimension argument.
 *   - K must be a positive multiple of 128. M == 0 or N == 0 is a no-op that
 *     returns FP8BS_OK.
 *   - Every matrix pointer (activations, weights, codes, metadata, outputs)
 *     must be 16-byte aligned; fp32 scale arrays and expert indices need
 *     4-byte alignment; UE8M0 scale-code arrays (bytes) need none.
 *   - Arguments are validated before anything is launched; on an error
 *     nothing is written and a nonzero FP8BS_ERR_* code is returned.
 *   - A launch failure returns FP8BS_ERR_CUDA. A kernel that gave up a bounded
 *     internal wait records FP8BS_ERR_DEVICE_TIMEOUT in a device error word,
 *     read by fp8bs_get_device_error().
 *   - Input and output buffers must not overlap.
 */
#ifndef FP8BS_H_
#define FP8BS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8BS_OK = 0,
  FP8BS_ERR_NULL = 1,           /* a required pointer is NULL */
  FP8BS_ERR_SHAPE = 2,          /* K % 128 != 0, K <= 0, M/N < 0, or a size too large */
  FP8BS_ERR_ALIGN = 3,          /* a pointer is not aligned (16 bytes; 4 for scales / indices) */
  FP8BS_ERR_WORKSPACE = 4,      /* workspace smaller than fp8bs_gemm_workspace_bytes() */
  FP8BS_ERR_CUDA = 5,           /* a CUDA runtime/driver call failed */
  FP8BS_ERR_DEVICE_TIMEOUT = 6, /* a kernel gave up a bounded wait */
  FP8BS_ERR_ARCH = 7,           /* the current device is not sm_100 */
  FP8BS_ERR_SCRATCH_LIMIT = 8   /* the problem needs more than the fixed no-allocation scratch */
} fp8bs_status;

/*
 * Dynamic per-token activation quantization in 1x128 groups along K
 * ("FP8 à granularité fine", opening bullets; "Chemin rapide de DeepGEMM").
 *
 *   x_bf16   [M][K] bf16, input.
 *   qa_e4m3  [M][K] E4M3 bytes, output: qa[m][k] = e4m3(x[m][k] / sa[m][k/128]).
 *   sa       [M][K/128] fp32, output: sa[m][g] = amax_{k in group g} |x[m][k]| / 448.
 */
int fp8_quant_act_group128(const void* x_bf16, int64_t M, int64_t K, void* qa_e4m3, float* sa,
                           void* stream);

/*
 * Weight quantization in 128x128 blocks ("FP8 à granularité fine", opening
 * bullets, weight_block_size=(128, 128)).
 *
 *   w_bf16   [N][K] bf16, input.
 *   qw_e4m3  [N][K] E4M3 bytes, output.
 *   sw       [ceil(N/128)][K/128] fp32, output: block amax / 448. The last row
 *            block covers only the valid rows when N % 128 != 0.
 */
int fp8_quant_weight_block128(const void* w_bf16, int64_t N, int64_t K, void* qw_e4m3, float* sw,
                              void* stream);

/*
 * 2:4 magnitude pruning along K, then block quantization and compression
 * ("Déployer la parcimonie 2:4 avec FP8 sur Hopper", steps 2, 4 and 6;
 * "Combiner élagage et quantification ...", section on 2:4 sparsity).
 *
 * In every group of 4 contiguous weights along K the two largest |w| are kept
 * (equal magnitudes: the lower index wins) and the other two become +0. The
 * pruned matrix is then quantized exactly like fp8_quant_weight_block128
 * (scales recomputed after pruning).
 *
 *   w_bf16         [N][K] bf16, input.
 *   vals_e4m3      [N][K/2] E4M3 bytes, output: the two kept codes of group g
 *                  at [n][2g] and [n][2g+1], in order of position.
 *   meta           [N][K/8] bytes, output: byte j holds group 2j in bits 0-3
 *                  and group 2j+1 in bits 4-7; each nibble is i0 | (i1 << 2)
 *                  with i0 < i1 the kept positions (0..3) within the group.
 *   sw             [ceil(N/128)][K/128] fp32, output.
 *   w_pruned_bf16  [N][K] bf16, optional output (may be NULL): the pruned
 *                  weights in bf16.
 */
int prune24_compress(const void* w_bf16, int64_t N, int64_t K, void* vals_e4m3, uint8_t* meta,
                     float* sw, void* w_pruned_bf16, void* stream);

/*
 * Block-scaled FP8 GEMM ("FP8 à granularité fine": 1x128 activation groups
 * against 128x128 weight blocks):
 *   y[m][n] = bf16_rn( sum_kb sa[m][kb] * sw[n/128][kb] * sum_{k in kb} qa[m][k] * qw[n][k] )
 * with fp32 accumulation.
 *
 *   qa  [M][K] E4M3, sa [M][K/128] fp32  (from fp8_quant_act_group128)
 *   qw  [N][K] E4M3, sw [ceil(N/128)][K/128] fp32  (from fp8_quant_weight_block128)
 *   y_bf16 [M][N] bf16, output. N must be a multiple of 8.
 *   workspace / workspace_bytes: scratch of at least
 *       fp8bs_gemm_workspace_bytes(M, N, K, 0) bytes (may be NULL when that is 0).
 * Results are deterministic: the same inputs give the same bytes every call.
 */
int fp8_block_gemm(const void* qa, const float* sa, const void* qw, const float* sw, void* y_bf16,
                   int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * fp8_block_gemm with the next layer's input quantization fused in: the same
 * y, and qy / sy = fp8_quant_act_group128(y) of that bf16 y, i.e. y's rows
 * cut into 1x128 groups along N ("FP8 à granularité fine": the output of one
 * linear is the activation of the next, quantized per token per 128
 * channels). For M > 256 the GEMM's epilogue quantizes its own tile (each
 * promotion thread holds one group); for M <= 16 with unsplit decode tiles
 * (N of at least 75 row blocks on 148 SMs) the decode-order epilogue
 * quantizes each token's staged group; otherwise y is written and then
 * quantized by the activation quantizer.
 *
 *   y_bf16  [M][N] bf16, output; may be NULL when M > 256 (then only the codes
 *           are written), required when M <= 256.
 *   qy_e4m3 [M][N] E4M3 codes, output; sy [M][N/128] fp32 scales, output.
 *   N must be a multiple of 128; the other arguments as fp8_block_gemm.
 * Returns FP8BS_ERR_SHAPE for N % 128 != 0 and FP8BS_ERR_NULL for a missing
 * qy / sy (or y with M <= 256).
 */
int fp8_block_gemm_quant(const void* qa, const float* sa, const void* qw, const float* sw,
                         void* y_bf16, void* qy_e4m3, float* sy, int64_t M, int64_t N, int64_t K,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The block-scaled GEMM with 2:4-compressed weights (vals, meta, sw as written
 * by prune24_compress). Same result definition as fp8_block_gemm with qw the
 * decompressed codes (pruned positions are code 0).
 */
int fp8_sparse24_gemm(const void* qa, const float* sa, const void* vals, const uint8_t* meta,
                      const float* sw, void* y_bf16, int64_t M, int64_t N, int64_t K,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * UE8M0 scale variant ("FP8 à granularité fine", section "Format d'échelle
 * UE8M0": scales stored as float8_e8m0fnu, a bare power of two). A scale is
 * kept as one code byte c standing for 2^(c - 127); it is the smallest power
 * of two s with 448 * s >= amax (so no element saturates), codes clamped to
 * 0..254, amax == 0 -> code 0. Elements are e4m3(x / s) as above (the quotient
 * by a power of two is exact unless it underflows).
 *
 *   fp8_quant_act_group128_ue8m0:    x_bf16 [M][K] -> qa_e4m3 [M][K], sa_ue8m0 [M][K/128]
 *   fp8_quant_weight_block128_ue8m0: w_bf16 [N][K] -> qw_e4m3 [N][K],
 *                                    sw_ue8m0 [ceil(N/128)][K/128]
 *   fp8_block_gemm_ue8m0: y = sum_kb 2^(sa - 127) 2^(sw - 127) (qa_kb . qw_kb^T),
 *       fp32 accumulation, bf16 out (N a multiple of 8); the tensor cores apply
 *       the scales themselves (block-scaled MMA), so there is no per-K-block
 *       promotion. Workspace as fp8_block_gemm (none needed).
 * Argument rules and errors as the fp32-scale entry points.
 */
int fp8_quant_act_group128_ue8m0(const void* x_bf16, int64_t M, int64_t K, void* qa_e4m3,
                                 uint8_t* sa_ue8m0, void* stream);
int fp8_quant_weight_block128_ue8m0(const void* w_bf16, int64_t N, int64_t K, void* qw_e4m3,
                                    uint8_t* sw_ue8m0, void* stream);
int fp8_block_gemm_ue8m0(const void* qa, const uint8_t* sa_ue8m0, const void* qw,
                         const uint8_t* sw_ue8m0, void* y_bf16, int64_t M, int64_t N, int64_t K,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Grouped (mixture-of-experts) block-scaled GEMMs ("FP8 à granularité fine",
 * section "Chemin rapide de DeepGEMM": the experts' products run through
 * grouped kernels; with UE8M0 scales on SM100 per section "Format d'échelle
 * UE8M0", with fp32 scales as a grouped matmul). The token rows are grouped
 * by expert in one matrix (the contiguous layout):
 *
 *   y[m][n] = sum_kb sa[m][kb] * sw[e][n/128][kb] * sum_{k in kb} qa[m][k] qw[e][n][k],
 *             e = m_indices[m]
 *
 *   qa [M][K] E4M3, sa [M][K/128] (fp32, or UE8M0 codes for the _ue8m0 form).
 *   qw [E][N][K] E4M3, sw [E][ceil(N/128)][K/128] (fp32, or UE8M0 codes).
 *   m_indices [M] int32, device memory: the expert of each row, or -1 for a
 *       padding row. Every aligned group of 128 rows (rows 128t .. 128t+127)
 *       must hold rows of a single expert plus padding rows: each expert's
 *       rows start at a multiple of 128. The expert of a tile is read from its
 *       first row; an index outside [0, E) there counts as expert 0.
 *   y_bf16 [M][N]: rows of real tokens are written; padding rows receive
 *       values with no defined meaning.
 * N a multiple of 8, K of 128, E >= 1. Same errors as fp8_block_gemm.
 */
int fp8_grouped_gemm(const void* qa, const float* sa, const void* qw, const float* sw,
                     const int32_t* m_indices, void* y_bf16, int64_t M, int64_t N, int64_t K,
                     int64_t E, void* workspace, size_t workspace_bytes, void* stream);
int fp8_grouped_gemm_ue8m0(const void* qa, const uint8_t* sa_ue8m0, const void* qw,
                           const uint8_t* sw_ue8m0, const int32_t* m_indices, void* y_bf16,
                           int64_t M, int64_t N, int64_t K, int64_t E, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * The gated MLP's gate+up GEMM with SwiGLU fused into its epilogue, keeping
 * both block scales (TensorRT-LLM docs, performance/fp8-quantization, section
 * "GEMM + SwiGLU Fusion in Gated-MLP": two matmuls and the SwiGLU in one
 * kernel), and the down projection's input quantization after it:
 *
 *   g, u = the block-scaled GEMM of qa with the gate rows [0, I) and the up
 *          rows [I, 2I) of qw_gate_up, in fp32;
 *   h    = bf16_rn( silu(g) * u ),  silu(g) = g / (1 + e^-g);
 *   qh, sh = fp8_quant_act_group128(h)   (1x128 groups along I).
 *
 *   qa [M][K], sa [M][K/128]           (the activations, as fp8_block_gemm)
 *   qw_gate_up [2I][K], sw_gate_up [2I/128][K/128]  ([W_gate; W_up] quantized
 *       with fp8_quant_weight_block128)
 *   h_bf16 [M][I] bf16, output, may be NULL; qh_e4m3 [M][I], sh [M][I/128].
 *   workspace: at least fp8bs_swiglu_workspace_bytes(M, I) bytes, 16-byte
 *       aligned (required for M <= 256 only, else may be NULL): there the
 *       call may run the decode-order GEMM of the 2I weight rows into this
 *       scratch (g and u rounded to bf16) and a second kernel that forms h and
 *       its codes; otherwise (M > 256, or M > 64 with 2I wide enough that
 *       tiles of 128 tokens x 256 weight rows fill at least three quarters of
 *       the GPU) one kernel does all of it from the fp32 accumulators. Both
 *       forms meet the same tolerance on h.
 *   I must be a positive multiple of 128. Same errors as fp8_block_gemm;
 *   FP8BS_ERR_WORKSPACE for a missing or short workspace.
 */
int fp8_gemm_swiglu_quant(const void* qa, const float* sa, const void* qw_gate_up,
                          const float* sw_gate_up, void* h_bf16, void* qh_e4m3, float* sh,
                          int64_t M, int64_t I, int64_t K, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Scratch bytes fp8_gemm_swiglu_quant needs for M tokens and intermediate size I. */
size_t fp8bs_swiglu_workspace_bytes(int64_t M, int64_t I);

/*
 * fp8_gemm_swiglu_quant without a workspace and without any device allocation
 * (no cudaMalloc / cudaFree, no allocating library call). The paper (the
 * pages this library follows) has no counterpart: it exists for callers that
 * cannot hand over or obtain device memory per call, such as a C host that
 * owns every buffer and passes only operands in and out (a plugin or
 * custom-op interface with no workspace slot), or a decode loop that must not
 * enter an allocator because
 * cudaMalloc / cudaFree may synchronise the device and fail once a memory
 * pool has reserved the free memory.
 *
 * Same operands, results and tolerance as fp8_gemm_swiglu_quant. For
 * M <= 256 the [M][2I] bf16 intermediate lives in one fixed device array of
 * FP8BS_NOALLOC_SCRATCH_BYTES (16 MiB) per device, reserved when the library's
 * module is loaded; calls needing more (M <= 256 and M * 2I * 2 bytes above
 * it: every M for I <= 16384; for I = 28672, M in 147 .. 256) return
 * FP8BS_ERR_SCRATCH_LIMIT before anything is launched. Nothing in the array
 * must start at zero: each call writes all of it that it reads. For M > 256
 * no scratch is used.
 *
 * Setup: the first call on a device (any M, including 0, with that device
 * current) looks up the array's address (cudaGetSymbolAddress) and caches it;
 * make it before any stream capture. Calls on one device share the array:
 * calls that overlap in time (other streams or host threads without ordering
 * between them) race on it and give wrong results.
 */
#define FP8BS_NOALLOC_SCRATCH_BYTES (16u << 20)
int fp8_gemm_swiglu_quant_noalloc(const void* qa, const float* sa, const void* qw_gate_up,
                                  const float* sw_gate_up, void* h_bf16, void* qh_e4m3,
                                  float* sh, int64_t M, int64_t I, int64_t K, void* stream);

/*
 * Output-column (N) split over P ranks (tensor parallelism; TensorRT-LLM docs,
 * performance/fp8-quantization: the Llama-3.3-70B case study runs tensor
 * parallel over 4 GPUs). Rank p holds weight rows [p Np, (p + 1) Np) (Np a
 * multiple of 128, so whole 128x128 blocks) and computes those columns of Y;
 * an all-gather over the ranks leaves them rank-major, [P][M][Np]. This call
 * turns that into the full rows: dst[m][p Np + j] = src[p][m][j].
 *   src_bf16 [P][M][Np], dst_bf16 [M][P Np], both bf16, no overlap;
 *   Np a multiple of 8.
 */
int fp8_gather_columns(const void* src_bf16, int64_t P, int64_t M, int64_t Np, void* dst_bf16,
                       void* stream);

/*
 * The input of a layer's FP8 linears from the residual stream: residual
 * addition, root-mean-square norm and dynamic 1x128 quantization in one pass.
 *
 *   r = bf16_rn(x + residual)   (r = x when residual_bf16 is NULL)
 *   n = r * w / sqrt(mean_k r^2 + eps)   in fp32, the mean over a row
 *   y = bf16_rn(n),  s[m][g] = amax_{k in group g} |n| / 448,  q = e4m3(n / s)
 *
 *   x_bf16 [M][K]; residual_bf16 [M][K] or NULL; weight_bf16 [K] or NULL (ones).
 *   residual_out_bf16 [M][K] or NULL: r. It may be the same pointer as
 *       residual_bf16 or x_bf16 (an update in place); no other two buffers may
 *       overlap.
 *   y_bf16 [M][K] or NULL (the router of a mixture of experts reads it).
 *   q_e4m3 [M][K], s [M][K/128] fp32 (the _ue8m0 form: codes, one byte each).
 *   eps >= 0 and finite. Finite rows may be of any size: squares beyond fp32 are
 *       no less exact. With eps = 0 a row of zeros gives NaN (0 / 0).
 * The codes come from the fp32 n (not from y). They are those of e4m3(n / s)
 * except where n / s lies within two fp32 ulps of the middle between two codes.
 * More rows than the GPU has SMs (148) take another kernel than fewer: the same
 * row can differ in such a code, and in the last bits of n, between the two.
 * K a positive multiple of 128, at most 65536. A group with an n that is NaN or
 * beyond fp32 gets the scale NaN (UE8M0: code 255). A row with a NaN is NaN
 * throughout; in one with an infinity n is NaN there and 0 elsewhere.
 */
int fp8_add_rmsnorm_quant(const void* x_bf16, const void* residual_bf16, const void* weight_bf16,
                          float eps, int64_t M, int64_t K, void* residual_out_bf16, void* y_bf16,
                          void* q_e4m3, float* s, void* stream);
int fp8_add_rmsnorm_quant_ue8m0(const void* x_bf16, const void* residual_bf16,
                                const void* weight_bf16, float eps, int64_t M, int64_t K,
                                void* residual_out_bf16, void* y_bf16, void* q_e4m3,
                                uint8_t* s_ue8m0, void* stream);

/*
 * The router's choice for a mixture-of-experts layer: the top_k of E experts of
 * every token from its logits, and their weights.
 *
 *   logits [M][E], fp32 (logits_bf16 == 0) or bf16 (!= 0).
 *   bias [E] fp32 or NULL: added to the scores for the choice only, not in the
 *       weights.
 *   scoring: FP8BS_ROUTE_SOFTMAX or FP8BS_ROUTE_SIGMOID.
 *   n_group, topk_group: with n_group > 1 the experts form n_group groups of
 *       E / n_group neighbours; a group scores the sum of its two largest keys
 *       (of its one, where only one is left) and only the experts of the
 *       topk_group best groups can be chosen. n_group == 1: no groups.
 *       A bias or groups need sigmoid scoring.
 *   ids [M][top_k] int32, weights [M][top_k] fp32, output, by key, largest first.
 *
 * The key of an expert is its logit; with a bias or with groups it is
 * sigmoid(logit) + bias, evaluated in double precision. Equal keys, and equal
 * group scores, go to the lower index. An expert whose logit or bias is -inf or
 * NaN is never chosen; a token left with fewer than top_k experts gets ids of -1
 * with weight 0 in the last places. weights[m][j] is the softmax (over all
 * experts whose logit is not -inf or NaN) or the sigmoid of the chosen logit;
 * with renormalize != 0 divided by their sum + 1e-20; times `scale`.
 *
 *   1 <= E <= 1024; 1 <= top_k <= min(E, 32); 1 <= n_group <= 32 divides E;
 *   1 <= topk_group <= n_group; top_k <= topk_group * (E / n_group). bf16 logits
 *   need 2-byte alignment, all other pointers 4.
 */
#define FP8BS_ROUTE_SOFTMAX 0
#define FP8BS_ROUTE_SIGMOID 1
int moe_route_topk(const void* logits, int logits_bf16, const float* bias, int scoring, int64_t M,
                   int64_t E, int64_t top_k, int64_t n_group, int64_t topk_group, int renormalize,
                   float scale, int32_t* ids, float* weights, void* stream);

/*
 * The whole expert MLP of a mixture-of-experts layer for a few tokens (decode):
 * gate+up, SwiGLU, quantization, down, and the weighted sum over a token's
 * experts. More than 128 tokens are refused: fp8_grouped_gemm has the products
 * then, but the grouping of the rows by expert, the SwiGLU between the two products
 * and the weighted sum are the caller's.
 *
 *   for token m and choice j with expert e = ids[m][j] - first_expert:
 *     g, u = the block-scaled products (as fp8_block_gemm, in fp32) of qa[m]
 *            with rows [0, I) and [I, 2I) of qw_gate_up[e]
 *     h    = silu(g) * u in fp32; qh, sh = its 1x128 codes and scales along I
 *     d_j  = the block-scaled product of qh with qw_down[e], in fp32
 *   y[m] = bf16_rn(sum_j weights[m][j] * d_j)
 *
 *   qa [M][K], sa [M][K/128]; ids [M][top_k] int32, weights [M][top_k] fp32
 *       (from moe_route_topk). A choice whose e is outside [0, E) adds nothing
 *       (an id of -1; an expert of another rank: the weights here are those of
 *       experts [first_expert, first_expert + E)); a token without a choice here
 *       gets zeros. A token may name an expert more than once: the weights add.
 *   qw_gate_up [E][2I][K], sw_gate_up [E][2I/128][K/128] ([W_gate; W_up]);
 *   qw_down [E][K][I], sw_down [E][K/128][I/128].
 *   y_bf16 [M][K], output; it and the workspace overlap no operand.
 *   workspace: at least fp8bs_moe_workspace_bytes(M, K, I, E, top_k) bytes, 16-byte
 *       aligned; its contents need no preparation and mean nothing afterwards. The
 *       size never falls with M, so that one workspace serves fewer tokens too. It
 *       is mostly fp32 partial sums, up to 32 MiB for each product and more only
 *       where a single set takes more: 17 to 71 MB for 1 to 128 tokens with 2
 *       choices of 4096 x 14336 (K x I) or 8 of 7168 x 2048, 650 MB for 128 tokens
 *       with 32 choices of 7168 x 14336.
 *       Calls that can run at the same time need workspaces of their own.
 *   0 <= M <= 128, 1 <= E <= 1024, 1 <= top_k <= 32, first_expert >= 0; K and I
 *   positive multiples of 128.
 * The _ue8m0 form takes all scales as UE8M0 codes (255: NaN) and quantizes h with
 * them.
 * A row whose h is not finite somewhere (NaN, or beyond fp32) gives NaN.
 * Results are deterministic: the same inputs give the same bytes every call. How
 * the sums are cut goes by the whole call: a token's row can differ in its rounding
 * from that of a call with other tokens.
 */
int fp8_moe_mlp(const void* qa, const float* sa, const int32_t* ids, const float* weights,
                const void* qw_gate_up, const float* sw_gate_up, const void* qw_down,
                const float* sw_down, void* y_bf16, int64_t M, int64_t K, int64_t I, int64_t E,
                int64_t top_k, int64_t first_expert, void* workspace, size_t workspace_bytes,
                void* stream);
int fp8_moe_mlp_ue8m0(const void* qa, const uint8_t* sa_ue8m0, const int32_t* ids,
                      const float* weights, const void* qw_gate_up,
                      const uint8_t* sw_gate_up_ue8m0, const void* qw_down,
                      const uint8_t* sw_down_ue8m0, void* y_bf16, int64_t M, int64_t K, int64_t I,
                      int64_t E, int64_t top_k, int64_t first_expert, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Scratch bytes fp8_moe_mlp and fp8_moe_mlp_ue8m0 need (0 for an invalid shape). */
size_t fp8bs_moe_workspace_bytes(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k);

/* Scratch bytes needed by the GEMMs for this shape (sparse != 0: the 2:4 GEMM). */
size_t fp8bs_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int sparse);

/*
 * Synchronises `stream`, then returns and clears the device error word of the
 * current device (FP8BS_OK if no kernel recorded an error).
 */
int fp8bs_get_device_error(void* stream);

/*
 * Upper bound, in SM clock cycles, of each internal wait of the GEMM kernels
 * (default about two seconds). cycles <= 0 restores the default. A wait that
 * runs out makes the kernel stop early and record FP8BS_ERR_DEVICE_TIMEOUT.
 * Intended for tests of the timeout path.
 */
void fp8bs_set_wait_limit(long long cycles);

/* Static description of a status code. */
const char* fp8bs_status_string(int status);

/* Library version, as MAJOR * 10000 + MINOR * 100 + PATCH. */
int fp8bs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_H_ */
