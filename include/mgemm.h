/*
 * mgemm.h -- C ABI of the GB300 (sm_103a) Mixture-of-Experts grouped GEMM.
 *
 * The hot path computes gmm(x, w, group_sizes): M token rows of x, stored
 * contiguously by expert (group e owns rows [offsets[e], offsets[e+1])), are
 * multiplied by per-expert weights w[E, K, N]; the group sizes stay in device
 * memory and no call ever waits on the host.  Sources, cited per entry point
 * below:
 *   [GRB]  "Support GPU-resident batch sizes" (tgale96/grouped_gemm PR #21):
 *          description and benchmark script; review of
 *          csrc/fill_arguments.cuh and csrc/grouped_gemm.cu.
 *   [SPM]  "F8I4 Grouped Gemm Optimization for Sparse M" (pytorch/FBGEMM PR
 *          #3854), Summary.
 *   [FP8]  "[moe training] Optimize FP8 MoE backward pass: fused colwise
 *          kernel + AMD tuning" (pytorch/ao commit 34322b5): commit message and
 *          bench_colwise_block_configs.py (_colwise_kernel, run_experiment).
 *   [CMM]  pytorch-labs/applied-ai issue 24, the column-major fused MoE script
 *          (built on vLLM's fused_moe.py): moe_align_block_size (docstring and
 *          worked example), fused_moe_kernel, fused_moe.
 *
 * Conventions (all entry points):
 *   - Every pointer argument is a DEVICE pointer owned by the caller; the
 *     library allocates nothing, keeps no reference after the call returns and
 *     never synchronizes: work is enqueued on `stream` (0 = legacy default).
 *   - Return value: MGEMM_OK (0) when the work was enqueued, or a negative
 *     MGEMM_E* code when a host-side check failed; then nothing is launched.
 *   - Errors found on the device (bad group sizes, a wait that timed out) are
 *     written to the int32 `status` word at the start of the args block (see
 *     below).  Every kernel that takes an args block reads `status` first and
 *     writes nothing when it is non-zero.  The caller reads the word whenever
 *     it chooses to synchronize.
 *   - Matrices are dense and row-major unless stated; "[R, C]" means R rows of
 *     C elements with row stride C.  bf16 is IEEE bfloat16 (2 bytes), fp8 is
 *     OCP/NVIDIA e4m3fn (1 byte, max 448, no infinities), scales are float32.
 *   - Base pointers must be 16-byte aligned and row strides multiples of 16
 *     bytes (the tensor-memory-accelerator rule): K and N multiples of 8 for
 *     bf16 operands, of 16 for fp8 operands.  1 <= E <= MGEMM_MAX_EXPERTS.
 *     M < 2^31.  Violations return MGEMM_EALIGN / MGEMM_EINVAL.
 */
#ifndef MGEMM_H_
#define MGEMM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA include. */
typedef struct CUstream_st *mgemm_stream_t;

/* Host-side return codes. */
#define MGEMM_OK 0
#define MGEMM_EINVAL (-1)   /* null pointer, bad size, bad dtype/flag */
#define MGEMM_EALIGN (-2)   /* pointer or stride breaks the 16-byte rule */
#define MGEMM_ETOOMANY (-3) /* E > MGEMM_MAX_EXPERTS */
#define MGEMM_ECUDA (-4)    /* a CUDA runtime/driver call failed (launch, tensor map) */
#define MGEMM_ENOTSUP (-5)  /* combination not provided (e.g. fp8 with w stored [E,K,N] in mgemm_fwd) */

/* Device-side status codes, written to args->status. */
#define MGEMM_STATUS_OK 0
#define MGEMM_STATUS_NEGATIVE_SIZE 1 /* some group_sizes[e] < 0 */
#define MGEMM_STATUS_SUM_MISMATCH 2  /* sum of group_sizes != M */
#define MGEMM_STATUS_TIMEOUT 4       /* a pipeline wait in a GEMM gave up (about 1 s) */

/* Operand types for the GEMM entry points. */
#define MGEMM_BF16 0
#define MGEMM_FP8_E4M3 1

/* One thread per expert in the single-CTA fill kernel [GRB description]. */
#define MGEMM_MAX_EXPERTS 1024
/* Rows per output tile; the fill kernel's tile prefix counts tiles of this height. */
#define MGEMM_TILE_M 128
/* Row padding of each group in the column-major FP8 layout (see mgemm_colwise_ld). */
#define MGEMM_COL_PAD 128

/*
 * Args block: a device buffer of mgemm_args_bytes(E) bytes, 16-byte aligned,
 * written by mgemm_fill_args and read by every other entry point that takes
 * `args`.  Byte layout (E = number of experts):
 *   [0]   int32  status        MGEMM_STATUS_*
 *   [4]   int32  n_active      number of non-empty groups (<= min(M, E))
 *   [8]   int32  E
 *   [12]  int32  work counter: mgemm_fill_args writes 0; mgemm_quant_colwise_grouped
 *                hands out its work items from it and leaves it at 0 again when it
 *                completes (calls that share an args block must not overlap on the GPU)
 *   [16]  int64  M
 *   [24]  int64  offsets[E+1]  exclusive prefix sum of group_sizes
 *   [A]   int32  active[E]     ids of the non-empty groups, ascending (first n_active valid)
 *   [T]   int32  mtile_start[E+1]  prefix over active groups of ceil(m_e / MGEMM_TILE_M)
 *   [W]   int32  wgrad_order[E]    all experts by m_e descending, ties by ascending id
 *   [P]   int64  poffsets[E+1] exclusive prefix sum of group_sizes each rounded up to
 *                MGEMM_COL_PAD: where group e starts in the padded column-major
 *                FP8 layout of mgemm_quant_colwise_grouped / mgemm_wgrad
 *   [Q]   int32  ptile_start[E+1]  prefix over active groups of ceil(m_e / (2 MGEMM_TILE_M))
 *                (the row-tile pairs of the FP8 GEMMs that run on CTA pairs)
 * with A = 24 + 8(E+1), T = A + 4E, W = T + 4(E+1), P = W + 4E rounded up to a
 * multiple of 8, Q = P + 8(E+1); mgemm_args_layout returns A, T and W.
 */
size_t mgemm_args_bytes(int E);
int mgemm_args_layout(int E, size_t *off_offsets, size_t *off_active, size_t *off_mtile_start,
                      size_t *off_wgrad_order);

/*
 * mgemm_fill_args -- turn device-resident group sizes into the args block.
 * [GRB description]: a single-threadblock kernel converts the batch sizes that
 * live on the GPU into GEMM arguments, removing the GPU->CPU->GPU roundtrip;
 * [GRB review, fill_arguments.cuh]: the block scan, and the sort of problems
 * by k descending when k is dynamic (wgrad_order here); [SPM Summary]: only
 * the min(total_M, groups) non-empty groups are scheduled (active, mtile_start).
 *   group_sizes  int64[E], device; group_sizes[e] rows belong to expert e
 *   E            number of experts, 1..MGEMM_MAX_EXPERTS
 *   M            total rows the caller expects (checked on the device), or -1:
 *                the rows are the sum of the sizes, which only the device
 *                knows (sizes written by another kernel, e.g. the padded
 *                group sizes of mgemm_moe_align); status 2 if it reaches 2^31
 *   args         device buffer of mgemm_args_bytes(E) bytes (output)
 * One launch of one CTA.  Invalid sizes set status 1 or 2 (the other fields
 * are then unspecified).
 */
int mgemm_fill_args(const int64_t *group_sizes, int E, int64_t M, void *args, mgemm_stream_t stream);

/*
 * mgemm_quant_rowwise -- fused per-row absmax scale and saturating e4m3 cast.
 * [FP8 commit message]: replaces tensor_to_scale(A, axiswise_dim=-1),
 * A_scaled = A.to(float32) * A_scales, A_fp8 = to_fp8_saturated(A_scaled) by
 * one launch.  Per row r: amax = max_c |in[r, c]|;
 * s = 2^floor(log2(fp32(448 / max(amax, 1e-12)))) (the scale rule of
 * _colwise_kernel, applied per row); out[r, c] = e4m3_rne_sat(in[r, c] * s).
 *   in      bf16 [R, C] with row stride ld_in elements (ld_in >= C, ld_in % 8 == 0)
 *   out     fp8  [R, C] with row stride ld_out bytes (ld_out >= C, ld_out % 16 == 0)
 *   scales  float32 [R]
 * C % 8 == 0.  R == 0 or C == 0 launches nothing.
 */
int mgemm_quant_rowwise(const void *in, int64_t R, int64_t C, int64_t ld_in, uint8_t *out, int64_t ld_out,
                        float *scales, mgemm_stream_t stream);

/*
 * mgemm_quant_mx -- MXFP8 block quantize: e4m3 codes with one e8m0 scale per
 * 32 consecutive elements of a row.  [FP8 commit message]: the MXFP8 grouped
 * MM path beside the FP8 one, with its token groups padded to 32; the page
 * prints no arithmetic.  Reading: per block b of row r (columns 32b..32b+31),
 * amax = max |in|; s = the power-of-two rule of mgemm_quant_rowwise applied to
 * that amax; out = e4m3_rne_sat(in * s); sf[r, b] = 127 - log2(s) (the e8m0
 * byte of the decode factor 1/s, always in 79..254).
 *   in   bf16 [R, C] with row stride ld_in elements (ld_in >= C, ld_in % 8 == 0)
 *   out  e4m3 [R, C] with row stride ld_out bytes (ld_out >= C, ld_out % 16 == 0)
 *   sf   e8m0 [R, ld_sf] bytes, ld_sf >= C / 32, ld_sf % 16 == 0 (bytes past
 *        C / 32 in each row are not written)
 * C % 32 == 0.  R == 0 or C == 0 launches nothing.  Errors: -1 (sizes), -2
 * (alignment).
 */
int mgemm_quant_mx(const void *in, int64_t R, int64_t C, int64_t ld_in, uint8_t *out, int64_t ld_out, uint8_t *sf,
                   int64_t ld_sf, mgemm_stream_t stream);

/*
 * mgemm_colwise_ld -- the smallest leading dimension (bytes per column) of the
 * padded column-major FP8 layout for M rows in E groups: M plus the padding of
 * up to min(M, E) non-empty groups, rounded up to MGEMM_COL_PAD.  Known on the
 * host without the group sizes.  Returns -1 for M < 0 or E outside 1..MGEMM_MAX_EXPERTS.
 * (An implementation choice, not in [FP8]: it sizes the layout below.)
 */
int64_t mgemm_colwise_ld(int64_t M, int E);

/*
 * mgemm_quant_colwise_grouped -- per-group, per-column scale and e4m3 cast,
 * column-major output; optionally two tensors in one launch (dual form).
 * [FP8 _colwise_kernel]: for group g (rows offsets[g]..offsets[g+1]) and
 * column c, amax over the group's rows, the same power-of-two scale rule, the
 * scale stored at index c + C * g, the cast clamp(x * s) -> e4m3;
 * [FP8 run_experiment]: the output is column-major;
 * [FP8 commit message]: the dual kernel quantizes grad_output and A together.
 *   args        args block from mgemm_fill_args (group offsets, status)
 *   E, M        experts and rows (must match the args block)
 *   in1         bf16 [M, C1] row-major
 *   out1        fp8, padded column-major: column c of group g occupies bytes
 *               out1[c * ld + poffsets[g] ...], m_g codes followed by zeros up
 *               to the next multiple of MGEMM_COL_PAD (C1 * ld bytes; bytes past
 *               poffsets[E] in a column are not written)
 *   sc1         float32 [E * C1], sc1[c + C1 * g]
 *   in2/out2/sc2/C2  the second tensor; in2 == NULL selects the single form
 *   ld          bytes per output column: >= mgemm_colwise_ld(M, E), % 16 == 0
 * C1, C2 % 8 == 0; out1, out2 16-byte aligned.  Empty groups get scale 2^48
 * (amax 0) and no data.  The padding keeps every group's codes aligned and
 * lets mgemm_wgrad contract whole 128-row blocks without masking (an
 * implementation choice; [FP8 run_experiment]'s layout is unpadded, strides (1, M)).
 */
int mgemm_quant_colwise_grouped(const void *args, int E, int64_t M, const void *in1, int64_t C1,
                                uint8_t *out1, float *sc1, const void *in2, int64_t C2, uint8_t *out2,
                                float *sc2, int64_t ld, mgemm_stream_t stream);

/*
 * mgemm_fwd -- out[r, :] = x[r, :] . w[e(r)] for every row r of every non-empty group.
 * [GRB benchmark script]: gmm(x, w, batch_sizes) with x[M, K], w[E, K, N];
 * [GRB review, grouped_gemm.cu]: the trans_b variant (w stored [E, N, K]);
 * [SPM Summary]: only non-empty groups are visited; [FP8 commit message]:
 * FP8 operands are A * scale, so the product is divided by the scales.
 *   dtype == MGEMM_BF16:
 *     x bf16 [M, K]; w bf16 [E, K, N] (trans_b = 0) or [E, N, K] (trans_b = 1);
 *     sx, sw ignored (may be NULL); out bf16 [M, N] (fp32 accumulation, RNE).
 *   dtype == MGEMM_FP8_E4M3 (trans_b must be 1):
 *     x fp8 [M, K] + sx float32 [M]; w fp8 [E, N, K] + sw float32 [E * N];
 *     out[r, n] = bf16( sum_k x[r,k] w[e,n,k] / (sx[r] * sw[e*N + n]) ).
 * Rows of empty groups do not exist; no other memory is written.
 */
int mgemm_fwd(const void *args, int dtype, int trans_b, const void *x, const float *sx, const void *w,
              const float *sw, void *out, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/*
 * mgemm_fwd_fp8_strided -- mgemm_fwd (dtype MGEMM_FP8_E4M3, w [E, N, K]) with
 * the e4m3 weights addressed through strides: w[e, n, k] at byte
 * e * ld_we + n * ld_wn + k.  With the weights' master copy stored [E, K, N]
 * (the layout of the GRIN benchmark script), the forward operand (one scale
 * per (e, n) over K) is mgemm_quant_colwise_grouped of w viewed [E * K, N]
 * with E groups of K rows ([FP8 commit message]: the per-group colwise
 * kernel): its padded column-major codes hold w[e, n, k] at
 * n * ld + e * ceil(K / 128) * 128 + k, i.e. ld_wn = ld (as passed to it),
 * ld_we = K rounded up to 128, and its scales [E * N] are this call's sw.  No
 * transposed copy of the weights is needed.
 *   ld_wn  >= K, % 16 == 0;  ld_we >= K (any value when E == 1), % 16 == 0
 *   the other arguments: as mgemm_fwd with dtype MGEMM_FP8_E4M3, trans_b = 1.
 * Errors as mgemm_fwd.
 */
int mgemm_fwd_fp8_strided(const void *args, const void *x, const float *sx, const void *w, int64_t ld_wn,
                          int64_t ld_we, const float *sw, void *out, int64_t M, int K, int N, int E,
                          mgemm_stream_t stream);

/*
 * mgemm_dgrad -- grad_x[r, :] = grad_out[r, :] . w[e(r)]^T (the backward pass
 * of gmm w.r.t. x).  [GRB benchmark script]: out.sum().backward();
 * [GRB review, grouped_gemm.cu]: the trans_b template; [FP8 commit message]:
 * grad_output is quantized rowwise for grad_A.
 *   grad_out  bf16 [M, N] (or fp8 [M, N] + sgo float32 [M])
 *   w         bf16 [E, K, N] (or fp8 [E, K, N] + sw float32 [E * K], one scale per (e, k))
 *   grad_x    bf16 [M, K]
 */
int mgemm_dgrad(const void *args, int dtype, const void *grad_out, const float *sgo, const void *w,
                const float *sw, void *grad_x, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/*
 * mgemm_fwd_mx -- the MXFP8 grouped GEMM: out[r, n] = sum_k xv[r, k] wv[e(r), n, k]
 * where xv, wv are the decoded block-scaled values (e4m3 value times
 * 2^(sf - 127) of its 32-element block; see mgemm_quant_mx).  [FP8 commit
 * message]: the MXFP8 grouped MM path; the block scales are applied by the
 * tensor cores (block-scaled MMA, one e8m0 scale per 32 contraction elements
 * of each row of either operand), accumulation in fp32, bf16 output (RNE).
 * The same call computes the MXFP8 dgrad: pass grad_out as x (contraction N)
 * and w stored [E, K, N] quantized along N as w.
 *   x    e4m3 [M, K] (row stride K bytes); sx e8m0 [M, ld_sf]
 *   w    e4m3 [E, N, K]; sw e8m0 [E * N, ld_sf]
 *   ld_sf  bytes per scale row, >= K / 32, % 16 == 0 (as written by mgemm_quant_mx)
 *   out  bf16 [M, N]
 * K % 128 == 0, N % 8 == 0.  Groups of any size (the blocks run along K).
 * Errors: -1 (sizes or NULL), -2 (alignment), -3 (E), -4 (CUDA).
 */
int mgemm_fwd_mx(const void *args, const uint8_t *x, const uint8_t *sx, const uint8_t *w, const uint8_t *sw,
                 int64_t ld_sf, void *out, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/*
 * mgemm_quant_colwise_mx -- per-group colwise MX blocks, the MXFP8 wgrad
 * operands (one or two tensors per launch).  Reading of [FP8]'s MXFP8 path
 * (groups padded to 32 rows): in group g and column c, blocks of 32
 * consecutive rows counted from the group's first row (a group's last block
 * may be short; its missing rows count as zeros); each block's scale and codes
 * follow mgemm_quant_mx.
 *   in1   bf16 [M, C1] row-major (C1 % 8 == 0); optionally in2 [M, C2] (dual)
 *   out1  e4m3 [C1, ld]: the padded column-major layout of
 *         mgemm_quant_colwise_grouped (group g's codes at column offset
 *         poffsets[g], zeros after them up to a multiple of MGEMM_COL_PAD)
 *   sf1   e8m0 [ld / 128][C1][4]: for padded row block j (rows 128 j .. 128 j +
 *         127) and column c, the 4 bytes of its four 32-row blocks
 *         ((ld / 128) * C1 * 4 bytes, 16-byte aligned)
 *   ld    bytes per column: >= mgemm_colwise_ld(M, E), % 128 == 0
 * Only bytes inside the padded total (poffsets[E]) are written.
 * Errors: -1 (sizes, NULL), -2 (alignment), -3 (E).
 */
int mgemm_quant_colwise_mx(const void *args, int E, int64_t M, const void *in1, int64_t C1, uint8_t *out1,
                           uint8_t *sf1, const void *in2, int64_t C2, uint8_t *out2, uint8_t *sf2, int64_t ld,
                           mgemm_stream_t stream);

/*
 * mgemm_wgrad_mx -- the MXFP8 wgrad: grad_w[e] = sum over the rows r of group e
 * of xv[r, :]^T gov[r, :], with the decoded block-scaled values of
 * mgemm_quant_colwise_mx (blocks of 32 rows of a group); zero for an empty
 * group.  Block-scaled tensor-core MMAs, fp32 accumulation, bf16 output.
 *   x, sx    x's codes [K, ld] and scale rows [ld / 128][K][4] (mgemm_quant_colwise_mx)
 *   grad_out, sgo   likewise [N, ld] and [ld / 128][N][4]
 *   grad_w   bf16 [E, K, N]; every element is written
 *   ld       as passed to mgemm_quant_colwise_mx
 * K % 16 == 0, N % 16 == 0.  Errors: -1, -2, -3, -4 as mgemm_wgrad.
 */
int mgemm_wgrad_mx(const void *args, const uint8_t *x, const uint8_t *sx, const uint8_t *grad_out,
                   const uint8_t *sgo, void *grad_w, int64_t M, int K, int N, int E, int64_t ld,
                   mgemm_stream_t stream);

/*
 * mgemm_wgrad -- grad_w[e] = x_e^T . grad_out_e, contracting over the m_e rows
 * of group e ("dynamic k"); grad_w[e] = 0 when m_e = 0.
 * [GRB review, fill_arguments.cuh]: problems sorted by k descending;
 * [GRB review, ZeroOutK0Outputs]: k = 0 problems produce zeros;
 * [FP8 commit message]: grad_B uses per-group colwise scales of grad_output and A.
 *   dtype == MGEMM_BF16: x bf16 [M, K], grad_out bf16 [M, N] (row-major).
 *   dtype == MGEMM_FP8_E4M3: x fp8 [K, ld] and grad_out fp8 [N, ld] in the
 *     padded column-major layout of mgemm_quant_colwise_grouped (rows of group
 *     e at poffsets[e], zero padding after them), sx float32 [E * K] and sgo
 *     float32 [E * N] its scales; ld as passed to it.
 *   ld        FP8: bytes per column of x and grad_out (% 16 == 0,
 *             >= mgemm_colwise_ld(M, E)); ignored for MGEMM_BF16.
 *   grad_w    bf16 [E, K, N]; every element is written.
 */
int mgemm_wgrad(const void *args, int dtype, const void *x, const float *sx, const void *grad_out,
                const float *sgo, void *grad_w, int64_t M, int K, int N, int E, int64_t ld, mgemm_stream_t stream);

/*
 * mgemm_dgrad_wgrad -- the bf16 backward of the grouped GEMM, both gradients:
 * grad_x exactly as mgemm_dgrad(MGEMM_BF16, grad_out, w [E, K, N]) and grad_w
 * exactly as mgemm_wgrad(MGEMM_BF16, x, grad_out), bit for bit ("Support
 * GPU-resident batch sizes", benchmark script: the backward of gmm after
 * out.sum()).  Where the groups are small enough that dgrad streams the
 * weights from HBM while wgrad is bound by its grad_w stores, both run in one
 * launch on disjoint sets of CTAs (a host-side model of the two sizes picks
 * the split) and overlap; otherwise the two calls run one after the other on
 * the stream.  Same args block as both; no other device memory.
 *   grad_out bf16 [M, N]; w bf16 [E, K, N]; x bf16 [M, K] (row-major)
 *   grad_x   bf16 [M, K]; grad_w bf16 [E, K, N] (every element written)
 * With M == 0 only grad_w is written (zeros) and grad_out, x, grad_x may be
 * NULL.  Errors as for the two calls (K % 8 == 0, N % 8 == 0, 16-byte aligned
 * pointers).
 */
int mgemm_dgrad_wgrad(const void *args, const void *grad_out, const void *w, const void *x, void *grad_x,
                      void *grad_w, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/* The number of CTAs mgemm_dgrad_wgrad gives to dgrad in its one-launch form
 * for these sizes (the rest of the SMs run wgrad), or 0 when it makes the two
 * calls in turn; negative MGEMM_E* for invalid sizes.  Host-side (reads the
 * current device's SM count once). */
int mgemm_dgrad_wgrad_split(int64_t M, int K, int N, int E);

/*
 * mgemm_fill_args_quant_rowwise -- mgemm_fill_args and mgemm_quant_rowwise of
 * the token rows in one launch (the two independent steps before an FP8
 * forward: "Support GPU-resident batch sizes", the argument fill; "[moe
 * training] Optimize FP8 MoE backward pass" commit message, the fused rowwise
 * scale + cast).  The args block is exactly mgemm_fill_args(group_sizes, E, M,
 * args); xq and sx exactly mgemm_quant_rowwise(x [M, K]).  One CTA fills the
 * args block while the others cast rows, so at sparse M the pair costs about
 * one launch instead of two.
 *   group_sizes int64[E], device; args as for mgemm_fill_args (M >= 0 here)
 *   x     bf16 [M, K], row stride ld_x elements; xq e4m3 [M, K], row stride ld_q
 *         bytes; sx fp32 [M]
 * K % 8 == 0, ld_x % 8 == 0, ld_q % 8 == 0.  Errors as for the two calls.
 */
int mgemm_fill_args_quant_rowwise(const int64_t *group_sizes, int E, int64_t M, void *args, const void *x, int64_t K,
                                  int64_t ld_x, uint8_t *xq, int64_t ld_q, float *sx, mgemm_stream_t stream);

/*
 * mgemm_fwd_fp8_sparse -- the FP8 forward for few token rows in one launch:
 * mgemm_fill_args + mgemm_quant_rowwise of x + mgemm_fwd (MGEMM_FP8_E4M3,
 * w [E, N, K]) ("F8I4 Grouped Gemm Optimization for Sparse M", Summary:
 * work only for the min(total_M, groups) non-empty groups; "[moe training]
 * Optimize FP8 MoE backward pass" commit message: the fused rowwise scale +
 * cast).  Every CTA scans the group sizes itself, casts the token rows it
 * needs (the rowwise rule: power-of-two scale from the row's magnitude
 * maximum, saturating e4m3) into shared memory and streams its share of the
 * touched experts' weights.  When the tiles of 128 output columns cover at
 * most half of the SMs (one token), pairs of CTAs split each tile's
 * contraction in two halves and add the second half's fp32 partial sums to
 * the first's; otherwise every output equals mgemm_fwd's bit for bit.
 *   group_sizes int64[E], device, summing to M
 *   x        bf16 [M, K] token rows sorted by expert, row stride ld_x elements
 *   w, sw    e4m3 [E, N, K] and fp32 [E * N] (as for mgemm_fwd)
 *   out      bf16 [M, N]; only the M rows are written
 *   status   int32, device, holding 0 or a negative value on entry (zeroed
 *            once, it stays 0 while calls succeed): the call raises it to
 *            MGEMM_STATUS_NEGATIVE_SIZE or MGEMM_STATUS_SUM_MISMATCH (then
 *            nothing else is written) or MGEMM_STATUS_TIMEOUT, else to 0; a
 *            caller that reads a nonzero status resets it before the next call
 * 1 <= M <= 16, E <= 1024, K % 128 == 0, N % 8 == 0, ld_x % 8 == 0, and the
 * token rows must fit on chip: ceil(M / 8) * 8 * K <= 150 KiB (else -1; use
 * the three calls).  Errors: -1 (sizes or NULL), -2 (alignment), -3 (E),
 * -4 (CUDA).
 */
int mgemm_fwd_fp8_sparse(const int64_t *group_sizes, int E, const void *x, int64_t ld_x, const void *w,
                         const float *sw, void *out, int *status, int64_t M, int K, int N, mgemm_stream_t stream);



/*
 * mgemm_quant_int4 -- the INT4 weights of the FP8 x INT4 grouped GEMM.
 * "F8I4 Grouped Gemm Optimization for Sparse M" (FBGEMM PR #3854), title and
 * Summary, names FP8 activations times INT4 weights and gives no format; this
 * library's reading: per row (e, n) of w [E, N, K] and block of 32 consecutive
 * k, s = 2^floor(log2(fp32(7 / max(amax, 1e-12)))) (the FP8 power-of-two rule
 * at the INT4 range), q = clamp(round_half_even(w * s), -8, 7).
 *   w       bf16 [E, N, K], row stride ld_in elements (>= K, % 8 == 0), device
 *   packed  uint8 [E, N, K / 2]: two's-complement nibbles, element 2i in the low
 *           nibble of byte i of its row (rows of K / 2 bytes, no padding)
 *   sf      uint8, E * (K / 128) * N * 4 bytes: the e8m0 byte 127 - log2(s) of
 *           each block (the decode factor 1 / s), contraction-block major:
 *           block j of row (e, n) at ((e * (K / 128) + j / 4) * N + n) * 4 + j % 4
 * K % 128 == 0.  Codes and bytes are unique (bit-exact against the oracle).
 * Errors: -1 (sizes or NULL), -2 (alignment), -4 (CUDA).
 */
int mgemm_quant_int4(const void *w, int E, int N, int K, int64_t ld_in, uint8_t *packed, uint8_t *sf,
                     mgemm_stream_t stream);

/*
 * mgemm_fwd_f8i4 -- the FP8 x INT4 grouped forward GEMM ("F8I4 Grouped Gemm
 * Optimization for Sparse M", FBGEMM PR #3854, Summary: tiles only for the
 * min(total_M, groups) non-empty groups):
 *   out[r, n] = sum_k (e4m3(x[r, k]) / sx[r]) * q[e(r), n, k] * 2^(b[e, n, k / 32] - 127)
 * in fp32 on the tensor cores (block-scaled MMA: x's row scale and the weight
 * blocks' bytes are both applied inside it), rounded once to bf16 (RNE).
 *   args     filled by mgemm_fill_args for these E group sizes and M
 *   x, sx    e4m3 [M, K] and fp32 [M] row scales (mgemm_quant_rowwise)
 *   w_packed, w_scales  as written by mgemm_quant_int4 for w [E, N, K]
 *   out      bf16 [M, N]; rows of empty groups do not exist, nothing else is written
 * K % 128 == 0, N % 8 == 0 (else -2).  Errors: -1 (sizes or NULL), -2
 * (alignment), -3 (E), -4 (CUDA); device-side errors in the args status word.
 */
int mgemm_fwd_f8i4(const void *args, const uint8_t *x, const float *sx, const uint8_t *w_packed,
                   const uint8_t *w_scales, void *out, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/*
 * mgemm_fwd_noalloc -- mgemm_fwd for callers that cannot allocate device memory.
 * The source pages have no counterpart to this call; it exists for callers
 * that may not call cudaMalloc (or any allocator) at the point where they run
 * the forward pass -- for example code inside another framework's launch
 * callback that has no allocator of its own, loops where an allocation could
 * synchronize the device, or runtimes that only provide a fixed workspace
 * chosen in advance.  Instead of a caller-provided args block it uses one held
 * in a static device array of this library, sized for MGEMM_NOALLOC_MAX_EXPERTS
 * experts (about 33 KB, kept on every GPU that loads the library until exit).
 *   group_sizes  int64[E], device (as for mgemm_fill_args)
 *   the other arguments are those of mgemm_fwd.
 * Makes every host check of mgemm_fill_args and mgemm_fwd first (same codes;
 * a rejected call launches nothing and leaves the array untouched; M must be
 * >= 0, and M == 0 returns MGEMM_OK at once), then runs mgemm_fill_args into
 * the static array and mgemm_fwd.  Allocates nothing.
 * E > MGEMM_NOALLOC_MAX_EXPERTS returns MGEMM_ETOOMANY.
 * The first call on each device looks up the array's device address (with
 * that device current); make that first call before any stream capture.  The
 * address is kept for the life of the process: do not use this call on a
 * device after cudaDeviceReset.
 * All calls share the array: calls whose work overlaps on the GPU race on it.
 * Device-side errors go to the status word of the static args block, which the
 * caller cannot read; check the group sizes beforehand when that matters.
 */
#define MGEMM_NOALLOC_MAX_EXPERTS 1024
int mgemm_fwd_noalloc(const int64_t *group_sizes, int E, int dtype, int trans_b, const void *x, const float *sx,
                      const void *w, const float *sw, void *out, int64_t M, int K, int N, mgemm_stream_t stream);

/*
 * mgemm_moe_align -- moe_align_block_size on the device [CMM]: the flat
 * (token, slot) entries of topk_ids are grouped by expert, each expert's list
 * padded up to a multiple of block_size, so that every block of the sorted list
 * belongs to one expert.
 *   topk_ids      int32 [numel]: expert of flat entry i (token i / top_k when
 *                 topk_ids is [T, top_k] row-major).  Entries outside [0, E)
 *                 are not placed.
 *   sorted_ids    int32 [numel + E * (block_size - 1)]: expert by expert in
 *                 ascending id, the expert's flat indices in ascending order,
 *                 then the pad id numel up to the expert's padded count; every
 *                 position from num_post_padded to the end also holds numel.
 *   expert_ids    int32 [(numel + E * (block_size - 1)) / block_size]: the
 *                 expert of each block of block_size positions; -1 past the
 *                 last block.
 *   num_post_padded  int32 [1]: the padded total (a multiple of block_size).
 *   group_sizes   int64 [E] or NULL: each expert's padded count (the group
 *                 sizes for mgemm_fill_args over the sorted, padded rows).
 *   workspace     mgemm_moe_align_workspace_bytes(numel, E) bytes, 16-byte
 *                 aligned, scratch for the duration of the call's kernels.
 * Limits: 1 <= E <= MGEMM_MAX_EXPERTS, 1 <= block_size <= 4096,
 * numel + E * (block_size - 1) < 2^31.  The result is unique (stable order), so
 * it is bit-for-bit reproducible.  Three kernels: per-chunk counts, one CTA
 * that turns them into positions and writes the padding and block experts,
 * and the stable placement.
 */
int64_t mgemm_moe_align_workspace_bytes(int64_t numel, int E);
int mgemm_moe_align(const int32_t *topk_ids, int64_t numel, int E, int block_size, int32_t *sorted_ids,
                    int32_t *expert_ids, int32_t *num_post_padded, int64_t *group_sizes, void *workspace,
                    mgemm_stream_t stream);

/*
 * mgemm_moe_route_align -- for decode-size batches, one launch doing the work
 * of mgemm_topk_softmax, mgemm_moe_align and mgemm_fill_args (M = -1) in
 * sequence [CMM]: every output is what those three calls write, bit for bit.
 *   gating        float32 [T, E] (as for mgemm_topk_softmax), or NULL: the
 *                 routing is skipped and topk_ids is read as the input ids
 *                 (as for mgemm_moe_align, entries outside [0, E) are not
 *                 placed); topk_weights is then not used
 *   topk_weights  float32 [T, top_k], written when gating is given
 *   topk_ids      int32 [T, top_k]: written when gating is given, read otherwise
 *   sorted_ids, expert_ids, num_post_padded, group_sizes (may be NULL):
 *                 as from mgemm_moe_align with numel = T * top_k
 *   args          mgemm_args_bytes(E) bytes, 16-byte aligned: the args block of
 *                 the padded group sizes (the sorted rows' grouped GEMMs)
 * Limits: 1 <= E <= MGEMM_MAX_EXPERTS; 1 <= top_k (<= E when gating is given);
 * T * top_k <= MGEMM_ROUTE_ALIGN_MAX_ENTRIES; 1 <= block_size <= 4096.  Larger
 * batches return MGEMM_EINVAL: use the three calls, whose kernels spread over
 * the SMs.  With T = 0 the gating, weights and ids may be NULL; the other
 * outputs are still written (no entries: padding ids, empty groups).  One CTA
 * of 1024 threads.
 */
#define MGEMM_ROUTE_ALIGN_MAX_ENTRIES 4096
int mgemm_moe_route_align(const float *gating, int64_t T, int E, int top_k, int renormalize, int block_size,
                          float *topk_weights, int32_t *topk_ids, int32_t *sorted_ids, int32_t *expert_ids,
                          int32_t *num_post_padded, int64_t *group_sizes, void *args, mgemm_stream_t stream);

/*
 * The routed (fused_moe) layer [CMM], built from mgemm_moe_align and these
 * calls: x rows are gathered into expert order, the grouped GEMM runs over the
 * sorted rows, and its epilogue scatters each row to its flat (token, slot)
 * entry, optionally times the routed weight -- the work of fused_moe_kernel,
 * whose masked loads read padding entries as zero rows and whose masked stores
 * skip them; then silu_and_mul, the second GEMM with MUL_ROUTED_WEIGHT, and the
 * sum over the top_k slots of each token.
 *
 * mgemm_gather_rows -- dst row s = src row sorted_ids[s] / top_k for every s
 * below min(*num_post_padded, dst_rows); zeros when sorted_ids[s] >= numel (a
 * padding entry) or names a row outside src.  Rows from *num_post_padded on
 * are not written.
 *   src  [src_rows] rows of row_bytes bytes, src_ld_bytes apart
 *   dst  [dst_rows] rows, dst_ld_bytes apart (row_bytes and both strides
 *        multiples of 16; src and dst 16-byte aligned)
 *   sorted_ids, num_post_padded, numel: as from mgemm_moe_align
 */
int mgemm_gather_rows(const void *src, int64_t src_rows, int64_t row_bytes, int64_t src_ld_bytes,
                      const int32_t *sorted_ids, const int32_t *num_post_padded, int64_t numel, int top_k,
                      void *dst, int64_t dst_rows, int64_t dst_ld_bytes, mgemm_stream_t stream);

/*
 * mgemm_fwd_scatter -- mgemm_fwd over rows sorted by expert, with each output
 * row stored at the row row_map names (fused_moe_kernel's c_ptrs), optionally
 * multiplied by its routed weight (MUL_ROUTED_WEIGHT: the fp32 accumulator row
 * times the weight, then one rounding to bf16).
 *   args        args block of the sorted rows: mgemm_fill_args over the padded
 *               group sizes of mgemm_moe_align, with M = -1
 *   x           bf16 [M, K]: the sorted rows (mgemm_gather_rows); M >= the
 *               padded total (e.g. the sorted_ids capacity)
 *   w           bf16 [E, N, K] (trans_b = 1, the layout of fused_moe) or [E, K, N]
 *   out         bf16 [map_limit, N]
 *   row_map     int32 [M]: output row of sorted row i (sorted_ids: flat entry
 *               ids); a row with row_map[i] < 0 or >= map_limit (padding) is
 *               not stored
 *   map_limit   rows of out (numel of topk_ids)
 *   row_weight  float32 [map_limit] or NULL
 * bf16 only (fp8 returns MGEMM_ENOTSUP).  Output rows no sorted row names are
 * left as they were.  With map_limit < 128 (decode-size batches: a group has
 * at most map_limit routed rows, at the start of its block) only those rows of
 * each block are loaded.
 */
int mgemm_fwd_scatter(const void *args, int dtype, int trans_b, const void *x, const void *w, void *out,
                      const int32_t *row_map, int64_t map_limit, const float *row_weight, int64_t M, int K, int N,
                      int E, mgemm_stream_t stream);

/*
 * mgemm_fwd_gated -- the first GEMM of fused_moe with silu_and_mul in its
 * epilogue: out[r, j] = silu(g) * u with g = x[r, :] . w[e(r), j, :] and
 * u = x[r, :] . w[e(r), F + j, :] (the gate and up halves of w1 [E, 2F, K],
 * vLLM's silu_and_mul convention), g and u in fp32, silu(g) = g / (1 + exp(-g)),
 * one rounding to bf16.  Each tile's weight stage holds matching gate and up
 * rows, so both halves of an output column meet in one accumulator.
 *   args, x [M, K], M, K, E: as for mgemm_fwd (bf16)
 *   w    bf16 [E, 2F, K];  out  bf16 [M, F] (F % 8 == 0)
 *   group_rows_max  an upper bound on the rows of any group that are not
 *        padding (the routed entries; they come first in each 128-row block,
 *        as mgemm_moe_align places them), or 0 if unknown.  Below 128 (decode-
 *        size batches) only those rows of each block are loaded and stored:
 *        the padding rows of out are then left as they were.
 */
int mgemm_fwd_gated(const void *args, const void *x, const void *w, void *out, int64_t M, int K, int F, int E,
                    int64_t group_rows_max, mgemm_stream_t stream);

/*
 * mgemm_fwd_gated_gather -- mgemm_fwd_gated whose sorted rows are read from
 * the token rows through the sorted entry ids, as fused_moe_kernel loads A
 * through sorted_token_ids [CMM]: sorted row i is x row sorted_ids[i] / top_k,
 * or a row of zeros when sorted_ids[i] >= numel (padding), so the gathered
 * copy of mgemm_gather_rows is not needed.  The outputs equal those of
 * mgemm_gather_rows followed by mgemm_fwd_gated, bit for bit.
 *   x           bf16 [x_rows, K] (the token rows), 16-byte aligned
 *   sorted_ids, numel, top_k: as from mgemm_moe_align (sorted_ids holds at
 *               least M entries)
 *   args, w, out, M, K, F, E, group_rows_max: as for mgemm_fwd_gated
 * For decode-size batches only: 1 <= group_rows_max <= 32 and K % 64 == 0;
 * other shapes return MGEMM_ENOTSUP.  The GEMM's producer copies the rows
 * itself (16-byte asynchronous copies into the swizzled operand layout).
 */
int mgemm_fwd_gated_gather(const void *args, const void *x, int64_t x_rows, const int32_t *sorted_ids, int64_t numel,
                           int top_k, const void *w, void *out, int64_t M, int K, int F, int E,
                           int64_t group_rows_max, mgemm_stream_t stream);

/*
 * mgemm_silu_and_mul -- out[r, j] = silu(in[r, j]) * in[r, F + j] for in bf16
 * [R, 2F] and out bf16 [R, F] (vLLM's silu_and_mul as fused_moe applies it to
 * the first GEMM's output), silu(v) = v / (1 + exp(-v)), computed in fp32 and
 * rounded to bf16 once.  F % 8 == 0; pointers 16-byte aligned.
 */
int mgemm_silu_and_mul(const void *in, int64_t R, int64_t F, void *out, mgemm_stream_t stream);

/*
 * mgemm_topk_sum -- out[t, :] = sum_j in[t * top_k + j, :] for in bf16
 * [T * top_k, H] and out bf16 [T, H] (fused_moe's final sum over the top_k
 * slots), accumulated in fp32 in ascending j and rounded to bf16 once.
 * H % 8 == 0; pointers 16-byte aligned.
 */
int mgemm_topk_sum(const void *in, int64_t T, int top_k, int64_t H, void *out, mgemm_stream_t stream);

/*
 * mgemm_topk_softmax -- fused_moe's routing [CMM] (its topk_softmax call and
 * renormalize step): per token t, p = softmax(gating[t, :]) over the E
 * experts; topk_ids[t, :] = the top_k experts, largest probability first;
 * topk_weights[t, :] = their probabilities, divided by their sum when
 * renormalize != 0.
 *   gating        float32 [T, E], finite
 *   topk_weights  float32 [T, top_k];  topk_ids  int32 [T, top_k]
 * The selection compares logits (softmax is increasing in each, so the same
 * experts, with no rounding ties); equal logits go to the lower id.  The
 * weights are exp(l - max) / sum in fp32.  1 <= top_k <= E <= MGEMM_MAX_EXPERTS.
 * One warp per token.
 */
int mgemm_topk_softmax(const float *gating, int64_t T, int E, int top_k, int renormalize, float *topk_weights,
                       int32_t *topk_ids, mgemm_stream_t stream);

/*
 * Choosing experts from router scores.  Where mgemm_topk_softmax takes the
 * top_k of a softmax, mgemm_route covers the routers of layers with many
 * experts: softmax or sigmoid scores, a balance bias that acts on the choice
 * only, experts in groups of which the best few are kept, renormalized and
 * scaled weights, experts that are switched off; and the gradient of the
 * logits.  (Not on the source pages: an addition of this library.)
 *
 * mgemm_route -- per token t, with l = logits[t, :]:
 *   scores   s = 1 / (1 + exp(-l)) (MGEMM_SCORE_SIGMOID) or softmax(l)
 *            (MGEMM_SCORE_SOFTMAX).  A logit at or below MGEMM_ROUTE_MASKED
 *            (-inf and the lowest value of either type) switches its expert
 *            off: score 0, chosen only after every other expert of the groups
 *            kept.
 *   order    c = s + bias[e] (bias may be NULL).  Softmax without bias compares
 *            the logits (the same order, without rounding ties).  Equal values
 *            go to the lower id; a NaN is the largest (its weight is NaN).
 *   groups   n_group > 1: experts g E / n_group .. form group g; its score is
 *            the largest c of its experts, or with group_top = 2 the sum of the
 *            two largest (softmax without bias: of exp(l - max l), the same
 *            order of groups as with the scores); experts that are off add
 *            nothing, and a group of only such experts comes last.  The
 *            topk_group best groups are kept (equal scores: the lower group).
 *   outputs  topk_ids[t, :] = the top_k experts by c in the groups kept, best
 *            first; topk_weights[t, j] = scale * r_j with r = s[ids], divided by
 *            their sum when renormalize != 0 (all 0 when that sum is 0).
 *   logits   float32 or bf16 (logits_bf16 != 0), rows of E values ld elements
 *            apart (ld >= E), naturally aligned;  bias float32 [E]
 *   topk_weights  float32 [T, top_k];  topk_ids  int32 [T, top_k]
 * Everything is computed in float32.  1 <= E <= MGEMM_MAX_EXPERTS; n_group
 * divides E, 1 <= topk_group <= n_group <= 64; group_top is 1 or 2;
 * 1 <= top_k <= min(MGEMM_ROUTE_MAX_TOPK, topk_group * E / n_group).
 *
 * mgemm_route_bwd -- grad_logits[t, e] = dL / dl for dL / dw = grad_weights[t, :]
 * (the choice of experts is constant, as is the bias): with f = sum_i g_i w_i /
 * scale,
 *   sigmoid, renormalized   w_j (1 - s_j) (g_j - f) at expert ids[j], 0 elsewhere
 *   sigmoid                 w_j (1 - s_j) g_j       likewise
 *   softmax, renormalized   w_j (g_j - f)           likewise
 *   softmax                 w_j g_j at ids[j], and everywhere - s_e sum_i g_i w_i
 *   topk_weights, topk_ids, logits, scoring, renormalize, scale: as given to and
 *   written by mgemm_route (scale != 0).  The logits are not read for softmax,
 *   renormalized (may be NULL).  An id outside [0, E) has no gradient.
 *   grad_logits  [T, E] of the logits' type, rows ld_grad elements apart; every
 *                element is written.
 */
#define MGEMM_SCORE_SOFTMAX 0
#define MGEMM_SCORE_SIGMOID 1
#define MGEMM_ROUTE_MASKED (-3.3e38f)
#define MGEMM_ROUTE_MAX_TOPK 32
int mgemm_route(const void *logits, int logits_bf16, int64_t ld, const float *bias, int64_t T, int E, int top_k,
                int scoring, int n_group, int topk_group, int group_top, int renormalize, float scale,
                float *topk_weights, int32_t *topk_ids, mgemm_stream_t stream);
int mgemm_route_bwd(const float *grad_weights, const void *logits, int logits_bf16, int64_t ld,
                    const float *topk_weights, const int32_t *topk_ids, int64_t T, int E, int top_k, int scoring,
                    int renormalize, float scale, void *grad_logits, int64_t ld_grad, mgemm_stream_t stream);

/*
 * The balance loss that trains a router, with the experts' counts.  (Not on the source
 * pages: an addition of this library, beside mgemm_route.)
 *
 * mgemm_balance -- for the tokens of a sequence (those rows of it that the mask keeps; n of
 * them, with top_k picks each, c_e of which are expert e):
 *   p_te = softmax(logits[t, :]) (MGEMM_SCORE_SOFTMAX), or the sigmoids over their sum
 *          (MGEMM_SCORE_SIGMOID); 0 for a logit at or below MGEMM_ROUTE_MASKED, and
 *          everywhere in a row whose scores are all 0 (sigmoids all below 2^-252)
 *          (scores below 2^-126 beside larger ones, a softmax's relative to its largest, are
 *          0: a p below 2^-86 may be, which no sum here notices)
 *   L_s  = sum_e (E c_e / (top_k n)) (sum_t p_te / n)
 *   loss = scale times the mean of L_s over the sequences with n > 0 (0 without any)
 *   logits    as for mgemm_route;  topk_ids  int32 [T, top_k] (ids outside [0, E) are not
 *             counted; the choice is constant in the gradient)
 *   offsets   int64 [S + 1], device, not decreasing, from 0 to T at most: sequence s is rows
 *             offsets[s] .. offsets[s + 1] - 1; rows of no sequence count nowhere.  NULL
 *             (S = 1): all T rows.  (Offsets that decrease give unspecified results.)
 *   mask      uint8 [T], 0: the row is not counted; or NULL
 *   loss      float32 [1];  counts  int64 [S, E]: c_e, the group sizes of a grouped GEMM
 *             over the picks when S = 1
 *   slopes    float32 [S * E + 1], what the backward pass reads: E c_e / (top_k n^2) (0
 *             where n = 0), and scale over the number of sequences; or NULL
 *   workspace mgemm_balance_workspace_bytes(T, E, S) bytes, 16-byte aligned, scratch
 * 1 <= E <= MGEMM_MAX_EXPERTS, 1 <= top_k <= MGEMM_MAX_EXPERTS, 1 <= S < 2^24, T * top_k < 2^31.
 * Sums are taken in a fixed order: the same bits on every call.
 *
 * mgemm_balance_bwd -- grad_logits[t, :] = *grad_loss dloss / dlogits, of the logits' type;
 * every element is written (0 for rows that do not count, and for experts that are off).
 *   grad_loss  float32 [1], device;  slopes, offsets, S, mask, scoring: as for mgemm_balance
 */
int64_t mgemm_balance_workspace_bytes(int64_t T, int E, int64_t S);
int mgemm_balance(const void *logits, int logits_bf16, int64_t ld, const int32_t *topk_ids, int top_k,
                  const int64_t *offsets, int64_t S, const uint8_t *mask, int64_t T, int E, int scoring, float scale,
                  float *loss, int64_t *counts, float *slopes, void *workspace, int64_t workspace_bytes,
                  mgemm_stream_t stream);
int mgemm_balance_bwd(const float *grad_loss, const void *logits, int logits_bf16, int64_t ld, const float *slopes,
                      const int64_t *offsets, int64_t S, const uint8_t *mask, int64_t T, int E, int scoring,
                      void *grad_logits, int64_t ld_grad, mgemm_stream_t stream);

/*
 * 4-bit block-scaled floats.  Codes are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives; bit 3 the sign), two to a byte, the even element in the low
 * nibble.  (Not on the source pages: an addition of this library, beside its
 * MXFP8 and INT4 formats; the scale rule is the same power-of-two rule.)
 *   MGEMM_MXFP4  one e8m0 byte per 32 elements of a row:
 *                s = 2^floor(log2(fp32(6 / max(amax, 1e-12)))), code =
 *                e2m1_rne_sat(x s), byte = 127 - log2(s); value code 2^(byte - 127)
 *   MGEMM_NVFP4  one e4m3 byte per 16 elements and one float32 per row:
 *                R = 2^floor(log2(fp32(2688 / max(row amax, 1e-12)))) (2688 = 6 x
 *                448), b = e4m3_rne(amax16 R / 6), code = e2m1_rne_sat(x R / b), 0
 *                where b = 0; value code b / R
 * (the sign of a zero is unspecified).  NaN and infinity show: a block (MXFP4) or
 * row (NVFP4) that holds one gets NaN scales (byte 0xFF; 0x7F and R = NaN) and
 * unspecified codes, its values are NaN, and so is every output of a product that
 * takes them.  Tensors from elsewhere may have row scales that are no powers of
 * two (positive, from 2^-120 to 2^120): mgemm_dequant_fp4 multiplies by their
 * reciprocals, correctly rounded, mgemm_fwd_fp4 by reciprocals within 2^-23.
 *
 * Scale bytes lie in tiles of 128 rows by one 4-byte word of each row, a word
 * being the row's scales of 128 (MXFP4) or 64 (NVFP4) consecutive elements:
 * block q of row r at byte ((r / 128 * W + q / 4) * 128 + (r % 32) * 4 +
 * (r % 128) / 32) * 4 + q % 4, W = ceil(K / word).  That is the order in which
 * tensor memory holds a tile's scale factors, so a GEMM stage's scales are
 * contiguous.  Every group of rows (an expert's weights, a group's tokens)
 * starts a tile: its tiles follow those of the group before.
 * mgemm_fp4_scale_bytes: bytes of the scales of `rows` rows of one group, -1 for
 * bad sizes; E groups of N rows take E times that.
 */
#define MGEMM_MXFP4 2
#define MGEMM_NVFP4 3
int64_t mgemm_fp4_scale_bytes(int fmt, int64_t rows, int K);

/*
 * mgemm_quant_fp4 -- cast E groups of N rows (weights [E, N, K]; E = 1: a matrix).
 *   in         bf16, row i (of E * N) at in + i * ld_in elements (ld_in >= K, % 8 == 0)
 *   codes      uint8 [E * N, K / 2]
 *   sf         uint8, E * mgemm_fp4_scale_bytes(fmt, N, K) bytes; every byte is
 *              written (zeros for rows past N and blocks past K)
 *   row_scale  float32 [E * N] (MGEMM_NVFP4), else ignored
 * K % 32 == 0.  E, N >= 0; nothing is launched when either is 0.
 * mgemm_dequant_fp4 -- the values the codes stand for, to bf16 (exact for the
 * casts' scales: a code times them has at most 6 significant bits; below 2^-133
 * they round, and past bf16's range they stay at its largest value).
 *   out        bf16, row i at out + i * ld_out elements (ld_out >= K, % 8 == 0)
 * Errors: -1 (sizes, format, NULL), -2 (alignment), -4 (CUDA).
 */
int mgemm_quant_fp4(const void *in, int E, int64_t N, int K, int64_t ld_in, int fmt, uint8_t *codes, uint8_t *sf,
                    float *row_scale, mgemm_stream_t stream);
int mgemm_dequant_fp4(const uint8_t *codes, const uint8_t *sf, const float *row_scale, int E, int64_t N, int K, int fmt,
                      void *out, int64_t ld_out, mgemm_stream_t stream);

/*
 * mgemm_quant_fp4_rows -- the cast of token rows in groups whose sizes live on
 * the device: the x operand of mgemm_fwd_fp4.
 *   args       filled by mgemm_fill_args for these E groups; the rows are those of
 *              its offsets, at most M
 *   in         bf16 [M, K], row stride ld_in elements
 *   codes      uint8 [M, K / 2];  row_scale  float32 [M] (MGEMM_NVFP4)
 *   sf         uint8, mgemm_fp4_scale_bytes(fmt, mgemm_colwise_ld(M, E), K) bytes;
 *              row i of group e lies at tile row poffsets[e] + i; scale rows
 *              that no token has are not written
 * With sorted_ids (the routed layer) the rows are gathered as by
 * mgemm_gather_rows: row i is in[sorted_ids[i] / top_k], zeros where
 * sorted_ids[i] >= numel or names no row below in_rows; M is then the capacity
 * of sorted_ids and the outputs, and the args block (M = -1) bounds the rows.
 * With gated != 0 (no sorted_ids), in is [M, 2 K] and row i is silu(in[i, :K]) *
 * in[i, K:], rounded to bf16 once, as by mgemm_silu_and_mul.
 */
int mgemm_quant_fp4_rows(const void *args, int E, int64_t M, const void *in, int64_t in_rows, int K, int64_t ld_in,
                         const int32_t *sorted_ids, int64_t numel, int top_k, int gated, int fmt, uint8_t *codes,
                         uint8_t *sf, float *row_scale, mgemm_stream_t stream);

/*
 * mgemm_fwd_fp4 -- the grouped product of 4-bit operands: out[r, n] = sum_k
 * xv[r, k] wv[e(r), n, k], xv and wv the values of the codes; block-scaled
 * tensor-core MMAs, float32 accumulation, one rounding to bf16.
 *   args       as for mgemm_fwd;  fmt  MGEMM_MXFP4 or MGEMM_NVFP4 (both operands)
 *   x, sx, rx  token rows from mgemm_quant_fp4_rows (rx: NVFP4 only)
 *   w, sw, rw  weights [E, N, K] from mgemm_quant_fp4 (rw: NVFP4 only)
 *   out        bf16 [M, N]
 *   row_map, map_limit, row_weight  NULL, or as for mgemm_fwd_scatter: row i goes
 *              to out[row_map[i]] (not stored outside [0, map_limit)), times
 *              row_weight[row_map[i]] before the rounding; out is [map_limit, N]
 * K % 32 == 0, N % 8 == 0.  Errors: -1, -2 (alignment), -3 (E), -4 (CUDA).
 */
int mgemm_fwd_fp4(const void *args, int fmt, const uint8_t *x, const uint8_t *sx, const float *rx, const uint8_t *w,
                  const uint8_t *sw, const float *rw, void *out, const int32_t *row_map, int64_t map_limit,
                  const float *row_weight, int64_t M, int K, int N, int E, mgemm_stream_t stream);

/*
 * mgemm_fp4_form -- how mgemm_fwd_fp4 and mgemm_gmm_fp4 tile a product on `sms` SMs
 * (0: those of the current device): returns the columns of a tile and sets *pairs
 * where pairs of CTAs compute 256 rows of them (else each its 128).  Host only; for
 * tests and measurements.
 */
int mgemm_fp4_form(int fmt, int64_t M, int K, int N, int E, int sms, int *pairs);

/*
 * mgemm_gmm_fp4 -- mgemm_fill_args, mgemm_quant_fp4_rows and mgemm_fwd_fp4 in one
 * call: out[rows of group e] = x[rows of group e] . w[e]^T for bf16 token rows.
 *   group_sizes  int64 [E], device, summing to M
 *   x            bf16 [M, K], row stride ld_x elements
 *   workspace    mgemm_gmm_fp4_workspace_bytes(fmt, M, K, E) bytes, 16-byte
 *                aligned, scratch of this call; it starts with the args block,
 *                whose status word tells of errors found on the device
 * M = 0 launches nothing.
 */
int64_t mgemm_gmm_fp4_workspace_bytes(int fmt, int64_t M, int K, int E);
int mgemm_gmm_fp4(const int64_t *group_sizes, int E, int fmt, const void *x, int64_t ld_x, const uint8_t *w,
                  const uint8_t *sw, const float *rw, void *out, int64_t M, int K, int N, void *workspace,
                  int64_t workspace_bytes, mgemm_stream_t stream);

/*
 * Weights in 4 bits with a scale for each group of a row's elements, and the product of
 * few bf16 token rows with them.  (Not on the source pages: an addition of this library,
 * beside mgemm_fwd_f8i4, whose token rows are FP8 and whose scales are powers of two.)
 *   codes   uint8 [E, N, K / 2]: q = 0 .. 15, two to a byte, the even element in the low
 *           nibble
 *   scales  bf16 [E, N, K / group], group 32, 64 or 128
 *   zeros   uint8 [E, N, K / group], 0 .. 15, or NULL: 8 everywhere
 * and w = (q - zero) scale.
 *
 * mgemm_quant_int4_groups -- cast `rows` rows (E * N) of K bf16 elements, ld_in apart
 * (% 8 == 0).  With zeros: lo = min(0, min), hi = max(0, max) of the group, scale =
 * bf16((hi / 2 - lo / 2) / 7.5), zero = clamp(rint(-lo / scale), 0, 15); without: scale =
 * bf16(max |w| / 7), zero 8.  A scale that is 0 becomes 1; q = clamp(rint(w / scale) + zero,
 * 0, 15).  A group that holds NaN or infinity gets a NaN scale.  K % group == 0, K up to 2^30.
 *
 * mgemm_gmm_int4 -- out[rows of group e] = x[rows of group e] . w[e]^T, each group's
 * products in float32, scaled and added in float32, rounded to bf16 once; the codes are
 * read in place.  Made for few rows of a group (decode): the weights are unpacked again
 * for every 8 to 24 rows of a group, so that many rows are right but slow.
 *   group_sizes  int64 [E], device, summing to M
 *   x       bf16 [M, K], row stride ld_x elements;  out  bf16 [M, N]
 *   status  int32 [1], device, or NULL: set to MGEMM_STATUS_OK, or to
 *           MGEMM_STATUS_NEGATIVE_SIZE or _SUM_MISMATCH, and then nothing else is written
 * K % group == 0, N % 8 == 0, M < 2^24, K and N up to 2^26.  M = 0 launches nothing.  One launch, no workspace.
 * Errors: -1 (sizes, group, NULL), -2 (K, N, alignment), -3 (E), -4 (CUDA).
 */
int mgemm_quant_int4_groups(const void *in, int64_t rows, int K, int64_t ld_in, int group, uint8_t *codes,
                            void *scales, uint8_t *zeros, mgemm_stream_t stream);
int mgemm_gmm_int4(const int64_t *group_sizes, int E, const void *x, int64_t ld_x, const uint8_t *codes,
                   const void *scales, const uint8_t *zeros, int group, void *out, int64_t M, int K, int N,
                   int *status, mgemm_stream_t stream);

/*
 * The norm in front of a routed layer: the residual's addition, the root mean
 * square norm, and its rows as the x operand of mgemm_fwd (e4m3 with a scale per
 * row) or mgemm_fwd_mx (e4m3 with an e8m0 scale per 32 elements) without a pass of
 * their own for the cast.  (Not on the source pages: an addition of this library.)
 *
 * mgemm_rms_norm -- per row:
 *   h = x + residual, rounded to the residual's type (without one, h = x)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * in float32; h is what the next layer reads, and the norm is that of the stored
 * values.  Rows whose squares, or their mean with eps, pass float32's range are scaled first.
 *   x         [T, C] of x_type (MGEMM_BF16 or MGEMM_F32), rows ld_x elements apart
 *   residual  [T, C] of r_type, rows ld_r apart, or NULL; MGEMM_F32 where x is
 *   weight    [C] of w_type, magnitudes below 2^60 (products h weight below 2^-126 lose bits)
 *   h         [T, C] of r_type (dense), with residual; else NULL
 *   out       bf16 [T, C] (dense): y rounded once; may be NULL where there are codes
 *   fmt       MGEMM_BF16: no codes.  MGEMM_FP8_E4M3: codes uint8 [T, C] = e4m3(y s),
 *             scales float32 [T] = s, the scale rule of mgemm_quant_rowwise on the
 *             row's largest |y|.  MGEMM_MXFP8: the rule of mgemm_quant_mx, scales
 *             uint8 [T, ld_sf] (bytes past C / 32 are not written).  The codes are
 *             cast from the float32 y, not from out.
 * 1 <= C <= MGEMM_NORM_MAX_COLUMNS, eps > 0, T < 2^31.  Without codes any C, row
 * stride and natural alignment will do (rows of 8 elements on 16-byte boundaries are
 * faster); with codes C % 16 == 0 (MXFP8: 32) and every pointer and row of x, residual,
 * weight, h, out and codes starts on a 16-byte boundary.  Outputs must not overlap
 * inputs.  Errors: -1 (sizes, types, NULL), -2 (alignment), -4 (CUDA), -5 (float32 x
 * with a bf16 residual).
 *
 * mgemm_rms_norm_bwd -- from grad_out = dL / dy (bf16) and grad_h = dL / dh (of h's
 * type, or NULL), with n = h / sqrt(mean(h^2) + eps):
 *   grad_stream  [T, C] of h_type: dL / d(x + residual) = (grad_out weight - n
 *                mean(grad_out weight n)) / sqrt(mean(h^2) + eps) + grad_h
 *   grad_x       the same in bf16, or NULL (x in bf16 under a float32 residual)
 *   grad_weight  [C] of w_type: the sum over rows of grad_out n, or NULL
 *   h, weight, eps   as written by and given to mgemm_rms_norm
 *   workspace    mgemm_rms_norm_bwd_workspace_bytes(T, C) bytes, 16-byte aligned,
 *                scratch of this call (NULL without grad_weight)
 * Sums of rows are taken in a fixed order (the same bits on every call).
 *
 * mgemm_dequant_fp8 -- the values of such codes (code / s, code 2^(byte - 127)) in
 * bf16: exact, but past bf16's range.  codes [T, C] dense, C up to 2^30; out bf16 [T, C] dense.
 */
#define MGEMM_F32 4
#define MGEMM_MXFP8 5
#define MGEMM_NORM_MAX_COLUMNS 16384
int mgemm_rms_norm(const void *x, int x_type, int64_t ld_x, const void *residual, int r_type, int64_t ld_r,
                   const void *weight, int w_type, int64_t T, int C, float eps, void *h, void *out, int fmt,
                   uint8_t *codes, void *scales, int64_t ld_sf, mgemm_stream_t stream);
int64_t mgemm_rms_norm_bwd_workspace_bytes(int64_t T, int C);
int mgemm_rms_norm_bwd(const void *grad_out, int64_t ld_g, const void *h, int h_type, int64_t ld_h, const void *weight,
                       int w_type, const void *grad_h, int64_t ld_gh, int64_t T, int C, float eps, void *grad_stream,
                       void *grad_x, void *grad_weight, void *workspace, int64_t workspace_bytes,
                       mgemm_stream_t stream);
int mgemm_dequant_fp8(const uint8_t *codes, const void *scales, int fmt, int64_t T, int C, int64_t ld_sf, void *out,
                      mgemm_stream_t stream);

/* Number of SMs of the current device (the persistent GEMM grid size), or < 0 on error. */
int mgemm_num_sms(void);
/* Static string naming a MGEMM_E* or MGEMM_STATUS_* code. */
const char *mgemm_error_string(int code);
/* Text describing the last CUDA failure that made a call return MGEMM_ECUDA
 * in the calling thread ("" if none); static per-thread storage, valid until
 * the next failing call from the same thread. */
const char *mgemm_last_error(void);
/* Library ABI version (major * 100 + minor). */
int mgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MGEMM_H_ */
