/*
 * q4gemv.h -- C ABI of a GB300 (sm_103a) library of memory-bound decode GEMVs over 4-bit block-quantized
 * weights.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All pointers are DEVICE pointers owned by the caller; the library never allocates, frees or keeps
 *    them. Outputs must not overlap inputs.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the legacy default stream) and returns
 *    as soon as the work is enqueued. Inputs must stay valid and unmodified until the work completes.
 *  - Return value: Q4_OK (0) when the work was enqueued, otherwise a negative code; nothing is enqueued when
 *    an argument is refused. The library refuses out-of-range arguments instead of clamping them.
 *      Q4_EINVAL       null required pointer, a size <= 0, M outside 1..16, K not a multiple of the block
 *                      size (32 for Q4, 256 for Q4_K), topk > E, eps negative or not finite
 *      Q4_EALIGN       a pointer below the alignment stated for it
 *      Q4_ECUDA        a CUDA call failed (launch error, no device, ...)
 *      Q4_EUNSUPPORTED the current device is not sm_103, or the staged input (M*K*4 bytes, T*K*4 for MoE)
 *                      does not fit in one CTA's shared memory next to the weight rings
 *    q4_last_error() describes the most recent refusal or failure of the calling thread.
 *  - Kernels never trap and contain no unbounded spin: each warp waits only for its own asynchronous copies
 *    (cp.async groups, or an mbarrier that its bulk or tensor copies complete). An mbarrier wait gives up after
 *    q4_set_wait_limit's cycles (default 4e9, about two seconds); the warp whose wait ran out then issues no
 *    further copies, stores NaN for every row it stores from then on (in the Q4_K row kernels, every row its CTA
 *    stores from then on), records Q4_FAULT_WAIT_TIMEOUT, and before exiting waits (bounded by 4e9 cycles) for
 *    the copies it had issued, so none lands in the shared memory of an exited CTA. Rows stored before the
 *    timeout keep their values.
 *  - Inputs are fp32 vectors, outputs fp32. Weights are packed as described per format below; multi-byte
 *    fields are little-endian.
 *
 * Formats
 * -------
 *  Q4 (planar; inferencelayer 0.2.13, src/bin/kernel_lab.rs, shader GEMV_F16S and its bindings
 *  `scales`/`quants`): a row of K weights is K/32 blocks. qs is uint8[N][K/32][16] and d is
 *  binary16[N][K/32] (raw bits in uint16). In block b, byte j holds weight 32b+j in its low nibble and
 *  weight 32b+j+16 in its high nibble; the weight is (q - 8) * d[n][b].
 *
 *  Q4_K (trueno-gpu 0.4.11, src/kernels/quantize/fused.rs, FusedRmsNormQ4KGemvKernel phase 3): a row is
 *  K/256 super-blocks of 144 bytes: binary16 d at byte 0, binary16 dmin at byte 2, 12 bytes of packed
 *  6-bit scales/mins at 4..15 and 128 quant bytes at 16..143. Sub-block j (weights 32j..32j+31) has
 *  scale sc and min m: for j < 4, sc = s[j] & 63 and m = s[j+4] & 63; for j >= 4,
 *  sc = (s[j+4] & 15) | ((s[j-4] >> 6) << 4) and m = (s[j+4] >> 4) | ((s[j] >> 6) << 4). Weight e is in
 *  quant byte 32*(e/64) + e%32, low nibble when e%64 < 32, else high nibble; its value is
 *  d*sc*q - dmin*m.
 *
 * Numerics: products and sums run in fp32 (packed fp32x2 FMAs), so results differ from exact arithmetic by
 * the order of summation; the library's tests hold every output within 1e-3 * sum_k |w_k||x_k| + 1e-5 of
 * an fp64 reference. The dequant entry points are bit-exact. Supported input range: the kernels stage each
 * 32-element block of x (or of the normalised x for Q4_K) scaled by a power of two chosen from its largest
 * magnitude; planar Q4 blocks must stay below 2^105 in magnitude and Q4_K blocks below 2^83, beyond which the
 * affected outputs are non-finite. Small inputs keep their relative accuracy down to the fp32 subnormal range.
 */
#ifndef Q4GEMV_H
#define Q4GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *q4_stream_t; /* the same type as cudaStream_t */

enum {
    Q4_OK = 0,
    Q4_EINVAL = -1,
    Q4_EALIGN = -2,
    Q4_ECUDA = -3,
    Q4_EUNSUPPORTED = -4
};

/* Fault bits reported by q4_device_faults. */
enum {
    Q4_FAULT_BAD_EXPERT = 4,   /* moe_q4_gemv, moe_q4_pure_read or moe_q4_down_gemv saw an expert id outside [0, E) */
    Q4_FAULT_WAIT_TIMEOUT = 8, /* a wait for a weight stage ran out of its cycle limit (rows written as NaN) */
    Q4_FAULT_COPY_LOST = 16,   /* even the final wait for a warp's issued copies ran out (not seen in practice) */
    Q4_FAULT_BAD_SLOT = 32,    /* kv4_write or kv4_read saw a slot >= num_pages * page_size */
    Q4_FAULT_BAD_PAGE = 64,    /* kv4_attention saw a page id outside [0, num_pages) */
    Q4_FAULT_BAD_LENGTH = 128, /* kv4_attention saw a length outside [0, max_pages * page_size] */
    Q4_FAULT_BAD_POSITION = 256 /* qk_norm_rope saw a position outside [0, max_pos) */
};

/*
 * y[n] = sum_k W[n][k] * x[k], W in planar Q4 (see Formats).
 * Source: inferencelayer kernel_lab.rs, shader GEMV_F16S (one column of its output).
 *   y   float[N]          output                       (4-byte aligned)
 *   qs  uint8[N][K/32][16] packed codes                (16-byte aligned)
 *   d   uint16[N][K/32]   binary16 block scales        (2-byte aligned; when 16-byte aligned and K % 256 == 0
 *                                                       the scales travel in the same 16-byte async copies
 *                                                       as the codes, otherwise each is read directly)
 *   x   float[K]          input                        (16-byte aligned)
 *   N >= 1; K >= 32 and K % 32 == 0.
 */
int q4_gemv(float *y, const uint8_t *qs, const uint16_t *d, const float *x, int N, int K, q4_stream_t stream);

/*
 * Y[m][n] = sum_k W[n][k] * X[m][k] for m < M, reading every weight byte once for all M rows.
 * Source: spark_model gemm_quant.rs, dense_gemv_batchm (the contract: one weight sweep for all M rows,
 * refusal of any M above the compiled maximum, which the page raises from 8 to 16 with every row bit-identical
 * to a single call); inferencelayer kernel_lab.rs, GEMV_F16S with KC columns per workgroup.
 *   Y float[M][N] (row-major), X float[M][K] (row-major, 16-byte aligned); other arguments as q4_gemv.
 *   1 <= M <= 16. Row m of Y equals q4_gemv on X[m] bit for bit (same per-row summation order and reduction
 *   tree for every M). The M staged input vectors (M*K*4 bytes) must fit in one CTA's shared memory beside the
 *   weight rings: all M <= 8 up to K = 4096 and M = 16 up to K = 2048; larger inputs return Q4_EUNSUPPORTED.
 */
int q4_gemv_batched(float *Y, const uint8_t *qs, const uint16_t *d, const float *X, int M, int N, int K,
                    q4_stream_t stream);

/*
 * y[n] = sum_k W[n][k] * xhat[k], xhat[k] = x[k] * r * gamma[k], r = 1 / sqrt(sum_k x[k]^2 / K + eps).
 * The normalised input stays in shared memory; it is never written to global memory.
 * Source: trueno-gpu fused.rs, FusedRmsNormQ4KGemvKernel (phases 1-3).
 *   y float[N]; w uint8[N][K/256][144] Q4_K (16-byte aligned); x, gamma float[K] (16-byte aligned);
 *   eps >= 0 and finite (1e-5 is the page's default). N >= 1; K >= 256 and K % 256 == 0.
 */
int fused_rmsnorm_q4k_gemv(float *y, const uint8_t *w, const float *x, const float *gamma, float eps, int N,
                           int K, q4_stream_t stream);

/*
 * Unfused Q4_K GEMV for M input rows: Y[m][n] = sum_k W[n][k] * X[m][k] for m < M, reading every weight byte
 * once for all M rows (no normalisation; M = 1 is the plain Q4_K GEMV).
 * Source: trueno-gpu fused.rs (the Q4_K format of FusedRmsNormQ4KGemvKernel phase 3; the page also names an
 * unfused Q4KGemvKernel); the batched contract of spark_model gemm_quant.rs, dense_gemv_batchm.
 *   Y float[M][N] (row-major), X float[M][K] (row-major, 16-byte aligned), w as fused_rmsnorm_q4k_gemv.
 *   1 <= M <= 8; N >= 1; K % 256 == 0. The M staged rows must fit in one CTA's shared memory beside the weight
 *   rings (M*K*4 + M*K/2 bytes: M = 8 up to K = 4096); larger inputs return Q4_EUNSUPPORTED. M = 1 runs the
 *   kernel of fused_rmsnorm_q4k_gemv without the normalisation, so its summation order differs from M >= 2.
 */
int q4k_gemv_batched(float *Y, const uint8_t *w, const float *X, int M, int N, int K, q4_stream_t stream);

/*
 * y_gate[n] = sum_k Wg[n][k] * xhat[k] and y_up[n] = sum_k Wu[n][k] * xhat[k] from one staged input.
 * gamma != NULL: xhat is the RMSNorm of x as in fused_rmsnorm_q4k_gemv; gamma == NULL: xhat = x.
 * Source: trueno-gpu fused.rs, FusedGateUpQ4KGemvKernel (with the full Q4_K decode for both projections).
 *   y_gate, y_up float[N]; w_gate, w_up uint8[N][K/256][144] (16-byte aligned); x float[K] and gamma
 *   float[K] or NULL (16-byte aligned). N >= 1; K >= 256 and K % 256 == 0; eps as above.
 */
int fused_gateup_q4k_gemv(float *y_gate, float *y_up, const uint8_t *w_gate, const uint8_t *w_up,
                          const float *x, const float *gamma, float eps, int N, int K, q4_stream_t stream);

/*
 * Expert-gathered MoE gate and up GEMV over planar Q4 expert stores.
 * For token t < T and slot s < topk with e = expert_ids[t*topk + s]:
 *   y_gate[(t*topk + s)*N + r] = sum_k Wg[e*N + r][k] * x[t][k],  likewise y_up with Wu, for r < N.
 * Each selected expert's rows are streamed once per call and applied to every token routed to it; the
 * routing is read on the device (no host synchronisation).
 * Source: inferencelayer kernel_lab.rs, moe_lab and the MoE ceiling shader (row = eid*MI + r, one output
 * per routed row, gate and up stores).
 *   qs_gate, qs_up uint8[E*N][K/32][16]; d_gate, d_up uint16[E*N][K/32]; x float[T][K] (16-byte aligned);
 *   expert_ids int32[T][topk] (device). 1 <= topk <= E; T*topk <= 512.
 *   A slot whose id is outside [0, E) gets NaN outputs and, when dev_status is not NULL, *dev_status is
 *   set to Q4_FAULT_BAD_EXPERT (dev_status is a device int32 the caller zeroes beforehand).
 */
int moe_q4_gemv(float *y_gate, float *y_up, const uint8_t *qs_gate, const uint16_t *d_gate, const uint8_t *qs_up,
                const uint16_t *d_up, const float *x, const int32_t *expert_ids, int T, int topk, int E, int N,
                int K, int32_t *dev_status, q4_stream_t stream);

/*
 * SwiGLU epilogue variants (one output instead of two):
 *   fused_gateup_swiglu_q4k_gemv: y[n] = silu(g[n]) * u[n] with g, u the two outputs of
 *     fused_gateup_q4k_gemv (same arguments, same RMSNorm rule);
 *   moe_q4_swiglu_gemv: y[(t*topk + s)*N + r] = silu(g) * u with g, u the two outputs of moe_q4_gemv for that
 *     routed row (same arguments, same routing, NaN for an invalid id, same dev_status rule).
 * silu(g) = g / (1 + exp(-g)). The pages show only that production MoE keeps one value per routed row; the
 * gated-linear-unit form is the standard one. Each call reads every weight byte once, as the two-output forms.
 *   y float[N] (gate+up) or float[T][topk][N] (MoE), 4-byte aligned.
 */
int fused_gateup_swiglu_q4k_gemv(float *y, const uint8_t *w_gate, const uint8_t *w_up, const float *x,
                                 const float *gamma, float eps, int N, int K, q4_stream_t stream);
int moe_q4_swiglu_gemv(float *y, const uint8_t *qs_gate, const uint16_t *d_gate, const uint8_t *qs_up,
                       const uint16_t *d_up, const float *x, const int32_t *expert_ids, int T, int topk, int E,
                       int N, int K, int32_t *dev_status, q4_stream_t stream);

/*
 * MoE router: gate GEMV over the experts fused with top-K softmax, for the decode tokens of one step.
 * Source: spark_model gemm_quant.rs, moe_gate_topk_fused (gate[e] = x . Wgate[e] for every expert, then the
 * top-K indices and softmax weights, `normalize` flag). Here the router rows are planar Q4 (the library's
 * format) and the inputs fp32. For token t < T:
 *   logits[t][e] = sum_k Wr[e][k] * x[t][k] for e < E (written when logits != NULL);
 *   expert_ids[t][i], i < topk: the experts of the topk largest logits in descending order, ties to the lower
 *     index (a NaN logit ranks below every other);
 *   expert_weights[t][i] = softmax over all E logits at expert_ids[t][i], divided by the sum over the topk
 *     picks when normalize != 0.
 * The ids can be passed straight to moe_q4_gemv / moe_q4_swiglu_gemv (same [T][topk] layout).
 *   expert_ids int32[T][topk], expert_weights float[T][topk], logits float[T][E] or NULL (4-byte aligned);
 *   qs uint8[E][K/32][16], d uint16[E][K/32] as q4_gemv; x float[T][K] (16-byte aligned).
 *   1 <= E <= 4096; 1 <= topk <= E; T >= 1; K % 32 == 0.
 */
int moe_router_q4(int32_t *expert_ids, float *expert_weights, float *logits, const uint8_t *qs, const uint16_t *d,
                  const float *x, int T, int E, int K, int topk, int normalize, q4_stream_t stream);

/*
 * ---- Between two projections of a decode step: q/k norm and rotation, the 4-bit cache, attention over it ----
 * (No counterpart in the source pages, whose kernels end at the projections.)
 *
 * Activations here are fp32, fp16 or bf16 (`dtype`, the same for every activation of a call); sums and statistics are
 * fp32, and values are rounded to the type once, when they are stored. (One product is narrower: kv4_attention rounds a
 * softmax weight times its value's scale to one fp16 for 16-bit types, 2^-11 of it, and to two, 2^-22, for fp32.) A
 * tensor of T tokens is rows of heads * D contiguous elements, `stride` elements from one token's row to the next (so q,
 * k and v may be columns of one projection output); every row must be 16-byte aligned.
 */
enum { Q4_F32 = 0, Q4_F16 = 1, Q4_BF16 = 2 };

/*
 * qk_norm_rope: RMSNorm of each query and key head and the rotary position rotation, in one pass.
 *   y_i = x_i * gamma_i / sqrt(sum_j x_j^2 / D + eps) for each head row x (gamma NULL: y = x), then each pair (a, b)
 *   of the first rot_dim elements becomes (a c - b s, b c + a s), c and s the cos and sin of the token's position.
 *   Pair i is (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved != 0. Elements from rot_dim on are not rotated.
 *   q, q_out [T][Hq][D], k, k_out [T][Hkv][D]; an output may be its input (same pointer and stride) or must not overlap
 *   any input; q_gamma, k_gamma float[D] or NULL; cos_sin float[max_pos][rot_dim]: row p holds cos for the rot_dim / 2
 *   pairs, then sin; positions int32[T] (device). gamma and cos_sin 16-byte aligned.
 *   The sum of squares is fp32: elements beyond about 1e18, or all below 1e-19 with an eps below 1e-38, leave its range.
 *   D a multiple of 32 up to 256; T * (Hq + Hkv) < 2^31; rot_dim a multiple of 16, 0..D (0: no rotation, cos_sin and positions unused).
 *   A token whose position is outside [0, max_pos) gets NaN heads and Q4_FAULT_BAD_POSITION is recorded.
 */
int qk_norm_rope(void *q_out, void *k_out, const void *q, const void *k, const float *q_gamma, const float *k_gamma,
                 float eps, const float *cos_sin, const int32_t *positions, int T, int Hq, int Hkv, int D, int rot_dim,
                 int max_pos, int interleaved, long long q_stride, long long k_stride, long long q_out_stride,
                 long long k_out_stride, int dtype, q4_stream_t stream);

/*
 * A paged key/value cache in planar Q4 (see Formats): a token's keys of one head are one row of head_dim weights.
 *   k_qs, v_qs uint8[num_pages][num_kv_heads][page_size][head_dim/2], k_d, v_d uint16[num_pages][num_kv_heads]
 *   [page_size][head_dim/32] (binary16), all 16-byte aligned device memory of the caller (so q4_dequant reads a cache
 *   as a matrix of num_pages * num_kv_heads * page_size rows). head_dim a multiple of 32 up to 256; page_size a power
 *   of two; at most 2^31 - 1 rows. Slot s is page s / page_size, offset s % page_size. The struct itself is host memory
 *   and is copied by the call.
 */
typedef struct {
    uint8_t *k_qs;
    uint16_t *k_d;
    uint8_t *v_qs;
    uint16_t *v_d;
    int num_pages, num_kv_heads, page_size, head_dim;
} kv4_cache;

/*
 * kv4_write: quantise the keys and values of T tokens into their slots. A 32-element block becomes
 *   d = binary16(min(max|x| / 7, 65504)), code = 8 + clamp(nearest(x / d), -7, 7) with ties to even (d = 0: codes 8);
 *   the nearest is exact, so equal inputs give equal bytes whatever the type they come in. A block that holds a NaN or
 *   an infinity is stored as d = NaN, codes 8 (it reads back as NaN).
 *   k, v [T][num_kv_heads][head_dim], T <= 2^30; slots int32[T] (device). A token whose slot is negative is skipped; one whose slot
 *   is past the cache is skipped and Q4_FAULT_BAD_SLOT recorded. The slots >= 0 of one call must be distinct (a slot
 *   given twice ends up with a mixture of the two rows).
 * kv4_read: the rows at T slots as values (code - 8) * d.
 *   k_out, v_out [T][num_kv_heads][head_dim], either may be NULL. A row whose slot is negative is left as it is; one
 *   whose slot is past the cache becomes NaN and Q4_FAULT_BAD_SLOT is recorded. A slot may be given more than once.
 */
int kv4_write(const kv4_cache *cache, const void *k, const void *v, const int32_t *slots, int T, long long k_stride,
              long long v_stride, int dtype, q4_stream_t stream);
int kv4_read(void *k_out, void *v_out, const kv4_cache *cache, const int32_t *slots, int T, long long k_stride,
             long long v_stride, int dtype, q4_stream_t stream);

/*
 * kv4_attention: attention of the M newest tokens of each of B sequences over the cache (their own keys and values are
 * in it already). Query m of a sequence of length n sits at position p = n - M + m and sees the tokens
 * max(0, p + 1 - window) <= t <= p (window 0: from token 0); token t of sequence b is at page
 * block_table[b][t / page_size], offset t % page_size. Query head h reads key head h / (Hq / num_kv_heads).
 *   out = sum_t softmax_t(scale * q . k_t) v_t;  lse = log sum_t exp(scale * q . k_t) (natural; written if not NULL).
 * A query that sees nothing (n = 0, or p < 0) gets zeros and lse = -infinity. Tokens that no query of the sequence sees
 * are not read, and what a query does not see does not enter its result, whatever bits it holds.
 *   q, out [B*M][Hq][head_dim] (token rows with strides as above); lse float[B*M][Hq]; block_table
 *   int32[B][max_pages], seq_lens int32[B] (device). 1 <= M <= 16; 1 <= B <= 1024; head_dim 64, 128 or 256;
 *   Hq a multiple of num_kv_heads; 0 < scale <= 1e30; max_pages * page_size <= 2^30.
 *   A sequence whose length is outside [0, max_pages * page_size], or that reads a page id outside [0, num_pages), gets
 *   NaN rows, and Q4_FAULT_BAD_LENGTH or Q4_FAULT_BAD_PAGE is recorded. A query row that holds a NaN or an infinity,
 *   or has a score (scale * q . k, times log2 e) above fp32's range, gives NaN; scores below its range count as minus
 *   infinity.
 *   workspace: device memory, 16-byte aligned, of at least the bytes that kv4_attention_workspace states for these
 *   sizes on the current device (whatever B and the lengths); its contents do not matter before or after. Calls that
 *   may run at the same time need a workspace each.
 *   A query element is held to 2^-34 of its row's largest (an fp32 one to 2^-22 of itself where that is more).
 *   The work is divided by the lengths of all sequences of the call, so a sequence's result may differ in the last bits
 *   when it is computed in another batch; the same call gives the same bits.
 */
int kv4_attention_workspace(size_t *bytes, int M, int Hq, int Hkv, int D, int dtype);
int kv4_attention(void *out, float *lse, const void *q, const kv4_cache *cache, const int32_t *block_table,
                  const int32_t *seq_lens, int B, int M, int Hq, int max_pages, long long q_stride, long long out_stride,
                  float scale, int window, int dtype, void *workspace, size_t workspace_bytes, q4_stream_t stream);

/*
 * ---- Around and inside a mixture-of-experts block ----
 * (No counterpart in the source pages.) Activations as in the section above: Q4_F32, Q4_F16 or Q4_BF16, rows of a token
 * `stride` elements apart and 16-byte aligned, fp32 sums, one rounding when a value is stored (for how the experts'
 * products hold their vectors see moe_q4_down_gemv).
 *
 * residual_norm: the norm behind a block, its gate and scales, the residual sum and the norm before the next block.
 *   b = x (post_gamma NULL) or x_i * post_gamma_i / sqrt(sum_j x_j^2 / K + eps);
 *   h = residual_scale * residual + branch_scale * gate * b;  y = h_i * pre_gamma_i / sqrt(sum_j h_j^2 / K + eps).
 *   h_out [T][K]; y_out [T][K], NULL exactly when pre_gamma is NULL; x [T][K]; residual [T][K] or NULL (no such term);
 *   gate NULL (1), or with gate_width K [T][K], with gate_width 1 [T] (a number per token; any alignment of its type), rows
 *   gate_stride elements apart (0: the same for every token); post_gamma, pre_gamma float[K] or NULL (16-byte aligned).
 *   y follows from the fp32 h, not from the stored one. h_out or y_out may be x or residual (same pointer and stride), and
 *   must otherwise not overlap an input or each other.
 *   T >= 1; K a multiple of 8 up to 32768; the scales finite. The sums of squares are fp32: elements beyond about 1e17, or
 *   all below 1e-19 with an eps below 1e-38, leave its range.
 */
int residual_norm(void *h_out, void *y_out, const void *x, const void *residual, const float *post_gamma, const void *gate,
                  const float *pre_gamma, float eps, float residual_scale, float branch_scale, int T, int K, int gate_width,
                  long long h_out_stride, long long y_out_stride, long long x_stride, long long residual_stride,
                  long long gate_stride, int dtype, q4_stream_t stream);

/*
 * moe_q4_down_gemv: the down projections of the selected experts and their weighted sum, behind moe_q4_swiglu_gemv.
 *   out[t][n] = residual[t][n] + sum_{s < topk} expert_weights[t][s] * sum_k W[e*N + n][k] * h[t][s][k],
 *   e = expert_ids[t*topk + s]. Each selected expert's rows are read once for up to 8 slots.
 *   out [T][N]; residual [T][N] or NULL, which out may be (same pointer and stride); qs uint8[E*N][K/32][16], d
 *   uint16[E*N][K/32]; h float[T][topk][K] (16-byte aligned); expert_ids int32[T][topk], expert_weights float[T][topk]
 *   (device). 1 <= topk <= E; T*topk <= 512; N a multiple of 8 up to 2^20; K % 32 == 0, K <= 65536;
 *   E*N < 2^31.
 *   A token with an id outside [0, E) gets a NaN row; Q4_FAULT_BAD_EXPERT is recorded and, when dev_status is not NULL,
 *   stored there. An expert may be given twice to a token.
 *   workspace: as for kv4_attention, of at least the bytes that moe_q4_down_workspace states for these sizes.
 *   A slot whose h holds a NaN or an infinity makes its token's row NaN. An element of h is held to 2^-33 of its slot's
 *   largest, or to 2^-22 of itself where that is more, whatever the type of out.
 */
int moe_q4_down_workspace(size_t *bytes, int T, int topk, int N, int K);
int moe_q4_down_gemv(void *out, const uint8_t *qs, const uint16_t *d, const float *h, const int32_t *expert_ids,
                     const float *expert_weights, const void *residual, int T, int topk, int E, int N, int K,
                     long long out_stride, long long residual_stride, int dtype, int32_t *dev_status, void *workspace,
                     size_t workspace_bytes, q4_stream_t stream);

/*
 * A mixture-of-experts layer's weights in planar Q4: router uint8[E][K/32][16] and uint16[E][K/32]; gate and up E*N rows of
 * K weights, down E*K rows of N weights (codes 16-byte aligned). Device memory of the caller; the struct itself is host
 * memory and is copied by the call.
 */
typedef struct {
    const uint8_t *router_qs;
    const uint16_t *router_d;
    const uint8_t *gate_qs;
    const uint16_t *gate_d;
    const uint8_t *up_qs;
    const uint16_t *up_d;
    const uint8_t *down_qs;
    const uint16_t *down_d;
    int E, N, K;
} moe_q4_weights;

/*
 * moe_q4_layer: the whole layer for T tokens.
 *   xn = x (gamma NULL) or its RMSNorm x_i * gamma_i / sqrt(sum_j x_j^2 / K + eps), in fp32; the router, its ties and
 *   weights as moe_router_q4 on xn; h = silu(Wg xn) * (Wu xn) of each pick, in fp32; out = residual + sum of weight * Wd h.
 *   out, x [T][K]; residual [T][K] or NULL. out may be x or residual, residual may be x (same pointers and strides).
 *   expert_ids int32[T][topk], expert_weights float[T][topk]: the picks, each written when not NULL.
 *   1 <= topk <= E <= 4096; T*topk <= 512; N % 32 == 0, N <= 65536; K % 32 == 0, K <= 32768; E*N, E*K < 2^31.
 *   A token whose x or h hold a NaN or an infinity, or whose logits hold a NaN or +infinity or are all -infinity, gets a NaN
 *   row (its ids are valid all the same); no other token is touched. A logit of -infinity beside others is a share of zero.
 *   With gamma the sum of squares is fp32, with residual_norm's range. workspace: as above, of the bytes that
 *   moe_q4_layer_workspace states; x and h are held as h is in moe_q4_down_gemv.
 */
int moe_q4_layer_workspace(size_t *bytes, int T, int topk, int E, int N, int K);
int moe_q4_layer(void *out, const void *x, const moe_q4_weights *weights, const float *gamma, float eps, const void *residual,
                 int32_t *expert_ids, float *expert_weights, int T, int topk, int normalize, long long out_stride,
                 long long x_stride, long long residual_stride, int dtype, void *workspace, size_t workspace_bytes,
                 q4_stream_t stream);

/*
 * Pure-read ceiling instruments: the same bytes, the same addressing and the same launch shape as the
 * matching GEMV, but no unpack and no dot products. Each output row receives the XOR of the 32-bit quant
 * words and zero-extended 16-bit scales (Q4) or of the 32-bit words of the super-blocks (Q4_K) of that
 * row, stored as raw bits in a float, so nothing can be optimised away and the result is checkable.
 * Source: inferencelayer kernel_lab.rs, the `pure_read` probe and MOE_PURE_READ ("pureread ~ kernel"
 * means the access pattern is the limit; "pureread >> kernel" means the arithmetic is).
 *   q4_pure_read:  sink float[N]; other arguments as q4_gemv.
 *   q4k_pure_read: sink float[N]; w as fused_rmsnorm_q4k_gemv.
 *   moe_q4_pure_read: sink_gate, sink_up float[T][topk][N]; other arguments as moe_q4_gemv; a slot with
 *   an id outside [0, E) gets NaN.
 */
int q4_pure_read(float *sink, const uint8_t *qs, const uint16_t *d, int N, int K, q4_stream_t stream);
int q4k_pure_read(float *sink, const uint8_t *w, int N, int K, q4_stream_t stream);
int moe_q4_pure_read(float *sink_gate, float *sink_up, const uint8_t *qs_gate, const uint16_t *d_gate,
                     const uint8_t *qs_up, const uint16_t *d_up, const int32_t *expert_ids, int T, int topk,
                     int E, int N, int K, int32_t *dev_status, q4_stream_t stream);

/*
 * FMA-ceiling instrument: at least `fmas` fp32 FMAs (packed fp32x2, a <- a * mul + add in eight independent
 * chains per thread) on one 512-thread CTA per SM, with no memory traffic but one float per CTA written to
 * sink. Its time is the floor for a call's FMA work alone: a batched call at M vectors does M FMAs per weight,
 * and at M = 8 the FMA pipe rather than HBM may bind.
 * Source: no page defines this instrument; it applies the idea of inferencelayer kernel_lab.rs's `pure_read`
 * probe (time one resource alone, here the FMA pipe instead of the weight stream).
 *   sink float[sink_len], sink_len >= the device's SM count; sink[b] = the sum of CTA b's chain ends.
 *   fmas >= 1; the FMAs run are rounded up to a whole number of rounds (SM count * 512 threads * 16), and the
 *   count run is stored in *fmas_done when fmas_done is not NULL (host pointer).
 *   With mul = 1 and add = 0 every chain keeps its start value: thread t's chains j = 0..7 start at
 *   ((t % 7) + j, (t % 5) + j), so sink[b] is the sum of those 8192 small integers (exact).
 */
int q4_fma_ceiling(float *sink, int sink_len, long long fmas, float mul, float add, long long *fmas_done,
                   q4_stream_t stream);

/*
 * Dequant dumps (debug): W[n][k] = the fp32 weight, bit-exact with the format definitions above
 * ((q - 8) * d for Q4; d*sc*q - dmin*m rounded once to fp32 for Q4_K).
 *   W float[N][K] (16-byte aligned); other arguments as q4_gemv / fused_rmsnorm_q4k_gemv.
 */
int q4_dequant(float *W, const uint8_t *qs, const uint16_t *d, int N, int K, q4_stream_t stream);
int q4k_dequant(float *W, const uint8_t *w, int N, int K, q4_stream_t stream);

/* Text of the calling thread's most recent refusal or failure ("" when none). Valid until the next call. */
const char *q4_last_error(void);

/*
 * Launch overlap (programmatic dependent launch; no counterpart in the source pages, which launch each
 * kernel on its own). Off by default. When on, every GEMV, fused and MoE call (not the dequant dumps) is
 * launched so that it may start while the kernel before it in the same stream is still running: the Q4
 * and Q4_K kernels issue their first weight copies at once, then wait for that kernel's completion (and
 * the visibility of its writes) before they read x, gamma or expert ids or write any output; the MoE kernel
 * waits before it reads the expert ids. The norm/rotation, cache and attention calls launch the same way and wait before
 * they read anything, so their caches and page tables may come from the call before. So a chain of calls where each x is the previous output stays
 * exact, and each call's weight streaming overlaps the previous call's tail. residual_norm, moe_q4_down_gemv and moe_q4_layer
 * likewise (the layer may read router weights before the wait). Those three are launched so in any case, but with the setting
 * off they touch nothing before the previous kernel has completed, so that it is free to write whatever they read.
 * Requirement while it is on: the kernel that runs directly before a call in the same stream must not
 * write that call's weight bytes (qs, d or the Q4_K blocks); weights written earlier in the stream, or on
 * another stream with ordinary event or stream synchronisation, are fine.
 * The setting is process-wide and read at each launch (a CUDA graph keeps the launches it captured).
 * q4_set_launch_overlap returns Q4_OK; q4_get_launch_overlap returns the current setting (0 or 1).
 */
int q4_set_launch_overlap(int enable);
int q4_get_launch_overlap(void);

/*
 * Limit, in SM cycles, of each kernel wait for a weight stage (no counterpart in the source pages). Process-wide,
 * read at each launch (a CUDA graph keeps the value it captured); default 4000000000 (about two seconds). 0 makes
 * every such wait give up at once without looking, which runs the timeout path (NaN rows, Q4_FAULT_WAIT_TIMEOUT)
 * on copies that still land. q4_set_wait_limit returns Q4_OK, or Q4_EINVAL for a negative limit;
 * q4_get_wait_limit returns the current limit.
 */
int q4_set_wait_limit(long long cycles);
long long q4_get_wait_limit(void);

/*
 * Synchronises the current device, then ORs the fault bits every kernel family recorded since the last
 * call into *faults and clears them. Returns Q4_OK or Q4_ECUDA.
 */
int q4_device_faults(unsigned *faults);

#ifdef __cplusplus
}
#endif

#endif /* Q4GEMV_H */
