/*
 * cpattn.h -- C ABI of libcpattn.so: causal scaled-dot-product attention
 * evaluated the ring way (context parallel / RingAttention) on one GPU.
 *
 * What is computed.  For every (batch b, head h) and query row i,
 *     O_i = sum_{j in A_i} softmax_j(scale * q_i . k_j) v_j,
 *     LSE_i = log sum_{j in A_i} exp(scale * q_i . k_j)      (natural log)
 * with A_i = { j <= i } when causal, all j otherwise.  "Configuring
 * RingAttention+FlashAttention for CP" (devpress.csdn.net), section 1: each
 * rank's Q takes turns against the K/V blocks of every rank and the results
 * are aggregated; section 3, note 2: the mask is exact, nothing leaks.
 *
 * How it is evaluated.  The sequence is split over cp_size virtual ranks.
 *   causal:     2*cp_size chunks of c = S / (2*cp_size) rows; rank r owns
 *               chunks r and 2*cp_size-1-r (the zigzag of the same page,
 *               section 5, item 1);
 *   non-causal: cp_size contiguous chunks of c = S / cp_size rows.
 * At ring step t rank r attends to the K/V of rank (r - t) mod cp_size (same
 * page, section 3 code).  A (q chunk a, kv chunk b) block is SKIP when a < b,
 * DIAG (masked j <= i) when a == b, FULL otherwise.  Each step yields a partial
 * (O, LSE) per row; partials are combined by the log-sum-exp merge
 *     L = max(La,Lb) + log(exp(La-M) + exp(Lb-M)),  O = e^(La-L) Oa + e^(Lb-L) Ob.
 * "Megatron-LM source analysis: Context Parallel" (mieleap.com), section 5:
 * the per-step attention call of the double-buffered ring loop.
 *
 * Conventions for every entry point.
 *   - Tensors are caller-owned DEVICE pointers, contiguous, layout [B][H][S][D]
 *     (LSE and per-row vectors [B][H][S]).  The library keeps no pointer after
 *     the call returns and allocates no device memory on any call.
 *   - dtype is cpattn_dtype: CPATTN_BF16 (bf16 in/out, fp32 accumulate) or
 *     CPATTN_FP32 (fp32 in/out, fp32 arithmetic throughout).
 *   - stream is a cudaStream_t (NULL = legacy default stream).  Work is
 *     enqueued asynchronously; argument and shape errors are returned before
 *     anything is enqueued.  In-kernel failures (a bounded wait that ran out)
 *     are recorded on the device and reported by cpattn_sync_status().
 *   - Preconditions (CPATTN_ERR_SHAPE otherwise): B, H >= 1; S >= 1;
 *     cp_size >= 1; D is 64 or 128; causal: S % (2*cp_size) == 0, non-causal:
 *     S % cp_size == 0 (any chunk length c).  bf16 problems with c % 128 == 0
 *     run on the tcgen05 tensor-core kernels, the rest (every fp32 problem,
 *     bf16 chunks of other lengths) on the CUDA-core kernels.
 *   - Pointers must be 16-byte aligned (CPATTN_ERR_ALIGN); scale must be
 *     finite and > 0 (CPATTN_ERR_ARG).
 *   - Sizes are not visible through plain pointers: every buffer must hold the
 *     elements its stated layout implies (the Python binding checks shapes and
 *     dtypes before calling).
 *   - Each entry point opens an NVTX range named after itself for the host
 *     side of the call (no-op without an attached profiler).
 */
#ifndef CPATTN_H
#define CPATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CPATTN_OK = 0,
    CPATTN_ERR_ARG = 1,       /* null pointer, bad scale, bad step, bad capacity */
    CPATTN_ERR_SHAPE = 2,     /* sizes violate the preconditions above */
    CPATTN_ERR_DTYPE = 3,     /* unknown dtype */
    CPATTN_ERR_ALIGN = 4,     /* a pointer is not 16-byte aligned */
    CPATTN_ERR_CUDA = 5,      /* a CUDA runtime call or launch failed */
    CPATTN_ERR_TIMEOUT = 6,   /* a bounded in-kernel wait ran out (reported later) */
    CPATTN_ERR_WORKSPACE = 7, /* workspace missing or smaller than required */
    CPATTN_ERR_PAGE = 8       /* a page number, slot or length outside of the paged cache (reported later) */
} cpattn_status;

typedef enum { CPATTN_BF16 = 0, CPATTN_FP32 = 1 } cpattn_dtype;

/* Element type of a paged cache beside the two above: e4m3 codes. */
enum { CPATTN_E4M3 = 2 };

/* Block kinds in a plan row. */
enum { CPATTN_SKIP = 0, CPATTN_FULL = 1, CPATTN_DIAG = 2 };

/* Number of int32 fields in one plan row. */
#define CPATTN_PLAN_FIELDS 6

/*
 * cpattn_plan -- host only, no GPU needed.
 * Writes the ring schedule: one row of CPATTN_PLAN_FIELDS int32 per
 * (rank r, step t, q slot, kv slot) in lexicographic order, SKIP rows included:
 *     (r, t, q_chunk a, kv_chunk b, src_rank, kind)
 * with src_rank = (r - t) mod cp_size, a the q slot's chunk of rank r and b
 * the kv slot's chunk of rank src_rank.  Rows: cp_size*cp_size*4 causal,
 * cp_size*cp_size non-causal.  out: host buffer of capacity rows
 * (capacity*CPATTN_PLAN_FIELDS int32).  *n_rows is always set to the number of
 * rows needed; CPATTN_ERR_ARG if capacity is too small (nothing written) or a
 * pointer is null, CPATTN_ERR_SHAPE if S is not a multiple of the chunk count.
 * Sources: ring rule and zigzag as cited at the top of this file.
 */
int cpattn_plan(int S, int cp_size, int causal, int32_t* out, int capacity, int* n_rows);

/*
 * cpattn_fwd -- the whole ring forward in one launch: every virtual rank, every
 * step, partials merged on chip by the online (log-sum-exp) rescale, SKIP
 * blocks never computed.
 *   q, k, v : [B][H][S][D] input dtype (read)
 *   o       : [B][H][S][D] input dtype (written)
 *   lse     : [B][H][S] fp32, natural-log LSE of scale*q.k (written)
 */
int cpattn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int S, int D, int cp_size, int causal, float scale, int dtype, void* stream);

/*
 * cpattn_fwd_step -- ring step `step` (0 <= step < cp_size) for all virtual
 * ranks at once: each row's partial against the K/V that its rank holds at
 * that step (both kv chunks of the source rank, SKIP blocks omitted).
 *   o_part  : [B][H][S][D] fp32, normalised partial output (written)
 *   lse_part: [B][H][S] fp32, partial LSE; -inf (and o_part = 0) where every
 *             block of the row is SKIP at this step (written)
 */
int cpattn_fwd_step(const void* q, const void* k, const void* v, float* o_part,
                    float* lse_part, int B, int H, int S, int D, int cp_size, int causal,
                    float scale, int step, int dtype, void* stream);

/*
 * cpattn_merge -- in place: (o_acc, lse_acc) <- merge((o_acc, lse_acc),
 * (o_part, lse_part)) for `rows` rows of D fp32 values, by the log-sum-exp
 * rule at the top of this file.  A side with LSE = -inf contributes nothing
 * (both -inf: o_acc and lse_acc unchanged).  The merge the pages leave
 * unwritten: their listing adds partial outputs, which is wrong; this is the
 * exact combination.  rows >= 0, D in {64, 128}.
 */
int cpattn_merge(float* o_acc, float* lse_acc, const float* o_part, const float* lse_part,
                 long rows, int D, void* stream);

/*
 * cpattn_finalize -- o[rows][D] (dtype) <- o_acc[rows][D] (fp32), rounding to
 * nearest-even for bf16.
 */
int cpattn_finalize(const float* o_acc, void* o, long rows, int D, int dtype, void* stream);

/*
 * cpattn_bwd_workspace_bytes -- bytes of device workspace cpattn_bwd needs for
 * this shape (two fp32 values per row: delta_i = dO_i . O_i and LSE_i in base
 * 2).  0 on bad sizes.
 */
size_t cpattn_bwd_workspace_bytes(int B, int H, int S, int D);

/*
 * cpattn_bwd -- recompute backward from (O, LSE): for every non-SKIP block,
 * P = exp(scale q.k - LSE) (DIAG masked), dV += P^T dO, dP = dO V^T,
 * dS = P (dP - delta) with delta_i = dO_i . O_i, dK += scale dS^T Q,
 * dQ += scale dS K.  The gradient is that of the same function the forward
 * computes ("Megatron-LM source analysis: Context Parallel", section 2: the
 * backward mirrors the forward's communication).
 *   q, k, v, o, dout : [B][H][S][D] dtype (read); lse: [B][H][S] fp32 from
 *                      cpattn_fwd (read)
 *   dq, dk, dv       : [B][H][S][D] dtype (written)
 *   workspace        : caller-owned device buffer of ws_bytes >=
 *                      cpattn_bwd_workspace_bytes(B, H, S, D), 256-byte aligned;
 *                      contents on entry are ignored
 */
int cpattn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
               const void* dout, void* dq, void* dk, void* dv, int B, int H, int S, int D,
               int cp_size, int causal, float scale, void* workspace, size_t ws_bytes,
               int dtype, void* stream);

/*
 * cpattn_bwd_accumulate -- the same backward as cpattn_bwd, but the block's
 * gradients are ADDED, in fp32 and without rounding to the input dtype, into
 * caller-owned fp32 accumulators:
 *     dq_acc += dQ,  dk_acc += dK,  dv_acc += dV      ([B][H][S][D] fp32 each)
 * For the multi-rank ring and all-gather drivers, which call the backward once
 * per (q chunk, kv chunk) block and sum the blocks' terms for every chunk
 * ("Megatron-LM source analysis: Context Parallel", section 2: the backward
 * mirrors the forward's exchange, every block adding to the gradients of its q
 * and kv chunks).  With bf16 inputs the sums then carry one rounding at the
 * end (the caller's cast) instead of one per block term.
 *   Arguments, workspace, preconditions and errors: as cpattn_bwd.  The
 *   accumulators must not alias each other or any input.  Every element of
 *   every accumulator is read and written exactly once per call (no atomics), so
 *   calls on one stream compose; calls that overlap on the GPU and share an
 *   accumulator race.
 */
int cpattn_bwd_accumulate(const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* dout, float* dq_acc, float* dk_acc,
                          float* dv_acc, int B, int H, int S, int D, int cp_size, int causal,
                          float scale, void* workspace, size_t ws_bytes, int dtype,
                          void* stream);

/*
 * FP8 (e4m3) forward.  "Megatron-LM source analysis: Context Parallel",
 * section 4: FP8 attention inputs combined with context parallelism, to save
 * memory.  The pages fix neither the format nor the scaling; this library
 * uses e4m3 ("fn": largest finite 448, no infinities) with one scale per
 * tensor:
 *     s = 448 / max|x|  (fp32; 1 for an all-zero tensor),
 *     code = e4m3(fp32(x * s)), round to nearest even, saturating to +-448,
 * and the value a code stands for is code / s.  The attention computed is the
 * attention of those values, with P = softmax rounded to e4m3 (scaled by 2^6)
 * before the P.V product; O is bf16, LSE fp32 as in cpattn_fwd.
 *
 * cpattn_amax -- *amax (device fp32) = max_i |x[i]| over n elements of dtype.
 *   amax must be 4-byte aligned; the call zeroes it first (cudaMemsetAsync on
 *   `stream`), so it needs no initialisation.
 * cpattn_quantize_e4m3 -- codes of x ([BH][S][D], dtype) with the scale
 *   derived from *amax (device, as written by cpattn_amax):
 *     transpose = 0: out [BH][S][D] bytes (the layout of q and k)
 *     transpose = 1: out [BH][D][S] bytes (V transposed per head); S % 64 == 0
 *   D in {64, 128}; x and out 16-byte aligned.
 * cpattn_fwd_fp8 -- the ring forward of cpattn_fwd on e4m3 inputs:
 *     q8, k8 : [B][H][S][D] codes;  vt8: [B][H][D][S] codes (V transposed)
 *     amax   : device float[3] = max|q|, max|k|, max|v| (the scales' source)
 *     o      : [B][H][S][D] bf16;   lse: [B][H][S] fp32 (written)
 *   Preconditions: those of cpattn_fwd, and D == 128 and a chunk length that
 *   is a multiple of 128 (CPATTN_ERR_SHAPE).  Pointers 16-byte aligned (amax:
 *   4).  One tcgen05 launch (kind::f8f6f4 MMAs).
 */
int cpattn_amax(const void* x, long n, int dtype, float* amax, void* stream);
int cpattn_quantize_e4m3(const void* x, int dtype, int BH, int S, int D, int transpose,
                         const float* amax, uint8_t* out, void* stream);
int cpattn_fwd_fp8(const uint8_t* q8, const uint8_t* k8, const uint8_t* vt8, const float* amax,
                   void* o, float* lse, int B, int H, int S, int D, int cp_size, int causal,
                   float scale, void* stream);

/* Size of the fixed device scratch array used by cpattn_bwd_noalloc (64 MiB). */
#define CPATTN_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * cpattn_bwd_noalloc -- the same backward as cpattn_bwd, for callers that
 * cannot allocate device memory (code running inside an allocator's own
 * callbacks, in a process whose memory pool belongs to another framework, or on
 * a path that cannot afford an allocation's synchronisation or failure).  The
 * pages have no counterpart: this is an interface convenience, not part of the
 * method.
 *   Arguments: as cpattn_bwd, minus the workspace.  The caller still passes
 *   every input and output.
 *   Scratch: a fixed CPATTN_NOALLOC_SCRATCH_BYTES array in device global
 *   memory that every device loading this library holds until the process
 *   exits.  The function itself allocates and frees nothing.
 *   Limits: shapes whose cpattn_bwd_workspace_bytes(B, H, S, D) exceeds
 *   CPATTN_NOALLOC_SCRATCH_BYTES are rejected with CPATTN_ERR_WORKSPACE before
 *   anything is enqueued (CPATTN_ERR_SHAPE for invalid sizes).
 *   Set-up: the first call on a device looks up the array's device address
 *   (with that device current) and keeps it for the life of the process;
 *   make that first call before any stream capture begins.  The address
 *   belongs to the device's current context: do not use the library across a
 *   cudaDeviceReset (or any other teardown of the primary context) in the same
 *   process.
 *   Sharing: all calls on a device use the same array, which keeps the last
 *   call's contents.  It holds two fp32 values per row, delta_i = dO_i . O_i
 *   and LSE_i * log2(e); the backward's preprocess kernel rewrites both for
 *   every row of the call before anything reads them, so leftovers of earlier
 *   calls are never used (dQ, dK and dV go straight to the caller's outputs).
 *   Calls that can overlap on the GPU -- on different streams, or from
 *   different host threads -- race on the array; serialise them.
 */
int cpattn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                       int H, int S, int D, int cp_size, int causal, float scale, int dtype,
                       void* stream);

/*
 * cpattn_accumulate -- acc[i] += x[i] for i < n, acc fp32, x of `dtype`: the
 * running gradient sums of the multi-rank ring backward, where every (q chunk,
 * kv chunk) block adds its dQ, dK, dV terms ("Megatron-LM source analysis:
 * Context Parallel", section 2: the backward mirrors the forward's exchange).
 * n must be a multiple of 4 (CPATTN_ERR_SHAPE), both pointers 16-byte aligned
 * (CPATTN_ERR_ALIGN); n = 0 does nothing.
 */
int cpattn_accumulate(float* acc, const void* x, long n, int dtype, void* stream);

/*
 * The attention layer around the ring attention ("Configuring
 * RingAttention+FlashAttention for CP", section 3 code): Q, K, V projections
 * of width E (nn.Linear with bias), the [B,S,E] -> [B,H,S,D] head split, the
 * ring attention (cpattn_fwd), the head merge and the output projection.
 * bf16 only; D = E / H must be 64 or 128 and the attention's own
 * preconditions apply to (B, H, S, D, cp_size, causal).
 *   Layouts (row-major, caller-owned device memory, 16-byte aligned):
 *     x, y, dy, dx           [B][S][E]
 *     w_qkv, dw_qkv          [3E][E]   rows = the q, k and v projection weights
 *                                      stacked (out features x in features)
 *     b_qkv, db_qkv          [3E]
 *     w_o, dw_o              [E][E];   b_o, db_o [E]
 *     q, k, v, o             [B][H][S][D] (bf16), lse [B][H][S] (fp32): saved
 *                                      by the forward for the backward
 *   The projections run on this library's tcgen05 GEMM (cpattn_gemm below:
 *   bf16, fp32 accumulation, the bias added in the GEMM epilogue); the head
 *   reshapes and the bias gradients are this library's kernels too.  B*S and E
 *   must be multiples of 8 (CPATTN_ERR_SHAPE).
 *   Workspace: cpattn_layer_workspace_bytes(B, S, E, H) bytes (0 for invalid
 *   sizes), used by both calls; its contents need not survive between them.
 *   Errors: CPATTN_ERR_SHAPE / ARG / ALIGN / WORKSPACE before anything is
 *   enqueued; CPATTN_ERR_CUDA when a launch fails.
 */
size_t cpattn_layer_workspace_bytes(int B, int S, int E, int H);

/* y = out_proj(merge_heads(attention(split_heads(x w_qkv^T + b_qkv)))) */
int cpattn_layer_fwd(const void* x, const void* w_qkv, const void* b_qkv, const void* w_o,
                     const void* b_o, void* y, void* q, void* k, void* v, void* o, float* lse,
                     int B, int S, int E, int H, int cp_size, int causal, float scale,
                     void* workspace, size_t ws_bytes, void* stream);

/*
 * Gradients of the layer for upstream gradient dy, from the forward's saved
 * q, k, v, o, lse: dx, dw_qkv, db_qkv, dw_o, db_o (all overwritten).
 */
int cpattn_layer_bwd(const void* x, const void* w_qkv, const void* w_o, const void* q,
                     const void* k, const void* v, const void* o, const float* lse,
                     const void* dy, void* dx, void* dw_qkv, void* db_qkv, void* dw_o,
                     void* db_o, int B, int S, int E, int H, int cp_size, int causal,
                     float scale, void* workspace, size_t ws_bytes, void* stream);

/*
 * cpattn_gemm -- the layer's projection GEMM on the tcgen05 tensor cores:
 *     C[M][N] = op(A) op(B) (+ bias[n] added to every row),
 * bf16 operands, bias and result (round to nearest even), fp32 accumulation,
 * all row-major and caller-owned device memory.  The products of the
 * attention layer's nn.Linear projections and their gradients ("Configuring
 * RingAttention+FlashAttention for CP", section 3 code: q/k/v_proj, out_proj).
 *   a_layout 0: A stored [M][K];   1: A stored [K][M] (A is its transpose)
 *   b_layout 0: B stored [N][K] (the nn.Linear weight layout, C = A B^T);
 *            1: B stored [K][N] (C = A B)
 *   bias: [N] or NULL.  C must not alias A, B or bias.
 *   M, N, K >= 1 and multiples of 8 (CPATTN_ERR_SHAPE); pointers 16-byte
 *   aligned (CPATTN_ERR_ALIGN); layouts other than 0 / 1: CPATTN_ERR_ARG.
 *   In-kernel bounded-wait failures are reported by cpattn_sync_status().
 */
int cpattn_gemm(const void* A, const void* B, const void* bias, void* C, int M, int N, int K,
                int a_layout, int b_layout, void* stream);

/*
 * The paged key-value cache: answering, token by token, from the long contexts
 * that the calls above train on and prefill.
 *
 *   k_cache, v_cache  [num_pages][Hkv][page_size][D] of cache_dtype: CPATTN_BF16
 *                     or CPATTN_FP32 with q, k, v of the same dtype, or
 *                     CPATTN_E4M3 (one byte per element) with bf16 q, k, v.
 *                     page_size is 16, 32, 64, 128 or 256; D is 64 or 128.
 *   k_bounds          [num_pages][Hkv][2][D] of cache_dtype: elementwise smallest
 *                     (row 0) and largest (row 1) key of each page, as stored
 *   kv_amax           device float[2], max|k| and max|v| that an e4m3 cache is
 *                     scaled by: code = e4m3(fp32(x * s)), saturating, with s =
 *                     448 * (1 / amax), both rounded to fp32 (448.0 / amax of a
 *                     PyTorch tensor; the last bit may differ from the one-step
 *                     quotient of cpattn_quantize_e4m3); NULL for the other types
 *   lens              [R] int32: tokens of request r that the cache holds
 *   block_table       [R][max_pages] int32: the page of tokens j * page_size ..
 *                     is block_table[r][j]; entries behind the last held page are
 *                     never read
 *   slot              page * page_size + row, int64: where one token's rows stand
 * Positions behind a request's length may hold anything, NaN included: they are
 * never part of a result.  R requests of which some have length 0 are a padded
 * batch.  A page number or slot outside of its range is not followed: the rows it
 * stands for are left out; of a length below 0 or above max_pages * page_size
 * cpattn_select_pages and cpattn_decode take that limit; and CPATTN_ERR_PAGE is
 * recorded in the device error word (cpattn_sync_status).  All sizes are read on the device, so
 * every call can be captured into a CUDA graph and replayed as lengths change.
 * Limits (CPATTN_ERR_SHAPE): max_pages * page_size < 2^31, at most 64 query
 * heads per kv head (Hq % Hkv == 0).
 */

/* Bits of a plan's verdict. */
enum {
    CPATTN_PLAN_SHORT = 1,      /* fewer free pages than the step needs */
    CPATTN_PLAN_BAD_LENGTH = 2, /* a length is, or would come to be, below 0 or above max_pages * page_size */
    CPATTN_PLAN_CAPACITY = 4,   /* more new tokens than `capacity` slots */
    CPATTN_PLAN_BAD_STATE = 8   /* the free pages' books do not balance */
};

/*
 * cpattn_cache_plan -- the books of one step, on the device.
 *   delta          [R] int32: new tokens of request r (> 0), or minus the tokens
 *                  to take back (< 0: rejected drafts, or -lens[r] for a request that ends)
 *   free_ring      [num_pages] int32, free_state int32[2] = {head, count}: the free
 *                  pages are free_ring[(head + i) % num_pages], i < count; taken
 *                  from the front, returned behind the last, requests in order
 *   lens_out       [R], free_state_out [2]: the new lengths and state (written);
 *                  may be the same memory as lens and free_state.  With other
 *                  memory the call can be repeated and gives the same again, and
 *                  larger steps are faster.  Nothing else that is written may overlap
 *                  anything that is read or written (CPATTN_ERR_ARG)
 *   block_table, free_ring: entries of pages taken and returned are written, the
 *                  others (those of returned pages too) left as they are
 *   cu_new         [R + 1]: first new token of request r in the packed order
 *   slots          [capacity] int64: slot of every new token, -1 behind the last
 *   verdict        int32[1]: 0, or CPATTN_PLAN_* bits; then nothing changes:
 *                  lens_out = lens, free_state_out = free_state, cu_new 0, slots -1
 * Pages returned by a call can be taken from the next call on.  Page numbers in the
 * table and the ring are the caller's: one outside of the pool that is taken or
 * returned is recorded (CPATTN_ERR_PAGE) and passed on, and its tokens get slot -1.
 * Workspace: cpattn_cache_plan_workspace_bytes(R, capacity), 16-byte aligned;
 * contents on entry are ignored; calls that can overlap on the GPU need one each.
 * 0 (and NULL) for steps of up to 1024 requests and 2048 tokens.  At most 2^30
 * requests (CPATTN_ERR_SHAPE).
 */
size_t cpattn_cache_plan_workspace_bytes(int R, long capacity);
int cpattn_cache_plan(const int32_t* lens, const int32_t* delta, int32_t* block_table, int R,
                      int max_pages, int page_size, int32_t* free_ring, const int32_t* free_state,
                      int num_pages, int32_t* lens_out, int32_t* free_state_out, int32_t* cu_new,
                      int64_t* slots, long capacity, int32_t* verdict, void* workspace,
                      size_t ws_bytes, void* stream);

/*
 * cpattn_cache_append -- rows k_new[i][h][:], v_new[i][h][:] (i < N, h < Hkv) into
 * slots[i] of the cache; negative slots are skipped.
 *   strides        of tokens and heads in elements, multiples of 16 bytes
 *                  (CPATTN_ERR_SHAPE; not looked at for one token or one head);
 *                  columns are contiguous.  K and V as the layer
 *                  saves them ([H][S][D]) have token stride D and head stride S * D
 *   k_bounds       kept up to date, or NULL.  A row in a page's first slot starts
 *                  the page's bounds afresh.  With k_bounds, the new tokens of one
 *                  page must stand next to one another, as cpattn_cache_plan lists
 *                  them: no token of another page and no skipped one between them
 *                  (their slots may leave gaps).  Bounds do not shrink when tokens are
 *                  taken back: they still cover the rows that were there.  NaN
 *                  keys are left out of them; NaN where a column holds no others
 * A slot may appear once only.  N = 0 does nothing.  At most 2^25 kv heads and 2^34
 * rows, N * Hkv (CPATTN_ERR_SHAPE).
 */
int cpattn_cache_append(const void* k_new, const void* v_new, long k_tok_stride, long k_head_stride,
                        long v_tok_stride, long v_head_stride, const int64_t* slots, long N,
                        void* k_cache, void* v_cache, void* k_bounds, int Hkv, int D, int page_size,
                        int num_pages, const float* kv_amax, int dtype, int cache_dtype, void* stream);

/*
 * cpattn_select_pages -- the pages that one new token per request attends to when
 * the context is too long to read whole.  For kv head h and page j
 *     score = max over the group's query heads i of sum_d max(q_id lo_d, q_id hi_d),
 * an upper bound of q.k over the page, summed in 64 bits and rounded to fp32.  Bounds
 * may be infinite (a zero of q counts as zero beside them); a head whose sum is NaN does
 * not count, and a page for which none counts ranks last.
 *   q              [R][Hq][D] dtype
 *   pages          [R][Hkv][budget] int32 (written): the `budget` pages with the
 *                  largest scores, ascending, ties to the lower page, -1 behind the
 *                  last; the newest page and the first keep_first pages are always
 *                  among them.  All pages where a request has no more than budget
 * Preconditions: budget > keep_first >= 0, max_pages <= 49152.
 */
int cpattn_select_pages(const void* q, const void* k_bounds, const int32_t* block_table,
                        const int32_t* lens, int32_t* pages, int R, int Hq, int Hkv, int D,
                        int page_size, int max_pages, int num_pages, int budget, int keep_first,
                        int dtype, int cache_dtype, void* stream);

/*
 * cpattn_decode -- attention of one new token per request over its cached keys:
 *     o = sum_j softmax_j(scale * q . k_j) v_j,  lse = log sum_j exp(scale * q . k_j)
 * over the lens[r] tokens of request r (the new token's own among them once it is
 * appended), or over those in the listed pages.  Query head i reads kv head
 * i / (Hq / Hkv).
 *   block_table    [R][max_pages]; short contexts are answered faster in a table
 *                  that is not much wider than they need
 *   q              [R][Hq][D] dtype
 *   pages          NULL, or [R][Hkv][budget] int32 as cpattn_select_pages writes it:
 *                  the first min(budget, held pages) entries are read, negative
 *                  ones are skipped, a page listed twice counts twice
 *   o              [R][Hq][D] of o_dtype (CPATTN_BF16 or CPATTN_FP32); lse [R][Hq] fp32.
 *                  Requests without a key: o = 0, lse = -inf.  fp32 results of
 *                  parts of one context (kept by several ranks) are combined by
 *                  cpattn_merge and rounded by cpattn_finalize
 * Scores, maxima and sums are fp32.  With bf16 and e4m3 caches a weight enters the
 * weighted sum as two 16-bit numbers, off by 2^-17 (bf16) or 2^-22 (e4m3; or 2^-39 of
 * the head's largest weight) relative: nothing in a bf16 result, the largest error of
 * an fp32 one.  Queries, keys, values and q . k before it is scaled are finite in fp32:
 * a key or value that is infinite or NaN makes its heads' results NaN or infinite.
 * Workspace: cpattn_decode_workspace_bytes(R, Hq, Hkv, D) (0 for invalid sizes),
 * 256-byte aligned; contents on entry are ignored; calls that can overlap on the
 * GPU need one each.  Results do not depend on it, nor on other requests' values.
 * Limits (CPATTN_ERR_SHAPE): a cache below 256 GB each for K and V, Hq * D <= 2^30, and
 * R * Hkv * (tokens of a table's row / 64 + 4) < 2^31.
 */
size_t cpattn_decode_workspace_bytes(int R, int Hq, int Hkv, int D);
int cpattn_decode(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_table, const int32_t* lens, const int32_t* pages, void* o,
                  float* lse, int R, int Hq, int Hkv, int D, int page_size, int max_pages,
                  int num_pages, int budget, float scale, const float* kv_amax, void* workspace,
                  size_t ws_bytes, int dtype, int cache_dtype, int o_dtype, void* stream);

/*
 * cpattn_sync_status -- synchronises `stream`, then returns and clears the
 * device-side error word of the current device (CPATTN_OK, CPATTN_ERR_TIMEOUT,
 * CPATTN_ERR_PAGE) or CPATTN_ERR_CUDA if the synchronisation itself failed.  The word's device
 * address is looked up once per device and kept: as for cpattn_bwd_noalloc,
 * do not use the library across a cudaDeviceReset in the same process.
 */
int cpattn_sync_status(void* stream);

/* Human-readable name of a status code (static string). */
const char* cpattn_status_str(int status);

/*
 * Diagnostics.
 * cpattn_launch_count: number of kernels this library has enqueued so far in
 *   this process (all devices).
 * cpattn_set_path: 0 = automatic (tcgen05 kernels where the shape allows),
 *   1 = force the CUDA-core kernels, 2 = tcgen05 kernels on one SM each (the
 *   two-SM dQ kernel off); any other value means 0.  Returns the previous
 *   setting.  For tests that compare the kernel families.
 * cpattn_last_path: kernel family used by the last fwd/bwd call
 *   (0 tcgen05, 1 CUDA cores).
 * cpattn_debug_stall: n > 0 makes the next n tcgen05 forward or cpattn_decode
 *   launches omit one K/V load, so the bounded waits run out and the call reports
 *   CPATTN_ERR_TIMEOUT through cpattn_sync_status; the device stays usable.
 *   For failure-detection tests only.
 */
long long cpattn_launch_count(void);
/*
 * cpattn_profile: on != 0 starts per-kernel timing (a CUDA event pair recorded
 *   on the launch stream around every kernel the library enqueues, up to 8192
 *   kernels) and discards earlier records; 0 stops recording.  Returns the
 *   previous setting.
 * cpattn_profile_read: total milliseconds and launch count of one kernel kind
 *   since the last cpattn_profile(1); waits for those events.  Kernel kinds:
 *   0 tcgen05 forward, 1 CUDA-core forward, 2 merge, 3 finalize, 4 backward
 *   preprocess (delta), 5 CUDA-core dK/dV, 6 CUDA-core dQ, 7 tcgen05 dK/dV,
 *   8 tcgen05 dQ, 9 layer head split / merge, 10 layer bias gradients,
 *   11 gradient accumulation (cpattn_accumulate), 12 GEMM (cpattn_gemm and
 *   the layer's projections), 13 tcgen05 e4m3 forward (cpattn_fwd_fp8),
 *   14 max|x| and e4m3 quantisation, 15 single-token attention over the paged
 *   cache, 16 the join of its partial results, 17 page and slot planning, 18
 *   append to the paged cache, 19 page selection.
 */
int cpattn_profile(int on);
int cpattn_profile_read(int kernel_kind, double* total_ms, long long* launches);
int cpattn_set_path(int path);
int cpattn_last_path(void);
int cpattn_debug_stall(int n);

#ifdef __cplusplus
}
#endif

#endif /* CPATTN_H */
