/*
 * mbt_ops.h -- kernel-level entry points of libmbt.so.
 *
 * Each call runs one kernel of the decode step (the same kernel and launch
 * geometry the step uses) on caller buffers, so that every stage can be checked
 * on its own at full model sizes. Conventions are those of mbt.h: 0 on success,
 * negative MBT_ERR_* codes, device pointers in CUDA device memory, asynchronous
 * on `stream`. Calls that need scratch space take it from the stream-ordered
 * allocator (cudaMallocAsync / cudaFreeAsync on `stream`). `err` is a device
 * uint32 the kernels OR MBT_DEV_* bits into (may be NULL).
 * BF16 arrays (weights, gains) are passed as uint16 bit patterns; activations
 * are fp32.
 */
#ifndef MBT_OPS_H_
#define MBT_OPS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MBT_EPI_PARTIAL 0   /* fp32 split-K partial sums out[split][B][N]              */
#define MBT_EPI_SWIGLU  1   /* act[B][N] = silu(gate) * up (fp32), W has 2N rows       */
#define MBT_EPI_ARGMAX  2   /* next_ids[B] = argmax_n (W x)_n, logits[B][N] if non-NULL */

/* op_embed_rmsnorm: r[b] = E[tokens[b]] (fp32), y[b] = r / sqrt(mean(r^2) + eps)
 * * gamma (fp32). RMSNorm as defined in "Root Mean Square Layer
 * Normalization" (reference 9 of "Kernel Fusion for Large-Scale LLM
 * Inference"). embed [vocab][H] and gamma [H] BF16; r, y [B][H] fp32; H a
 * multiple of 4. */
int op_embed_rmsnorm(int B, int H, int vocab, const int32_t* tokens, const uint16_t* embed,
                     const uint16_t* gamma, float eps, float* r, float* y, uint32_t* err,
                     void* stream);

/* op_add_rmsnorm: r[b] += sum_s delta[s][b]; y[b] = rmsnorm(r[b]) * gamma
 * ("Kernels, Fusion & CUDA Graphs", "Fix 1: kernel fusion": residual add +
 * RMSNorm in one pass). delta [n_delta][B][H] fp32 (n_delta may be 0); r, y
 * fp32; gamma BF16. */
int op_add_rmsnorm(int B, int H, float* r, const float* delta, int n_delta,
                   const uint16_t* gamma, float eps, float* y, void* stream);

/* op_gemv_nsplit: split-K count op_gemv uses for this shape (1 unless PARTIAL). */
int op_gemv_nsplit(int epi, int w_dtype, int B, int N, int K);

/* op_gemv: the weight-streaming projection for B rows (any B >= 1; rows are
 * processed 8 at a time). W [rows][K] row-major, BF16 or e4m3 codes (w_dtype
 * MBT_DTYPE_BF16 / MBT_DTYPE_E4M3) with fp32 per-row scales (NULL for BF16);
 * x [B][K] fp32; K a multiple of 16.
 *   PARTIAL: out [nsplit][B][N] fp32, nsplit = op_gemv_nsplit(...) unless
 *            force_nsplit > 0 (clamped to K / 8 for BF16, K / 16 for e4m3);
 *            *nsplit_used receives it (may be NULL).
 *   SWIGLU:  W has 2N rows (gate rows then up rows); act [B][N] fp32.
 *   ARGMAX:  next_ids [B] int32; logits [B][N] fp32 or NULL.
 * Dequantisation is fused into the projection ("Kernel Fusion for Large-Scale
 * LLM Inference", section 11, "Epilogue and dequant fusion"). */
int op_gemv(int epi, int w_dtype, const void* W, const float* scales, int N, int K,
            const float* x, int B, int force_nsplit, float* out, float* act,
            float* logits, int32_t* next_ids, int* nsplit_used, uint32_t* err, void* stream);

/* op_gemv_sched_ints: ints of work-queue counters op_gemv_ex may use for this
 * shape (the projections split their tail into row groups claimed at run
 * time from one counter per launch and K split). */
int op_gemv_sched_ints(int epi, int w_dtype, int B, int N, int K);

/* op_gemv_ex: op_gemv with caller-owned work-queue counters: sched_ints
 * (device, op_gemv_sched_ints(...) ints) must be zero when the call is issued
 * and is zero again when it completes, so one array serves any number of
 * calls issued in order on one stream (not calls that run concurrently).
 * NULL: the counters are allocated and zeroed per call, as op_gemv does. The
 * pages have no counterpart: it exists so that back-to-back launches (timing
 * one projection, for one) carry no memset between them. */
int op_gemv_ex(int epi, int w_dtype, const void* W, const float* scales, int N, int K,
               const float* x, int B, int force_nsplit, float* out, float* act,
               float* logits, int32_t* next_ids, int* nsplit_used, int* sched_ints, uint32_t* err,
               void* stream);

/* op_gemv_norm_sched_ints: ints of work-queue counters op_gemv_norm may use. */
int op_gemv_norm_sched_ints(int epi, int w_dtype, int B, int N, int K);

/* op_gemv_norm: the projection as the decode step launches it at batch 1..15,
 * with the residual add + RMSNorm as its prologue ("Kernels, Fusion & CUDA
 * Graphs", "Fix 1: kernel fusion": residual add + RMSNorm in one pass, fused
 * here into the projection that consumes it): every CTA forms
 * x[b] = rmsnorm(r_in[b] + sum_s delta[s][b]) * gamma into its own tile and
 * the call stores the new residual r_in[b] + sum_s delta[s][b] to r_out[b].
 * r_in, r_out [B][K] fp32 (distinct buffers); delta [n_delta][B][K] fp32 or
 * NULL with n_delta = 0; gamma [K] BF16; eps inside the square root. No K
 * split: PARTIAL writes out [1][B][N]. Other arguments as op_gemv_ex
 * (sched_ints from op_gemv_norm_sched_ints, or NULL). Launch geometry and
 * shared-memory carveout are those of an 8B-class model's step. */
int op_gemv_norm(int epi, int w_dtype, const void* W, const float* scales, int N, int K,
                 const float* r_in, const float* delta, int n_delta, const uint16_t* gamma, float eps,
                 float* r_out, int B, float* out, float* act, float* logits, int32_t* next_ids,
                 int* sched_ints, uint32_t* err, void* stream);

/* op_gemm_tc: the tensor-core (tcgen05) projection the decode step uses from
 * 2 rows on with BF16 weights: W [rows][K] BF16 (K a multiple of 16, >= 64),
 * x [B][K] fp32 with 1 <= B <= 128, split internally into BF16 high/low rows
 * so that the product keeps near-fp32 accuracy; launches of at most 64 rows,
 * each CTA taking an equal share of the (tile, K) work and the fp32 sums kept
 * in registers. Epilogues as op_gemv: PARTIAL out [B][N] (complete sums:
 * `ksplit` is accepted and ignored), SWIGLU act [B][N] fp32 (W has 2N rows),
 * ARGMAX next_ids [B] (+ logits [B][N] if non-NULL). Returns
 * MBT_ERR_UNSUPPORTED where the tensor-map encoder is unavailable. ("GPU
 * Inference Internals", "Roofline: Why Decode Is Memory-Bound": at batch B the
 * weight-only intensity is 2B / b_w FLOP per byte.) */
int op_gemm_tc(int epi, const void* W, const float* scales, int N, int K, const float* x, int B,
               int ksplit, float* out, float* act, float* logits, int32_t* next_ids, uint32_t* err,
               void* stream);

/* op_gemm_tc_e4m3: as op_gemm_tc for e4m3 weights W [rows][K] (codes) with
 * fp32 per-row scales (required): x is split internally into four e4m3 terms
 * per value with a power-of-two scale per row (x = s (c0 + c1/16 + c2/256 +
 * c3/4096), within 2^-16 of |x| plus 2^-29 of the row's largest value), the
 * codes are multiplied as they are (e4m3 x e4m3 products, fp32 sums), and the
 * row scales are applied in the epilogue ("Kernel Fusion for Large-Scale LLM
 * Inference", section 11, FP8 weights and "Epilogue and dequant fusion"). The
 * SWIGLU rows pass through FP16 high/low pairs before act. K a multiple of 16,
 * >= 64; 1 <= B <= 128. */
int op_gemm_tc_e4m3(int epi, const void* W, const float* scales, int N, int K, const float* x, int B,
                    int ksplit, float* out, float* act, float* logits, int32_t* next_ids, uint32_t* err,
                    void* stream);

/* op_rope_kv_write: rotate q and k of qkv [B][(nq + 2 nkv) d] (fp32; q heads,
 * then k heads, then v heads) at positions[b] with the rotate-half pairing
 * (element i with i + d/2, angle p * theta^(-2i/d)), write rotated q to q_out
 * [B][nq][d] fp32, and store k / k_scale and v / v_scale, rounded to the cache
 * format (BF16 or e4m3), at block bt[b][p / 16], slot p % 16 of the pools
 * kpool, vpool [num_blocks + 1][nkv][16][d]. ("Kernels, Fusion & CUDA Graphs",
 * "Fix 1: kernel fusion": RoPE + KV-cache write.) */
int op_rope_kv_write(int B, const float* qkv, int nq, int nkv, int d, const int32_t* positions,
                     const int32_t* bt, int bt_stride, int max_pos, float theta, void* kpool,
                     void* vpool, int num_blocks, int kv_dtype, float k_scale, float v_scale,
                     float* q_out, uint32_t* err, void* stream);

/* op_paged_attention: out[b][h] = sum_t softmax_t(q[b][h] . K_t / sqrt(d)) V_t
 * over t < seq_lens[b], K_t and V_t (times k_scale, v_scale) gathered through
 * bt; query head h reads KV head h / (nq / nkv). q [B][nq][d] fp32; out
 * [B][nq * d] fp32. Split-K over the context with the launch geometry the
 * decode step uses for a table of bt_stride entries. ("GPU Inference
 * Internals", "The KV-Cache Ledger" and "Kernels: FlashAttention and the Memory
 * Hierarchy".) */
int op_paged_attention(int B, const float* q, int nq, int nkv, int d, const void* kpool,
                       const void* vpool, int kv_dtype, float k_scale, float v_scale,
                       const int32_t* bt, int bt_stride, const int32_t* seq_lens, int num_blocks,
                       float* out, uint32_t* err, void* stream);

/* Size in bytes of the device array op_paged_attention_noalloc works in. */
#define MBT_NOALLOC_SCRATCH_BYTES (8u << 20)

/* op_paged_attention_noalloc: op_paged_attention for callers that cannot
 * allocate device memory when they run attention -- processes that reserve
 * nearly all HBM for their KV pool up front (a new allocation would fail or
 * fragment it), latency-critical paths where cudaMalloc / cudaFree may
 * synchronise the device, runtimes that forbid allocation after start-up. The
 * paper has no counterpart; this is a property of the library, not of the
 * method.
 * Same arguments, result and launch geometry as op_paged_attention, but its
 * scratch (split partials, (max, sum) pairs, merge tickets) is a file-scope
 * device array of MBT_NOALLOC_SCRATCH_BYTES that every GPU loading the library
 * holds until the process exits; it calls no cudaMalloc, cudaFree or other
 * allocating routine. The scratch needed is about B * nq * splits * (4 d + 8)
 * bytes (splits as op_paged_attention chooses them); a call needing more than
 * the array returns MBT_ERR_SCRATCH before doing any work.
 * All calls share the array and it keeps the last call's contents (the
 * tickets are cleared at every call): calls that overlap on the GPU race, so
 * keep them in one stream order. The first call on a device also does the
 * set-up (looks up the array's device address with that device current); make
 * it before any stream capture. */
int op_paged_attention_noalloc(int B, const float* q, int nq, int nkv, int d, const void* kpool,
                               const void* vpool, int kv_dtype, float k_scale, float v_scale,
                               const int32_t* bt, int bt_stride, const int32_t* seq_lens,
                               int num_blocks, float* out, uint32_t* err, void* stream);

/* op_paged_attention_noalloc_limit: MBT_NOALLOC_SCRATCH_BYTES, as built. */
size_t op_paged_attention_noalloc_limit(void);

/* ---- 4-bit paged KV cache and prompt attention --------------------------- *
 * A third cache format beside BF16 and e4m3 (MBT_DTYPE_E2M1), for 0.28 of the
 * BF16 bytes: value = e2m1(code) * e4m3(scale) * g, one 4-bit e2m1 code per
 * value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), one e4m3 scale per 16
 * neighbouring channels of a token's head, and the fp32 scale g of the K or V
 * tensor (k_scale, v_scale). A pool is [num_blocks + 1][nkv][unit]; the unit
 * of a (block, KV head) is 9 d bytes: the codes of its 16 tokens [16][d / 2]
 * (channel 2j in the low half of byte j), then their scales [16][d / 16]. K and
 * V have a pool each. ("Kernel Fusion for Large-Scale LLM Inference", section
 * 11, "FP8 weights and KV cache": a narrow paged cache; the pages stop at 8
 * bits.)
 * Of these entry points, all take any 16-byte aligned pools, head sizes 64 and
 * 128; the attention ones up to 16 query heads per KV head. Scales are between
 * 2^-64 and 2^64, tables up to 2^26 blocks wide. Scores have to stay in fp32's
 * range. They keep nothing between calls, so calls on several streams and
 * captured graphs that run at the same time do not disturb one another as long
 * as their outputs differ. */

/* op_kv_unit_bytes: bytes of one (block, KV head) of a K or V pool for a head
 * size and cache format (MBT_DTYPE_BF16, _E4M3 or _E2M1); 0 for any other. */
size_t op_kv_unit_bytes(int d, int kv_dtype);

/* op_rope_table: the table op_rope_kv_write_fp4 reads: [max_pos][d / 2] pairs
 * (cos, sin) of the angle p * theta^(-2i/d), evaluated in double precision and
 * rounded to fp32 (device memory). Set-up: computes on the host and
 * synchronises `stream`; keep the table for all calls. */
int op_rope_table(int max_pos, int d, float theta, float* table, void* stream);

/* op_rope_kv_write_fp4: op_rope_kv_write for the 4-bit cache, n rows of any
 * sequences: rotate the q and k heads of row i of qkv [n][ld_qkv] (fp32; q
 * heads, then k heads, then v heads; ld_qkv a multiple of 4) at positions[i],
 * write the rotated q to q_out [n][nq][d] fp32, and store k and v at block
 * bt[row_seq[i]][p / 16], slot p % 16. row_seq NULL: row i is sequence i (nseq
 * >= n). bt [nseq][bt_stride]. Over each 16 channels
 *   scale = e4m3(max |x| / (6 g)),  code = e2m1(x / (scale g)),
 * to nearest (ties to even) and saturating, decided for the exact x (the
 * rotation of the fp32 inputs by the fp32 table). A group with a NaN reads as
 * NaN; an infinity saturates its group (its finite values are then small
 * beside the scale). A row whose position is outside [0, max_pos) sets
 * MBT_DEV_POS_RANGE, one whose sequence or block id is out of range
 * MBT_DEV_BLOCK_RANGE; neither is stored (its q_out row is rotated at position
 * 0 in the first case). Padding rows name block num_blocks, the null block.
 * Rows of one call that name the same slot leave its contents unspecified (the
 * null block's among them); every other byte of the pools stays as it was. */
int op_rope_kv_write_fp4(int n, const float* qkv, int ld_qkv, int nq, int nkv, int d, const int32_t* positions,
                         const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride, const float* rope,
                         int max_pos, void* kpool, void* vpool, int num_blocks, float k_scale, float v_scale,
                         float* q_out, uint32_t* err, void* stream);

/* op_kv_read_fp4: the values the cache holds for n (sequence, position) rows:
 * k_out, v_out [n][nkv][d] fp32. row_seq, nseq and bt as above. A row whose
 * position or sequence is outside the table (MBT_DEV_POS_RANGE) or whose block
 * id is out of range (MBT_DEV_BLOCK_RANGE) reads as zeros. */
int op_kv_read_fp4(int n, const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                   int nkv, int d, const void* kpool, const void* vpool, int num_blocks, float k_scale, float v_scale,
                   float* k_out, float* v_out, uint32_t* err, void* stream);

/* op_paged_attention_fp4: op_paged_attention over the 4-bit cache. q [B][nq][d]
 * fp32, out [B][nq * d] fp32, seq_lens[b] tokens of bt [B][bt_stride]. A row
 * with seq_len < 1 or beyond its table sets MBT_DEV_SEQLEN_RANGE and is 0; an
 * out-of-range block id sets MBT_DEV_BLOCK_RANGE and reads the null block.
 * Cache contents past seq_len never reach the output, NaN scales included. */
int op_paged_attention_fp4(int B, const float* q, int nq, int nkv, int d, const void* kpool, const void* vpool,
                           float k_scale, float v_scale, const int32_t* bt, int bt_stride, const int32_t* seq_lens,
                           int num_blocks, float* out, uint32_t* err, void* stream);

/* op_prompt_attention: causal attention of packed prompts over the paged cache
 * (kv_dtype MBT_DTYPE_BF16, _E4M3 or _E2M1) that already holds their K and V
 * ("GPU Inference Internals", "Roofline: Why Decode Is Memory-Bound": prefill
 * works on the whole prompt at once). Rows cu_seqlens[s] .. cu_seqlens[s + 1]
 * - 1 of q [n][nq][d] (fp32, rotated) are the last tokens of sequence s, whose
 * ctx_lens[s] tokens (those before the prompt included) are in the blocks
 * bt[s][0 ..]; the row at position p attends over tokens 0 .. p. out [n][nq * d]
 * fp32. cu_seqlens has nseq + 1 device ints, non-decreasing from 0 to at most
 * n; a sequence may have no rows. Rows past the last sequence are left as they
 * are. A row whose position is negative (ctx_lens[s] smaller than its prompt)
 * attends over nothing and is 0; ctx_lens[s] < 0 or beyond the table sets
 * MBT_DEV_SEQLEN_RANGE and the sequence's rows are 0; an out-of-range block id
 * sets MBT_DEV_BLOCK_RANGE and reads the null block. Tokens after a row's own
 * never reach it, whatever they hold. A query that is not finite makes its row
 * NaN in that head, a key that is not the rows that attend to it; an infinity
 * or a NaN in V reaches them in its channel. Queries and probabilities are
 * exact to 2^-22, probabilities below 2^-17 of the row's largest to 2^-39 of
 * that. Values of a BF16 cache are exact down to 2^-29 of the largest that the
 * row attends to among their block's 16 tokens of a head, and 2^-30 of it
 * (2^-126 at least) off below; where V's blocks differ in size, 2^-39 of the
 * largest |V| that the row attends to is the smallest share that counts. */
int op_prompt_attention(int n, const float* q, int nq, int nkv, int d, int nseq, const int32_t* cu_seqlens,
                        const int32_t* ctx_lens, const void* kpool, const void* vpool, int kv_dtype, float k_scale,
                        float v_scale, const int32_t* bt, int bt_stride, int num_blocks, float* out, uint32_t* err,
                        void* stream);

/* ---- attention over selected blocks of the paged cache -------------------- *
 * Long contexts make a decode step read all of their K and V ("GPU Inference
 * Internals", "The KV-Cache Ledger"). These entry points let every query read
 * k blocks per KV head instead, chosen by a bound on its scores that costs 1/32
 * of the BF16 cache's bytes, and lay out a step's rows on the GPU. In the order
 * of a serving step: op_kv_extend (blocks and rows for the new tokens), the
 * cache write, op_key_bounds (the ranges of the blocks written to),
 * op_block_select, op_block_attention. The write is op_rope_kv_write_fp4 for a
 * 4-bit cache. op_rope_kv_write has no row_seq: it fits a step in which every
 * sequence gets one token, so that row i is sequence i; the k and v of any other
 * step's rows the caller stores in a BF16 or e4m3 cache, at slots[i].
 * All take cache formats, head sizes, groups, scales and table widths as the
 * 4-bit section above says, up to 2^30 rows, 2^16 KV heads and 2^26 chosen
 * blocks per row and head (the last two entry points fewer than 2^28 products of
 * rows, KV heads and groups of eight query heads), and rows of any sequences: row
 * i is at positions[i] of sequence row_seq[i] (NULL: sequence i, nseq >= n) of bt
 * [nseq][bt_stride].
 * A row whose position or sequence is outside the table sets MBT_DEV_POS_RANGE;
 * an out-of-range block id sets MBT_DEV_BLOCK_RANGE. They keep nothing between
 * calls, and but for op_block_select's long tables use no scratch memory. */

/* op_kv_extend: block tables and row layout for a step's new tokens, from the
 * sequences' lengths ("Kernels, Fusion & CUDA Graphs", "The serving engine's
 * kernel stack": the paged cache behind block tables). Sequence s holds
 * ctx_lens[s] tokens and gets new_lens[s] more: its table entries from
 * ceil(ctx / 16) on are taken, sequences in order, from free_blocks[free_at[0]
 * ..] of nfree ids; *free_next is where the next call goes on. Outputs:
 *   held[nseq]          tokens afterwards
 *   cu_seqlens[nseq+1]  first packed row of each sequence's new tokens
 *   positions, row_seq, slots [n]: position, sequence and cache slot (block id *
 *                       16 + position % 16, for writes of the caller's own) of
 *                       each packed row. Rows from
 *                       cu_seqlens[nseq] on are padding: sequence nseq,
 *                       position 0, slot num_blocks * 16 (the null block; a table
 *                       with one more row that names it makes the other entry
 *                       points write and read there).
 * held may be ctx_lens and free_next may be free_at (in place), so that a
 * captured graph advances by replaying; the other arrays must be distinct. A
 * sequence whose blocks or rows no longer fit (counting those of all before it)
 * gets none and keeps its table: MBT_DEV_BLOCK_RANGE or MBT_DEV_POS_RANGE. One
 * with a negative length or beyond its table gets none: MBT_DEV_SEQLEN_RANGE. A
 * free_at[0] outside [0, nfree] sets MBT_DEV_BLOCK_RANGE and no blocks are
 * taken. Ids outside [0, num_blocks] are entered as they are, set
 * MBT_DEV_BLOCK_RANGE and make their rows' slots -1. free_blocks may be NULL if
 * nfree is 0. */
int op_kv_extend(int nseq, const int32_t* ctx_lens, const int32_t* new_lens, int32_t* bt, int bt_stride, int num_blocks,
                 const int32_t* free_blocks, int nfree, const int32_t* free_at, int n, int32_t* held, int32_t* cu_seqlens,
                 int32_t* positions, int32_t* row_seq, int64_t* slots, int32_t* free_next, uint32_t* err, void* stream);

/* op_key_bounds: for each block that the rows are in, and each KV head, a range
 * per channel that holds the keys of its tokens up to the row's own. With M the
 * largest magnitude among them (in the cache's units: k_scale is a factor of
 * all scores alike) and e the smallest exponent >= -100 with M <= 127 * 2^e,
 *   bounds[block][head][0][i] = floor(min k_i / 2^e),
 *   bounds[block][head][1][i] = ceil(max k_i / 2^e),   scales[block][head] = 2^e;
 * scale 0 where M is 0, +infinity (and codes 0) where a key is not finite.
 * bounds [num_blocks + 1][nkv][2][d] int8, scales [num_blocks + 1][nkv] fp32.
 * A row leaves its block to the next row when that is in the same block of the
 * same sequence, so a sequence's rows come in increasing order, one after
 * another; rows that are in one block otherwise must have the same position, or
 * which of them counts is unspecified. A row with an error is left
 * out; every other range stays as it was. */
int op_key_bounds(int n, const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                  int nkv, int d, const void* kpool, int kv_dtype, int num_blocks, int8_t* bounds, float* scales,
                  uint32_t* err, void* stream);

/* op_block_select_scratch: bytes of scratch that op_block_select works in for
 * these sizes on the current device; 0 up to tables of 4096 blocks. */
size_t op_block_select_scratch(int n, int nkv, int bt_stride, int k);

/* op_block_select: per row and KV head the k blocks of the row's context (tokens
 * 0 .. positions[i]) that can hold the largest scores. Over the group's query
 * heads q_g and with 2^x the smallest power of two above their largest
 * magnitude,
 *   u_gi = rint(q_gi * 2^(10 - x)),  P_i = sum_g max(u_gi, 0),  N_i = sum_g min(u_gi, 0),
 *   score = fp32(sum_i P_i high_i + N_i low_i) * scale
 * (all u are 0 where a query is not finite): above the sum of the group's scores
 * with any key of the block, up to the rounding of u. The integer sum is exact,
 * so the choice does not depend on an order of summation. A block whose scale is
 * not finite scores +infinity. The first keep_first and the last keep_last
 * blocks of the context are taken in any case (keep_last >= 1: a row sees itself;
 * keep_first + keep_last <= k), then the largest scores; of equal ones the
 * earlier block. sel [n][nkv][k] int32: the taken blocks' places in the table,
 * ascending, then -1 where the context has fewer than k blocks. q [n][nq][d]
 * fp32. An out-of-range id counts with the null block's range; a row outside
 * its table gets -1 throughout. scratch (device, 16-byte aligned) has at least
 * op_block_select_scratch(..) bytes, or the call returns MBT_ERR_SCRATCH; calls
 * that may overlap need one each. NULL: taken from the stream-ordered allocator. */
int op_block_select(int n, const float* q, int nq, int nkv, int d, const int8_t* bounds, const float* scales,
                    const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                    int num_blocks, int keep_first, int keep_last, int k, int32_t* sel, void* scratch, size_t scratch_bytes,
                    uint32_t* err, void* stream);

/* op_block_attention: softmax attention of n rows over selected blocks of the
 * cache: out[i][h] = sum_t softmax_t(q[i][h] . K_t / sqrt(d)) V_t over the tokens
 * t <= positions[i] of the blocks sel[i][KV head of h][0 .. k). Negative entries
 * of sel are skipped; one beyond the row's context sets MBT_DEV_BLOCK_RANGE and
 * is skipped. Entries may come in any order; a block entered twice counts twice.
 * A row that is left with no token, or outside its table, is 0 whatever its
 * query. q [n][nq][d] fp32, out [n][nq * d] fp32. An out-of-range id reads the
 * null block. Cache contents past a row's position never reach it. A query that
 * is not finite makes its row, if that has a token, NaN in that head, a key that
 * is not the rows that attend to it; an infinity or a NaN in V reaches them in its
 * channel. Twice sum_i |q_i k_i| over a key as the cache holds it (before
 * k_scale) has to stay in fp32's range, and so has the sum of a BF16 cache's
 * values over the row's tokens. Queries and probabilities enter the products to
 * 2^-24 over a BF16 cache and to 2^-22 over the others, probabilities below 2^-17
 * of the row's largest to 2^-39 of that. Scores are sums in fp32, off by about
 * 2^-22 of sum_i |q_i k_i| / sqrt(d); a probability is off by 2^-22 of itself, for
 * the exponential, and by 2^-21 for every factor of e between it and the row's
 * largest, for its argument's roundings. */
int op_block_attention(int n, const float* q, int nq, int nkv, int d, const void* kpool, const void* vpool, int kv_dtype,
                       float k_scale, float v_scale, const int32_t* positions, const int32_t* row_seq, int nseq,
                       const int32_t* bt, int bt_stride, const int32_t* sel, int k, int num_blocks, float* out,
                       uint32_t* err, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MBT_OPS_H_ */
