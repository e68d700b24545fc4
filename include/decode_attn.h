/*
 * decode_attn.h — C ABI of the split-KV GQA decode-attention library (GB300, sm_103a).
 *
 * One query token per sequence attends over that sequence's bf16 KV cache.  For
 * sequence b, query head h and KV head g = h / G (G = Hq / Hkv; the G query heads
 * of a KV head are consecutive), over the L_b cached tokens t:
 *
 *     s_t = scale * <q[b,h,:], k[b,t,g,:]>,   out[b,h,:] = sum_t softmax(s)_t * v[b,t,g,:]
 *
 * in fp32 on the GPU, rounded once to bf16.  The G query heads of a KV head share
 * every K/V tile they read (head packing, AstrAI commit 988e013 "csrc", MMA decode
 * items).  The token range of each (sequence, KV head) is cut into pieces processed
 * by different CTAs; each piece leaves unnormalised partials (acc, m, l) and a
 * log-sum-exp combine merges them (AstrAI commit 988e013, split-KV items; merge
 * order as in "perf(qwen3.8): split the flash-decode KV range across warp-groups",
 * section "Mechanism").  Paged caches are read through a page table (AstrAI commit
 * 69fecaf "csrc/tests", paged decode items).
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    allocates nothing, keeps no per-call state, never synchronises the stream and
 *    enqueues its kernels on `stream` (a cudaStream_t; NULL = legacy default stream)
 *    of the current device.
 *  - bf16 tensors are passed as `void*` (__nv_bfloat16 elements); fp32 as float*.
 *  - q, k, v, k_pool, v_pool, out must be 16-byte aligned; part_acc and part_ml
 *    16-byte and 8-byte aligned.
 *  - Every argument is checked on the host first; a bad argument returns
 *    DA_ERR_INVALID_ARG or DA_ERR_UNSUPPORTED and launches nothing.  A launch
 *    failure returns DA_ERR_CUDA (the CUDA error is cleared).
 *  - Supported: head_dim in {32, 64, 128, 256}; Hq % Hkv == 0; 1 <= G <= 64;
 *    1 <= num_splits <= DA_MAX_SPLITS; page_size a multiple of 16.
 *  - Device waits are bounded: a kernel that waits too long sets a device error
 *    word and returns; decode_device_error() reads it.
 *
 * The split plan.  Work is counted in 16-token blocks, n_b = ceil(L_b / 16).
 * The query heads of one KV head form ceil(G / 8) equal sub-groups of at most 8
 * rows; one pass over the KV head runs ngp of them (the largest power of two that
 * divides their number, at most 2 for head_dim 128 and 4 otherwise), so a
 * sequence has U = Hkv * ceil(G / 8) / ngp segment slots (U = Hkv when G <= 8).
 * The segments (b, u) lie end to end on one line in (u, b) order (slot-major);
 * segment (b, u) takes w_b = c + 4*ceil(n_b / 4) positions, c = 4*ceil((2816 /
 * head_dim) / 4) of them without blocks (they stand for the fixed cost of a
 * piece), then its n_b blocks, then padding to whole 64-token units; an empty
 * sequence takes none.  P_b = w_0 + ... + w_{b-1}; segment (b, u) starts at
 * u*P_B + P_b; NB = U * P_B positions in all.
 *   num_splits == 1: every segment is computed whole and written directly.
 *   num_splits >= 2: the line is cut into ranges of q positions, q = ceil(NB / R)
 *     with R = (num_splits - 1) * U, rounded up to a multiple of 4 (at least 4);
 *     each range is one CTA's work; the pieces of a segment are the non-empty sets
 *     of its blocks that share a range (index j = r - range of its first block),
 *     at most num_splits of them.  A segment with one piece is written directly;
 *     one with several leaves partials in slots j = 0..pieces-1, which are merged
 *     into the output by the CTA that finishes its last piece (found with the
 *     segment's counter) when there are at most 8, else by a combine kernel that
 *     follows as a programmatic dependent launch (one CTA alone would need several
 *     dependent rounds of L2 reads for a long run of partials); an empty sequence
 *     (L_b == 0) gets a zero output.
 *   decode_plan_pieces reports this partition, and what every partial slot holds
 *   when a call returns, for any shape (host only).
 */
#ifndef DECODE_ATTN_H
#define DECODE_ATTN_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DA_OK = 0,
  DA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, negative size, Hq % Hkv != 0, ... */
  DA_ERR_UNSUPPORTED = 2,  /* head_dim, page_size, group size or batch outside the built kernels */
  DA_ERR_WORKSPACE = 3,    /* num_splits >= 2 but part_acc / part_ml / seg_counters missing */
  DA_ERR_CUDA = 4,         /* a CUDA call or launch failed (error cleared) */
  DA_ERR_TIMEOUT = 5       /* a kernel gave up on a bounded wait (see decode_device_error) */
} da_status;

#define DA_MAX_SPLITS 1024
#define DA_MAX_QLEN 16  /* query tokens per sequence of decode_attn_multi_* */

/*
 * decode_num_splits — the split count for a decode shape (host only, pure).
 *
 * The pages choose a split count that fills the device, capped by the tile count
 * (AstrAI commit 988e013, split-KV items; AstrAI commit 69fecaf, planner items).
 * Here it is the number of partial slots that lets every CTA of the persistent
 * grid own one range: S = ceil(C / num_kv_heads) + 1 with C = num_sms (one CTA per
 * SM), capped by ceil(max_seq_len / 16) and DA_MAX_SPLITS; S = 1 when
 * max_seq_len <= 16.  batch is accepted for interface stability and does not
 * change the result.  num_sms <= 0 queries the current device.
 * Returns S >= 1, or -DA_ERR_INVALID_ARG / -DA_ERR_CUDA.
 */
int decode_num_splits(int batch, int num_kv_heads, int max_seq_len, int head_dim, int num_sms);

/*
 * decode_attn_contig — decode attention over a contiguous cache.
 *
 *  q        bf16 [batch, num_q_heads, head_dim]
 *  k, v     bf16 [batch, max_ctx, num_kv_heads, head_dim]  (token-major rows)
 *  seq_lens int32 [batch] on the device, or NULL (every sequence has max_ctx tokens);
 *           values are clamped to [0, max_ctx]
 *  scale    finite float multiplying q.k (applied in fp32 after the dot product)
 *  num_splits, part_acc float [batch, num_q_heads, num_splits, head_dim],
 *           part_ml float [batch, num_q_heads, num_splits, 2] = (m, l) with m in
 *           natural-log units of the scaled score: caller-owned scratch, unused
 *           (may be NULL) when num_splits == 1.  Slots the plan does not use are not
 *           written.
 *  seg_counters  uint64 [batch * num_kv_heads * ceil(G / 8)] (at least batch * U entries are
 *           used): caller-owned, zeroed once before the first call and then
 *           reusable by every later call (each call tags its updates with its own
 *           epoch, and a value left by another call counts as zero, so no reset is
 *           needed, even after a failed call); unused (may be NULL) when
 *           num_splits == 1.  Calls that share partial buffers or counters must
 *           not overlap on the GPU.  A call may be captured in a CUDA graph and
 *           replayed: a completed call leaves each counter it used holding a value
 *           that every later call, replays included, counts as zero.  Only after a
 *           call that ended in DA_ERR_TIMEOUT must the counters be zeroed again
 *           before a captured graph that uses them is replayed.
 *  Batch limit: the split kernel keeps 8 bytes of plan per sequence in shared
 *           memory, so batch is at most decode_max_batch(...) for the shape
 *           (1159 for bf16 head_dim 128 with G <= 8); a larger batch returns
 *           DA_ERR_UNSUPPORTED and launches nothing.
 *  out      bf16 [batch, num_q_heads, head_dim]
 *  stream   cudaStream_t
 * Enqueues the split kernel, and the combine kernel when num_splits > 8.
 */
int decode_attn_contig(const void* q, const void* k, const void* v, const int* seq_lens,
                       int batch, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx,
                       float scale, int num_splits, float* part_acc, float* part_ml,
                       unsigned long long* seg_counters, void* out, void* stream);

/*
 * decode_attn_paged — decode attention over a paged cache.
 *
 *  k_pool, v_pool bf16 [num_pages, page_size, num_kv_heads, head_dim]
 *  page_table     int32 [batch, max_pages_per_seq] on the device: token t of
 *                 sequence b is row t % page_size of page page_table[b, t / page_size].
 *                 Entries past ceil(L_b / page_size) are never read.  Entries that
 *                 are read must lie in [0, num_pages); one that does not sets bit 2
 *                 of the device error word (decode_device_error) and reads page 0.
 *  seq_lens       int32 [batch] on the device (required); clamped to
 *                 [0, min(max_seq_len, max_pages_per_seq * page_size)]
 *  Other arguments as for decode_attn_contig.  Each 16-token block is fetched from
 *  its page with one tile copy, so page_size must be a multiple of 16.
 */
int decode_attn_paged(const void* q, const void* k_pool, const void* v_pool,
                      const int* page_table, const int* seq_lens,
                      int batch, int num_q_heads, int num_kv_heads, int head_dim,
                      int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                      float scale, int num_splits, float* part_acc, float* part_ml,
                      unsigned long long* seg_counters, void* out, void* stream);

/*
 * decode_combine — stand-alone log-sum-exp merge of split partials.
 *
 * For each (b, h): M = max over slots j < num_splits with l_j > 0 of m_j,
 * w_j = exp(m_j - M), out = sum_j w_j acc_j / sum_j w_j l_j, summed in a fixed
 * order (bitwise reproducible); slots with l_j == 0 are skipped and a row with no
 * live slot is written as zeros
 * ("perf(qwen3.8): split the flash-decode KV range across warp-groups", section
 * "Mechanism"; AstrAI commit 988e013, combine kernel).  Every slot is read, so
 * unused slots must hold l == 0.  Layouts as in decode_attn_contig.
 */
int decode_combine(const float* part_acc, const float* part_ml, int batch, int num_q_heads,
                   int head_dim, int num_splits, void* out, void* stream);

/*
 * decode_attn_contig_noalloc — decode_attn_contig for callers that cannot allocate.
 *
 * For callers that may not allocate device memory or hold any workspace of
 * their own: a runtime with a fixed device-memory budget that hands its plugins
 * only input and output buffers, or a serving loop that must not call cudaMalloc
 * (which can synchronise the device) between steps.  The source pages have no
 * such entry point; it is specific to this library.  Arguments are those of
 * decode_attn_contig without num_splits, part_acc, part_ml and seg_counters: the
 * split count is decode_num_splits(batch, num_kv_heads, max_ctx, head_dim, <SMs of
 * the device>), and the segment counters and partials live in an 8 MiB array
 * inside the library (every GPU that loads the library holds it until exit).
 * The array holds at most 16384 segments (batch * num_kv_heads * ceil(G / 8)) and
 * batch * num_q_heads * S * head_dim * 4 bytes of partial values (rounded up to
 * 256) plus batch * num_q_heads * S * 8 bytes of (m, l) in 8 MiB - 128 KiB;
 * larger shapes return DA_ERR_WORKSPACE and launch nothing.  Argument errors
 * return the status decode_attn_contig returns for them.  The first call on a
 * device looks up the array's device address (no allocation); make that first
 * call before any stream capture.  Calls share the array: calls that overlap on
 * the GPU race.  Calls no cudaMalloc, cudaFree or allocating library routine.
 */
int decode_attn_contig_noalloc(const void* q, const void* k, const void* v, const int* seq_lens,
                               int batch, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx,
                               float scale, void* out, void* stream);

/*
 * decode_num_splits_multi — the split count for a shape given its query heads and
 * query tokens per sequence (host only, pure): decode_num_splits with the KV
 * heads counted once per pass.  The G * q_len rows of a KV head form ceil(G*q_len/8)
 * sub-groups of at most 8 rows; one pass over the KV head runs ngp of them, the
 * largest power of two that divides their number, at most 2 for head_dim 128 and
 * 4 otherwise; so a sequence has num_kv_heads * (sub-groups / ngp) segments.
 * Gives the same value as decode_num_splits when G * q_len <= 8.  Returns
 * -DA_ERR_INVALID_ARG / -DA_ERR_UNSUPPORTED for bad shapes.
 */
int decode_num_splits_multi(int batch, int q_len, int num_q_heads, int num_kv_heads, int max_seq_len,
                            int head_dim, int num_sms);

/*
 * decode_plan_pieces — the partition of a decode call into pieces (host only, pure).
 *
 * Reports, for a call with these sizes, host copies of its sequence lengths and
 * num_splits, every piece the split kernel computes: the same plan code runs
 * here on the host.  The pages fix only caps on the split count (AstrAI commit
 * 988e013 "csrc", split-KV items: at most the tile count and 32 splits); the
 * partition itself is this library's (see "The split plan" above), and any
 * partition of each segment into at most num_splits pieces gives the same
 * attention output.
 *  seq_lens   int32 [batch] on the HOST, or NULL (every sequence max_len tokens);
 *             clamped to [0, max_len]
 *  q_len      query tokens per sequence (1 for decode_attn_contig / _paged);
 *             rows of a sequence are num_q_heads * q_len (head-major)
 *  max_len    the call's length cap: max_ctx (contiguous) or
 *             min(max_pages_per_seq * page_size, max_seq_len) (paged)
 *  records    int32 [capacity][9], one record per piece in CTA walk order:
 *             (b, row0, nrows, j, npieces, t0, t1, held_t0, held_t1): sequence b,
 *             rows row0 .. row0 + nrows - 1 of the pass (query heads x q_len
 *             rows, head-major), partial slot j of npieces, tokens [t0, t1), and
 *             the token range whose partial slot j holds when the call returns
 *             ([t0, t1); held_t0 == held_t1 == 0 when the segment has one piece,
 *             which is written straight to the output).  Empty sequences
 *             have no pieces.
 * *count receives the number of pieces; at most capacity records are written.
 * Returns DA_OK, DA_ERR_WORKSPACE (capacity < *count; *count is still set),
 * DA_ERR_INVALID_ARG or DA_ERR_UNSUPPORTED.
 */
int decode_plan_pieces(const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                       int max_len, int num_splits, int* records, int capacity, int* count);

/*
 * decode_max_batch — the largest batch the decode kernels accept for a shape
 * (host only, pure): the split kernel keeps two ints of plan per sequence in
 * shared memory beside its K/V stages.  q_len and the heads are as for
 * decode_num_splits_multi; kv_int8 != 0 for the int8 cache entry points, paged
 * != 0 for paged caches.  Returns the limit, or -DA_ERR_INVALID_ARG /
 * -DA_ERR_UNSUPPORTED.
 */
int decode_max_batch(int q_len, int num_q_heads, int num_kv_heads, int head_dim, int kv_int8, int paged);

/*
 * decode_attn_multi_contig / decode_attn_multi_paged — multi-query decode, the
 * verification step of speculative decoding scored on "perf(dspark): overlap KV
 * staging with compute via cp.async", section "sparkinfer DSpark auto-eval —
 * eval-dspark:XL" (a draft block of 7): every sequence scores q_len new tokens at once, the last q_len of its
 * L_b cached tokens, causally within the block.  Query token i (0-based) of
 * sequence b attends to cached tokens [0, L_b - q_len + 1 + i); a token that
 * sees none (L_b < q_len - i) gets a zero output.  q_len == 1 is exactly
 * decode_attn_contig / decode_attn_paged.
 *  q, out        bf16 [batch, num_q_heads, q_len, head_dim] (head-major: the q_len
 *                rows of one head are consecutive)
 *  part_acc      float [batch, num_q_heads, q_len, num_splits, head_dim];
 *  part_ml       float [batch, num_q_heads, q_len, num_splits, 2]
 *  seg_counters  uint64 [batch * num_kv_heads * ceil(G * q_len / 8)], zeroed once
 *  Every other argument as for decode_attn_contig / decode_attn_paged (the same
 *  split plan, with G * q_len rows per KV head in sub-groups of at most 8).
 *  1 <= q_len <= DA_MAX_QLEN and G * q_len <= 64, else DA_ERR_INVALID_ARG /
 *  DA_ERR_UNSUPPORTED.  num_splits: decode_num_splits_multi(batch, q_len, ...).
 */
int decode_attn_multi_contig(const void* q, const void* k, const void* v, const int* seq_lens, int batch,
                             int q_len, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx, float scale,
                             int num_splits, float* part_acc, float* part_ml, unsigned long long* seg_counters,
                             void* out, void* stream);
int decode_attn_multi_paged(const void* q, const void* k_pool, const void* v_pool, const int* page_table,
                            const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads,
                            int head_dim, int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                            float scale, int num_splits, float* part_acc, float* part_ml,
                            unsigned long long* seg_counters, void* out, void* stream);

/*
 * decode_attn_int8_contig / decode_attn_int8_paged — decode over an int8 KV cache.
 * "perf(dspark): overlap KV staging with compute via cp.async", section "Cost and
 * fallbacks", names an int8 pool read through a dequant-into-shared-memory path; its
 * format is not given there.  Here K and V are symmetric int8 values with one fp32
 * scale per (token, KV head): K[t, g, :] = k_i8[t, g, :] * k_scale[g, t] (V likewise).
 *  k_i8, v_i8       int8 [batch, max_ctx, num_kv_heads, head_dim] (16-byte aligned)
 *  k_scale, v_scale float [batch, num_kv_heads, max_ctx], head-major (16-byte aligned;
 *                   max_ctx a multiple of 4)
 *  paged:  k_pool_i8, v_pool_i8 int8 [num_pages, page_size, num_kv_heads, head_dim],
 *          k_scale_pool, v_scale_pool float [num_pages, num_kv_heads, page_size]
 *  Every other argument, the split plan, the partials and the error behaviour are
 *  those of decode_attn_contig / decode_attn_paged.  The MMA warps widen the int8
 *  operands of each 16-token block to f16 in registers (exact) and multiply in f16
 *  with fp32 accumulation; K's scale multiplies a token's score and V's scale its
 *  probability.  q is converted to f16, exact for |q| in [2^-14, 65504].
 */
int decode_attn_int8_contig(const void* q, const void* k_i8, const void* v_i8, const float* k_scale,
                            const float* v_scale, const int* seq_lens, int batch, int num_q_heads, int num_kv_heads,
                            int head_dim, int max_ctx, float scale, int num_splits, float* part_acc, float* part_ml,
                            unsigned long long* seg_counters, void* out, void* stream);
int decode_attn_int8_paged(const void* q, const void* k_pool_i8, const void* v_pool_i8, const float* k_scale_pool,
                           const float* v_scale_pool, const int* page_table, const int* seq_lens, int batch,
                           int num_q_heads, int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq,
                           int num_pages, int max_seq_len, float scale, int num_splits, float* part_acc,
                           float* part_ml, unsigned long long* seg_counters, void* out, void* stream);

/*
 * prefill_attn_contig / prefill_attn_paged — causal GQA attention of a chunk of
 * q_len new tokens per sequence (prefill when the chunk is the whole sequence,
 * chunked prefill otherwise).  "gqa_prefill_attn" on the AstrAI commit page
 * ("csrc", commit 988e013) is a tiled shared-memory kernel with mask support; the
 * pages fix no layout, so: sequence b holds L_b cached tokens (its chunk included,
 * already written to the cache), the chunk is its last q_len tokens, and query
 * token i (position L_b - q_len + i) attends to positions 0 .. L_b - q_len + i.  A
 * query that sees no token (L_b < q_len - i) gives zeros.  Query head h reads KV
 * head h / G.
 *  q, out   bf16 [batch, q_len, num_q_heads, head_dim], token-major (16-byte aligned)
 *  k, v     the decode cache: contiguous [batch, max_ctx, num_kv_heads, head_dim]
 *           (seq_lens may be NULL: every sequence max_ctx tokens), or pools
 *           [num_pages, page_size, num_kv_heads, head_dim] with page_table
 *           int32 [batch, max_pages_per_seq] (page_size a multiple of 16)
 *  seq_lens int32 [batch], clamped to [0, max_ctx] (paged: to
 *           min(max_pages_per_seq * page_size, max_seq_len))
 *  head_dim 32, 64, 128 or 256; G = num_q_heads / num_kv_heads <= 64.
 *  scale    any finite value (a positive one is applied in the exponent's fma).
 * Softmax in fp32 (log2 units), P rounded to bf16 for the P V product, fp32
 * accumulation, output rounded to bf16.  head_dim 64, 128 and 256 run on the
 * tcgen05 tensor cores with the S and O accumulators in tensor memory; head_dim
 * 32 on warp-level MMAs.  No workspace; the library allocates nothing.  Argument
 * errors return DA_ERR_INVALID_ARG / DA_ERR_UNSUPPORTED before any launch; so
 * does a build whose tensor-core kernel was compiled with fewer registers per
 * thread than its warpgroup split needs (DA_ERR_UNSUPPORTED).  Page-table entries
 * outside [0, num_pages) set bit 2 of the device error word (decode_device_error)
 * and read page 0 instead.
 */
int prefill_attn_contig(const void* q, const void* k, const void* v, const int* seq_lens, int batch, int q_len,
                        int num_q_heads, int num_kv_heads, int head_dim, int max_ctx, float scale, void* out,
                        void* stream);
int prefill_attn_paged(const void* q, const void* k_pool, const void* v_pool, const int* page_table,
                       const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                       int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, float scale, void* out,
                       void* stream);

/*
 * Rotary positions.
 *
 * Pair j of a head, j < rot_dim / 2, is turned by position * inv_freq[j] radians:
 *
 *     a' = magnitude (a cos - b sin),   b' = magnitude (a sin + b cos)
 *
 * (a, b) are elements rot_offset + (2j, 2j + 1) of the head when interleaved is 1, or
 * rot_offset + (j, j + rot_dim / 2) when it is 0; the rest of the head is unchanged.
 * inv_freq is a float64 array on the device, finite; angles are exact to 2e-7 radians
 * + position * inv_freq * 2^-52 at any 32-bit position, negative ones included, and the
 * rotation runs in fp32 with one rounding to the tensor's type.
 */
typedef enum { DA_BF16 = 0, DA_F16 = 1, DA_F32 = 2 } da_dtype;
typedef enum {
  DA_ROPE_PLAIN = 0,    /* w_j = base^(-2j / rot_dim) */
  DA_ROPE_LINEAR = 1,   /* w_j / factor: positions squeezed into the original context */
  DA_ROPE_BASE = 2,     /* base * factor^(rot_dim / (rot_dim - 2)): the slowest pair stretched by
                           factor, the fastest kept */
  DA_ROPE_BY_PARTS = 3  /* pairs of more than high_turns turns over original_ctx positions kept, of
                           fewer than low_turns divided by factor, in between mixed linearly in the
                           turns.  A model that mixes linearly in the pair's index needs its own table. */
} da_rope_scaling;

/*
 * rope_inv_freq — the frequencies of a rotary embedding (host only, pure): writes
 * rot_dim / 2 values to inv_freq (HOST memory); the magnitude that goes with a scaling is
 * the caller's.  base > 1; factor >= 1 (unused when
 * plain); original_ctx > 0 and 0 <= low_turns < high_turns (by parts only).
 */
int rope_inv_freq(double* inv_freq, int rot_dim, double base, int scaling, double factor, double original_ctx,
                  double low_turns, double high_turns);

/*
 * rope_apply — rotates the heads of tokens, or the gradient through them.
 *  x, out     [tokens, num_heads, head_dim] of dtype, elements of a head consecutive, with the
 *             given strides (in elements).  Rows of out may not share elements.  out may be x itself
 *             with the same strides (in place), and may not overlap it otherwise.  16-byte
 *             accesses are used when pointers, strides, rot_offset and the rotated part allow.
 *  positions  int32 [tokens]
 *  backward   0: out = magnitude R x; otherwise its gradient, out = magnitude R^T x.
 *  rot_dim    even, rot_offset + rot_dim <= head_dim, at most 2048
 */
int rope_apply(const void* x, void* out, const int* positions, const double* inv_freq, long long tokens,
               int num_heads, int head_dim, int rot_offset, int rot_dim, int interleaved, float magnitude,
               int backward, int dtype, long long x_token_stride, long long x_head_stride,
               long long out_token_stride, long long out_head_stride, void* stream);

/*
 * kv_write_contig / kv_write_paged / kv_write_int8_contig / kv_write_int8_paged — write
 * the last q_len tokens of every sequence into the cache that the attention calls read.
 * As for prefill_attn_*, seq_lens counts a sequence's tokens with the new ones, so new
 * token i of sequence b is position L_b - q_len + i.  Positions below 0 are skipped (a
 * padded batch: a sequence of L_b < q_len tokens brings only the last L_b of its rows).
 * A position at or past the capacity (max_ctx, or min(max_seq_len, max_pages_per_seq *
 * page_size)) is not written and sets bit 3 of the device error word; one whose page-table
 * entry lies outside [0, num_pages) is not written and sets bit 2.  Nothing else in the
 * cache changes.  Sequences whose new tokens fall on the same cache row race; new tokens
 * and caches that overlap are refused.
 *  k_new, v_new  bf16 [batch, q_len, num_kv_heads, head_dim], k_stride / v_stride elements
 *                from one token to the next (a multiple of 8, at least num_kv_heads *
 *                head_dim: a slice of a fused projection will do); 16-byte aligned
 *  inv_freq      NULL, or the frequencies by which keys are rotated first, as in rope_apply,
 *                at their positions (rot_offset a multiple of 8, rot_dim of 16); in fp32,
 *                without a rounding in between (not for a cache that kv_evict_* has cut: see there)
 *  v_new, v      both NULL: only keys are written (a latent cache, num_kv_heads 1)
 *  bf16 caches   as decode_attn_contig / _paged read them (latent_attn_*: num_kv_heads 1,
 *                head_dim latent_dim + 64); head_dim a multiple of 8 up to 1024
 *  int8 caches   as decode_attn_int8_* read them: scale = max|x| / 127 over the row's
 *                head_dim elements (1 for a row of zeros, and no smaller than the smallest normal
 *                float), value = x / scale rounded to nearest even; head_dim a multiple of 16.
 *                A row with an infinity or a NaN gets a NaN scale and zeros.
 *  seq_lens      int32 [batch] on the device (contiguous: may be NULL, every sequence
 *                max_ctx tokens)
 */
int kv_write_contig(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                    const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim, int max_ctx,
                    const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                    void* k, void* v, void* stream);
int kv_write_paged(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                   const int* page_table, const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim,
                   int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, const double* inv_freq,
                   int rot_offset, int rot_dim, int interleaved, float magnitude, void* k_pool, void* v_pool,
                   void* stream);
int kv_write_int8_contig(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                         const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim, int max_ctx,
                         const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                         void* k_i8, void* v_i8, float* k_scale, float* v_scale, void* stream);
int kv_write_int8_paged(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                        const int* page_table, const int* seq_lens, int batch, int q_len, int num_kv_heads,
                        int head_dim, int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                        const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                        void* k_pool_i8, void* v_pool_i8, float* k_scale_pool, float* v_scale_pool, void* stream);

/*
 * kv_read_paged / kv_read_int8_contig / kv_read_int8_paged — a cache's tokens as
 * contiguous bf16 (an int8 cache for prefill_attn_contig, the pages of a latent cache
 * for its expansion).  Output row i of sequence b is position starts[b] + i, widened as
 * int8 * scale in fp32 and rounded once; rows whose position is negative or at or past
 * L_b, and rows of a page-table entry outside [0, num_pages) (which sets bit 2 of the
 * device error word), are left as they were.
 *  k_out, v_out  bf16 [batch, n_tokens, num_kv_heads, head_dim] (v_out NULL with v NULL)
 *  starts        int32 [batch] on the device, or NULL (0)
 *  seq_lens      int32 [batch], clamped to the capacity; contiguous: may be NULL (max_ctx)
 */
int kv_read_paged(const void* k_pool, const void* v_pool, const int* page_table, const int* starts,
                  const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim, int page_size,
                  int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out, void* v_out, void* stream);
int kv_read_int8_contig(const void* k_i8, const void* v_i8, const float* k_scale, const float* v_scale,
                        const int* starts, const int* seq_lens, int batch, int n_tokens, int num_kv_heads,
                        int head_dim, int max_ctx, void* k_out, void* v_out, void* stream);
int kv_read_int8_paged(const void* k_pool_i8, const void* v_pool_i8, const float* k_scale_pool,
                       const float* v_scale_pool, const int* page_table, const int* starts, const int* seq_lens,
                       int batch, int n_tokens, int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq,
                       int num_pages, int max_seq_len, void* k_out, void* v_out, void* stream);

/*
 * kv_read_paged_filled / kv_read_int8_contig_filled / kv_read_int8_paged_filled — the same, but
 * the outputs' rows that kv_read_* leaves as they were are zeros: every row is written.
 */
int kv_read_paged_filled(const void* k_pool, const void* v_pool, const int* page_table, const int* starts,
                         const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim, int page_size,
                         int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out, void* v_out, void* stream);
int kv_read_int8_contig_filled(const void* k_i8, const void* v_i8, const float* k_scale, const float* v_scale,
                               const int* starts, const int* seq_lens, int batch, int n_tokens, int num_kv_heads,
                               int head_dim, int max_ctx, void* k_out, void* v_out, void* stream);
int kv_read_int8_paged_filled(const void* k_pool_i8, const void* v_pool_i8, const float* k_scale_pool,
                              const float* v_scale_pool, const int* page_table, const int* starts, const int* seq_lens,
                              int batch, int n_tokens, int num_kv_heads, int head_dim, int page_size,
                              int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out, void* v_out,
                              void* stream);

/*
 * latent_attn_contig / latent_attn_paged — attention over a cache of one shared latent
 * vector a token, in its absorbed form: the up-projections of keys and values are folded
 * into the queries and the output, so every head attends to the cached vector itself.
 * With c_t the cached row of latent_dim + 64 elements (the latent, then the rotated part
 * that all heads share), for query token i (of the last q_len tokens, as in
 * decode_attn_multi_*: it sees the first L_b - q_len + 1 + i cached tokens) and head h:
 *
 *     s_t = scale * <q[b,i,h,:], c_t>,   out[b,i,h,:] = sum_t softmax(s)_t * c_t[0 : latent_dim]
 *
 * A query that sees no token gives zeros.
 *  q          bf16 [batch, q_len, num_heads, latent_dim + 64], token-major
 *  cache      bf16 [batch, max_ctx, latent_dim + 64], or a pool [num_pages, page_size,
 *             latent_dim + 64] with page_table int32 [batch, max_pages_per_seq] (page_size a
 *             multiple of 16; kv_write_* with num_kv_heads 1 and no values writes either).  Rows at
 *             positions below L_b are finite; what lies past them is never used.
 *  seq_lens   int32 [batch], clamped to the capacity (contiguous: may be NULL, max_ctx)
 *  out        bf16 [batch, q_len, num_heads, latent_dim]
 *  workspace  latent_workspace_bytes(...) bytes, 16-byte aligned, of any content; calls that share
 *             it must not overlap on the GPU (two captured graphs included)
 *  latent_dim 128, 256 or 512; num_heads up to DA_MAX_LATENT_HEADS; 1 <= q_len <= DA_MAX_QLEN;
 *             batch up to latent_max_batch(...).  scale: finite.
 * Softmax in fp32, weights rounded to bf16 for the product with the latents and summed as
 * rounded, fp32 accumulation, one rounding of the output.  Results are bitwise reproducible.
 * Page-table entries outside [0, num_pages) set bit 2 of the device error word and read
 * page 0 instead.  DA_ERR_WORKSPACE: the workspace is missing or too small.
 */
#define DA_MAX_LATENT_HEADS 256
int latent_attn_contig(const void* q, const void* cache, const int* seq_lens, int batch, int q_len, int num_heads,
                       int latent_dim, int max_ctx, float scale, void* workspace, long long workspace_bytes,
                       void* out, void* stream);
int latent_attn_paged(const void* q, const void* pool, const int* page_table, const int* seq_lens, int batch,
                      int q_len, int num_heads, int latent_dim, int page_size, int max_pages_per_seq, int num_pages,
                      int max_seq_len, float scale, void* workspace, long long workspace_bytes, void* out,
                      void* stream);

/*
 * latent_workspace_bytes — the workspace of a latent_attn_* call on a device of num_sms
 * SMs (<= 0: the current device); latent_max_batch — the largest batch it accepts (host
 * only, pure).  Negative da_status for shapes outside those above.
 */
long long latent_workspace_bytes(int batch, int q_len, int num_heads, int latent_dim, int num_sms);
int latent_max_batch(int q_len, int num_heads, int latent_dim);

/*
 * latent_prefill_contig — causal prefill of the last q_len tokens over keys and values
 * expanded from the latent vectors (the expanded form, for many query tokens: fewer
 * operations a key than the absorbed one).  Head h's key at token t is [k_nope[b,t,h,:],
 * k_rope[b,t,:]]; causality, lengths and empty rows as for prefill_attn_contig.
 *  q          bf16 [batch, q_len, num_heads, head_dim + 64], token-major
 *  k_nope, v  bf16 [batch, max_ctx, num_heads, head_dim] with the given strides in elements, the
 *             same for both (multiples of 8; a batch entry is max_ctx tokens): one product may
 *             expand a token's keys and values side by side
 *  k_rope     bf16 [batch, max_ctx, 64] with rope_token_stride elements between tokens (a multiple
 *             of 8): the last 64 columns of a latent cache will do
 *  out        bf16 [batch, q_len, num_heads, head_dim]
 *  head_dim   64 or 128; seq_lens int32 [batch] clamped to [0, max_ctx], or NULL (max_ctx); max_ctx
 *             below 2^31 - 256
 *  workspace  NULL, or latent_prefill_workspace_bytes(...) bytes, 16-byte aligned, of any content:
 *             with it, the keys of few query blocks are split over CTAs and joined in fp32.  Calls
 *             that share it must not overlap on the GPU (two captured graphs included).
 * Keys and values at positions below L_b are finite; what lies past them is never used.
 * Numerics as for prefill_attn_*.  DA_ERR_WORKSPACE: a workspace that is too small.
 */
int latent_prefill_contig(const void* q, const void* k_nope, const void* k_rope, const void* v, const int* seq_lens,
                          int batch, int q_len, int num_heads, int head_dim, int max_ctx,
                          long long kv_token_stride, long long kv_head_stride, long long rope_token_stride,
                          float scale, void* workspace, long long workspace_bytes, void* out, void* stream);

/*
 * latent_prefill_workspace_bytes — the workspace with which latent_prefill_contig splits
 * keys on a device of num_sms SMs (<= 0: the current device); 0 where it would not (host
 * only, pure).  Negative da_status for shapes outside those above.
 */
long long latent_prefill_workspace_bytes(int batch, int q_len, int num_heads, int head_dim, int max_ctx, int num_sms);

/* Human-readable name of a da_status value (static string). */
const char* decode_status_string(int status);

/*
 * Attention behind a shared prefix.
 *
 * prefix_attn_contig / prefix_attn_paged — attention of the last q_len tokens of every
 * sequence of a batch whose sequences begin with the same prefix_len tokens.  The prefix is
 * read once for the whole batch, the rest of each sequence once for that sequence, and the
 * two parts are joined by their softmax sums.  Query token i of sequence b (position L_b -
 * q_len + i, L_b prefix included) attends to tokens 0 .. L_b - q_len + i, prefix and rest
 * alike; one that sees none (a batch entry of length 0, say) gives zeros.  Query head h reads
 * KV head h / G, G = num_q_heads / num_kv_heads <= 64.
 *  q, out   bf16 [batch, q_len, num_q_heads, head_dim], token-major; head_dim 64, 128 or 256
 *  k_prefix, v_prefix  contiguous: bf16 [prefix_len, num_kv_heads, head_dim]
 *  k, v     contiguous: bf16 [batch, max_ctx, num_kv_heads, head_dim], row t - prefix_len holds token t;
 *           paged: pools [num_pages, page_size, num_kv_heads, head_dim], page_size a multiple of 16
 *  prefix_table  int32, the prefix's ceil(prefix_len / page_size) pages
 *  page_table    int32 [batch, max_pages_per_seq] of the whole sequences: entry t / page_size is token t's
 *           page for t >= prefix_len; the entries of the prefix's whole pages are not read, so the prefix
 *           may end inside a page
 *  seq_lens int32 [batch], clamped to [0, prefix_len + max_ctx], or to what the table and max_seq_len hold;
 *           NULL (contiguous only): all prefix_len + max_ctx
 *  workspace  prefix_attn_workspace_bytes(...) bytes, 16-byte aligned; contents need not be kept, calls that
 *           share one must not overlap on the GPU.  num_sms <= 0: of the current device.
 * Softmax in fp32, the weights rounded to bf16 for the product with V, fp32 sums, one rounding of the output.
 * Made for few new tokens a sequence: their own tokens are read once for every 8 or 16 query rows, so prompts of more
 * than about 100 tokens are faster as whole sequences in prefill_attn_* (8 x 128 tokens behind 2048, 32/8 heads of 128:
 * 107 us against 43; 8 x 64 behind 8192: 91 against 131).
 * What lies past a sequence's end may hold anything, and infinities and NaN, of the prefix too, reach only the rows
 * that see them.
 * Pages outside [0, num_pages) set bit 2 of the device error word and read page 0 instead.  Outputs may not
 * overlap inputs.
 */
long long prefix_attn_workspace_bytes(int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                                      int num_sms);
int prefix_attn_contig(const void* q, const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                       const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                       int prefix_len, int max_ctx, float scale, void* workspace, long long workspace_bytes, void* out,
                       void* stream);
int prefix_attn_paged(const void* q, const void* k_pool, const void* v_pool, const int* prefix_table, int prefix_len,
                      const int* page_table, const int* seq_lens, int batch, int q_len, int num_q_heads,
                      int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                      int max_seq_len, float scale, void* workspace, long long workspace_bytes, void* out, void* stream);

/*
 * Attention over selected blocks.
 *
 * A sequence's cache is taken as blocks of block_size tokens (block j: tokens j block_size ..).
 *
 * block_means_contig / block_means_paged — the mean keys of the blocks that hold the last q_len
 * tokens of each sequence (q_len >= the length: of all its blocks; after the keys are written):
 * means[b, h, j] = the mean of the block's keys below the length, summed in fp32, rounded once.
 * Other blocks' means stay as they were.
 *  k        bf16 cache or pool as above; head_dim a multiple of 8
 *  means    bf16 [batch, num_kv_heads, max_blocks, head_dim]; max_blocks * block_size must cover max_ctx (paged:
 *           what the table and max_seq_len hold); block_size <= 65536; a pool of less than 2^32 tokens
 */
int block_means_contig(const void* k, const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim,
                       int max_ctx, int block_size, int max_blocks, void* means, void* stream);
int block_means_paged(const void* k_pool, const int* page_table, const int* seq_lens, int batch, int q_len,
                      int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                      int max_seq_len, int block_size, int max_blocks, void* means, void* stream);
/*
 * block_select — the blocks that each of the last q_len tokens attends to, for every KV head.  Token i of
 * sequence b, at position p = L_b - q_len + i, sees blocks 0 .. p / block_size.  It takes the first `first` and
 * the last `recent` (>= 1) of them, and of the others those with the largest max over the group's heads of
 * <q, mean>, until it has n_select (>= first + recent) or all.  Scores are compared to 2^-42 of |q| |mean| (ties:
 * the lower block; a head whose score is NaN counts as lowest).  Blocks whose scores lie within fp32's error of the
 * last one taken are compared pairwise: a few as a rule, but a cache of many equal means takes long (512 of them 0.15
 * ms, 8192 14 ms).
 *  q        bf16 [batch, q_len, num_q_heads, head_dim], head_dim 64, 128 or 256
 *  means    as block_means writes them, max_blocks <= 8192; seq_lens is clamped to max_blocks * block_size (NULL:
 *           that length)
 *  out      int32 [batch, q_len, num_kv_heads, n_select], ascending, -1 behind the last
 */
int block_select(const void* q, const void* means, const int* seq_lens, int batch, int q_len, int num_q_heads,
                 int num_kv_heads, int head_dim, int block_size, int max_blocks, int n_select, int first, int recent,
                 int* out, void* stream);
/*
 * sparse_attn_contig / sparse_attn_paged — attention of the last q_len tokens over the listed blocks: query
 * token i attends to the tokens of its blocks up to its own position.  An entry that is negative or past the
 * position lists nothing, one that is listed twice counts twice, the order is free; a token whose blocks hold
 * nothing gives zeros.
 *  q, out, k, v, page_table, seq_lens, scale  as prefix_attn without a prefix
 *  blocks   int32 [batch, q_len, num_kv_heads, n_select]; block_size a multiple of 16, of any relation to page_size
 */
int sparse_attn_contig(const void* q, const void* k, const void* v, const int* blocks, const int* seq_lens, int batch,
                       int q_len, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx, int block_size,
                       int n_select, float scale, void* out, void* stream);
int sparse_attn_paged(const void* q, const void* k_pool, const void* v_pool, const int* blocks, const int* page_table,
                      const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                      int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, int block_size, int n_select,
                      float scale, void* out, void* stream);

/*
 * Weights and eviction.
 *
 * kv_weights_contig / kv_weights_paged / kv_weights_int8_* — what attention weight the last q_len tokens give
 * each cached token: out[b, h, t] = decay * prior[b, h, t] + sum over the q_len tokens and the G heads of group h
 * of softmax_t(scale <q, k>), causal as in prefix_attn without a prefix, for t < L_b; entries at and past L_b are
 * neither read nor written.  Softmax and sums in fp32.
 *  q        bf16 [batch, q_len, num_q_heads, head_dim], head_dim 64, 128 or 256, q_len * G <= 1024
 *  k        bf16 or int8 cache or pool as for decode_attn_*, page_size a multiple of 16; k_scale fp32 [batch, num_kv_heads, max_ctx] or
 *           [num_pages, num_kv_heads, page_size]
 *  prior, out  fp32, laid out like k_scale; prior may be out, or NULL (zeros), and may not overlap it otherwise
 *  workspace  kv_weights_workspace_bytes(...) bytes, 16-byte aligned; max_len: max_ctx, or what the table and
 *           max_seq_len hold.  With up to 16 rows a KV head (q_len * G) it holds their scores over the whole
 *           capacity, whatever the lengths: batch * num_kv_heads * max_len * 4 bytes a row (rows rounded up to 4's),
 *           2.1 GB for 64 sequences of 8 heads and 8 rows that can grow to 131072 tokens.
 * Sequences may not share pages.  A page outside the pool is flagged (bit 2), read as page 0, and not written.
 */
long long kv_weights_workspace_bytes(int batch, int q_len, int num_q_heads, int num_kv_heads, int max_len, int num_sms);
int kv_weights_contig(const void* q, const void* k, const int* seq_lens, int batch, int q_len, int num_q_heads,
                      int num_kv_heads, int head_dim, int max_ctx, float scale, float decay, const float* prior,
                      void* workspace, long long workspace_bytes, float* out, void* stream);
int kv_weights_paged(const void* q, const void* k_pool, const int* page_table, const int* seq_lens, int batch, int q_len,
                     int num_q_heads, int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq,
                     int num_pages, int max_seq_len, float scale, float decay, const float* prior, void* workspace,
                     long long workspace_bytes, float* out, void* stream);
int kv_weights_int8_contig(const void* q, const void* k_i8, const float* k_scale, const int* seq_lens, int batch,
                           int q_len, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx, float scale,
                           float decay, const float* prior, void* workspace, long long workspace_bytes, float* out,
                           void* stream);
int kv_weights_int8_paged(const void* q, const void* k_pool_i8, const float* k_scale_pool, const int* page_table,
                          const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                          int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, float scale, float decay,
                          const float* prior, void* workspace, long long workspace_bytes, float* out, void* stream);
/*
 * kv_evict_contig / kv_evict_paged / kv_evict_int8_* — cuts each sequence down to `keep` tokens, KV head by KV
 * head: of a sequence longer than that the first `first`, the last `recent`, and of the others those of the
 * largest weights (ties: the lower position; NaN lowest, -0 as 0), first + recent <= keep; a shorter one keeps all.
 * The kept tokens' keys, values, scales and weights move together to positions 0, 1, ... in their order.
 * kept[b, h, i] is the old position of the token now at i, -1 behind the last; new_lens[b] = min(L_b, keep).
 *  k, v, k_scale, v_scale  the cache or pools (v and v_scale may be NULL: keys only); head_dim * (2 or, int8, 1) a
 *           multiple of 16 bytes, page_size any
 *  weights  fp32, laid out like k_scale
 *  seq_lens int32 [batch], clamped to the capacity; NULL (contiguous only): all max_ctx.  Not written.
 *  k_out, v_out, k_scale_out, v_scale_out, weights_out  all NULL: the cache is compacted in place, and weights
 *           [new_len, L_b) become 0.  Otherwise contiguous [batch, out_ctx, num_kv_heads, head_dim] and [batch,
 *           num_kv_heads, out_ctx], out_ctx >= keep: rows past new_lens stay as they were, weights there
 *           become 0.  weights_out may be NULL (not wanted) next to a k_out.
 *  kept     int32 [batch, num_kv_heads, keep]; new_lens int32 [batch]
 * In place, sequences may not share pages.  A page outside the pool is flagged (bit 2); rows from it are zeros,
 * rows to it are not written.
 * After an eviction a token's place in the cache is no longer its position in the sequence, and the places of a
 * position differ from KV head to KV head.  Kept keys keep the rotation that they were written with, while kv_write_*
 * with inv_freq rotates a new key by its place: turn new keys and queries by rope_apply, with the positions that the
 * program counts, and write with inv_freq NULL.  Block means of the cache are to be made again.
 */
int kv_evict_contig(void* k, void* v, float* weights, const int* seq_lens, int batch, int num_kv_heads, int head_dim,
                    int max_ctx, int keep, int first, int recent, void* k_out, void* v_out, float* weights_out,
                    int out_ctx, int* kept, int* new_lens, void* stream);
int kv_evict_paged(void* k_pool, void* v_pool, float* weights_pool, const int* page_table, const int* seq_lens,
                   int batch, int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                   int max_seq_len, int keep, int first, int recent, void* k_out, void* v_out, float* weights_out,
                   int out_ctx, int* kept, int* new_lens, void* stream);
int kv_evict_int8_contig(void* k_i8, void* v_i8, float* k_scale, float* v_scale, float* weights, const int* seq_lens,
                         int batch, int num_kv_heads, int head_dim, int max_ctx, int keep, int first, int recent,
                         void* k_out, void* v_out, float* k_scale_out, float* v_scale_out, float* weights_out,
                         int out_ctx, int* kept, int* new_lens, void* stream);
int kv_evict_int8_paged(void* k_pool_i8, void* v_pool_i8, float* k_scale_pool, float* v_scale_pool, float* weights_pool,
                        const int* page_table, const int* seq_lens, int batch, int num_kv_heads, int head_dim,
                        int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, int keep, int first,
                        int recent, void* k_out, void* v_out, float* k_scale_out, float* v_scale_out,
                        float* weights_out, int out_ctx, int* kept, int* new_lens, void* stream);

/*
 * decode_device_error — synchronise `stream`, then read and clear the device error
 * word of the current device.  *flags receives the word: bit 0 a kernel gave up on
 * a bounded wait, bit 1 a segment-counter update gave up, bit 2 a page-table entry
 * read by a paged attention call (decode_attn_*, prefill_attn_*, latent_attn_*, prefix_attn_*, sparse_attn_*) or by
 * block_means_* or kv_weights_* was outside [0, num_pages) (those tokens were read from page 0 instead, so the affected
 * results are wrong but no copy leaves the pool; kv_write_* and kv_read_* skip such rows, kv_weights_* writes nothing
 * for them, kv_evict_* takes zeros from them and writes none), bit 3 a token at or
 * past the cache's capacity that kv_write_* did not write.  Returns DA_OK when flags == 0, DA_ERR_TIMEOUT otherwise,
 * or DA_ERR_CUDA.
 */
int decode_device_error(void* stream, unsigned int* flags);

/*
 * decode_selftest_bounded_wait — diagnostic of the bounded waits that every
 * kernel of this library uses (the pages have no counterpart).  Enqueues on
 * `stream` one CTA that waits on a shared-memory mbarrier that nothing ever
 * completes; the wait gives up after timeout_ns nanoseconds of the GPU's global
 * timer, sets bit 0 of the device error word and the kernel returns normally, so
 * the context stays usable.  decode_device_error() then reports DA_ERR_TIMEOUT
 * with flags bit 0 set.  timeout_ns must be in (0, 10^9]; returns DA_OK,
 * DA_ERR_INVALID_ARG or DA_ERR_CUDA (launch failure).
 */
int decode_selftest_bounded_wait(unsigned long long timeout_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H */
