/*
 * mips.h -- C ABI of the MI355X (gfx950) exhaustive inner-product top-K library.
 *
 * The operation is the serving step of two-tower retrieval: a batch of L2-normalised
 * user embeddings queries[B, D] is scored by dot product against a precomputed,
 * L2-normalised candidate index corpus[N, D], and each user gets its K best candidates
 * (Phoenix README, "How Retrieval Works", steps 1-4; `RecsysTwoTowerModel.forward` in
 * recsys_two_tower_model.py, x-algorithm Phoenix, which scores the users against the
 * whole index, masks it with one shared type mask and takes a sorted top-min(k, N)).
 * The score matrix is never written to memory.
 *
 * Entry points: mips_l2_normalize and mips_prepare_corpus (normalisation, index build);
 * mips_topk (one result set per query), mips_topk_ranges (one per id range) and
 * mips_topk_masks (one per exclusion mask, from one pass over the index), with their
 * workspace sizes; mips_topk_noalloc (mips_topk with library-held scratch);
 * mips_merge_topk and mips_merge_interests (merges of sorted result lists);
 * mips_type_bitmap (per-type exclusion bitmaps); status strings and a timing hook.
 * For training and evaluation: mips_logprobs and its gradient
 * mips_logprobs_backward; mips_embedding_lookup and mips_embedding_grad, mips_clip_grad_norm. For
 * a user tower that reads a history of events: mips_gated_scan with its gradient
 * mips_gated_scan_backward and its form for single events mips_gated_step, mips_dropout,
 * mips_pool_normalize and mips_pool_normalize_backward.
 *
 * Conventions shared by every entry point:
 *  - All buffers are caller-owned (except the static scratch array of
 *    mips_topk_noalloc). Pointers marked "device" are HIP device memory; the library
 *    never allocates, frees or synchronises. Work is enqueued on
 *    `stream` (a hipStream_t; NULL is the default stream) and the call returns after
 *    enqueueing. Results are visible once the stream has reached that point.
 *  - Arguments are validated on the host before anything is enqueued. On any error
 *    nothing is enqueued and no output is touched. A failed launch returns
 *    MIPS_ERR_HIP; mips_last_hip_error() then gives the HIP error code (per thread).
 *    Faults inside kernels surface at the caller's next synchronisation.
 *  - Inputs must be finite. NaN and infinities are not supported.
 *  - Element types: MIPS_F32 (IEEE binary32), MIPS_BF16 (the upper 16 bits of a
 *    binary32), MIPS_FP8_E4M3 (OCP 8-bit float E4M3: bias 7, 3 mantissa bits, no
 *    infinities, max 448) and MIPS_INT8 (two's complement, -127..127), the last two
 *    always with one float scale per row.
 */
#ifndef MIPS_H
#define MIPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Entry points are the only symbols the shared library exports. */
#define MIPS_API __attribute__((visibility("default")))

#define MIPS_F32 0
#define MIPS_BF16 1
#define MIPS_FP8_E4M3 2
#define MIPS_INT8 3

#define MIPS_OK 0
#define MIPS_ERR_INVALID_ARG 1
#define MIPS_ERR_UNSUPPORTED 2
#define MIPS_ERR_WORKSPACE 3
#define MIPS_ERR_HIP 4

/* Largest supported K. */
#define MIPS_K_MAX 1024

/* Largest supported number of result lists per call: b for mips_topk, mips_topk_ranges and
 * the merges, b * nmasks for mips_topk_masks. Each list is one 256-thread workgroup of a
 * launch, whose work-item count must stay below 2^32. */
#define MIPS_B_MAX 8388608

/*
 * Packed corpus layout ("fragment-tiled"). Rows are grouped in blocks of 32
 * (N is padded up to a multiple of 32 with zero rows). Block g covers rows
 * 32g..32g+31 and occupies 32*D*E bytes (E = 4, 2 or 1 bytes per element), split into
 * 1 KiB chunks of 64 slots x 16 bytes. Slot s of chunk c holds row 32g + (s & 31) and
 * the following dimensions, with h = s >> 5 and t the element index inside the slot:
 *   MIPS_F32      (4 per slot):  dim = 8c + 2t + h
 *   MIPS_BF16     (8 per slot):  dim = 16c + 8h + t
 *   MIPS_FP8_E4M3 (16 per slot): dim = 64(c >> 1) + 32h + 16(c & 1) + t
 *   MIPS_INT8     (16 per slot): dim = 32c + 16h + t
 * Every 16-byte slot is exactly one lane's operand of the gfx950 32x32 MFMA, so the
 * score kernel streams the corpus from HBM with fully coalesced 1 KiB wave loads and
 * no LDS transpose. For MIPS_FP8_E4M3 and MIPS_INT8 the per-row scale array has one
 * float per padded row (see mips_prepare_corpus); fp8 scales are powers of two.
 */

/* Bytes of a packed corpus of n rows (n >= 1) and width d; -1 if unsupported. */
MIPS_API int64_t mips_corpus_bytes(int64_t n, int32_t d, int32_t dtype);

/* Number of floats in the per-row scale array of an n-row corpus (n rounded up to 32). */
MIPS_API int64_t mips_scale_count(int64_t n);

/*
 * mips_l2_normalize -- y = x / sqrt(max(sum_d x^2, 1e-12)) per row, the form of
 * `_l2_normalize_candidates` and of the user-representation normalisation in
 * recsys_two_tower_model.py. Computed in fp32; the bf16 output is rounded to nearest
 * even.
 *   src   device, float [rows, d] row-major, finite.
 *   rows  >= 0 (0 enqueues nothing); d in [1, 4096].
 *   out_dtype  MIPS_F32 or MIPS_BF16.
 *   dst   device, [rows, d] row-major of out_dtype; may not alias src.
 * Errors: INVALID_ARG for NULL pointers, rows < 0, d out of range, misaligned pointers
 * (4 bytes for float, 2 for bf16); UNSUPPORTED for another out_dtype.
 */
MIPS_API int mips_l2_normalize(const float *src, int64_t rows, int32_t d, int32_t out_dtype, void *dst,
                      void *stream);

/*
 * mips_prepare_corpus -- the offline index build: normalise raw rows as
 * mips_l2_normalize does and pack them into the fragment-tiled layout ("normalise once
 * at index time; store f16/int8", "Two-tower retrieval", mhtirogla.ai, section
 * "Implementation notes"; the bf16 `post_embeddings` index of recsys_two_tower_model.py).
 *   src         device, float [rows, d] row-major: logical rows
 *               row_offset .. row_offset+rows-1 of the corpus.
 *   row_offset  multiple of 32 (lets a large corpus be packed in chunks).
 *   rows        >= 1. If rows is not a multiple of 32, this must be the last chunk: the
 *               rest of the last block is written as zero rows (with a zero row's
 *               scale: 1 for fp8, 1e-12 for int8).
 *   d           16, 32, 64, 128 or 256 (MIPS_F32: up to 128; MIPS_FP8_E4M3: 64, 128,
 *               256; MIPS_INT8: 32 .. 256).
 *   dtype       MIPS_F32 (rounded to nearest), MIPS_BF16 (nearest even),
 *               MIPS_FP8_E4M3: per row, scale s = the smallest power of two with
 *               max|y| <= 448 s (1 for a zero row) and codes = E4M3(y / s), nearest even,
 *               saturating; or MIPS_INT8: per row, scale s = max(max|y| / 127, 1e-12)
 *               and codes = y / s rounded to nearest (ties to even), clipped to
 *               [-127, 127] -- the per-row rule of the quantised scoring branch of
 *               `RecsysTwoTowerModel.forward` (recsys_two_tower_model.py).
 *   dst         device, packed corpus of at least mips_corpus_bytes(row_offset + rows).
 *   row_scale   device float [mips_scale_count(row_offset + rows)] for MIPS_FP8_E4M3 and
 *               MIPS_INT8 (entries row_offset.. are written), NULL otherwise.
 * Errors: INVALID_ARG (NULL, rows < 1, row_offset < 0 or not a multiple of 32, dst not
 * 16-byte aligned, row_scale missing for fp8 or int8), UNSUPPORTED (d or dtype).
 */
MIPS_API int mips_prepare_corpus(const float *src, int64_t rows, int64_t row_offset, int32_t d,
                        int32_t dtype, void *dst, float *row_scale, void *stream);

/*
 * mips_topk_workspace_size -- bytes of device workspace mips_topk needs for these
 * sizes with its default candidate capacity (about max(16 k, 32768) per query, at most
 * the corpus). A larger workspace raises the per-query candidate capacity; see
 * mips_topk. Returns 0 for unsupported arguments. The size depends on the current
 * device's compute-unit count (the candidate lists are split into one segment per
 * corpus slice, at most one slice per compute unit).
 */
MIPS_API size_t mips_topk_workspace_size(int32_t b, int64_t n, int32_t d, int32_t k,
                                int32_t query_dtype, int32_t corpus_dtype);

/*
 * mips_topk_workspace_size_for -- as mips_topk_workspace_size, for a candidate capacity
 * of at least candidates_per_query (>= 1) per query instead of the default. A capacity
 * below the number of candidates a query produces makes mips_topk rescan that query
 * (slower, same result). Returns 0 for unsupported arguments.
 */
MIPS_API size_t mips_topk_workspace_size_for(int32_t b, int64_t n, int32_t d, int32_t k,
                                    int32_t query_dtype, int32_t corpus_dtype,
                                    int64_t candidates_per_query);

/*
 * mips_topk -- exact top-k by inner product of every query against every corpus row
 * that the exclusion bitmap does not mask ("already seen"), with ties broken by
 * score descending, then id ascending.
 *   queries      device, [b, d] row-major, query_dtype MIPS_F32 or MIPS_BF16, assumed
 *                L2-normalised (use mips_l2_normalize); 4-byte aligned.
 *   b            1 .. MIPS_B_MAX.
 *   corpus       device, packed by mips_prepare_corpus (n rows, width d, corpus_dtype);
 *                16-byte aligned.
 *   row_scale    device, per-row scales for MIPS_FP8_E4M3 and MIPS_INT8 (NULL
 *                otherwise).
 *   corpus_dtype with query_dtype: F32/F32, BF16 with F32 or BF16 queries (queries are
 *                rounded to bf16), FP8_E4M3 with F32 or BF16 queries (each query row is
 *                quantised to E4M3 with its own power-of-two scale, the rule of
 *                mips_prepare_corpus), INT8 with F32 or BF16 queries (each query row is
 *                quantised to int8 with its own scale max|q| / 127, as the quantised
 *                branch of `RecsysTwoTowerModel.forward` does; the int32 dot product of
 *                the codes is scaled by the row scale, then by the query scale).
 *   n            1 .. 2^31 - 64.  d: as mips_prepare_corpus.
 *   exclude      device or NULL: bit (i & 31) of word (i >> 5) set means id i is never
 *                returned. With exclude_row_words == 0, one uint32 [ceil(n/32)] bitmap
 *                serves the whole batch; with exclude_row_words = w > 0, query q's own
 *                bitmap starts at word q * w (uint32 [b, w], w >= ceil(n/32)): a
 *                per-user set, such as the engagement history that hard-negative
 *                mining removes from each user's retrieved top-k ("Two-Tower Retrieval
 *                at Industrial Scale", section "When hard is too hard"). The sampled thresholds ignore per-query bitmaps, so
 *                a query whose own bitmap removes many of its best rows is rescued (exact,
 *                slower).
 *   exclude_row_words  0 or >= ceil(n/32), as above; > 0 needs a non-NULL exclude.
 *   k            1 .. MIPS_K_MAX.
 *   out_scores   device float [b, k]; out_ids device int32 [b, k]. Row q holds query q's
 *                min(k, eligible) best (score, id) pairs, score descending then id
 *                ascending; remaining slots are (-INFINITY, -1). Scores are fp32
 *                accumulations of the stored operands (no temperature is applied).
 *   workspace    device, 256-byte aligned; the fixed part plus at least one candidate
 *                per query and list segment (mips_topk_workspace_size gives the default,
 *                mips_topk_workspace_size_for any other capacity); its contents are
 *                undefined between calls, except two diagnostic counts (uint32) that the
 *                call's last pass leaves in bytes 0..7: the result lists queued for the
 *                rescue pass, and the lists resolved by the exact one-workgroup rescan
 *                (slow; 0 unless a rescue pass also overflows). Calls that share a
 *                workspace must be ordered on one stream.
 * Errors: INVALID_ARG (NULL where a buffer is required, b/n/k out of range, fp8 or int8
 * without row_scale, misalignment), UNSUPPORTED (d, k > MIPS_K_MAX, b > MIPS_B_MAX, dtype
 * pair), WORKSPACE (workspace_bytes too small), HIP (a launch failed); INVALID_ARG also for
 * exclude_row_words < 0, or > 0 with a NULL exclude or below ceil(n/32).
 */
MIPS_API int mips_topk(const void *queries, int32_t query_dtype, int32_t b, const void *corpus,
              const float *row_scale, int32_t corpus_dtype, int64_t n, int32_t d,
              const uint32_t *exclude, int64_t exclude_row_words, int32_t k,
              float *out_scores, int32_t *out_ids, void *workspace, size_t workspace_bytes,
              void *stream);

/*
 * mips_topk_noalloc -- mips_topk for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation): the same
 * search, arguments, ordering, padding and errors, with no workspace argument. Its scratch
 * is a device array held by the library, MIPS_NOALLOC_SCRATCH_BYTES per device, from the
 * first call on a device until the process ends; the call allocates and frees nothing.
 * Every call on one device shares that device's array: calls that overlap on a device (on
 * different streams, or from several threads without ordering) race and give undefined
 * results. The array keeps the last call's contents; a call reads nothing it did not write.
 * Errors: as mips_topk; WORKSPACE when mips_topk_workspace_size for the same arguments
 * exceeds MIPS_NOALLOC_SCRATCH_BYTES (e.g. b = 256, n = 10^7, d = 128, k = 500 fits, about
 * 76 MB; b = 1024, n = 10^8 does not); HIP when the array's address cannot be had.
 */
#define MIPS_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
MIPS_API int mips_topk_noalloc(const void *queries, int32_t query_dtype, int32_t b,
                               const void *corpus, const float *row_scale, int32_t corpus_dtype,
                               int64_t n, int32_t d, const uint32_t *exclude,
                               int64_t exclude_row_words, int32_t k, float *out_scores,
                               int32_t *out_ids, void *stream);

/*
 * mips_topk_ranges -- mips_topk restricted to id ranges, one result set per range: for
 * range r = [ranges[2r], ranges[2r+1]), the exact top-k of the non-excluded rows with ids
 * in the range (the dataset_ranges path of `RecsysTwoTowerModel.forward` in
 * recsys_two_tower_model.py, which slices the scores to [start, end), takes a sorted
 * top-k and adds start to the indices). Each range's pass reads only the blocks that hold
 * its rows, so disjoint ranges read the corpus once in all.
 *   ranges       host int64 [nranges][2]: 0 <= start < end <= n; ranges may overlap.
 *   nranges      >= 1.
 *   out_scores   device float [nranges, b, k]; out_ids device int32 [nranges, b, k]:
 *                range r's result, as mips_topk's, with absolute ids.
 *   The other arguments, the ordering, the padding and the workspace are as mips_topk's
 *   (the workspace for the whole corpus serves every range; ranges run one after the
 *   other on the stream).
 * Errors: as mips_topk, plus INVALID_ARG for a NULL ranges, nranges < 1 or a range outside
 * [0, n) or empty.
 */
MIPS_API int mips_topk_ranges(const void *queries, int32_t query_dtype, int32_t b, const void *corpus,
                              const float *row_scale, int32_t corpus_dtype, int64_t n, int32_t d,
                              const uint32_t *exclude, int64_t exclude_row_words,
                              const int64_t *ranges, int32_t nranges,
                              int32_t k, float *out_scores, int32_t *out_ids, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * mips_topk_masks -- several result sets from one pass over the corpus: for each of the
 * nmasks exclusion masks, every query's exact top-k of the rows that mask does not
 * exclude. This is the per-type loop of `RecsysTwoTowerModel.forward`
 * (recsys_two_tower_model.py), which scores the batch once and takes one masked top-k per
 * target type; here each score is computed once and tested against the threshold of each
 * mask that admits its row. Masks may overlap.
 *   masks        device uint32 [nmasks][mask_words]: bit (i & 31) of word (i >> 5) of row t
 *                set means id i is not in result set t (mips_type_bitmap builds one per
 *                item type, with a shared exclusion folded in).
 *   nmasks       1 .. MIPS_MAX_MASKS.  mask_words >= ceil(n/32).
 *   out_scores   device float [nmasks, b, k]; out_ids device int32 [nmasks, b, k]: result
 *                set t of query q at [t][q], as mips_topk's row q.
 *   workspace    mips_topk_masks_workspace_size bytes: the fixed part and candidate lists
 *                per mask and query, of candidates_per_list entries each (< 1: the default
 *                capacity, as mips_topk_workspace_size; 0 returned for invalid sizes).
 *   The other arguments, the ordering and the padding are as mips_topk's.
 * Errors: as mips_topk; INVALID_ARG for a NULL or misaligned masks, nmasks < 1 or
 * mask_words < ceil(n/32); UNSUPPORTED for nmasks > MIPS_MAX_MASKS or b * nmasks >
 * MIPS_B_MAX.
 */
#define MIPS_MAX_MASKS 4
MIPS_API size_t mips_topk_masks_workspace_size(int32_t b, int64_t n, int32_t d, int32_t k,
                                               int32_t query_dtype, int32_t corpus_dtype,
                                               int32_t nmasks, int64_t candidates_per_list);
MIPS_API int mips_topk_masks(const void *queries, int32_t query_dtype, int32_t b, const void *corpus,
                             const float *row_scale, int32_t corpus_dtype, int64_t n, int32_t d,
                             const uint32_t *masks, int32_t nmasks, int64_t mask_words, int32_t k,
                             float *out_scores, int32_t *out_ids, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * mips_type_bitmap -- the exclusion bitmap of a search restricted to one item type: id i
 * is excluded when item_types[i] != target or exclude marks it (the per-type mask of
 * `RecsysTwoTowerModel.forward`, recsys_two_tower_model.py, one result set per target
 * type). Feed the result to mips_topk, or one row per type to mips_topk_masks; excluded
 * ids are never returned, so every id a type-restricted search returns has that type.
 *   item_types   device int32 [n]; n >= 1.
 *   exclude      device uint32 [ceil(n/32)] or NULL: ids excluded in any case.
 *   out_bitmap   device uint32 [ceil(n/32)]; bits of ids >= n are set. May alias exclude.
 * Errors: INVALID_ARG (NULL, n < 1, misaligned pointers), HIP (the launch failed).
 */
MIPS_API int mips_type_bitmap(const int32_t *item_types, int64_t n, int32_t target,
                              const uint32_t *exclude, uint32_t *out_bitmap, void *stream);

/*
 * mips_merge_topk -- merge of p sorted result lists per query into one top-k_out: the
 * fresh-shard pattern of "Two-Tower Retrieval at Industrial Scale" (engineeringmaxxing.com:
 * a small fresh index is searched beside the base index and the result lists are merged
 * by score), and the exchange step of a corpus split by rows across devices.
 *   in_scores    device float [p, b, k_in] (list-major): list l, query q, rank j.
 *   in_ids       device int32 [p, b, k_in]: ids local to list l's index; id < 0 is
 *                padding and is skipped (as mips_topk pads with (-INFINITY, -1)).
 *   offsets      host int64 [p], each in [0, 2^31): list l's ids are shifted by
 *                offsets[l]. Shifted ids must be distinct across lists (disjoint
 *                indexes) and below 2^31.
 *   p            1 .. 64 lists; b 1 .. MIPS_B_MAX queries; k_in >= 1; k_out 1 .. MIPS_K_MAX.
 *   out_scores   device float [b, k_out]; out_ids device int32 [b, k_out]: per query the
 *                k_out best real entries of all lists, score descending then id
 *                ascending, then (-INFINITY, -1). Exact for its inputs: when each list is
 *                its index's exact top-k_out, the result is the exact top-k_out of the
 *                union of the indexes.
 * Errors: INVALID_ARG (NULL, p/b/k out of range, an offset out of range, misaligned
 * pointers), UNSUPPORTED (k_out > MIPS_K_MAX or b > MIPS_B_MAX), HIP (the launch failed).
 */
MIPS_API int mips_merge_topk(const float *in_scores, const int32_t *in_ids, const int64_t *offsets,
                             int32_t p, int32_t b, int32_t k_in, int32_t k_out, float *out_scores,
                             int32_t *out_ids, void *stream);

/*
 * mips_merge_interests -- per user, the merge of its m interest vectors' result lists:
 * a user with several interest vectors matches an item by the best of them ("Two-Tower
 * Retrieval at Industrial Scale", engineeringmaxxing.com, section "Beyond Dot Products":
 * one search per interest vector, results merged by the maximum). An id returned for
 * several of the user's vectors keeps its highest score; the best k_out ids follow, score
 * descending then id ascending, then (-INFINITY, -1). When each list is its vector's exact
 * top-k_out (mips_topk over the b * m vectors), the result is the exact top-k_out by the
 * maximum over the user's vectors.
 *   in_scores    device float [b, m, k_in] (user-major: rows u*m .. u*m+m-1 of a mips_topk
 *                output); in_ids device int32 [b, m, k_in], id < 0 is padding.
 *   b 1 .. MIPS_B_MAX users, m >= 1 vectors per user, k_in >= 1 with m * k_in <= 2048,
 *   k_out 1 .. MIPS_K_MAX.
 *   out_scores   device float [b, k_out]; out_ids device int32 [b, k_out].
 * Errors: INVALID_ARG (NULL, b/m/k < 1, misaligned pointers), UNSUPPORTED (m * k_in > 2048,
 * k_out > MIPS_K_MAX or b > MIPS_B_MAX), HIP (the launch failed).
 */
MIPS_API int mips_merge_interests(const float *in_scores, const int32_t *in_ids, int32_t b, int32_t m,
                                  int32_t k_in, int32_t k_out, float *out_scores, int32_t *out_ids,
                                  void *stream);

/* ---------------------------------------------------------------------------------------
 * Training: the steps around the search that make and use the vectors. The conventions
 * above hold, with these of their own: matrices are row-major with a row stride in
 * elements; NaN and infinities are allowed and propagate as in the formulas, or as each entry
 * point says.
 */

/* Largest width of an embedding row, and most tokens of one mips_embedding_grad call. */
#define MIPS_EMBEDDING_D_MAX 16384
#define MIPS_TOKENS_MAX 1073741824

/*
 * mips_embedding_lookup -- out[i] = scale * table[ids[i]], computed in binary32 and rounded
 * once to the table's type; a row of zeros for an id outside [0, rows) (padding).
 *   table       device, [rows, d] of dtype MIPS_F32 or MIPS_BF16, row_stride >= d.
 *   rows        >= 1.  d 1 .. MIPS_EMBEDDING_D_MAX.
 *   ids         device, int32 or int64 [t] (id_bits 32 or 64); t >= 0 (0 enqueues nothing).
 *   out         device, [t, d] contiguous, of dtype; may not overlap the table.
 * Rows that are 16-byte multiples at 16-byte aligned addresses (table, out and row_stride)
 * move in 16-byte units, others one element at a time.
 * Errors: INVALID_ARG (NULL, t < 0, rows < 1, d < 1, row_stride < d, a pointer not aligned
 * to its element), UNSUPPORTED (dtype, id_bits, d), HIP.
 */
MIPS_API int mips_embedding_lookup(const void *table, int32_t dtype, int64_t rows, int32_t d,
                                   int64_t row_stride, const void *ids, int32_t id_bits, int64_t t,
                                   float scale, void *out, void *stream);

/*
 * mips_embedding_grad -- the gradient of mips_embedding_lookup for the table:
 * out[v] = scale * sum of grad[i] over the tokens i with ids[i] = v, zero rows for ids that
 * no token has. Sums are in binary32 without atomics, in an order that follows from the call's
 * ids, sizes and device alone (a hot id's tokens are added in several parts): the same call gives
 * the same bits. Ids outside [0, rows) take no part.
 *   grad        device, [t, d] of grad_dtype MIPS_F32 or MIPS_BF16, grad_stride >= d.
 *   ids         device, int32 or int64 [t]; t 0 .. MIPS_TOKENS_MAX.
 *   rows        1 .. 2^31 - 64.
 *   accumulate  nonzero: the sums are added to out (rows without a token stay as they are);
 *               zero: out is written whole.
 *   out         device, [rows, d] of grad_dtype, or MIPS_F32 with bf16 gradients;
 *               out_stride >= d; may not overlap grad.
 *   workspace   device, 256-byte aligned, mips_embedding_grad_workspace_size bytes (0 is
 *               returned for unsupported sizes). Calls that share one must be ordered.
 * Errors: INVALID_ARG (NULL, sizes or strides below their minima, misaligned pointers),
 * UNSUPPORTED (dtypes, id_bits, d, t or rows above the limits), WORKSPACE, HIP.
 */
MIPS_API size_t mips_embedding_grad_workspace_size(int64_t t, int64_t rows, int32_t d);
MIPS_API int mips_embedding_grad(const void *grad, int32_t grad_dtype, int64_t t, int32_t d,
                                 int64_t grad_stride, const void *ids, int32_t id_bits,
                                 int64_t rows, float scale, int32_t accumulate, void *out,
                                 int32_t out_dtype, int64_t out_stride, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * mips_clip_grad_norm -- the 2-norm over all elements of several tensors, and the tensors
 * scaled by min(1, max_norm / (norm + 1e-6)). Squares are summed in binary64, the scaling is
 * one binary32 product rounded to the tensor's type. A NaN among the elements makes the norm
 * and every output NaN; an infinite one makes the factor 0.
 *   tensors, outs, counts, dtypes   host arrays of ntensors >= 1 entries: device pointers,
 *               element counts (0 .. 2^38) and MIPS_F32 or MIPS_BF16. outs[i] may equal
 *               tensors[i] (scaled in place; not written when the factor is 1) and may not
 *               otherwise overlap any tensor. 16-byte aligned pairs move in 16-byte units.
 *   max_norm    >= 0; infinity only takes the norm (and copies): the factor is 1, whatever the
 *               norm, infinite and NaN ones included.
 *   out_norm    device float [1].
 *   workspace   device, 256-byte aligned, mips_clip_workspace_size(ntensors) bytes.
 * Errors: INVALID_ARG, UNSUPPORTED (a dtype), WORKSPACE, HIP.
 */
MIPS_API size_t mips_clip_workspace_size(int32_t ntensors);
MIPS_API int mips_clip_grad_norm(const void *const *tensors, void *const *outs,
                                 const int64_t *counts, const int32_t *dtypes, int32_t ntensors,
                                 float max_norm, float *out_norm, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * mips_logprobs -- log probabilities under the softmax of a batch of queries over an item
 * table: with s_bj = queries[b] . items[j] accumulated in binary32,
 *   l_bj = fl(fl(s_bj * scale) + bias[j])    (fl(s_bj * scale) without a bias),
 *   lse_b = log sum over the eligible items j of exp(l_bj),
 *   out_logprobs[b][i] = l_bj - lse_b for j = ids[b][i],
 *   out_entropy[b] = - sum_j p_bj log p_bj,  p_bj = exp(l_bj - lse_b),
 *   alternatives: the k eligible items of the largest l_bj, ties by the lowest id; an item whose
 *   logit is NaN or below -6e29 (-INFINITY among them) is none.
 * A logit that is NaN or +INFINITY makes its query's lse, entropy and log probabilities NaN.
 * The scores are never written to memory. scale is 1 / temperature; the bias is, for
 * instance, - log q of a sampled softmax ("Two-Tower Retrieval at Industrial Scale", the logQ
 * correction).
 *   queries      device, [b, d] row-major of dtype, query_stride elements apart.
 *   b            1 .. MIPS_B_MAX.
 *   items        device; layout MIPS_ROWS: [n, d] row-major of dtype, item_stride elements
 *                apart; MIPS_PACKED: packed by mips_prepare_corpus (dtype, n, d; item_stride
 *                is not used).
 *   n            1 .. 2^31 - 64.
 *   d            a multiple of 16 bytes, up to 128 (MIPS_F32) or 256 (MIPS_BF16); for
 *                MIPS_PACKED as mips_prepare_corpus. Rows are 16-byte aligned (base and
 *                stride) and at most 2^25 bytes apart.
 *   dtype        MIPS_F32 or MIPS_BF16, of queries and items.
 *   bias         device float [n] or NULL. -INFINITY and the lowest float mask an item: p = 0.
 *   exclude, exclude_row_words   as mips_topk: ids whose bit is set have probability 0,
 *                whatever their rows hold (NaN and infinities included).
 *   scale        MIPS_SCALE_MIN .. MIPS_SCALE_MAX.
 *   ids          device, int32 or int64 (id_bits) [b, g], g >= 0. An id outside [0, n) is
 *                padding: log probability 0. An excluded one has -INFINITY.
 *   k            0 .. MIPS_ALTERNATIVES_MAX.
 *   out_logprobs device float [b, g]; out_lse device float [b]; out_entropy device float [b]
 *                or NULL; out_alt_ids device int32 [b, k] and out_alt_logprobs device float
 *                [b, k]: largest first, missing ones (-1, -INFINITY).
 *                A query without an eligible item, or whose eligible logits are all below -6e29
 *                (-INFINITY among them), has lse and log probabilities -INFINITY and entropy 0.
 *   workspace    device, 256-byte aligned, mips_logprobs_workspace_size bytes (it depends on
 *                the device's compute units; 0 for unsupported sizes). Calls that share one
 *                must be ordered.
 * Errors: INVALID_ARG (NULL, sizes, scale, strides, alignment, exclude_row_words as
 * mips_topk), UNSUPPORTED (dtype, d, n, b or k above their limits, id_bits), WORKSPACE, HIP.
 */
#define MIPS_ROWS 0
#define MIPS_PACKED 1
#define MIPS_ALTERNATIVES_MAX 64
#define MIPS_SCALE_MIN 1e-6f
#define MIPS_SCALE_MAX 1e6f
MIPS_API size_t mips_logprobs_workspace_size(int32_t b, int64_t n, int32_t d, int32_t dtype,
                                             int32_t k);
MIPS_API int mips_logprobs(const void *queries, int64_t query_stride, int32_t b, const void *items,
                           int32_t layout, int64_t item_stride, int64_t n, int32_t d,
                           int32_t dtype, const float *bias, const uint32_t *exclude,
                           int64_t exclude_row_words, float scale, const void *ids,
                           int32_t id_bits, int32_t g, int32_t k, float *out_logprobs,
                           float *out_lse, float *out_entropy, int32_t *out_alt_ids,
                           float *out_alt_logprobs, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * mips_logprobs_backward -- the gradient of mips_logprobs (MIPS_ROWS) for queries, items and
 * bias, given those of the log probabilities (G, [b, g]) and, optionally, of the entropies (H', [b]):
 *   w_bj = sum_i G_bi [ids_bi = j] - p_bj (sum_i G_bi + H'_b (log p_bj + entropy_b)),
 *   grad_queries[b] = scale sum_j w_bj items[j],  grad_items[j] = scale sum_b w_bj queries[b],
 *   grad_bias[j] = sum_b w_bj,
 * over the eligible items; padding and excluded targets, and queries of lse -INFINITY, have no
 * gradient, and p log p is 0 where p is. The scores are computed again, once for each of the two
 * sums, and never written. Sums are in binary32 in a fixed order (the same call gives the same
 * bits). With MIPS_BF16 the weights are rounded to bf16 before they multiply the rows, those of
 * targets excepted, and the gradients to bf16 at the end.
 *   queries .. g   as the forward call's; g at most MIPS_TARGETS_MAX, n at most 2^30. An item that
 *               the shared bitmap excludes may hold anything; with one bitmap per query, the rows
 *               must be finite (a row may be excluded for some queries and not for others).
 *   lse, entropy   device float [b], the forward call's (entropy only with grad_entropy).
 *   grad_logprobs  device float [b, g]; grad_entropy device float [b] or NULL.
 *   grad_queries   device, [b, d] contiguous of dtype, or NULL: not wanted; grad_items device,
 *               [n, d] contiguous of dtype, or NULL; grad_bias device float [n] or NULL. One of
 *               them at least. Gradients are written whole (not accumulated), 16-byte aligned.
 *   workspace   device, 256-byte aligned, mips_logprobs_backward_workspace_size bytes (0 for
 *               unsupported sizes). Calls that share one must be ordered.
 * Errors: as mips_logprobs; INVALID_ARG without any output, or grad_entropy without entropy;
 * UNSUPPORTED for g > MIPS_TARGETS_MAX or n > 2^30.
 */
#define MIPS_TARGETS_MAX 64
MIPS_API size_t mips_logprobs_backward_workspace_size(int32_t b, int64_t n, int32_t d,
                                                      int32_t dtype, int32_t g);
MIPS_API int mips_logprobs_backward(const void *queries, int64_t query_stride, int32_t b,
                                    const void *items, int64_t item_stride, int64_t n, int32_t d,
                                    int32_t dtype, const float *bias, const uint32_t *exclude,
                                    int64_t exclude_row_words, float scale, const void *ids,
                                    int32_t id_bits, int32_t g, const float *lse,
                                    const float *entropy, const float *grad_logprobs,
                                    const float *grad_entropy, void *grad_queries,
                                    void *grad_items, float *grad_bias, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------
 * Histories: the user tower's operators over sequences of events. The conventions of the training
 * entry points hold. A sequence's rows come in one of three forms:
 *   dense    [b, t, d]: b sequences of t rows (offsets and lengths NULL);
 *   padded   the same with lengths, int32 or int64 [b] on the device, clamped to [0, t]: rows behind
 *            a sequence's length are padding;
 *   packed   [n, d], sequence s having the rows offsets[s] .. offsets[s + 1] - 1: offsets int32
 *            or int64 [b + 1] on the device, not decreasing, in [0, n]. Rows before the first
 *            offset and behind the last one are padding. Offsets outside [0, n] are clamped;
 *            decreasing ones give meaningless results (no access leaves the buffers).
 * Padding is never read as data (it may hold anything, NaN included); in outputs it is 0. Outputs
 * overlap neither inputs nor one another unless said otherwise.
 */
typedef struct mips_sequences {
  int32_t b;           /* sequences, 1 .. MIPS_B_MAX */
  int32_t index_bits;  /* 32 or 64, of offsets or lengths */
  int64_t t;           /* dense and padded: rows a sequence, >= 1; b * t <= MIPS_TOKENS_MAX */
  int64_t n;           /* packed: rows, 0 .. MIPS_TOKENS_MAX */
  const void *offsets; /* device, or NULL */
  const void *lengths; /* device, or NULL; not with offsets */
} mips_sequences;

/* An input tensor over such rows: unit stride along d, row_stride >= d elements from a row to the
 * next one (packed: at most MIPS_PACKED_STRIDE_MAX), seq_stride >= d (dense and padded) from a
 * sequence to the next one. */
#define MIPS_PACKED_STRIDE_MAX 524288
typedef struct mips_rows {
  const void *data; /* device */
  int64_t row_stride;
  int64_t seq_stride;
} mips_rows;

/*
 * mips_gated_scan -- a gated linear recurrence along each sequence, per channel, in binary32:
 *   h_r = a_r h_{r-1} + b_r x_r,  a = sigmoid(forget),  b = sigmoid(gate), or 1 - a without a gate,
 * from initial (or 0) before the first row. Rows are cut into tiles whose states are joined in an
 * order that follows from the sizes alone: the same call gives the same bits. A state that is not
 * finite makes those behind it in its sequence and channel not finite. Gates are off by up to
 * (2 |logit| + 8) 2^-24 of their value; those below 2^-126 may be 0, and sigmoid(-inf) is.
 *   x, forget, gate   rows of dtype MIPS_F32 or MIPS_BF16; gate may be NULL.  d 1 .. 16384.
 *   initial      device float [b, d] or NULL.
 *   states       device, contiguous rows of dtype in the layout of the input ([b, t, d] or [n, d]):
 *                every h, rounded once; or NULL.
 *   last         device float [b, d]: the state behind the last row; initial (or 0) without rows.
 *   carries      device float [mips_gated_scan_carries(seq, d, dtype), d]: states between short runs of
 *                rows, for the gradient (left as they were for runs of padding alone); or NULL. The
 *                number follows from the sizes and dtype.
 *   workspace    device, 256-byte aligned, mips_gated_scan_workspace_size bytes (0: none is needed, or
 *                sizes are unsupported). Calls that share one must be ordered.
 * Rows whose elements lie in aligned groups of four (d, strides and pointers) are the fastest.
 * Errors: INVALID_ARG (NULL, sizes, strides, alignment), UNSUPPORTED (dtype, index_bits, d, b or
 * rows above their limits), WORKSPACE, HIP.
 */
MIPS_API int64_t mips_gated_scan_carries(const mips_sequences *seq, int32_t d, int32_t dtype);
MIPS_API size_t mips_gated_scan_workspace_size(const mips_sequences *seq, int32_t d, int32_t dtype);
MIPS_API int mips_gated_scan(const mips_sequences *seq, int32_t d, int32_t dtype, const mips_rows *x,
                             const mips_rows *forget, const mips_rows *gate, const float *initial,
                             void *states, float *last, float *carries, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * mips_gated_scan_backward -- the gradient of mips_gated_scan. With G the gradient of the states and,
 * added at a sequence's last row, of the last one, D_r = G_r + a_{r+1} D_{r+1}:
 *   grad_x = D b,  grad_forget = D (h_{r-1} - x) a (1 - a) without a gate,  D h_{r-1} a (1 - a)
 *   and grad_gate = D x b (1 - b) with one,  grad_initial = a D at the first row (grad_last
 *   without rows).
 * States are computed again in binary32 from the inputs and the carries, not read.
 *   seq .. initial, carries   as the forward call's (d, sizes and lengths decide the carries' places).
 *   grad_states   rows of dtype or NULL; grad_last  device float [b, d] or NULL; one of them at least.
 *   grad_x, grad_forget, grad_gate   device, contiguous rows of dtype, written whole (grad_gate
 *                 with a gate only); grad_initial  device float [b, d] or NULL: not wanted.
 *   workspace     as mips_gated_scan.
 * Errors: as mips_gated_scan; INVALID_ARG without any gradient.
 */
MIPS_API int mips_gated_scan_backward(const mips_sequences *seq, int32_t d, int32_t dtype, const mips_rows *x,
                                      const mips_rows *forget, const mips_rows *gate, const float *initial,
                                      const mips_rows *grad_states, const float *grad_last,
                                      const float *carries, void *grad_x, void *grad_forget, void *grad_gate,
                                      float *grad_initial, void *workspace, size_t workspace_bytes,
                                      void *stream);

/*
 * mips_gated_step -- the recurrence for single events against a table of states: for events e in
 * order, with r = ids[e], state[r] = a_e state[r] + b_e x_e and out[e] = state[r]. Events of one row
 * are applied one after another in their order. An id outside [0, rows) is padding: out[e] = 0.
 *   x, forget, gate   device, [b, d] of dtype, strides >= d; gate may be NULL.
 *   b            0 .. MIPS_EVENTS_MAX (0 enqueues nothing).
 *   state        device float [rows, d], state_stride >= d.
 *   out_state    device float [rows, d]: the rows that events name are written, others are left as
 *                they are; either `state` itself with the same stride, or no overlap (INVALID_ARG, also
 *                for tables that lie within one another otherwise than as columns of one tensor,
 *                all its rows or some at a stride).
 *   ids          device, int32 or int64 [b].
 *   out          device, [b, d] contiguous of dtype.
 * Errors: INVALID_ARG (NULL, sizes, strides, alignment), UNSUPPORTED (dtype, id_bits, d > 16384,
 * b > MIPS_EVENTS_MAX), HIP.
 */
#define MIPS_EVENTS_MAX 65536
MIPS_API int mips_gated_step(const void *x, int64_t x_stride, const void *forget, int64_t forget_stride,
                             const void *gate, int64_t gate_stride, int32_t dtype, int32_t b, int32_t d,
                             const float *state, int64_t state_stride, float *out_state, int64_t out_stride,
                             int64_t rows, const void *ids, int32_t id_bits, void *out, void *stream);

/*
 * mips_dropout -- out = residual + (kept ? x * 65536 / (65536 - c) : 0), c = p * 65536 rounded to
 * the nearest integer (p is taken in steps of 2^-16). The ratio is rounded to binary32, product and sum
 * together once more, and then to dtype. Element i is kept if its 16 random bits are at
 * least c: half-word i % 8, low halves first, of the four words of Philox4x32-10 with the counter
 * (i / 8 mod 2^32, i / 8 / 2^32, offset mod 2^32, offset / 2^32) and the key (seed mod 2^32, seed / 2^32).
 * The same call on the gradient is the gradient for x. Dropped elements count as 0 whatever they hold.
 *   x, out       device, [n] of dtype; out may be x or residual.  n 0 .. 2^40.
 *   p            0 .. 1; all elements are dropped at 1.
 *   counter      device uint64 [1], added to the offset (mod 2^64) when the kernel runs, or NULL: a
 *                captured graph draws new numbers when it is replayed with another value there.
 *   residual     device, [n] of dtype, or NULL.
 * Errors: INVALID_ARG (NULL, n, p, alignment), UNSUPPORTED (dtype, n), HIP.
 */
MIPS_API int mips_dropout(const void *x, int32_t dtype, int64_t n, double p, uint64_t seed, uint64_t offset,
                          const uint64_t *counter, const void *residual, void *out, void *stream);

/*
 * mips_pool_normalize -- per sequence the mean m of its rows (0 without rows), and, with normalize,
 * m / sqrt(max(sum m^2, 1e-12)) as mips_l2_normalize's rows. Sums in binary32, in an order that
 * follows from sizes, offsets and lengths.
 *   x            rows of dtype MIPS_F32 or MIPS_BF16.  d 1 .. 16384.
 *   vectors      device, [b, d] contiguous of dtype; mean device float [b, d]; norm device float
 *                [b]: the root (1 without normalize). The latter two are what the gradient needs.
 *   workspace    device, 256-byte aligned, mips_pool_workspace_size bytes (0: none is needed, or sizes
 *                are unsupported). Calls that share one must be ordered.
 * mips_pool_normalize_backward -- its gradient: with g that of the vectors and u = m / norm,
 *   grad_x = (g - u (u . g)) / norm / rows of the sequence (g / norm / rows where the sum is below
 *   1e-12; g / rows without normalize), one row for all of a sequence's.
 *   grad         device, [b, d] of dtype, grad_stride >= d.
 *   grad_x       device, contiguous rows of dtype, written whole.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP as above.
 */
MIPS_API size_t mips_pool_workspace_size(const mips_sequences *seq, int32_t d);
MIPS_API int mips_pool_normalize(const mips_sequences *seq, int32_t d, int32_t dtype, const mips_rows *x,
                                 int32_t normalize, void *vectors, float *mean, float *norm, void *workspace,
                                 size_t workspace_bytes, void *stream);
MIPS_API int mips_pool_normalize_backward(const mips_sequences *seq, int32_t d, int32_t dtype, const void *grad,
                                          int64_t grad_stride, int32_t normalize, const float *mean,
                                          const float *norm, void *grad_x, void *stream);

/*
 * mips_set_timing_events -- profiling hook (host, per calling thread). When both are
 * non-NULL, later mips_topk calls on this thread launch the main score kernel so that its
 * dispatch records `before` (a hipEvent_t) at the kernel's start and `after` at its end,
 * on the call's stream (no packets of their own, so no gap between the call's kernels).
 * Pass NULL, NULL to stop. Returns MIPS_OK.
 */
MIPS_API int mips_set_timing_events(void *before, void *after);

/* Human-readable name of a status code (host, static storage). */
MIPS_API const char *mips_status_string(int status);

/* HIP error code of the last MIPS_ERR_HIP returned on this thread (host). */
MIPS_API int mips_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MIPS_H */
