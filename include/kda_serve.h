/*
 * kda_serve.h — C ABI of the single-token (serving) operators: what a hybrid
 * of KDA layers and full-attention layers runs after kda_chunk_fwd has taken
 * the prompt.
 *
 *   kda_step          a few tokens (usually one) on the fp32 KDA states, in place
 *   kda_cache_append  new keys and values into a paged cache, keys and queries
 *                     rotated by their position on the way
 *   kda_cache_attend  attention of one new token per sequence over that cache
 *                     (_sinks: a window and a few first rows)
 *   kda_cache8_*      the same on a cache in 8 bits with a scale for each block
 *   kda_cache_resize  pages for new lengths: page tables, slots and offsets
 *
 * Conventions are those of kda.h: device pointers owned by the caller and
 * 16-byte aligned (int32 arrays: 4-byte, int64 arrays: 8-byte), no allocation,
 * no synchronisation, kernels enqueued on `stream`, argument errors returned
 * before any launch, outputs fully overwritten, bit-identical reruns.
 *
 * Indices that live on the device (slots, page tables, lengths, offsets of
 * packed sequences) cannot be checked by the host. The kernels check each
 * before it is used: what it would have reached is not touched, and the
 * optional device word `status` receives KDA_ERR_INVALID_ARG. The word is only
 * ever set, never cleared: the caller zeroes it and reads it when it wants to
 * know. A negative slot or length is no error: it marks an inactive row of a
 * padded batch.
 */
#ifndef KDA_GB300_SERVE_H
#define KDA_GB300_SERVE_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The recurrent form of KDA on T tokens of each of N sequences:
 *   S <- Diag(e^g) S;  d = beta (v - S^T k);  S <- S + k d^T;  o = scale S^T q
 * K, V must be 64 or 128, HV a multiple of H. dtype is that of q, k, v, beta
 * and o. num_slots is the number of states that `state` holds.
 */
typedef struct {
    int32_t N, T, H, HV, K, V;
    int32_t num_slots;
    int32_t dtype;
    float scale;
} kda_step_dims;

/*
 *   q, k    [N, T, H, K]         v, o  [N, T, HV, V]
 *   g       [N, T, HV, K] fp32   beta  [N, T, HV]       (as in kda_chunk_fwd)
 *   state   [num_slots, HV, K, V] fp32, updated in place (kda_chunk_fwd's ht
 *           layout: its ht is a valid state)
 *   slots   int32 [N], nullable: the state of sequence n is state[slots[n]]
 *           (NULL: state[n], and num_slots >= N). Negative: the row is
 *           inactive, o is 0 there and no state changes. Two rows with the
 *           same slot race on it.
 *   status  int32, nullable: set when a slot is >= num_slots (o is 0 there).
 * N == 0 or T == 0 is KDA_OK and launches nothing.
 * Errors: KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED before any launch;
 * KDA_ERR_CUDA if the launch fails.
 */
kda_status kda_step(const kda_step_dims* dims, const void* q, const void* k, const void* v, const float* g,
                    const void* beta, float* state, const int32_t* slots, void* o, int32_t* status,
                    kda_stream_t stream);

/*
 * A paged cache of keys and values: num_pages pages of page_size rows, HKV
 * heads. Row r of head h of page p starts at
 *   k + p * k_page + r * k_row + h * k_head      (strides in elements)
 * and holds K contiguous channels; v likewise with V. Strides are
 * non-negative multiples of 16 bytes, so pages may hold rows of heads or
 * heads of rows, and keys and values may share a pool. K and V must be 64 or
 * 128; page_size is any positive number.
 */
typedef struct {
    void* k;
    void* v;
    int64_t k_page, k_row, k_head;
    int64_t v_page, v_row, v_head;
    int32_t num_pages, page_size;
    int32_t HKV, K, V;
    int32_t dtype;
} kda_cache;

/*
 * Appends R new rows of N sequences. Row r of sequence n goes to position
 * pos = kv_lens[n] + (its index among the sequence's new rows), that is to row
 * pos % page_size of page page_table[n][pos / page_size].
 *   k [R, HKV, K], v [R, HKV, V], row strides k_stride, v_stride (elements,
 *     multiples of 16 bytes; the heads of a row are contiguous)
 *   q [R, HQ, K] with row stride q_stride, and q_out [R, HQ, K] contiguous:
 *     both NULL (with HQ == 0) to append only. q_out may be q where q is
 *     contiguous; otherwise the two do not overlap.
 *   cu_seqlens  int64 [N + 1], non-decreasing, from 0 to R: the rows of each
 *     sequence; NULL: R / N rows each (R % N == 0).
 *   rope        fp32 [rope_len, rope_dim], nullable: for each position,
 *     rope_dim / 2 cosines, then as many sines. rope_dim is a multiple of 16
 *     and at most K; channels from rope_dim on are copied. With interleaved
 *     == 0 channel i turns with i + rope_dim / 2, otherwise 2i with 2i + 1.
 *     Products and sums are fp32, rounded once.
 *   page_table  int32 [N, max_pages] with row stride table_stride
 *   kv_lens     int32 [N]: rows already in the cache; not changed. Negative:
 *     the sequence is inactive (nothing is appended, its q_out rows are 0).
 *   status      nullable: set where a position needs a page beyond max_pages,
 *     a page outside [0, num_pages) or a rope row beyond rope_len, and where
 *     a row lies outside its sequence in cu_seqlens; such a row is not
 *     appended and its q_out row is 0.
 * R == 0 is KDA_OK and launches nothing. R is at most 2^31 - 1 and HQ + 2 HKV
 * less than 2^26 - 32 (else KDA_ERR_UNSUPPORTED).
 * Errors: KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED before any launch;
 * KDA_ERR_CUDA if the launch fails.
 */
kda_status kda_cache_append(const kda_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const void* q, int64_t q_stride, void* q_out, int32_t HQ, int32_t N, int64_t R,
                            const int64_t* cu_seqlens, const float* rope, int32_t rope_len, int32_t rope_dim,
                            int32_t interleaved, const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                            const int32_t* kv_lens, int32_t* status, kda_stream_t stream);

/*
 * The same for lengths that were granted (kda_cache_resize): a row whose
 * position is granted[n] or more (int32 [N]; NULL: no such limit) is not
 * appended and its q_out row is 0, as in an inactive sequence; no error. So a
 * sequence that got no pages keeps its cache as it is, also where its last page
 * has room for some of the rows.
 */
kda_status kda_cache_append_granted(const kda_cache* cache, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ, int32_t N,
                                    int64_t R, const int64_t* cu_seqlens, const float* rope, int32_t rope_len,
                                    int32_t rope_dim, int32_t interleaved, const int32_t* page_table, int64_t table_stride,
                                    int32_t max_pages, const int32_t* kv_lens, const int32_t* granted, int32_t* status,
                                    kda_stream_t stream);

/*
 * Attention of one token of each of N sequences over its cached rows:
 *   o[n, h] = sum_t p_t V[t],  p = softmax_t(scale q[n, h] . K[t]),
 * t from max(0, kv_lens[n] - window) (window > 0; else from 0) to kv_lens[n]
 * - 1, head h reading cache head h / (HQ / HKV). The new token's own row is
 * one of them when it was appended before.
 *   q    [N, HQ, K], row stride q_stride (elements, a multiple of 16 bytes)
 *   o    [N, HQ, V] contiguous, in the cache's dtype
 *   lse  fp32 [N, HQ], nullable: the natural log of the softmax's denominator
 * Where nothing is left to attend (kv_lens[n] <= 0, or every score is -inf)
 * o is 0 and lse is -inf. Rows outside the range are never read, whatever
 * they hold. Softmax statistics, weights and sums are held in fp32 (with a bf16
 * cache the weights enter the products as three bf16 values that add up to
 * them within 2^-21.9), and each output is rounded once.
 * Values that are not finite come out as the sum says: an infinite one makes
 * its channel infinite, a NaN, or infinities of both signs, make it NaN. (A
 * weight below 2^-90 of the largest may count as 0, and 0 times an infinite
 * value is NaN.)
 *   status  nullable: set where kv_lens[n] needs more than max_pages pages
 *     (only the rows of the table are attended) or a page is outside
 *     [0, num_pages) (its rows are left out).
 *   ws / ws_bytes: device workspace of at least
 *     kda_cache_attend_workspace_bytes; its contents do not matter. Calls
 *     that overlap on the GPU with the same workspace race.
 * N == 0 is KDA_OK and launches nothing. N and HQ are at most 65535, N * HQ at
 * most 2^24 and max_pages * page_size at most 2^30 (else KDA_ERR_UNSUPPORTED).
 * Errors: KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE before
 * any launch; KDA_ERR_CUDA if a launch fails.
 */
kda_status kda_cache_attend(const kda_cache* cache, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                            const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                            const int32_t* kv_lens, int32_t window, float scale, void* o, float* lse, int32_t* status,
                            void* ws, size_t ws_bytes, kda_stream_t stream);

/*
 * Bytes of workspace kda_cache_attend needs for these sizes on the present
 * device (0 if they are invalid): KDA_ATTEND_WORKSPACE_MIN, which is then
 * neither read nor written, or more.
 */
#define KDA_ATTEND_WORKSPACE_MIN 256
size_t kda_cache_attend_workspace_bytes(const kda_cache* cache, int32_t HQ, int32_t N, int32_t max_pages,
                                        int32_t window);

/*
 * The same, with the first `sinks` rows of each sequence visible beside a
 * window: t runs over 0 .. sinks - 1 and kv_lens[n] - window .. kv_lens[n] - 1,
 * each row once. Without a window (0) all rows are visible, and sinks says
 * nothing. The rows keep the positions that they were rotated by.
 */
kda_status kda_cache_attend_sinks(const kda_cache* cache, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                  const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                  const int32_t* kv_lens, int32_t window, int32_t sinks, float scale, void* o, float* lse,
                                  int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream);
size_t kda_cache_attend_sinks_workspace_bytes(const kda_cache* cache, int32_t HQ, int32_t N, int32_t max_pages,
                                              int32_t window, int32_t sinks);

/*
 * A paged cache in 8 bits: values in e4m3 (4 bits of exponent, 3 of mantissa,
 * no infinity), in units of a scale for each block of `block` rows of a page
 * and head. cache.dtype is KDA_DTYPE_E4M3, its strides multiples of 16. Block b
 * of a page, rows b block .. (b + 1) block - 1, has for head h the scale
 *   k_scale[p * k_scale_page + b * k_scale_block + h * k_scale_head]
 * (strides in elements, non-negative; to append, blocks do not share a scale);
 * v_scale likewise. `block` divides
 * page_size. `dtype` is that of the rows appended, of q and of o.
 */
#define KDA_DTYPE_E4M3 2
typedef struct {
    kda_cache cache;
    float* k_scale;
    float* v_scale;
    int64_t k_scale_page, k_scale_block, k_scale_head;
    int64_t v_scale_page, v_scale_block, v_scale_head;
    int32_t block, dtype;
} kda_cache8;

/*
 * kda_cache_append into such a cache; arguments and errors are the same. Keys
 * are rotated in fp32, each product and each sum rounded by itself, and go from
 * there to 8 bits; q_out is in `dtype`. A block's scale is the smallest power
 * of two, 2^-126 at least, by which its finite values come to 448 at most, and
 * a value is stored as x / scale, rounded to the nearest e4m3 (ties to even);
 * what is not finite becomes a NaN. Of a block that has rows already
 * (positions below kv_lens[n]) the scale only grows, to what the new rows want
 * (a scale that is not a power of two: to the next one, 2^126 at most, beyond
 * which values become a NaN too); its rows are then
 * written again in the new units, rounded once more where they fall below
 * e4m3's normal values. Scales of blocks without rows are not read. Rows that
 * are dropped count for nothing. Where cu_seqlens does not go from 0 to R,
 * status is set; the rows of a sequence that begins before row 0 are dropped,
 * those up to R of one that ends behind it are appended. Two sequences that
 * append to the same page race.
 */
kda_status kda_cache8_append(const kda_cache8* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* q, int64_t q_stride, void* q_out, int32_t HQ, int32_t N, int64_t R,
                             const int64_t* cu_seqlens, const float* rope, int32_t rope_len, int32_t rope_dim,
                             int32_t interleaved, const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                             const int32_t* kv_lens, int32_t* status, kda_stream_t stream);
kda_status kda_cache8_append_granted(const kda_cache8* cache, const void* k, int64_t k_stride, const void* v,
                                     int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ, int32_t N,
                                     int64_t R, const int64_t* cu_seqlens, const float* rope, int32_t rope_len,
                                     int32_t rope_dim, int32_t interleaved, const int32_t* page_table,
                                     int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                                     const int32_t* granted, int32_t* status, kda_stream_t stream);

/*
 * kda_cache_attend_sinks over such a cache: K[t] and V[t] are the values that
 * the rows stand for, e4m3 times the block's scale (of any sign and size; not
 * only those that kda_cache8_append leaves). Scores are sums of exact products
 * q . K8 in fp32 (which have to be finite there before the scales count), of
 * bf16 queries as they are down to 2^-31 of the head's largest value, of fp32
 * queries to 22 bits, or 2^-39 of the largest (both of heads whose largest value
 * is 2^-100 or more). Weights times the scales of V enter the products as two
 * fp16 values, to 2^-22, or 2^-35 of the largest (scales of 2^-100 and more); a
 * weight below 2^-90 of the largest may count as 0, however large its row's
 * scale. A scale of K is a factor of its row's score; an infinite one of V makes
 * its rows' values infinite (NaN where they are 0). q and o are in `dtype`;
 * arguments, limits and errors are otherwise the same.
 */
kda_status kda_cache8_attend(const kda_cache8* cache, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                             const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                             int32_t window, int32_t sinks, float scale, void* o, float* lse, int32_t* status, void* ws,
                             size_t ws_bytes, kda_stream_t stream);
size_t kda_cache8_attend_workspace_bytes(const kda_cache8* cache, int32_t HQ, int32_t N, int32_t max_pages,
                                         int32_t window, int32_t sinks);

/*
 * Pages for new lengths of N sequences, from a list of free pages and back to
 * it, and where their new rows go. Sequence n holds the pages of its
 * kv_lens[n] rows, ceil(kv_lens[n] / page_size) entries of its row of the page
 * table; new_lens[n] rows want ceil(new_lens[n] / page_size). A negative length
 * counts as 0. In this order:
 *   1. pages beyond the new length go back: those of sequence 0 first, each
 *      sequence's in the order of its rows; their entries become -1;
 *   2. missing pages are taken, for sequence 0 first and in the order of its
 *      rows. A sequence is served if its pages and those of all before it are
 *      there, and it wants no more than max_pages; if not it gets none, keeps
 *      those it has, and status is set.
 *   page_table  int32 [N, max_pages], row stride table_stride; other entries
 *               stay as they are. A page is in one place: held by one
 *               sequence, or free (one that two sequences share goes back twice)
 *   free_pages  int32 [num_pages], of which the first free_count[0] are the
 *               free pages; pages come from its end and go to its end. An entry
 *               that goes back is moved as it is (status is set where it is no
 *               page of [0, num_pages), or the list has no room for it: then it
 *               is dropped); one that is taken and is no page becomes -1, and
 *               status is set.
 *   cu_seqlens  int64 [N + 1], nullable: the new rows of each sequence,
 *               max(0, new_lens[n] - kv_lens[n]) of them, one sequence after the
 *               other, as kda_cache_append takes them; those of a sequence that
 *               was not served among them, so append with `granted`
 *               (kda_cache_append_granted), or its last page takes as many of
 *               them as it has room for
 *   slots       int64 [rows], nullable: of each new row, its page * page_size
 *               plus its row in the page; -1 where it has no page or its
 *               sequence was not served, and behind the last new row. Where
 *               there are more than `rows`, status is set. (For a caller's own
 *               kernels: kda_cache_append goes by the table.)
 *   granted     int32 [N], nullable: new_lens[n], or kv_lens[n] where the
 *               sequence was not served. It overlaps neither of them.
 *   status      int32, nullable
 *   ws          kda_cache_resize_workspace_bytes(N, max_pages, rows) bytes, 16-byte
 *               aligned (NULL where that is 0)
 * Kernel launches only: nothing waits for the host. Overlapping calls on the
 * same table, list or workspace race. N == 0 is KDA_OK; cu_seqlens and slots are
 * written all the same. N is at most 65535, N * max_pages at most 2^30 and rows
 * at most 2^31 - 1 (else KDA_ERR_UNSUPPORTED). Errors: KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED,
 * KDA_ERR_WORKSPACE before any launch; KDA_ERR_CUDA if a launch fails.
 */
kda_status kda_cache_resize(int32_t* page_table, int64_t table_stride, int32_t max_pages, int32_t N, int32_t page_size,
                            const int32_t* kv_lens, const int32_t* new_lens, int32_t* free_pages, int32_t num_pages,
                            int32_t* free_count, int64_t* cu_seqlens, int64_t* slots, int64_t rows, int32_t* granted,
                            int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream);
size_t kda_cache_resize_workspace_bytes(int32_t N, int32_t max_pages, int64_t rows);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_SERVE_H */
