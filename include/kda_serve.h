/*
 * kda_serve.h — C ABI of the single-token (serving) operators: what a hybrid
 * of KDA layers and full-attention layers runs after kda_chunk_fwd has taken
 * the prompt.
 *
 *   kda_step          a few tokens (usually one) on the fp32 KDA states, in place
 *   kda_cache_append  new keys and values into a paged cache, keys and queries
 *                     rotated by their position on the way
 *   kda_cache_attend  attention of one new token per sequence over that cache
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

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_SERVE_H */
