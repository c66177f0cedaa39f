// kda_cache_append: new keys and values into a paged cache, keys and queries
// rotated by their position on the way. Declared in include/kda_serve.h.
//
// A rotation turns each pair of channels by the position's angle for that pair,
//   x' = x cos - y sin,   y' = y cos + x sin,
// in fp32, rounded once to the cache's type. A thread moves 16-byte units; one
// that turns channel i with channel i + rope_dim / 2 takes the unit of each.
//
// Bound: every new row is read once and written once; for one token a sequence
// it is the latency of a launch. A CTA has one row, so that its sequence, page
// and angles are found by uniform instructions; what is left of it is loads and
// stores, and the CTA's size decides how many rows an SM has under way:
//   many rows: the fewest threads, from 64 on, that fill the SMs. 16 packed prompts
//     of U[1,4096] tokens, 32 query and 8 cache heads of 128, bf16 (822 MB): 64
//     threads, 122 us, 6.74 TB/s, the rate of a plain copy; with 128 threads 124
//     us, 256: 131, 512: 236. 3000 rows of 128 and 16 heads: 128 threads, 17.2 us;
//     64 leave SMs half empty, and took half as long again.
//   up to two rows an SM: 512 threads, one unit each. One token 2.1 us (64 threads:
//     4.2), 128 tokens 2.6 us (7.2); 512 tokens already 4.5 (256 threads: 4.0).
//   rows of 64 units or fewer share a CTA of 256 threads: 33,000 rows of two
//     heads of 64 take 11.9 us, and 33.5 us with a CTA each (1 ns a CTA).
// Units that turn and units that are copied are separate loops, the copies two at a
// time (the prompts without a rotation 139 -> 120 us, with half of each head turned
// 169 -> 124); 24 CTAs of 64 threads fit an SM (40 registers; with 47: 126 us).
// Several rows to a thread, their loads ahead of their sums, was slower (150 to
// 226 us for the prompts): the angles take the registers that more CTAs need.
#include "kda_cache.cuh"

namespace kda {
namespace {

struct AppendArgs {
    kda_cache c;
    const void *k, *v, *q;
    void* q_out;
    int64_t k_stride, v_stride, q_stride, table_stride;
    int HQ, N;
    unsigned R, per;  // new rows; of a sequence, where there is no cu
    const int64_t* cu;
    const float* rope;
    int rope_len, rope_dim, interleaved;
    const int32_t *table, *kv_lens, *granted;
    int max_pages;
    int32_t* status;
    unsigned lanes, rows;  // short rows: threads of a row, rows of a CTA
};

// The sequence of new row r: the last n with cu[n] <= r.
__device__ __forceinline__ int seq_of(const int64_t* cu, int N, unsigned r) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cu[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// GRANTED: rows have lengths to keep to. (A kernel of its own: to ask whether they have takes 0.1 us of a token's 2.2.)
template <typename TI, bool SHORT, int MOST, bool GRANTED>
__global__ void __launch_bounds__(MOST, SHORT ? 6 : MOST == 64 ? 24 : 2) k_append(AppendArgs a) {
    constexpr int E = Unit<TI>::n, kBatch = SHORT ? 1 : 2;  // units of a row; copies that a thread has under way
    after_previous();
    int64_t r = blockIdx.x;
    int lane = threadIdx.x;
    if constexpr (SHORT) {
        const unsigned in = lane / a.lanes;
        r = r * a.rows + in;
        lane -= in * a.lanes;
        if (in >= a.rows || r >= a.R) return;
    }
    unsigned n, idx;
    bool ok = true;
    if (a.cu) {
        n = seq_of(a.cu, a.N, (unsigned)r);
        const int64_t begin = a.cu[n];
        ok = begin <= r && r < a.cu[n + 1];
        idx = (unsigned)(r - begin);
    } else {
        n = (unsigned)r / a.per;
        idx = (unsigned)r - n * a.per;
    }
    const int len = a.kv_lens[n];
    const unsigned at_pos = (unsigned)len + idx, pg = at_pos / (unsigned)a.c.page_size;
    const int64_t pos = at_pos, row = at_pos - pg * a.c.page_size;
    int64_t page = -1;
    // (a row that was not granted is dropped like one of an inactive sequence)
    if (len >= 0 && !(GRANTED && ok && at_pos >= (unsigned)max(a.granted[n], 0))) {
        ok = ok && pg < (unsigned)a.max_pages && (!a.rope || pos < (unsigned)a.rope_len);
        if (ok) page = a.table[n * a.table_stride + pg];
        if (page < 0 || page >= a.c.num_pages) {
            page = -1;
            if (a.status && lane == 0) *a.status = KDA_ERR_INVALID_ARG;
        }
    }
    const int lanes = SHORT ? a.lanes : blockDim.x;
    const int heads = a.HQ + a.c.HKV, rot = a.rope_dim / E;  // query heads, then key heads; a head's units that turn
    // row r of head h, from channel `at` on: where it is, and where it goes (null: it is dropped)
    const auto from = [&](int h, int at) {
        return h < a.HQ ? (const TI*)a.q + r * a.q_stride + (int64_t)h * a.c.K + at
                        : (const TI*)a.k + r * a.k_stride + (int64_t)(h - a.HQ) * a.c.K + at;
    };
    const auto to = [&](int h, int at) -> TI* {
        if (h < a.HQ) return (TI*)a.q_out + (r * a.HQ + h) * a.c.K + at;
        if (page < 0) return nullptr;
        return (TI*)a.c.k + page * a.c.k_page + row * a.c.k_row + (h - a.HQ) * a.c.k_head + at;
    };
    // the units that turn: two of them, half of rope_dim apart, or one with its channels in pairs
    const int per = a.interleaved ? rot : rot / 2, turning = heads * per;
    const float* cs = a.rope + pos * a.rope_dim;
    for (int i = lane; i < turning; i += lanes) {
        const int h = i / per, at = (i - h * per) * E, other = at + a.rope_dim / 2;
        TI* dst = to(h, at);
        if (!dst) continue;
        float x[E], y[E];
        if (page < 0) {  // a query row of a dropped or inactive token
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
            Unit<TI>::store(dst, x);
            if (!a.interleaved) Unit<TI>::store(dst + a.rope_dim / 2, x);
        } else if (a.interleaved) {
            Unit<TI>::load(from(h, at), x);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float co = cs[(at + e) / 2], si = cs[(a.rope_dim + at + e) / 2], t = x[e];
                x[e] = t * co - x[e + 1] * si;
                x[e + 1] = x[e + 1] * co + t * si;
            }
            Unit<TI>::store(dst, x);
        } else {
            Unit<TI>::load(from(h, at), x);
            Unit<TI>::load(from(h, other), y);
            float co[E], si[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                co[e] = cs[at + e];
                si[e] = cs[other + e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float t = x[e];
                x[e] = t * co[e] - y[e] * si[e];
                y[e] = y[e] * co[e] + t * si[e];
            }
            Unit<TI>::store(dst, x);
            Unit<TI>::store(dst + a.rope_dim / 2, y);
        }
    }
    // the units that are copied, some at a time; the threads that had the fewest to turn begin
    const int rest = a.c.K / E - rot, uv = a.c.V / E, of_heads = heads * rest, copied = of_heads + a.c.HKV * uv;
    int first = lane - turning % lanes;
    if (first < 0) first += lanes;
    for (int i = first; i < copied; i += kBatch * lanes) {
        uint4 x[kBatch];
        TI* dst[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int j = i + b * lanes;
            dst[b] = nullptr;
            if (j < of_heads) {
                const int h = j / rest, at = (rot + j - h * rest) * E;
                dst[b] = to(h, at);
                x[b] = page < 0 ? make_uint4(0, 0, 0, 0) : *(const uint4*)from(h, at);
            } else if (j < copied && page >= 0) {
                const int h = (j - of_heads) / uv, at = (j - of_heads - h * uv) * E;
                dst[b] = (TI*)a.c.v + page * a.c.v_page + row * a.c.v_row + h * a.c.v_head + at;
                x[b] = *(const uint4*)((const TI*)a.v + r * a.v_stride + (int64_t)h * a.c.V + at);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (dst[b]) *(uint4*)dst[b] = x[b];
    }
}

template <typename TI, bool GRANTED> void (*kernel_of(bool few, int most))(AppendArgs) {
    return few          ? k_append<TI, true, 256, GRANTED>
           : most == 64 ? k_append<TI, false, 64, GRANTED>
                        : k_append<TI, false, 512, GRANTED>;
}
template <typename TI> void (*kernel_of(bool few, int most, bool granted))(AppendArgs) {
    return granted ? kernel_of<TI, true>(few, most) : kernel_of<TI, false>(few, most);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_cache_append(const kda_cache* c, const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ,
                                       int32_t N, int64_t R, const int64_t* cu_seqlens, const float* rope,
                                       int32_t rope_len, int32_t rope_dim, int32_t interleaved,
                                       const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                       const int32_t* kv_lens, int32_t* status, kda_stream_t stream) {
    return kda_cache_append_granted(c, k, k_stride, v, v_stride, q, q_stride, q_out, HQ, N, R, cu_seqlens, rope, rope_len,
                                    rope_dim, interleaved, page_table, table_stride, max_pages, kv_lens, nullptr, status,
                                    stream);
}

extern "C" kda_status kda_cache_append_granted(const kda_cache* c, const void* k, int64_t k_stride, const void* v,
                                               int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ,
                                               int32_t N, int64_t R, const int64_t* cu_seqlens, const float* rope,
                                               int32_t rope_len, int32_t rope_dim, int32_t interleaved,
                                               const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                               const int32_t* kv_lens, const int32_t* granted, int32_t* status,
                                               kda_stream_t stream) {
    const kda_status s = check_cache(c);
    if (s != KDA_OK) return s;
    const int64_t unit = c->dtype == KDA_DTYPE_BF16 ? 8 : 4;
    const AppendCall x{k, k_stride, v, v_stride, q, q_stride, q_out, HQ, N, R, cu_seqlens, rope, rope_len, rope_dim,
                       page_table, table_stride, max_pages, kv_lens, granted, status};
    const kda_status checked = check_append(c, x, unit);
    if (checked != KDA_OK || R == 0) return checked;
    const int64_t uk = (c->K - (interleaved ? 0 : rope_dim / 2)) / unit;
    const int64_t units = (HQ + c->HKV) * uk + c->HKV * (c->V / unit);  // of a row
    const bool few = units <= 64;
    const int sms = sm_count();
    int most = few ? 256 : R <= 2 * sms ? 512 : 64;  // threads of a CTA; measured: see the top of this file
    while (most < 256 && R * most < sms * (int64_t)2048) most *= 2;
    const int64_t turns = (units + most - 1) / most;
    const int lanes = (int)((units + turns - 1) / turns), rows = few ? most / lanes : 1;
    const int threads = (lanes * rows + 31) / 32 * 32;
    const AppendArgs a{*c, k, v, q, q_out, k_stride, v_stride, q_stride, table_stride, HQ, N, (unsigned)R,
                       (unsigned)(R / N), cu_seqlens, rope, rope_len, rope_dim, interleaved, page_table, kv_lens,
                       granted, max_pages, status, (unsigned)lanes, (unsigned)rows};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    void (*const kernel)(AppendArgs) =
        c->dtype == KDA_DTYPE_BF16 ? kernel_of<__nv_bfloat16>(few, most, granted) : kernel_of<float>(few, most, granted);
    const cudaError_t e = launch_after(kernel, a, (unsigned)((R + rows - 1) / rows), threads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_append", st);
    return KDA_OK;
}
