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
//     us, 256: 131, 512: 236. 3000 rows of 128 and 16 heads: 128 threads, 21.7 us;
//     with 64, which leave SMs half empty, 33.6.
//   up to two rows an SM: 512 threads, one unit each. One token 2.1 us (64 threads:
//     4.2), 128 tokens 3.0 us (7.2); 512 tokens already 4.5 (256 threads: 4.0).
//   rows of 64 units or fewer share a CTA of 256 threads: 33,000 rows of two
//     heads of 64 take 10.2 us, and 33.5 us with a CTA each (1 ns a CTA).
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
    const int32_t *table, *kv_lens;
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

template <typename TI, bool SHORT, int MOST>
__global__ void __launch_bounds__(MOST) k_append(AppendArgs a) {
    constexpr int E = Unit<TI>::n;
    after_previous();
    unsigned r = blockIdx.x;
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
        n = seq_of(a.cu, a.N, r);
        const int64_t first = a.cu[n];
        ok = first <= r;
        idx = r - (unsigned)first;
    } else {
        n = r / a.per;
        idx = r - n * a.per;
    }
    const int len = a.kv_lens[n];
    const unsigned pos = (unsigned)len + idx, pg = pos / (unsigned)a.c.page_size, row = pos - pg * a.c.page_size;
    int page = -1;
    if (len >= 0) {
        ok = ok && pg < (unsigned)a.max_pages && (!a.rope || pos < (unsigned)a.rope_len);
        if (ok) page = a.table[n * a.table_stride + pg];
        if (page < 0 || page >= a.c.num_pages) {
            page = -1;
            if (a.status && lane == 0) *a.status = KDA_ERR_INVALID_ARG;
        }
    }
    // units of a head: the pairs of units that turn together, then the rest
    const int half = a.interleaved ? 0 : a.rope_dim / 2 / E;
    const int uk = a.c.K / E - half, uv = a.c.V / E;
    const int units_q = a.HQ * uk, units_k = a.c.HKV * uk, units = units_q + units_k + a.c.HKV * uv;
    for (int i = lane; i < units; i += SHORT ? a.lanes : blockDim.x) {
        if (i >= units_q + units_k) {
            const int j = i - units_q - units_k, h = j / uv, u = j % uv;
            if (page >= 0) {
                const TI* src = (const TI*)a.v + (int64_t)r * a.v_stride + h * a.c.V + u * E;
                TI* dst = (TI*)a.c.v + (int64_t)page * a.c.v_page + row * a.c.v_row + h * a.c.v_head + u * E;
                *(uint4*)dst = *(const uint4*)src;
            }
            continue;
        }
        const bool is_q = i < units_q;
        const int j = is_q ? i : i - units_q, h = j / uk, u = j % uk;
        if (!is_q && page < 0) continue;
        const TI* src = is_q ? (const TI*)a.q + (int64_t)r * a.q_stride + h * a.c.K
                             : (const TI*)a.k + (int64_t)r * a.k_stride + h * a.c.K;
        TI* dst = is_q ? (TI*)a.q_out + ((int64_t)r * a.HQ + h) * a.c.K
                       : (TI*)a.c.k + (int64_t)page * a.c.k_page + row * a.c.k_row + h * a.c.k_head;
        float x[E], y[E];
        if (page < 0) {  // a query row of a dropped or inactive token
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
            if (u < half) Unit<TI>::store(dst + u * E, x);
            Unit<TI>::store(dst + (u + half) * E, x);
            continue;
        }
        const float* cs = a.rope + (int64_t)pos * a.rope_dim;
        if (u < half) {
            Unit<TI>::load(src + u * E, x);
            Unit<TI>::load(src + (u + half) * E, y);
            float co[E], si[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                co[e] = cs[u * E + e];
                si[e] = cs[a.rope_dim / 2 + u * E + e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float t = x[e];
                x[e] = t * co[e] - y[e] * si[e];
                y[e] = y[e] * co[e] + t * si[e];
            }
            Unit<TI>::store(dst + u * E, x);
            Unit<TI>::store(dst + (u + half) * E, y);
            continue;
        }
        const int at = (u + half) * E;
        Unit<TI>::load(src + at, x);
        if (a.interleaved && at < a.rope_dim) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float co = cs[(at + e) / 2], si = cs[a.rope_dim / 2 + (at + e) / 2], t = x[e];
                x[e] = t * co - x[e + 1] * si;
                x[e + 1] = x[e + 1] * co + t * si;
            }
        }
        Unit<TI>::store(dst + at, x);
    }
}

template <typename TI> void (*kernel_of(bool few, int most))(AppendArgs) {
    return few ? k_append<TI, true, 256> : most == 64 ? k_append<TI, false, 64> : k_append<TI, false, 512>;
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
    const kda_status s = check_cache(c);
    if (s != KDA_OK) return s;
    const int64_t unit = c->dtype == KDA_DTYPE_BF16 ? 8 : 4;
    if (N < 0 || R < 0 || HQ < 0 || max_pages < 0 || table_stride < 0) return KDA_ERR_INVALID_ARG;
    if (R > 0 && (N == 0 || (!cu_seqlens && R % N != 0))) return KDA_ERR_INVALID_ARG;
    if ((HQ > 0) != (q != nullptr) && R > 0) return KDA_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr)) return KDA_ERR_INVALID_ARG;
    if (k_stride < (int64_t)c->HKV * c->K || v_stride < (int64_t)c->HKV * c->V || k_stride % unit || v_stride % unit)
        return KDA_ERR_INVALID_ARG;
    if (q && (q_stride < (int64_t)HQ * c->K || q_stride % unit)) return KDA_ERR_INVALID_ARG;
    if (q && q == q_out && q_stride != (int64_t)HQ * c->K) return KDA_ERR_INVALID_ARG;
    if (rope_dim < 0 || rope_dim % 16 != 0 || rope_dim > c->K || rope_len < 0 || (rope != nullptr) != (rope_dim > 0))
        return KDA_ERR_INVALID_ARG;
    if (R == 0) return KDA_OK;
    if (!k || !v || !kv_lens || (!page_table && max_pages > 0)) return KDA_ERR_INVALID_ARG;
    for (const void* x : {k, v, q, (const void*)q_out, (const void*)rope})
        if (!aligned16(x)) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)page_table & 3u) || ((uintptr_t)kv_lens & 3u) || ((uintptr_t)status & 3u) ||
        ((uintptr_t)cu_seqlens & 7u))
        return KDA_ERR_INVALID_ARG;
    if (R > INT32_MAX || ((int64_t)HQ + 2 * (int64_t)c->HKV) * 32 > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const int64_t uk = (c->K - (interleaved ? 0 : rope_dim / 2)) / unit;
    const int64_t units = (HQ + c->HKV) * uk + c->HKV * (c->V / unit);  // of a row
    const bool few = units <= 64;
    int most = few ? 256 : R <= 2 * 152 ? 512 : 64;  // threads of a CTA; measured: see the top of this file
    while (most < 256 && R * most < 152 * 2048) most *= 2;
    const int64_t turns = (units + most - 1) / most;
    const int lanes = (int)((units + turns - 1) / turns), rows = few ? most / lanes : 1;
    const int threads = (lanes * rows + 31) / 32 * 32;
    const AppendArgs a{*c, k, v, q, q_out, k_stride, v_stride, q_stride, table_stride, HQ, N, (unsigned)R,
                       (unsigned)(R / N), cu_seqlens, rope, rope_len, rope_dim, interleaved, page_table, kv_lens, max_pages,
                       status, (unsigned)lanes, (unsigned)rows};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    void (*const kernel)(AppendArgs) =
        c->dtype == KDA_DTYPE_BF16 ? kernel_of<__nv_bfloat16>(few, most) : kernel_of<float>(few, most);
    const cudaError_t e = launch_after(kernel, a, (unsigned)((R + rows - 1) / rows), threads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_append", st);
    return KDA_OK;
}
