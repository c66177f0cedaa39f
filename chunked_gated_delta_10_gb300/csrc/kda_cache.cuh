// Shared definitions of the paged-cache operators (kda_cache_append, kda_cache_attend).
#pragma once
#include "../../include/kda_serve.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "serve_common.cuh"

namespace kda {

// The host-side checks that all operators make of the cache description, but for its type; `unit`: elements of 16 bytes.
inline kda_status check_cache(const kda_cache* c, int64_t unit) {
    if (c->num_pages < 1 || c->page_size < 1 || c->HKV < 1) return KDA_ERR_INVALID_ARG;
    if (!((c->K == 64 || c->K == 128) && (c->V == 64 || c->V == 128))) return KDA_ERR_UNSUPPORTED;
    for (const int64_t s : {c->k_page, c->k_row, c->k_head, c->v_page, c->v_row, c->v_head})
        if (s < 0 || s % unit != 0) return KDA_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}
inline kda_status check_cache(const kda_cache* c) {
    if (!c || (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_F32)) return KDA_ERR_INVALID_ARG;
    return check_cache(c, c->dtype == KDA_DTYPE_BF16 ? 8 : 4);
}
inline kda_status check_cache(const kda_cache8* c) {
    if (!c || c->cache.dtype != KDA_DTYPE_E4M3 || (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_F32))
        return KDA_ERR_INVALID_ARG;
    const kda_status s = check_cache(&c->cache, 16);
    if (s != KDA_OK) return s;
    if (c->block < 1 || c->cache.page_size % c->block != 0 || !c->k_scale || !c->v_scale ||
        ((uintptr_t)c->k_scale & 3u) || ((uintptr_t)c->v_scale & 3u))
        return KDA_ERR_INVALID_ARG;
    for (const int64_t x : {c->k_scale_page, c->k_scale_block, c->k_scale_head, c->v_scale_page, c->v_scale_block,
                            c->v_scale_head})
        if (x < 0) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// What an append is given besides the cache.
struct AppendCall {
    const void* k;
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    const void* q;
    int64_t q_stride;
    const void* q_out;
    int32_t HQ, N;
    int64_t R;
    const int64_t* cu_seqlens;
    const float* rope;
    int32_t rope_len, rope_dim;
    const int32_t* page_table;
    int64_t table_stride;
    int32_t max_pages;
    const int32_t *kv_lens, *granted, *status;
};
// Its checks (`unit`: elements of 16 bytes of the rows).
inline kda_status check_append(const kda_cache* c, const AppendCall& x, int64_t unit) {
    if (x.N < 0 || x.R < 0 || x.HQ < 0 || x.max_pages < 0 || x.table_stride < 0) return KDA_ERR_INVALID_ARG;
    if (x.R > 0 && (x.N == 0 || (!x.cu_seqlens && x.R % x.N != 0))) return KDA_ERR_INVALID_ARG;
    if ((x.HQ > 0) != (x.q != nullptr) && x.R > 0) return KDA_ERR_INVALID_ARG;
    if ((x.q != nullptr) != (x.q_out != nullptr)) return KDA_ERR_INVALID_ARG;
    if (x.k_stride < (int64_t)c->HKV * c->K || x.v_stride < (int64_t)c->HKV * c->V || x.k_stride % unit || x.v_stride % unit)
        return KDA_ERR_INVALID_ARG;
    if (x.q && (x.q_stride < (int64_t)x.HQ * c->K || x.q_stride % unit)) return KDA_ERR_INVALID_ARG;
    if (x.q && x.q == x.q_out && x.q_stride != (int64_t)x.HQ * c->K) return KDA_ERR_INVALID_ARG;
    if (x.rope_dim < 0 || x.rope_dim % 16 != 0 || x.rope_dim > c->K || x.rope_len < 0 || (x.rope != nullptr) != (x.rope_dim > 0))
        return KDA_ERR_INVALID_ARG;
    if (x.R == 0) return KDA_OK;
    if (!x.k || !x.v || !x.kv_lens || (!x.page_table && x.max_pages > 0)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {x.k, x.v, x.q, (const void*)x.q_out, (const void*)x.rope})
        if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)x.page_table & 3u) || ((uintptr_t)x.kv_lens & 3u) || ((uintptr_t)x.granted & 3u) ||
        ((uintptr_t)x.status & 3u) || ((uintptr_t)x.cu_seqlens & 7u))
        return KDA_ERR_INVALID_ARG;
    // (a row's units are counted in 32 bits, in steps of 1024 at most)
    if (x.R > INT32_MAX || ((int64_t)x.HQ + 2 * (int64_t)c->HKV) * 32 > INT32_MAX - 1024) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// 16 bytes of a row as fp32 values, and back.
template <typename TI> struct Unit;
template <> struct Unit<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void load(const void* p, float (&x)[8]) {
        const uint4 u = *(const uint4*)p;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(void* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *(const uint32_t*)&b;
        }
        *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Unit<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void load(const void* p, float (&x)[4]) {
        const float4 u = *(const float4*)p;
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
    static __device__ __forceinline__ void store(void* p, const float (&x)[4]) {
        *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
    }
};

}  // namespace kda
