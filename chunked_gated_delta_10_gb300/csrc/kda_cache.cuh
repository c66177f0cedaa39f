// Shared definitions of the paged-cache operators (kda_cache_append, kda_cache_attend).
#pragma once
#include "../../include/kda_serve.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "serve_common.cuh"

namespace kda {

// The host-side checks that both operators make of the cache description.
inline kda_status check_cache(const kda_cache* c) {
    if (!c || c->num_pages < 1 || c->page_size < 1 || c->HKV < 1) return KDA_ERR_INVALID_ARG;
    if (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARG;
    if (!((c->K == 64 || c->K == 128) && (c->V == 64 || c->V == 128))) return KDA_ERR_UNSUPPORTED;
    const int64_t unit = c->dtype == KDA_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
    for (const int64_t s : {c->k_page, c->k_row, c->k_head, c->v_page, c->v_row, c->v_head})
        if (s < 0 || s % unit != 0) return KDA_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return KDA_ERR_INVALID_ARG;
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
