// kda_cache8_attend: attention of one new token per sequence over a paged cache in 8 bits. Declared in
// include/kda_serve.h.
//
// With K[t] = sk[t] K8[t] and V[t] = sv[t] V8[t] (e4m3 values, scales of the rows' blocks),
//   s_t = scale sk[t] (q . K8[t]),   p_t = 2^(s_t - m),   l = sum p_t,   acc = sum (p_t sv[t]) V8[t],
// so the scales go to the scores and to the weights, one number a row each, and the cached values enter the tensor
// cores as they are: an e4m3 value is an fp16 value, and one instruction turns two of them into two.
//
// fp16 has five bits of exponent, so what the values meet there is held near the top of its range:
//   - q times a power of two that brings the head's largest value to [2^14, 2^15): bf16's eight bits then are exact in
//     fp16 down to 2^-31 of the largest. An fp32 query is two such values, 22 bits.
//   - the weights p sv times 2^(m - M + 11), M a running whole number like the maximum m itself, raised where one of them
//     passes 2^15. Each is two fp16 values: to 2^-22 of itself, or 2^-35 of the largest.
// m and M are whole numbers (log2 units), so that rescaling l and acc rounds nothing.
#include <cuda_fp16.h>

#include "kda_attend.cuh"

namespace kda {
namespace attend {
namespace {

// How far above the running maximum a score, or a weighted scale, may lie (log2 units) before l and acc are rescaled; and
// the power of two that a weight at the running maximum has in fp16.
constexpr float kSlack8 = 3.f;
constexpr int kTop8 = 11;
constexpr float kMost8 = 32768.f;  // of a weight in fp16, which holds 65504

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 values, the lower or upper two bytes, as two fp16 values.
__device__ __forceinline__ uint32_t lower2(uint32_t x) {
    uint32_t y;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t upper2(uint32_t x) {
    uint32_t y;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&h;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x) { return __half22float2(*(const __half2*)&x); }
// 2^x of a whole number x, 0 below 2^-126; x is at most 127. (-inf: 0)
__device__ __forceinline__ float power(float x) {
    return __int_as_float(((int)fmaxf(x, -127.f) + 127) << 23);
}
__device__ __forceinline__ float max_of_rows(float x) {
#pragma unroll
    for (int w = 4; w < 32; w *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
    return x;
}
// 8 bytes of a row.
__device__ __forceinline__ uint2 load8(const void* p, bool ok) {
    uint2 x = make_uint2(0, 0);
    if (ok) x = __ldcs((const uint2*)p);
    return x;
}

// CTAs of k_attend8 to an SM.
constexpr int ctas8(int NT, int K, int V) { return (K + V == 128 ? 5 : 4) - NT; }

// Channels of a query in fp32.
template <typename TI> __device__ __forceinline__ void load4(const TI* p, bool ok, float (&x)[4]) {
    if constexpr (sizeof(TI) == 2) {
        uint2 u = make_uint2(0, 0);
        if (ok) u = *(const uint2*)p;
        x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float4 u = ok ? *(const float4*)p : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
}

// A unit has up to 8 NT query heads, each warp a tile of 32 rows at a time, a lane looking up one. The products are taken
// transposed, as over a cache in 16 bits (k_attend_mma): S^T [32 rows x 8 heads] = K8 Q^T, O^T [V x 8 heads] += V8^T P^T.
//   - lane 4 g + t loads 16-byte units t, t + 4, .. of rows g, g + 8, .. of K8; four channels of two rows are one product's
//     share of the lane, and Q has the same order.
//   - of V8 it loads V / 8 channels, from V / 8 g on, of rows 2 t, 2 t + 1, 2 t + 8, ..; a byte permutation pairs the
//     rows, and row i of the j-th product is channel V / 8 (i % 8) + j.
template <typename TI, int K, int V, int NT, bool SHARES>
__global__ void __launch_bounds__(kWarps * 32, ctas8(NT, K, V)) k_attend8(AttendArgs a) {
    constexpr int KI = K / 64, CW = V / 8, VJ = V / 16, HT = 8 * NT, QP = sizeof(TI) / 2;
    __shared__ Partial<HT, V> sm;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    if (!SHARES && a.split == kCluster) cluster_started();
    after_previous();
    typedef Work<32, HT, SHARES, true> Wk;
    Wk wk;
    __shared__ typename Wk::Share share;
#pragma unroll 1
    for (bool more = wk.start(a, share); more; more = wk.next(a, share)) {
        const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
        Rows<32, true>& rows = wk.rows;
        uint32_t q[NT][QP][KI][4][2];
        float qf[NT][2];  // what the scores of heads 2 t, 2 t + 1 are multiplied by
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float x[KI][4][4], top = 0.f;
#pragma unroll
            for (int i = 0; i < KI; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    load4((const TI*)a.q + (int64_t)wk.n * a.q_stride + (h0 + 8 * j + g) * K + (4 * i + t) * 16 + 4 * w,
                          8 * j + g < heads, x[i][w]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[i][w][e]));
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // (an infinite value stays infinite, and the others finite; below 2^-100 a query has fewer bits)
            const int up = 14 - min(max((__float_as_int(top) >> 23) - 127, -100), 127);
            const float f = __int_as_float((up + 127) << 23);
#pragma unroll
            for (int i = 0; i < KI; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float lo = x[i][w][2 * e] * f, hi = x[i][w][2 * e + 1] * f;
                        q[j][0][i][w][e] = pack_f16(lo, hi);
                        if constexpr (QP == 2) {
                            const float2 y = unpack_f16(q[j][0][i][w][e]);
                            // (an infinite part leaves nothing)
                            q[j][1][i][w][e] = pack_f16(isinf(y.x) ? 0.f : lo - y.x, isinf(y.y) ? 0.f : hi - y.y);
                        }
                    }
            const float down = a.scale_log2 * __int_as_float((127 - up) << 23);
            qf[j][0] = __shfl_sync(0xffffffffu, down, 8 * t);
            qf[j][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
        }
        float acc[NT][VJ][4], m[NT][2], l[NT][2], big[NT][2], pf[NT][2];  // big: M; pf: 2^(m - M + kTop8)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[j][e] = big[j][e] = -INFINITY;
                l[j][e] = pf[j][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VJ; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
        }
        const char* kh = (const char*)a.c.k + wk.hkv * a.c.k_head + t * 16;
        const char* vh = (const char*)a.c.v + wk.hkv * a.c.v_head + g * CW;
        const float *ksh = a.k_scale + wk.hkv * a.ks_head, *vsh = a.v_scale + wk.hkv * a.vs_head;
        uint4 kr[4][KI], vr[8][(CW + 15) / 16];
        uint2 vh8[CW == 8 ? 8 : 1];
        float ks, vs;  // the scales of this lane's row
        auto load_k = [&]() {
            const bool mine = rows.valid >> lane & 1;
            const int64_t block = a.block(rows.at_off);
            ks = mine ? ksh[rows.at * a.ks_page + block * a.ks_block] : 0.f;
            vs = mine ? vsh[rows.at * a.vs_page + block * a.vs_block] : 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const char* p = kh + rows.k_of(g + 8 * r);
                const bool ok = rows.valid >> (g + 8 * r) & 1;
#pragma unroll
                for (int i = 0; i < KI; ++i) kr[r][i] = load16(p + 64 * i, ok);
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int at = 2 * t + (r & 1) + 4 * (r & 2) + 4 * (r & 4);
                const char* p = vh + rows.v_of(at);
                const bool ok = rows.valid >> at & 1;
                if constexpr (CW == 16)
                    vr[r][0] = load16(p, ok);
                else
                    vh8[r] = load8(p, ok);
            }
        };
        rows.next(a);
        load_k();
        load_v();
#pragma unroll 1
        for (int left = wk.left; left > 0; left -= a.step) {
            float s[NT][2][4];  // of rows g, g + 8 (and 16 more) and heads 2 t, 2 t + 1
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int j = 0; j < NT; ++j) s[j][b][0] = s[j][b][1] = s[j][b][2] = s[j][b][3] = 0.f;
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    const uint32_t* r0 = (const uint32_t*)&kr[2 * b][i];
                    const uint32_t* r1 = (const uint32_t*)&kr[2 * b + 1][i];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = lower2(r0[w]), a1 = lower2(r1[w]), a2 = upper2(r0[w]), a3 = upper2(r1[w]);
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < QP; ++c)
                                mma_f16(s[j][b], a0, a1, a2, a3, q[j][c][i][w][0], q[j][c][i][w][1]);
                    }
                }
            }
            float vf[4];
            const unsigned in = rows.valid;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float kf = __shfl_sync(0xffffffffu, ks, g + 8 * r);
                vf[r] = __shfl_sync(0xffffffffu, vs, g + 8 * r);
                const bool ok = in >> (g + 8 * r) & 1;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = s[j][r / 2][2 * (r % 2) + e];
                        x = ok ? x * qf[j][e] * kf : -INFINITY;
                    }
            }
            rows.next(a);
            load_k();
            // weights (p), and what they are times the scales of V (w)
            float p[NT][4][2], w[NT][4][2];
            bool higher = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = s[j][r / 2][2 * (r % 2) + e];
                        p[j][r][e] = ex2(x - finite_base(m[j][e]));
                        w[j][r][e] = p[j][r][e] * pf[j][e] * vf[r];
                        higher |= x > m[j][e] + kSlack8 || fabsf(w[j][r][e]) > kMost8;
                    }
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = -INFINITY, most = 0.f;
#pragma unroll
                        for (int r = 0; r < 4; ++r) top = fmaxf(top, s[j][r / 2][2 * (r % 2) + e]);
                        top = fmaxf(m[j][e], ceilf(max_of_rows(top)));
                        const float base = finite_base(top);
                        l[j][e] *= power(m[j][e] - base);
                        m[j][e] = top;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            p[j][r][e] = ex2(s[j][r / 2][2 * (r % 2) + e] - base);
                            most = fmaxf(most, fabsf(p[j][r][e] * vf[r]));
                        }
                        // 2^(exponent of `most`, rounded up), as far from m as fp32 holds 2^(m - M + kTop8)
                        const int up = ((__float_as_int(max_of_rows(most)) + 0x7fffff) >> 23) - 127;
                        const float to =
                            top == -INFINITY ? big[j][e] : fmaxf(big[j][e], base + (float)max(up, kTop8 - 126));
                        const float f = power(big[j][e] - to);
                        big[j][e] = to;
                        pf[j][e] = power(fmaxf(base - to + kTop8, -126.f));
#pragma unroll
                        for (int i = 0; i < VJ; ++i) {
                            acc[j][i][e] *= f;
                            acc[j][i][e + 2] *= f;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) w[j][r][e] = p[j][r][e] * pf[j][e] * vf[r];
                    }
            }
            uint32_t pt[NT][2][4];  // the two parts of P^T, 8 rows each
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    l[j][0] += p[j][r][0];
                    l[j][1] += p[j][r][1];
                    const uint32_t hi = pack_f16(w[j][r][0], w[j][r][1]);
                    const float2 y = unpack_f16(hi);
                    pt[j][0][r] = transpose8(hi);
                    pt[j][1][r] = transpose8(pack_f16(w[j][r][0] - y.x, w[j][r][1] - y.y));
                }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int c = 0; c < VJ / 4; ++c) {
                    // four products: rows 0-7 of the j-th are channels CW g + j, rows 8-15 channels CW g + j + CW / 2
                    uint32_t x[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int word = c + (e & 1) * (VJ / 4), r = 4 * b + (e & 2);
                        uint32_t even, odd;
                        if constexpr (CW == 16) {
                            even = ((const uint32_t*)&vr[r][0])[word];
                            odd = ((const uint32_t*)&vr[r + 1][0])[word];
                        } else {
                            even = ((const uint32_t*)&vh8[r])[word];
                            odd = ((const uint32_t*)&vh8[r + 1])[word];
                        }
                        const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
                        x[0][e] = lower2(lo);
                        x[1][e] = upper2(lo);
                        x[2][e] = lower2(hi);
                        x[3][e] = upper2(hi);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_f16(acc[j][4 * c + i], x[i][0], x[i][1], x[i][2], x[i][3], pt[j][part][2 * b],
                                        pt[j][part][2 * b + 1]);
                }
            load_v();
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * j + 2 * t + e;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], d);
                if (g == 0) {
                    sm.m[warp][h] = m[j][e];
                    sm.l[warp][h] = l[j][e] * kAtMostOne;
                }
                // relative to m as the join wants it, in two steps that fp32 holds
                const float apart = m[j][e] == -INFINITY ? 0.f : big[j][e] - m[j][e] - kTop8, half = rintf(0.5f * apart);
                const float f0 = power(half) * kAtMostOne, f1 = power(apart - half);
                float* row = (float*)sm.acc[warp][h] + CW * g;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < VJ; i += 4)
                        *(float4*)(row + VJ * r + i) =
                            make_float4(acc[j][i][e + 2 * r] * f0 * f1, acc[j][i + 1][e + 2 * r] * f0 * f1,
                                        acc[j][i + 2][e + 2 * r] * f0 * f1, acc[j][i + 3][e + 2 * r] * f0 * f1);
            }
        join<TI, V, HT, SHARES, Wk>(a, share, sm);
        if constexpr (!SHARES) return;
        __syncthreads();  // the shared memory is free for the next unit
    }
}

template <int K, int V> Kernel kernel_of(bool bf16, int ht, Split split) {
    using B = __nv_bfloat16;
    if (!bf16) return ht == 8 ? k_attend8<float, K, V, 1, false> : k_attend8<float, K, V, 2, false>;
    if (split == kShares) return ht == 8 ? k_attend8<B, K, V, 1, true> : k_attend8<B, K, V, 2, true>;
    return ht == 8 ? k_attend8<B, K, V, 1, false> : k_attend8<B, K, V, 2, false>;
}
Kernel kernel_of(const kda_cache8& c, int ht, Split split) {
    const bool bf16 = c.dtype == KDA_DTYPE_BF16;
    const int K = c.cache.K, V = c.cache.V;
    return K == 128 ? (V == 128 ? kernel_of<128, 128>(bf16, ht, split) : kernel_of<128, 64>(bf16, ht, split))
                    : (V == 128 ? kernel_of<64, 128>(bf16, ht, split) : kernel_of<64, 64>(bf16, ht, split));
}

kda_status plan_for(const kda_cache8* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks, Plan& plan) {
    static std::atomic<int> known[2][2][2][2][kDevices];
    kda_status s = check_cache(c);
    if (s == KDA_OK) s = check_sizes(&c->cache, HQ, N, max_pages, window, sinks);
    if (s != KDA_OK) return s;
    const int K = c->cache.K, V = c->cache.V, ht = HQ / c->cache.HKV <= 8 ? 8 : 16, device = present_device();
    const bool bf16 = c->dtype == KDA_DTYPE_BF16;
    const Form form{ht, 32, ctas8(ht / 8, K, V), bf16};
    const Gpu gpu{sm_count(device), largest_cluster(device, (const void*)kernel_of(*c, ht, kCluster), kWarps * 32,
                                                    kMaxCluster, known[bf16][ht / 16][K / 128][V / 128])};
    plan = plan_of(&c->cache, HQ, N, max_pages, window, sinks, form, gpu);
    return KDA_OK;
}

}  // namespace
}  // namespace attend
}  // namespace kda

using namespace kda;
using namespace kda::attend;

extern "C" size_t kda_cache8_attend_workspace_bytes(const kda_cache8* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                    int32_t window, int32_t sinks) {
    Plan plan;
    return plan_for(c, HQ, N, max_pages, window, sinks, plan) == KDA_OK ? plan.ws_bytes : 0;
}

extern "C" kda_status kda_cache8_attend(const kda_cache8* c, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                        const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                        const int32_t* kv_lens, int32_t window, int32_t sinks, float scale, void* o,
                                        float* lse, int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream) {
    Plan plan;
    kda_status s = plan_for(c, HQ, N, max_pages, window, sinks, plan);
    if (s != KDA_OK) return s;
    const bool bf16 = c->dtype == KDA_DTYPE_BF16;
    const Call x{q, q_stride, HQ, N, page_table, table_stride, max_pages, kv_lens, window, sinks, scale, o, lse, status, ws,
                 ws_bytes, (cudaStream_t)stream};
    s = check_call(&c->cache, x, bf16 ? 8 : 4);
    if (s != KDA_OK || N == 0) return s;
    if (!ws || !aligned16(ws) || ws_bytes < plan.ws_bytes) return KDA_ERR_WORKSPACE;
    AttendArgs a = args_of(&c->cache, x, plan);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.ks_page = c->k_scale_page, a.ks_block = c->k_scale_block, a.ks_head = c->k_scale_head;
    a.vs_page = c->v_scale_page, a.vs_block = c->v_scale_block, a.vs_head = c->v_scale_head;
    a.block = Divisor(c->block);
    static const char* const names[] = {"cache8_attend", "cache8_attend_cluster", "cache8_attend_parts",
                                        "cache8_attend_shares"};
    return launch(a, plan, kernel_of(*c, plan.ht, plan.split), bf16, names, x.stream);
}
