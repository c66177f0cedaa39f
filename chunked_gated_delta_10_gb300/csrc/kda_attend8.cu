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
//     fp16 down to 2^-31 of the largest. An fp32 query is two such values, 22 bits, or 2^-39 of the largest.
//   - the weights p sv times 2^(m - M + 11), M a running whole number like the maximum m itself, raised where one of them
//     passes 2^15. Each is two fp16 values: to 2^-22 of itself, or 2^-35 of the largest.
// m and M are whole numbers (log2 units), so that rescaling l and acc rounds nothing.
//
// Bound: the cached values are read once. Measured on one GB300 (time of a call in a graph; GB/s of the cached rows and
// scales), bf16 queries, K = V = 128:
//   64 sequences of U[1,8192] rows, 32 query heads on 8: 87 to 89 us, 6.0 TB/s (77 at a plain copy's rate); of 32768 rows
//     each 622 us, 6.9 TB/s. The start (lengths, shares, pages, first rows), uneven SMs and the second kernel take 10 us.
//     570 instructions of a warp to 8 KB, 39 % of the issue slots; tensor cores busy 26 % of the time;
//   one of 65536 rows, 16 heads on 2: 12.9 us (5.0 at that rate); one of 2048 rows, 32 heads on 8: 6.0 us; both latency;
//   with 16 heads to a cache head, twice the products and weights to a byte, 113 us for the first of these: two CTAs an SM,
//     whose instructions wait for one another (41 % of the issue slots, tensor cores busy 41 % of the time).
// Where the rows come from matters more than how many are under way: the heads of a sequence take the same rows at the same
// time (shares of all heads together: 93 -> 87 us; pages of 512 rows instead of 64 gain 3 %), and one tile of a warp under
// way is faster than two (87 and 92 us, 12 warps to an SM; 8 warps of two tiles 95, 16 of one tile 95). Rows in registers, as
// k_attend_mma holds them, took 92 us, with 720 instructions to a tile: 24 shuffles of addresses, now read from shared
// memory, and loads of 16 bytes with a condition each, now asked only of tiles with a row that is not there.
#include <cuda_fp16.h>

#include <cfloat>

#include "kda_attend.cuh"

namespace kda {
namespace attend {
namespace {

// How large a weight, relative to the running maximum, may be before l and acc are rescaled; the power of two that one times
// its scale has in fp16 where it is at the running maximum of these; and the most that it may have.
constexpr float kMostP8 = 8.f;  // 2^3
constexpr int kTop8 = 11;
constexpr float kMost8 = 32768.f;  // of a weight in fp16, which holds 65504
// The least exponent of scaled weights that M follows (relative to m), so that 2^(m - M + kTop8) is 2^124 at most: times a
// weight of kMostP8 it is finite in fp32, also where all scales so far were 0 (infinity times a scale of 0 is a NaN). The
// largest scaled weight has all its bits from 2^-113 on.
constexpr int kLeast8 = kTop8 - 124;
constexpr float kNone8 = -FLT_MAX;  // of the maximum, before any score

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
// Two fp32 values to an instruction.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, const Two& b) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ Two operator+(Two a, const Two& b) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x) { return __half22float2(*(const __half2*)&x); }
// What two fp32 values are beyond two fp16 values. It is 16 at most (of kMost8), but for an infinite value, of which
// infinity - infinity is left: -64 in its place keeps it infinite.
__device__ __forceinline__ uint32_t rest_f16(float lo, float hi, uint32_t of) {
    const float2 y = unpack_f16(of);
    uint32_t x = pack_f16(lo - y.x, hi - y.y);
    asm("max.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xd400d400u));  // (of a NaN and a number: the number)
    return x;
}
// 2^x of a whole number x, 0 below 2^-126; x is at most 127. (-inf: 0)
__device__ __forceinline__ float power(float x) {
    return __int_as_float(((int)fmaxf(x, -127.f) + 127) << 23);
}
__device__ __forceinline__ float max_of_rows(float x) {
#pragma unroll
    for (int w = 4; w < 32; w *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
    return x;
}
// A warp's tile of 32 rows in shared memory: K8, V8, the scales of K and of V, and the addresses of the rows. The units of 16
// bytes of a row are permuted so that eight lanes that read together find all banks.
template <int K, int V> struct Tile {
    static constexpr int kScales = 32 * (K + V), kPlaces = kScales + 2 * 32 * 4, kWarp = kPlaces + 2 * 32 * 8,
                         kBytes = kWarps * kWarp;
    // K8: lanes read unit t of rows g; V8: unit g of rows 2 t
    __device__ __forceinline__ static int k_at(int row, int unit) {
        return row * K + (K == 128 ? unit ^ (row & 1) << 2 : unit) * 16;
    }
    __device__ __forceinline__ static int v_at(int row, int unit) {
        if constexpr (V == 128) return 32 * K + row * V + (unit ^ (row & 6)) * 16;
        return 32 * K + (row ^ (row >> 1 & 1)) * V + (unit ^ (row >> 1 & 2)) * 16;
    }
};
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void sts8(uint32_t at, const char* x) {
    asm volatile("st.shared.b64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}
// 16 or 4 bytes to shared memory; zeros if not `ok`.
__device__ __forceinline__ void fetch16(uint32_t to, const char* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void fetch16(uint32_t to, const char* from, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch4(uint32_t to, const float* from, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(ok ? 4 : 0) : "memory");
}
// The units of 16 bytes of a tile's rows, whose addresses lie at `places`, to where `at` says; rows that are not valid as
// zeros. D / 16 lanes to a row, and as many rows to a lane, whose addresses it reads two at a time.
template <int D, typename At> __device__ __forceinline__ void fetch_rows(uint32_t places, unsigned valid, At at) {
    constexpr int U = D / 16;
    const int lane = threadIdx.x % 32, unit = lane % U, first = lane / U * U;
    const auto address = [&](uint32_t lo, uint32_t hi) { return (const char*)((uint64_t)hi << 32 | lo) + unit * 16; };
    if (valid == 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < U; i += 2) {
            const uint4 x = lds16(places + (first + i) * 8);
            fetch16(at(first + i, unit), address(x.x, x.y));
            fetch16(at(first + i + 1, unit), address(x.z, x.w));
        }
    } else {
#pragma unroll
        for (int i = 0; i < U; i += 2) {
            const uint4 x = lds16(places + (first + i) * 8);
            fetch16(at(first + i, unit), address(x.x, x.y), valid >> (first + i) & 1);
            fetch16(at(first + i + 1, unit), address(x.z, x.w), valid >> (first + i + 1) & 1);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All groups but the newest N are there, of every lane.
template <int N> __device__ __forceinline__ void await() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
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
//   - lane 4 g + t has 16-byte units t, t + 4, .. of rows g, g + 8, .. of K8; four channels of two rows are one product's
//     share of the lane, and Q has the same order.
//   - of V8 it has V / 8 channels, from V / 8 g on, of rows 2 t, 2 t + 1, 2 t + 8, ..; a byte permutation pairs the rows,
//     and row i of the j-th product is channel V / 8 (i % 8) + j.
// The rows come through shared memory: K8 of the next tile is asked for once the scores of this one are there, V8 once its
// sums are.
template <typename TI, int K, int V, int NT, bool SHARES>
__global__ void __launch_bounds__(kWarps * 32, ctas8(NT, K, V)) k_attend8(AttendArgs a) {
    constexpr int KI = K / 64, CW = V / 8, VJ = V / 16, HT = 8 * NT, QP = sizeof(TI) / 2;
    typedef Tile<K, V> T;
    extern __shared__ uint4 shared[];
    Partial<HT, V>& sm = *(Partial<HT, V>*)shared;  // (once the rows are done with)
    __shared__ Inbox<HT, V> in;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    if (!SHARES && a.split == kCluster) cluster_started();
    after_previous();
    typedef Work<32, HT, SHARES, true, true> Wk;
    Wk wk;
    __shared__ typename Wk::Share share;
#pragma unroll 1
    for (bool more = wk.start(a, share); more; more = wk.next(a, share)) {
        const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
        Rows<32, true>& rows = wk.rows;
        const uint32_t tile = (uint32_t)__cvta_generic_to_shared(shared) + warp * T::kWarp;
        const char *kh = (const char*)a.c.k + wk.hkv * a.c.k_head, *vh = (const char*)a.c.v + wk.hkv * a.c.v_head;
        const float *ksh = a.k_scale + wk.hkv * a.ks_head, *vsh = a.v_scale + wk.hkv * a.vs_head;
        // the next tile: K8 and the scales, then V8
        auto fetch_k = [&]() {
            rows.next(a);
            const bool mine = rows.valid >> lane & 1;
            const uint32_t page = (uint32_t)rows.at, block = a.block(rows.at_off);
            const uint32_t places = tile + T::kPlaces, scale = tile + T::kScales + (4 * (lane % 8) + lane / 8) * 4;
            sts8(places + lane * 8, kh + rows.k_off);
            sts8(places + 256 + lane * 8, vh + rows.v_off);
            fetch4(scale, ksh + ((uint64_t)page * (uint64_t)a.ks_page + (uint64_t)block * (uint64_t)a.ks_block), mine);
            fetch4(scale + 128, vsh + ((uint64_t)page * (uint64_t)a.vs_page + (uint64_t)block * (uint64_t)a.vs_block), mine);
            __syncwarp();
            fetch_rows<K>(places, rows.valid, [&](int row, int unit) { return tile + T::k_at(row, unit); });
        };
        auto fetch_v = [&]() {
            fetch_rows<V>(tile + T::kPlaces + 256, rows.valid, [&](int row, int unit) { return tile + T::v_at(row, unit); });
        };
        fetch_k();
        fetch_v();
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
        // (M is held relative to m: scores may lie where fp32 has steps of more than one)
        float acc[NT][VJ][4], m[NT][2], l[NT][2], big[NT][2], pf[NT][2];  // big: M - m; pf: 2^(m - M + kTop8)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[j][e] = big[j][e] = kNone8;
                l[j][e] = pf[j][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VJ; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
        }
#pragma unroll 1
        for (int left = wk.left; left > 0; left -= a.step) {
            float s[NT][2][4];  // of rows g, g + 8 (and 16 more) and heads 2 t, 2 t + 1
            await<1>();
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) s[j][b][0] = s[j][b][1] = s[j][b][2] = s[j][b][3] = 0.f;
            // Products that follow one another go to different sums. How a tensor core rounds what it adds to a sum is not
            // specified, so the two parts of an fp32 query have sums of their own, joined by an fp32 addition: the median error
            // of 4000 drawn cases (1 to 65536 rows) fell from 4.0e-7 to 2.4e-7, and no time that was measured grew.
            float more[QP == 2 ? NT : 1][2][4];  // of the second parts of fp32 queries
            if constexpr (QP == 2) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) more[j][b][0] = more[j][b][1] = more[j][b][2] = more[j][b][3] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                uint32_t x[4][4];  // unit 4 i + t of rows g, g + 8, ..
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint4 y = lds16(tile + T::k_at(g + 8 * r, 4 * i + t));
                    x[r][0] = y.x, x[r][1] = y.y, x[r][2] = y.z, x[r][3] = y.w;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int c = 0; c < QP; ++c)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma_f16(c == 0 ? s[j][b] : more[QP == 2 ? j : 0][b], lower2(x[2 * b][w]), lower2(x[2 * b + 1][w]),
                                        upper2(x[2 * b][w]), upper2(x[2 * b + 1][w]), q[j][c][i][w][0], q[j][c][i][w][1]);
            }
            if constexpr (QP == 2) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[j][b][e] += more[j][b][e];
            }
            const uint4 k4 = lds16(tile + T::kScales + g * 16), v4 = lds16(tile + T::kScales + 128 + g * 16);
            const float kf[4] = {__uint_as_float(k4.x), __uint_as_float(k4.y), __uint_as_float(k4.z), __uint_as_float(k4.w)};
            const float vf[4] = {__uint_as_float(v4.x), __uint_as_float(v4.y), __uint_as_float(v4.z), __uint_as_float(v4.w)};
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float* x = s[j][r / 2] + 2 * (r % 2);
                    (Two(x[0], x[1]) * Two(qf[j][0], qf[j][1]) * Two(kf[r], kf[r])).get(x[0], x[1]);
                }
            if (rows.valid != 0xffffffffu) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!(rows.valid >> (g + 8 * r) & 1)) {
#pragma unroll
                        for (int j = 0; j < NT; ++j) s[j][r / 2][2 * (r % 2)] = s[j][r / 2][2 * (r % 2) + 1] = -INFINITY;
                    }
            }
            __syncwarp();  // (the tile's K8 and scales, and the last tile's places, are read)
            fetch_k();
            // weights (p), and what they are times the scales of V (w)
            float p[NT][4][2], w[NT][4][2], most_p = 0.f, most_w = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float* x = s[j][r / 2] + 2 * (r % 2);
                    float d[2];
                    (Two(x[0], x[1]) + Two(-m[j][0], -m[j][1])).get(d[0], d[1]);
                    p[j][r][0] = ex2(d[0]);
                    p[j][r][1] = ex2(d[1]);
                    (Two(p[j][r][0], p[j][r][1]) * Two(pf[j][0], pf[j][1]) * Two(vf[r], vf[r])).get(w[j][r][0], w[j][r][1]);
                    most_p = fmaxf(most_p, fmaxf(p[j][r][0], p[j][r][1]));
                    most_w = fmaxf(most_w, fmaxf(fabsf(w[j][r][0]), fabsf(w[j][r][1])));
                }
            if (__any_sync(0xffffffffu, most_p > kMostP8 || most_w > kMost8)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = -INFINITY, most = 0.f;
#pragma unroll
                        for (int r = 0; r < 4; ++r) top = fmaxf(top, s[j][r / 2][2 * (r % 2) + e]);
                        top = fmaxf(m[j][e], ceilf(max_of_rows(top)));
                        const float down = m[j][e] - top, was = big[j][e] + down;
                        l[j][e] *= power(down);
                        m[j][e] = top;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            p[j][r][e] = ex2(s[j][r / 2][2 * (r % 2) + e] - top);
                            most = fmaxf(most, fabsf(p[j][r][e] * vf[r]));
                        }
                        // 2^(exponent of `most`, rounded up)
                        const int up = ((__float_as_int(max_of_rows(most)) + 0x7fffff) >> 23) - 127;
                        const float to = fmaxf(was, (float)max(up, kLeast8)), f = power(was - to);
                        big[j][e] = to;
                        pf[j][e] = power(kTop8 - to);  // (to: kLeast8 to 128)
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
                    pt[j][0][r] = transpose8(hi);
                    pt[j][1][r] = transpose8(rest_f16(w[j][r][0], w[j][r][1], hi));
                }
            await<1>();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t vr[4][CW / 4];  // rows 16 b + 2 t, + 1, + 8, + 9
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * b + 2 * t + (r & 1) + 4 * (r & 2);
                    if constexpr (CW == 16) {
                        const uint4 x = lds16(tile + T::v_at(row, g));
                        vr[r][0] = x.x, vr[r][1] = x.y, vr[r][CW / 8] = x.z, vr[r][CW / 4 - 1] = x.w;
                    } else {
                        const uint2 x = lds8(tile + T::v_at(row, g / 2) + g % 2 * 8);
                        vr[r][0] = x.x, vr[r][1] = x.y;
                    }
                }
#pragma unroll
                for (int c = 0; c < VJ / 4; ++c) {
                    // four products: rows 0-7 of the j-th are channels CW g + j, rows 8-15 channels CW g + j + CW / 2
                    uint32_t x[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int word = c + (e & 1) * (VJ / 4);
                        const uint32_t even = vr[e & 2][word], odd = vr[(e & 2) + 1][word];
                        const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
                        x[0][e] = lower2(lo);
                        x[1][e] = upper2(lo);
                        x[2][e] = lower2(hi);
                        x[3][e] = upper2(hi);
                    }
                    if constexpr (QP == 2) {
                        // Sums of 16 rows, added to acc in fp32 and not by the tensor core, as above: the largest error of
                        // those cases fell from 2.4e-6 to 1.1e-6, for 1 % of the time with 4 heads to a cache head (4 % with 64
                        // channels) and 4 % with 16. bf16 queries have their sums run on in the tensor core, over all of a
                        // warp's rows: about 1e-5 of a sum over thousands of rows, where o's own rounding is 2^-9 to 2^-8 (of
                        // outputs over 4096 to 32768 rows 0.1 to 0.25 % are not the exact value's rounding; of sums in fp32
                        // at most 0.05 %).
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            float sum[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
#pragma unroll
                            for (int part = 1; part >= 0; --part)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_f16(sum[i], x[i][0], x[i][1], x[i][2], x[i][3], pt[j][part][2 * b], pt[j][part][2 * b + 1]);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[j][4 * c + i][e] += sum[i][e];
                        }
                    } else {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int j = 0; j < NT; ++j)
                                    mma_f16(acc[j][4 * c + i], x[i][0], x[i][1], x[i][2], x[i][3], pt[j][part][2 * b],
                                            pt[j][part][2 * b + 1]);
                    }
                }
            }
            __syncwarp();  // (the tile's V8 is read)
            fetch_v();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // (all rows are done with)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * j + 2 * t + e;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], d);
                if (g == 0) {
                    sm.m[warp][h] = m[j][e] == kNone8 ? -INFINITY : m[j][e];
                    sm.l[warp][h] = l[j][e] * kAtMostOne;
                }
                // relative to m as the join wants it, in two steps that fp32 holds
                const float apart = m[j][e] == kNone8 ? 0.f : big[j][e] - kTop8, half = rintf(0.5f * apart);
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
        join<TI, V, HT, SHARES, Wk>(a, share, sm, in);
        if constexpr (!SHARES) return;
        __syncthreads();  // the shared memory is free for the next unit
    }
}

template <typename TI, int K, int V> Kernel kernel_of(int ht, Split split) {
    if (split == kShares) return ht == 8 ? k_attend8<TI, K, V, 1, true> : k_attend8<TI, K, V, 2, true>;
    return ht == 8 ? k_attend8<TI, K, V, 1, false> : k_attend8<TI, K, V, 2, false>;
}
template <int K, int V> Kernel kernel_of(bool bf16, int ht, Split split) {
    return bf16 ? kernel_of<__nv_bfloat16, K, V>(ht, split) : kernel_of<float, K, V>(ht, split);
}
Kernel kernel_of(const kda_cache8& c, int ht, Split split) {
    const bool bf16 = c.dtype == KDA_DTYPE_BF16;
    const int K = c.cache.K, V = c.cache.V;
    return K == 128 ? (V == 128 ? kernel_of<128, 128>(bf16, ht, split) : kernel_of<128, 64>(bf16, ht, split))
                    : (V == 128 ? kernel_of<64, 128>(bf16, ht, split) : kernel_of<64, 64>(bf16, ht, split));
}

template <int K, int V> constexpr size_t shared8(int ht) {
    const size_t results = ht == 8 ? sizeof(Partial<8, V>) : sizeof(Partial<16, V>);
    return results > Tile<K, V>::kBytes ? results : Tile<K, V>::kBytes;
}
size_t shared8(int ht, int K, int V) {
    return K == 128 ? (V == 128 ? shared8<128, 128>(ht) : shared8<128, 64>(ht)) : (V == 128 ? shared8<64, 128>(ht) : shared8<64, 64>(ht));
}

}  // namespace

// (The kernels of a form are allowed the shared memory that they ask for once on each device.)
kda_status plan_for8(const kda_cache8* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks, Gpu gpu,
                     Plan& plan) {
    static std::atomic<int> known[2][2][2][2][kDevices];
    static std::atomic<bool> allowed[2][2][2][2][kDevices];
    kda_status s = check_cache(c);
    if (s == KDA_OK) s = check_sizes(&c->cache, HQ, N, max_pages, window, sinks);
    if (s != KDA_OK) return s;
    const int K = c->cache.K, V = c->cache.V, ht = HQ / c->cache.HKV <= 8 ? 8 : 16, device = present_device();
    const bool bf16 = c->dtype == KDA_DTYPE_BF16;
    // (the costs of the joins: fitted to times of all splits of 23,000 sizes, and on average 2 % above the best split)
    const Form form{ht, 32, ctas8(ht / 8, K, V), true, shared8(ht, K, V), true, 2.6, 1.4, 1.8, 2.7, 5.6};
    if (device >= 0) {
        std::atomic<bool>* done = device < kDevices ? &allowed[bf16][ht / 16][K / 128][V / 128][device] : nullptr;
        if (!done || !done->load(std::memory_order_relaxed)) {
            for (const Split split : {kCluster, kShares}) {
                const cudaError_t e = cudaFuncSetAttribute(kernel_of(*c, ht, split), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           (int)form.shared);
                if (e != cudaSuccess) return cuda_fail(e);
            }
            if (done) done->store(true, std::memory_order_relaxed);
        }
    }
    if (gpu.sms == 0)
        gpu = {sm_count(device), largest_cluster(device, (const void*)kernel_of(*c, ht, kCluster), kWarps * 32, kMaxCluster,
                                                 known[bf16][ht / 16][K / 128][V / 128], form.shared)};
    plan = plan_of(&c->cache, HQ, N, max_pages, window, sinks, form, gpu);
    return KDA_OK;
}

}  // namespace attend
}  // namespace kda

using namespace kda;
using namespace kda::attend;

extern "C" size_t kda_cache8_attend_workspace_bytes(const kda_cache8* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                    int32_t window, int32_t sinks) {
    Plan plan;
    return plan_for8(c, HQ, N, max_pages, window, sinks, Gpu{}, plan) == KDA_OK ? plan.ws_bytes : 0;
}

extern "C" kda_status kda_cache8_attend(const kda_cache8* c, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                        const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                        const int32_t* kv_lens, int32_t window, int32_t sinks, float scale, void* o,
                                        float* lse, int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream) {
    Plan plan;
    kda_status s = plan_for8(c, HQ, N, max_pages, window, sinks, Gpu{}, plan);
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
