// Kernels of attention over a paged cache in 16 or 32 bits.
#pragma once
#include "kda_attend.cuh"

namespace kda {
namespace attend {

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&b;
}
// The three parts of a weight above 0 are all above 0: the first two are cut off a little below what is left, not rounded.
// A part of 0, or one of the other sign, would make a NaN of an infinite value of V. What is left for the third part
// is less than 2^-13.9 of the weight, so rounding it loses 2^-21.9 at most. (Weights of 2^-100 and more keep to that.)
constexpr float kBelow = 1.f - 0x1p-12f;

// CTAs of k_attend_mma to an SM.
constexpr int mma_ctas(int NT, int K, int V) { return K + V == 128 ? 4 : 4 - NT; }

// Tensor-core kernel: a unit has up to 8 NT query heads, each warp a tile of 16 rows at a time. The products are taken
// transposed,
//   S^T [16 rows x 8 heads] = K Q^T,     O^T [V x 8 heads] += V^T P^T,
// so that the rows of the cache are the 16-row operand and a group's few heads the 8 columns. The cache goes from
// memory straight to the registers in which mma.sync wants it, with no copy in shared memory:
//   - lane 4 g + t loads 16-byte units t, t + 4, .. of rows g and g + 8 of K. The order of the channels within the
//     contraction is free as long as Q has the same.
//   - of V it loads unit g (and g + 8) of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9; a byte permutation pairs the rows, and
//     row i of the product is channel 8 (i % 8) + j of the j-th product.
//   - P^T comes from S^T by an 8 x 8 transposition in registers; it is split into three bf16 values, which hold the 24
//     bits of fp32. (With two of them, 16 to 18 bits, 646 of the 262144 outputs of 64 sequences of U[1,8192] rows were not
//     the exact result's rounding; with three 349, of elementary operations in fp32 225. The third product costs 0 to 3 %
//     where memory is the bound, 10 % where a CTA's few turns are, 4000 rows 8.3 -> 9.1 us, and 12 % with 9 to 16 heads
//     of K = V = 64.)
// Groups of 9 to 16 heads take two such columns of heads (NT = 2) at two CTAs an SM: reading the rows twice instead
// takes 81 us where this takes 51 (64 sequences of 8000 rows, 16 heads on one). K = V = 64 leaves registers for four CTAs
// (40 sequences of U[1,8000] rows, 16 heads on 16: 94.1 us; with five, which spill, 95.5; with three, whose rows under way
// are too few, 99.8. 128 of 1000 rows, eight heads on two: 14.4 and 16.2 us with four and five).
// A tensor core of the fifth generation wants its operands in shared memory and 128 rows in a product; here 8 to 16
// columns of the product are of use, and with the memory at its rate the tensor cores are busy 19 % of the time as it is.
template <int K, int V, int NT, bool SHARES, bool SINKS>
__global__ void __launch_bounds__(kWarps * 32, mma_ctas(NT, K, V)) k_attend_mma(AttendArgs a) {
    using TI = __nv_bfloat16;
    constexpr int KI = K / 32, VC = V / 64, VJ = V / 16, HT = 8 * NT;
    __shared__ Partial<HT, V> sm;
    __shared__ Inbox<HT, V> in;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    if (!SHARES && a.split == kCluster) cluster_started();
    after_previous();
    typedef Work<16, HT, SHARES, SINKS, SINKS> Wk;
    Wk wk;
    __shared__ typename Wk::Share share;
#pragma unroll 1
    for (bool more = wk.start(a, share); more; more = wk.next(a, share)) {
        const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
        Rows<16, SINKS>& rows = wk.rows;
        uint4 q[NT][KI];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < KI; ++i)
                q[j][i] = load16((const TI*)a.q + (int64_t)wk.n * a.q_stride + (h0 + 8 * j + g) * K + (4 * i + t) * 8,
                                 8 * j + g < heads);
        float acc[NT][VJ][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            m[j][0] = m[j][1] = -INFINITY;
            l[j][0] = l[j][1] = 0.f;
#pragma unroll
            for (int i = 0; i < VJ; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
        }
        const TI* kh = (const TI*)a.c.k + wk.hkv * a.c.k_head + t * 8;
        const TI* vh = (const TI*)a.c.v + wk.hkv * a.c.v_head + g * 8;
        uint4 kr[2][KI], vr[4][VC];
        auto load_k = [&]() {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const TI* p = kh + rows.k_of(g + 8 * r);
                const bool ok = rows.valid >> (g + 8 * r) & 1;
#pragma unroll
                for (int i = 0; i < KI; ++i) kr[r][i] = load16(p + 32 * i, ok);
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = 2 * t + (r & 1) + 4 * (r & 2);
                const TI* p = vh + rows.v_of(at);
                const bool ok = rows.valid >> at & 1;
#pragma unroll
                for (int i = 0; i < VC; ++i) vr[r][i] = load16(p + 64 * i, ok);
            }
        };
        rows.next(a);
        load_k();
        load_v();
#pragma unroll 1
        for (int left = wk.left; left > 0; left -= a.step) {
            float s[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float s1[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    mma(s[j], kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, q[j][i].x, q[j][i].y);
                    mma(s1, kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, q[j][i].z, q[j][i].w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] += s1[e];
            }
            const bool in0 = rows.valid >> g & 1, in1 = rows.valid >> (g + 8) & 1;
            rows.next(a);
            load_k();
            bool higher = false;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][e] = (e < 2 ? in0 : in1) ? s[j][e] * a.scale_log2 : -INFINITY;
                    higher |= s[j][e] > m[j][e & 1] + kSlack;
                }
            }
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(m[j][e], fmaxf(s[j][e], s[j][e + 2]));
#pragma unroll
                        for (int w = 4; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                        const float f = ex2(m[j][e] - finite_base(top));
                        m[j][e] = top;
                        l[j][e] *= f;
#pragma unroll
                        for (int i = 0; i < VJ; ++i) {
                            acc[j][i][e] *= f;
                            acc[j][i][e + 2] *= f;
                        }
                    }
            }
            uint32_t pt[NT][3][2];  // the parts of P^T
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float b0 = finite_base(m[j][0]), b1 = finite_base(m[j][1]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float p0 = ex2(s[j][2 * r] - b0) * kAtMostOne, p1 = ex2(s[j][2 * r + 1] - b1) * kAtMostOne;
                    l[j][0] += p0;
                    l[j][1] += p1;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t x = __byte_perm(__float_as_uint(p0 * kBelow), __float_as_uint(p1 * kBelow), 0x7632);
                        pt[j][c][r] = transpose8(x);
                        p0 -= __uint_as_float(x << 16);
                        p1 -= __uint_as_float(x & 0xffff0000u);
                    }
                    pt[j][2][r] = transpose8(pack(p0, p1));
                }
            }
#pragma unroll
            for (int i = 0; i < VJ; ++i) {
                // product i: rows 0-7 are channels 8 g + i (V = 64: 8 g + i), rows 8-15 channels 64 + 8 g + i (8 g + i + 4)
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = VC == 2 ? e & 1 : 0, j = VC == 2 ? i : i + 4 * (e & 1), r = e & 2;
                    const uint32_t* even = (const uint32_t*)&vr[r][c];
                    const uint32_t* odd = (const uint32_t*)&vr[r + 1][c];
                    x[e] = __byte_perm(even[j / 2], odd[j / 2], j % 2 ? 0x7632 : 0x5410);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int c = 0; c < 3; ++c) mma(acc[j][i], x[0], x[1], x[2], x[3], pt[j][c][0], pt[j][c][1]);
                }
            }
            load_v();
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * j + 2 * t + e;
#pragma unroll
                for (int w = 4; w < 32; w *= 2) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], w);
                if (g == 0) {
                    sm.m[warp][h] = m[j][e];
                    sm.l[warp][h] = l[j][e];
                }
                float* row = (float*)sm.acc[warp][h] + 8 * g;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < VJ; i += 4)
                        *(float4*)(row + (VC == 2 ? 64 : 4) * r + i) =
                            make_float4(acc[j][i][e + 2 * r], acc[j][i + 1][e + 2 * r], acc[j][i + 2][e + 2 * r],
                                        acc[j][i + 3][e + 2 * r]);
            }
        join<TI, V, HT, SHARES, Wk>(a, share, sm, in);
        if constexpr (!SHARES) return;
        __syncthreads();  // the shared memory is free for the next unit
    }
}

// ------------------------------------------------------------------ fp32

// CTAs of k_attend_simt to an SM, and rows of a warp's tile.
constexpr int simt_ctas(int HT, int K, int V) { return (HT == 1 ? 4 : 3) + (HT == 4 ? K + V < 256 : V == 64); }
constexpr int simt_rows(int ht) { return ht == 8 ? 4 : 8; }

// FFMA kernel (fp32): a unit has up to HT query heads, each warp R rows at a time, a
// lane holding K / 32 and V / 32 channels of each row and of every head. The R HT scores are sums over the lanes: a
// butterfly that halves the values with the lanes leaves value i, summed, in the lanes l with l % (R HT) == i.
// 8 sequences of U[1,8000] rows, K = V = 128: 16 heads on 16 99 us (102 at a plain copy's rate), on 4 32 us (25), 32 on
// 4 49 us (25): with eight heads the scores' sums over the lanes take as many issue slots as the products, and 48 KB of
// rows under way on an SM are too few to hide them.
template <int K, int V, int HT, int R, bool SINKS>
__global__ void __launch_bounds__(kWarps * 32, simt_ctas(HT, K, V)) k_attend_simt(AttendArgs a) {
    constexpr int KL = K / 32, VL = V / 32, NV = R * HT;
    __shared__ Partial<HT, V> sm;
    __shared__ Inbox<HT, V> in;
    const int lane = threadIdx.x % 32;
    if (a.split == kCluster) cluster_started();
    after_previous();
    typedef Work<R, HT, false, SINKS> Wk;
    Wk wk;
    __shared__ typename Wk::Share share;
    if (!wk.start(a, share)) return;
    const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
    Rows<R, SINKS>& rows = wk.rows;
    float q[HT][KL], acc[HT][VL];
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
        for (int i = 0; i < KL; ++i)
            q[h][i] = h < heads ? ((const float*)a.q)[(int64_t)wk.n * a.q_stride + (h0 + h) * K + lane * KL + i] : 0.f;
#pragma unroll
        for (int i = 0; i < VL; ++i) acc[h][i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;  // of head lane % HT
    const float* kh = (const float*)a.c.k + wk.hkv * a.c.k_head + lane * KL;
    const float* vh = (const float*)a.c.v + wk.hkv * a.c.v_head + lane * VL;
    float kr[R][KL], vr[R][VL];
    auto load_k = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) load_channels<KL>(kh + rows.k_of(r), rows.valid >> r & 1, kr[r]);
    };
    auto load_v = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) load_channels<VL>(vh + rows.v_of(r), rows.valid >> r & 1, vr[r]);
    };
    rows.next(a);
    load_k();
    load_v();
#pragma unroll 1
    for (int left = wk.left; left > 0; left -= a.step) {
        float s[NV];  // value r HT + h
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                s[r * HT + h] = q[h][0] * kr[r][0];
#pragma unroll
                for (int i = 1; i < KL; ++i) s[r * HT + h] = fmaf(q[h][i], kr[r][i], s[r * HT + h]);
            }
        const bool in = rows.valid >> (lane % NV / HT) & 1;
        rows.next(a);
        load_k();
#pragma unroll
        for (int w = NV / 2; w > 0; w /= 2)
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float mine = lane & w ? s[i + w] : s[i], other = lane & w ? s[i] : s[i + w];
                s[i] = mine + __shfl_xor_sync(0xffffffffu, other, w);
            }
#pragma unroll
        for (int w = NV; w < 32; w *= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], w);
        const float score = in ? s[0] * a.scale_log2 : -INFINITY;
        if (__any_sync(0xffffffffu, score > m + kSlack)) {
            float top = fmaxf(m, score);
#pragma unroll
            for (int w = HT; w < NV; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float f = exp2f(m - finite_base(top));
            m = top;
            l *= f;
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float fh = __shfl_sync(0xffffffffu, f, h);
#pragma unroll
                for (int i = 0; i < VL; ++i) acc[h][i] *= fh;
            }
        }
        const float p = ex2(score - finite_base(m)) * kAtMostOne;
        l += p;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float ph = __shfl_sync(0xffffffffu, p, r * HT + h);
#pragma unroll
                for (int i = 0; i < VL; ++i) acc[h][i] = fmaf(ph, vr[r][i], acc[h][i]);
            }
        load_v();
    }
#pragma unroll
    for (int w = HT; w < NV; w *= 2) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (lane < HT) {
        sm.m[warp][lane] = m;
        sm.l[warp][lane] = l;
    }
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < VL; ++i) ((float*)sm.acc[warp][h])[lane * VL + i] = acc[h][i];
    join<float, V, HT, false, Wk>(a, share, sm, in);
}

// ------------------------------------------------------------------ which

template <int K, int V, bool SINKS> Kernel kernel_of(bool bf16, int ht, Split split) {
    if (bf16 && split == kShares) return ht == 8 ? k_attend_mma<K, V, 1, true, SINKS> : k_attend_mma<K, V, 2, true, SINKS>;
    if (bf16) return ht == 8 ? k_attend_mma<K, V, 1, false, SINKS> : k_attend_mma<K, V, 2, false, SINKS>;
    return ht == 1   ? k_attend_simt<K, V, 1, simt_rows(1), SINKS>
           : ht == 4 ? k_attend_simt<K, V, 4, simt_rows(4), SINKS>
                     : k_attend_simt<K, V, 8, simt_rows(8), SINKS>;
}
template <bool SINKS> Kernel kernel_of(const kda_cache& c, int ht, Split split) {
    const bool bf16 = c.dtype == KDA_DTYPE_BF16;
    return c.K == 128 ? (c.V == 128 ? kernel_of<128, 128, SINKS>(bf16, ht, split) : kernel_of<128, 64, SINKS>(bf16, ht, split))
                      : (c.V == 128 ? kernel_of<64, 128, SINKS>(bf16, ht, split) : kernel_of<64, 64, SINKS>(bf16, ht, split));
}

}  // namespace attend
}  // namespace kda
