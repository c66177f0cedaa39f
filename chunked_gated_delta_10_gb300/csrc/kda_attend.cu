// kda_cache_attend: attention of one new token per sequence over a paged
// cache. Declared in include/kda_serve.h.
//
// One pass over the cached rows with the running maximum m and sum l of the
// softmax (in log2 units): a row's score s raises m to m' = max(m, s), and
//   l <- l 2^(m - m') + 2^(s - m'),   acc <- acc 2^(m - m') + 2^(s - m') V.
// Partial results over disjoint rows join by the same rule.
//
// Bound: the cached keys and values are read once.
#include "kda_cache.cuh"

namespace kda {
namespace {

struct AttendArgs {
    kda_cache c;
    const void* q;
    int64_t q_stride, table_stride;
    int HQ, N, max_pages, window;
    const int32_t *table, *kv_lens;
    float scale_log2;
    void* o;
    float* lse;
    int32_t* status;
    int cluster, slices;  // CTAs of a slice, slices of a sequence's rows
    float* part_acc;      // [N, HQ, slices, V]: each slice's weighted sum, relative to its maximum
    float2* part_ml;      // [N, HQ, slices]: its maximum (log2 units) and its sum of weights
};

// The rows [begin, end) that sequence n attends.
__device__ __forceinline__ void kv_range(const AttendArgs& a, int64_t n, int& begin, int& end) {
    const int64_t len = a.kv_lens[n], room = (int64_t)a.max_pages * a.c.page_size;
    if (len > room && a.status && threadIdx.x == 0) *a.status = KDA_ERR_INVALID_ARG;
    begin = a.window > 0 && len > a.window ? (int)(len - a.window) : 0;
    end = (int)max(min(len, room), (int64_t)0);
}

// The value that exponents are taken relative to: the maximum, or 0 where no score is above -inf, so that a
// weight there is 2^-inf = 0 and a NaN score stays a NaN.
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

#ifndef WANT
#define WANT (152 * 12)
#endif
#ifndef MAXC
#define MAXC 8
#endif
#ifndef SLICE_ROWS
#define SLICE_ROWS 512
#endif
constexpr int kWarps = 4;
constexpr int kMaxCluster = MAXC;
constexpr int kPartRows = 64;  // a part's rows are a multiple: a tile of 16 for each warp

// ------------------------------------------------------------------ split
//
// The rows of a sequence are cut into equal parts, a CTA each. `cluster` neighbouring parts are a slice: a cluster of
// CTAs that join their results in shared memory. Where a sequence has more than one slice in use, each leaves its
// result in the workspace and a second kernel joins those. How many parts and slices there are is the host's choice (it
// knows the sizes but not the lengths); how a sequence's own rows fill them follows from its length on the device.

// Rows [lo, hi) of part s, and the number of parts that hold any.
__device__ __forceinline__ int part_rows(int begin, int end, int parts, int s, int& lo, int& hi) {
    const int len = end - begin;
    int per = (len + parts - 1) / parts;
    per = (max(per, 1) + kPartRows - 1) / kPartRows * kPartRows;
    lo = (int)min(begin + (int64_t)s * per, (int64_t)end);
    hi = (int)min((int64_t)lo + per, (int64_t)end);
    return max((len + per - 1) / per, 1);
}

// ------------------------------------------------------------------ rows of a tile
//
// R rows in a warp's tile: lane l looks up row l % R. Pages may be of any size, so every row has its own; the lookup
// of the next tile's pages is in flight while a tile is computed.
template <int R> struct Rows {
    const int32_t* table;
    int hi, row, pg, off, page;      // the next tile's row of this lane
    int step_pg, step_off, step;
    int64_t k_off, v_off;            // this tile's row of this lane
    unsigned valid;                  // bit r: row r is in range and its page exists

    __device__ __forceinline__ Rows(const AttendArgs& a, int64_t n, int lo, int hi_, int stride)
        : table(a.table + n * a.table_stride), hi(hi_), row(lo + threadIdx.x % 32 % R), step(stride) {
        pg = row / a.c.page_size;
        off = row - pg * a.c.page_size;
        step_pg = stride / a.c.page_size;
        step_off = stride - step_pg * a.c.page_size;
        page = row < hi ? table[pg] : -1;
    }
    __device__ __forceinline__ void next(const AttendArgs& a, int hkv) {
        const bool in = row < hi, ok = (unsigned)page < (unsigned)a.c.num_pages;
        if (in && !ok && a.status) *a.status = KDA_ERR_INVALID_ARG;
        valid = __ballot_sync(0xffffffffu, ok);
        const int64_t p = ok ? page : 0;
        k_off = p * a.c.k_page + off * a.c.k_row;
        v_off = p * a.c.v_page + off * a.c.v_row;
        row += step;
        pg += step_pg;
        off += step_off;
        if (off >= a.c.page_size) {
            off -= a.c.page_size;
            ++pg;
        }
        page = row < hi ? table[pg] : -1;
    }
    __device__ __forceinline__ int64_t k_of(int r) const { return __shfl_sync(0xffffffffu, k_off, r); }
    __device__ __forceinline__ int64_t v_of(int r) const { return __shfl_sync(0xffffffffu, v_off, r); }
};

__device__ __forceinline__ uint4 load16(const void* p, bool ok) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (ok) x = __ldcs((const uint4*)p);
    return x;
}

template <int C> __device__ __forceinline__ void load_channels(const float* p, bool ok, float (&x)[C]) {
    if constexpr (C == 4) {
        const float4 y = ok ? __ldcs((const float4*)p) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    } else {
        const float2 y = ok ? __ldcs((const float2*)p) : make_float2(0.f, 0.f);
        x[0] = y.x, x[1] = y.y;
    }
}

// ------------------------------------------------------------------ joins

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The value at shared-memory address p of this cluster's CTA `rank`.
__device__ __forceinline__ float load_of(const float* p, uint32_t rank) {
    uint32_t at;
    float x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}

// The results of a CTA's warps for HT heads: maxima m, sums of weights l, and weighted sums acc relative to m.
template <int HT, int V> struct Partial {
    float m[kWarps][HT], l[kWarps][HT], acc[kWarps][HT][V + 4];
    float cta_m[HT], cta_l[HT];
};

// Joins the warps of a CTA, then the CTAs of its cluster, and writes the result for `heads` heads: the operator's, or,
// where the sequence has more than one slice in use, this slice's. The order of the sums is fixed.
template <typename TI, int V, int HT>
__device__ __forceinline__ void join_slice(const AttendArgs& a, int64_t n, int h0, int heads, int slice, int slices_used,
                                           Partial<HT, V>& p) {
    auto write = [&](int h, int d, float m, float l, float x) {
        const int64_t at = n * a.HQ + h0 + h;
        if (slices_used == 1) {
            ((TI*)a.o)[at * V + d] = from_f<TI>(l == 0.f ? 0.f : x / l);
            if (d == 0 && a.lse) a.lse[at] = (finite_base(m) + log2f(l)) * kLn2;
        } else {
            a.part_acc[(at * a.slices + slice) * V + d] = x;
            if (d == 0) a.part_ml[at * a.slices + slice] = make_float2(m, l);
        }
    };
    __syncthreads();
    for (int i = threadIdx.x; i < heads * V; i += kWarps * 32) {
        const int h = i / V, d = i % V;
        float m = p.m[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, p.m[w][h]);
        const float base = finite_base(m);
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(p.m[w][h] - base);
            l = fmaf(p.l[w][h], f, l);
            x = fmaf(p.acc[w][h][d], f, x);
        }
        if (a.cluster == 1) {
            write(h, d, m, l, x);
        } else {
            p.acc[0][h][d] = x;  // read by this thread only, above
            if (d == 0) {
                p.cta_m[h] = m;
                p.cta_l[h] = l;
            }
        }
    }
    if (a.cluster == 1) return;
    cluster_sync();
    const int rank = blockIdx.x % a.cluster;
    for (int i = rank * kWarps * 32 + threadIdx.x; i < heads * V; i += a.cluster * kWarps * 32) {
        const int h = i / V, d = i % V;
        float mc[kMaxCluster], m = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            mc[c] = c < a.cluster ? load_of(&p.cta_m[h], c) : -INFINITY;
            m = fmaxf(m, mc[c]);
        }
        const float base = finite_base(m);
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c < a.cluster) {
                const float f = exp2f(mc[c] - base);
                l = fmaf(load_of(&p.cta_l[h], c), f, l);
                x = fmaf(load_of(&p.acc[0][h][d], c), f, x);
            }
        }
        write(h, d, m, l, x);
    }
    cluster_sync();  // the others may still read this CTA's shared memory
}

// The slices of one query head, joined in order.
template <typename TI, int V>
__global__ void __launch_bounds__(128) k_attend_join(AttendArgs a) {
    constexpr int G = 128 / (V / 4);  // groups of threads, each taking every G-th part
    __shared__ float4 sx[G][V / 4];
    __shared__ float sl[G];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t at = blockIdx.x, n = at / a.HQ;
    int begin, end, lo, hi;
    kv_range(a, n, begin, end);
    const int used = (part_rows(begin, end, a.cluster * a.slices, 0, lo, hi) + a.cluster - 1) / a.cluster;
    if (used == 1) return;
    const float2* ml = a.part_ml + at * a.slices;
    float m = -INFINITY;
    for (int s = threadIdx.x % 32; s < used; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int w = 16; w > 0; w /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float base = finite_base(m);
    const int g = threadIdx.x / (V / 4), c = threadIdx.x % (V / 4);
    const float4* acc = (const float4*)(a.part_acc + at * a.slices * V) + c;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int s = g; s < used; s += G) {
        const float2 e = ml[s];
        const float4 y = acc[s * (V / 4)];
        const float f = exp2f(e.x - base);
        l = fmaf(e.y, f, l);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
    }
    sx[g][c] = x;
    if (c == 0) sl[g] = l;
    __syncthreads();
    if (threadIdx.x < V) {
        const int d = threadIdx.x;
        float total = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            total += sl[i];
            y += ((const float*)&sx[i][d / 4])[d % 4];
        }
        ((TI*)a.o)[at * V + d] = from_f<TI>(total == 0.f ? 0.f : y / total);
        if (d == 0 && a.lse) a.lse[at] = (base + log2f(total)) * kLn2;
    }
}

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values (lane 4 i + j holds columns 2 j, 2 j + 1 of row i), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&b;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How far above the running maximum a score may lie (log2 units) before acc and l are rescaled: up to 2^8 is no loss
// in fp32 or in a pair of bf16 values, and most tiles then only ask whether any score is higher.
constexpr float kSlack = 8.f;

// Tensor-core kernel: one CTA per (part, up to 8 NT query heads of one cache head, sequence), each warp a tile of 16
// rows at a time. The products are taken transposed,
//   S^T [16 rows x 8 heads] = K Q^T,     O^T [V x 8 heads] += V^T P^T,
// so that the rows of the cache are the 16-row operand and a group's few heads the 8 columns. The cache goes from
// memory straight to the registers in which mma.sync wants it, with no copy in shared memory:
//   - lane 4 g + t loads 16-byte units t, t + 4, .. of rows g and g + 8 of K. The order of the channels within the
//     contraction is free as long as Q has the same.
//   - of V it loads unit g (and g + 8) of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9; a byte permutation pairs the rows, and
//     row i of the product is channel 8 (i % 8) + j of the j-th product.
//   - P^T comes from S^T by an 8 x 8 transposition in registers; it is split into a pair of bf16 values (2^-16).
// A tensor core of the fifth generation wants its operands in shared memory and 128 rows in a product; with at most 16
// query heads against it, the memory's time would cover none of that traffic.
template <int K, int V, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) k_attend_mma(AttendArgs a) {
    using TI = __nv_bfloat16;
    constexpr int KI = K / 32, VC = V / 64, VJ = V / 16, HT = 8 * NT;
    __shared__ Partial<HT, V> sm;
    const int parts = a.cluster * a.slices, part = blockIdx.x % parts, slice = part / a.cluster;
    const int group = a.HQ / a.c.HKV, tiles = (group + HT - 1) / HT;
    const int64_t unit = blockIdx.x / parts, n = unit / (a.c.HKV * tiles);
    const int hkv = (int)(unit / tiles % a.c.HKV), qt = (int)(unit % tiles);
    const int h0 = hkv * group + qt * HT, heads = min(HT, group - qt * HT);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    int begin, end, lo, hi;
    kv_range(a, n, begin, end);
    const int used = part_rows(begin, end, parts, part, lo, hi);
    asm volatile("griddepcontrol.launch_dependents;");
    if (slice * a.cluster >= used) return;  // so does the whole cluster

    uint4 q[NT][KI];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < KI; ++i)
            q[j][i] = load16((const TI*)a.q + n * a.q_stride + (h0 + 8 * j + g) * K + (4 * i + t) * 8, 8 * j + g < heads);
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
    const TI* kh = (const TI*)a.c.k + hkv * a.c.k_head + t * 8;
    const TI* vh = (const TI*)a.c.v + hkv * a.c.v_head + g * 8;
    uint4 kr[2][KI], vr[4][VC];
    Rows<16> rows(a, n, lo + warp * 16, hi, kWarps * 16);
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
    rows.next(a, hkv);
    load_k();
    load_v();
    for (int first = lo + warp * 16; first < hi; first += kWarps * 16) {
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                mma(s[j], kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, q[j][i].x, q[j][i].y);
                mma(s[j], kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, q[j][i].z, q[j][i].w);
            }
        }
        const bool in0 = rows.valid >> g & 1, in1 = rows.valid >> (g + 8) & 1;
        rows.next(a, hkv);
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
        uint32_t hi_p[NT][2], lo_p[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float b0 = finite_base(m[j][0]), b1 = finite_base(m[j][1]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float p0 = ex2(s[j][2 * r] - b0), p1 = ex2(s[j][2 * r + 1] - b1);
                l[j][0] += p0;
                l[j][1] += p1;
                const uint32_t h = pack(p0, p1);
                hi_p[j][r] = transpose8(h);
                lo_p[j][r] = transpose8(pack(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u)));
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
                mma(acc[j][i], x[0], x[1], x[2], x[3], hi_p[j][0], hi_p[j][1]);
                mma(acc[j][i], x[0], x[1], x[2], x[3], lo_p[j][0], lo_p[j][1]);
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
            float* row = &sm.acc[warp][h][8 * g];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < VJ; i += 4)
                    *(float4*)(row + (VC == 2 ? 64 : 4) * r + i) =
                        make_float4(acc[j][i][e + 2 * r], acc[j][i + 1][e + 2 * r], acc[j][i + 2][e + 2 * r],
                                    acc[j][i + 3][e + 2 * r]);
        }
    join_slice<TI, V, HT>(a, n, h0, heads, slice, (used + a.cluster - 1) / a.cluster, sm);
}

// ------------------------------------------------------------------ fp32

// FFMA kernel: one CTA per (part, up to HT query heads of one cache head, sequence), each warp R rows at a time, a
// lane holding K / 32 and V / 32 channels of each row and of every head. The R HT scores are sums over the lanes: a
// butterfly that halves the values with the lanes leaves value i, summed, in the lanes l with l % (R HT) == i.
template <int K, int V, int HT, int R>
__global__ void __launch_bounds__(kWarps * 32) k_attend_simt(AttendArgs a) {
    constexpr int KL = K / 32, VL = V / 32, NV = R * HT;
    __shared__ Partial<HT, V> sm;
    const int parts = a.cluster * a.slices, part = blockIdx.x % parts, slice = part / a.cluster;
    const int group = a.HQ / a.c.HKV, tiles = (group + HT - 1) / HT;
    const int64_t unit = blockIdx.x / parts, n = unit / (a.c.HKV * tiles);
    const int hkv = (int)(unit / tiles % a.c.HKV), qt = (int)(unit % tiles);
    const int h0 = hkv * group + qt * HT, heads = min(HT, group - qt * HT);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int begin, end, lo, hi;
    kv_range(a, n, begin, end);
    const int used = part_rows(begin, end, parts, part, lo, hi);
    asm volatile("griddepcontrol.launch_dependents;");
    if (slice * a.cluster >= used) return;  // so does the whole cluster

    float q[HT][KL], acc[HT][VL];
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
        for (int i = 0; i < KL; ++i)
            q[h][i] = h < heads ? ((const float*)a.q)[n * a.q_stride + (h0 + h) * K + lane * KL + i] : 0.f;
#pragma unroll
        for (int i = 0; i < VL; ++i) acc[h][i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;  // of head lane % HT
    const float* kh = (const float*)a.c.k + hkv * a.c.k_head + lane * KL;
    const float* vh = (const float*)a.c.v + hkv * a.c.v_head + lane * VL;
    float kr[R][KL], vr[R][VL];
    Rows<R> rows(a, n, lo + warp * R, hi, kWarps * R);
    auto load_k = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) load_channels<KL>(kh + rows.k_of(r), rows.valid >> r & 1, kr[r]);
    };
    auto load_v = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) load_channels<VL>(vh + rows.v_of(r), rows.valid >> r & 1, vr[r]);
    };
    rows.next(a, hkv);
    load_k();
    load_v();
    for (int first = lo + warp * R; first < hi; first += kWarps * R) {
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
        rows.next(a, hkv);
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
        const float p = exp2f(score - finite_base(m));
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
        for (int i = 0; i < VL; ++i) sm.acc[warp][h][lane * VL + i] = acc[h][i];
    join_slice<float, V, HT>(a, n, h0, heads, slice, (used + a.cluster - 1) / a.cluster, sm);
}

// ------------------------------------------------------------------ launch

// Query heads that a CTA takes together.
int head_tile(const kda_cache* c, int HQ) {
    const int group = HQ / c->HKV;
    if (c->dtype == KDA_DTYPE_BF16) return group <= 8 ? 8 : 16;
    return group == 1 ? 1 : group <= 4 ? 4 : 8;
}

// The split of each sequence's rows: CTAs to a cluster, and clusters.
struct Plan {
    int cluster, slices;
};
Plan plan_of(const kda_cache* c, int HQ, int N, int max_pages, int window) {
    const int group = HQ / c->HKV, ht = head_tile(c, HQ);
    const int64_t units = (int64_t)(N > 0 ? N : 1) * c->HKV * ((group + ht - 1) / ht);
    int64_t rows = (int64_t)max_pages * c->page_size;
    if (window > 0 && window < rows) rows = window;
    const int64_t most = (rows + kPartRows - 1) / kPartRows, want = (WANT + units - 1) / units;
    Plan p{1, 1};
    while (p.cluster < kMaxCluster && p.cluster < want && p.cluster < most) p.cluster *= 2;
    int64_t slices = want / p.cluster;
    const int64_t fill = rows / ((int64_t)p.cluster * SLICE_ROWS);
    if (slices > fill) slices = fill;
    if (slices > 1) p.slices = (int)slices;
    return p;
}

cudaError_t launch_in(void (*kernel)(AttendArgs), const AttendArgs& a, unsigned grid, int cluster, bool after,
                      cudaStream_t st) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (after) {  // may be set up while the kernel before it runs; it waits for that one's end itself
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    if (cluster > 8) {
        const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

typedef void (*Kernel)(AttendArgs);

template <int K, int V> Kernel kernel_of(bool bf16, int ht) {
    if (bf16) return ht == 8 ? k_attend_mma<K, V, 1> : k_attend_mma<K, V, 2>;
    return ht == 1 ? k_attend_simt<K, V, 1, 8> : ht == 4 ? k_attend_simt<K, V, 4, 8> : k_attend_simt<K, V, 8, 4>;
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    const bool bf16 = a.c.dtype == KDA_DTYPE_BF16;
    const int ht = head_tile(&a.c, a.HQ), group = a.HQ / a.c.HKV, K = a.c.K, V = a.c.V;
    const unsigned grid = (unsigned)((int64_t)a.N * a.c.HKV * ((group + ht - 1) / ht) * a.cluster * a.slices);
    const Kernel kernel = K == 128 ? (V == 128 ? kernel_of<128, 128>(bf16, ht) : kernel_of<128, 64>(bf16, ht))
                                   : (V == 128 ? kernel_of<64, 128>(bf16, ht) : kernel_of<64, 64>(bf16, ht));
    cudaError_t e = launch_in(kernel, a, grid, a.cluster, false, st);
    if (e != cudaSuccess) return e;
    note_launch("cache_attend", st);
    if (a.slices == 1) return cudaSuccess;
    const Kernel join = bf16 ? (V == 128 ? k_attend_join<__nv_bfloat16, 128> : k_attend_join<__nv_bfloat16, 64>)
                             : (V == 128 ? k_attend_join<float, 128> : k_attend_join<float, 64>);
    if ((e = launch_in(join, a, (unsigned)((int64_t)a.N * a.HQ), 1, true, st)) != cudaSuccess) return e;
    note_launch("cache_attend_join", st);
    return cudaSuccess;
}

kda_status check_sizes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window) {
    const kda_status s = check_cache(c);
    if (s != KDA_OK) return s;
    if (N < 0 || HQ < 1 || HQ % c->HKV != 0 || max_pages < 0 || window < 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)N * HQ > INT32_MAX || (int64_t)max_pages * c->page_size > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_cache_attend_workspace_bytes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                   int32_t window) {
    if (check_sizes(c, HQ, N, max_pages, window) != KDA_OK) return 0;
    const int64_t slices = plan_of(c, HQ, N, max_pages, window).slices;
    return slices == 1 ? 256 : 256 + (size_t)N * HQ * slices * ((size_t)c->V * sizeof(float) + sizeof(float2));
}

extern "C" kda_status kda_cache_attend(const kda_cache* c, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                       const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                       const int32_t* kv_lens, int32_t window, float scale, void* o, float* lse,
                                       int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream) {
    const kda_status s = check_sizes(c, HQ, N, max_pages, window);
    if (s != KDA_OK) return s;
    const int64_t unit = c->dtype == KDA_DTYPE_BF16 ? 8 : 4;
    if (q_stride < (int64_t)HQ * c->K || q_stride % unit || table_stride < 0) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    if (!q || !o || !kv_lens || (!page_table && max_pages > 0)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || ((uintptr_t)lse & 3u) || ((uintptr_t)page_table & 3u) ||
        ((uintptr_t)kv_lens & 3u) || ((uintptr_t)status & 3u))
        return KDA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws) || ws_bytes < kda_cache_attend_workspace_bytes(c, HQ, N, max_pages, window))
        return KDA_ERR_WORKSPACE;
    const Plan plan = plan_of(c, HQ, N, max_pages, window);
    AttendArgs a{*c, q, q_stride, table_stride, HQ, N, max_pages, window, page_table, kv_lens, scale * kLog2e, o, lse,
                 status, plan.cluster, plan.slices, nullptr, nullptr};
    a.part_acc = (float*)ws;
    a.part_ml = (float2*)(a.part_acc + (int64_t)N * HQ * a.slices * c->V);
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const cudaError_t e = launch_attend(a, st);
    if (e != cudaSuccess) return cuda_fail(e);
    return KDA_OK;
}
