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

#ifdef TUNE
#include <stdlib.h>
#endif
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
    int parts;        // CTAs over a sequence's rows
    int cluster;      // whether the parts of a sequence are a cluster of CTAs, which joins them
    int turn;         // rows that a CTA takes at a time
    float* part_acc;  // [N, HQ, parts, V]: each part's weighted sum, relative to its maximum
    float2* part_ml;  // [N, HQ, parts]: its maximum (log2 units) and its sum of weights
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

// ------------------------------------------------------------------ split
//
// A CTA takes W R rows at a time, R for each of its W warps, and the CTAs of a sequence, its parts, take them in turn:
// CTA i the turns i, i + parts, .. So parts are equal whatever the length, and the first rows of a CTA do not depend on
// it: their pages are looked up while the length is on its way. Where a sequence has more than one part in use, each
// leaves its result in the workspace and a second kernel joins those. How many parts there are is the host's choice (it
// knows the sizes but not the lengths).

constexpr int kMaxCluster = 16;

// The parts of a sequence that hold any rows (one at least, which writes the result of a sequence without).
__device__ __forceinline__ int parts_used(const AttendArgs& a, int rows, int turn) {
    return max(1, min(a.parts, (rows + turn - 1) / turn));
}

// ------------------------------------------------------------------ rows of a tile
//
// R rows in a warp's tile: lane l looks up row l % R. Pages may be of any size, so every row has its own; the lookup
// of the next tile's pages is in flight while a tile is computed.
template <int R> struct Rows {
    const int32_t* table;
    int end, row, pg, off, page;     // the next tile's row of this lane
    int step_pg, step_off, step;
    int64_t k_off, v_off;            // this tile's row of this lane
    unsigned valid;                  // bit r: row r is in range and its page exists

    // Rows from `first` on, `stride` apart; without a window neither depends on the sequence's length.
    __device__ __forceinline__ void start(const AttendArgs& a, int64_t n, int first, int stride) {
        table = a.table + n * a.table_stride;
        row = first + threadIdx.x % 32 % R;
        step = stride;
        pg = (unsigned)row / (unsigned)a.c.page_size;
        off = row - pg * a.c.page_size;
        step_pg = (unsigned)stride / (unsigned)a.c.page_size;
        step_off = stride - step_pg * a.c.page_size;
        page = pg < a.max_pages ? __ldg(table + pg) : -1;
    }
    __device__ __forceinline__ void next(const AttendArgs& a) {
        const bool in = row < end, ok = in && (unsigned)page < (unsigned)a.c.num_pages;
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
        page = row < end ? __ldg(table + pg) : -1;
    }
    __device__ __forceinline__ int64_t k_of(int r) const { return __shfl_sync(0xffffffffu, k_off, r); }
    __device__ __forceinline__ int64_t v_of(int r) const { return __shfl_sync(0xffffffffu, v_off, r); }
};

// What a CTA works on, and the rows of this warp: the first lookup is issued before the length is read.
template <int W, int R, int HT> struct Work {
    int64_t n;
    int hkv, h0, heads, part, used, warp, first, end;
    Rows<R> rows;

    __device__ __forceinline__ bool start(const AttendArgs& a) {
        const unsigned parts = a.parts, unit = blockIdx.x / parts;
        const unsigned group = (unsigned)a.HQ / a.c.HKV, tiles = (group + HT - 1) / HT, per = a.c.HKV * tiles;
        const unsigned qt = unit % tiles;
        n = unit / per;
        hkv = unit / tiles % a.c.HKV;
        h0 = hkv * group + qt * HT;
        heads = min(HT, (int)(group - qt * HT));
        part = blockIdx.x % parts;
        warp = threadIdx.x / 32;
        first = (part * W + warp) * R;
        rows.start(a, n, first, parts * W * R);
        int begin;
        kv_range(a, n, begin, end);
        if (begin > 0) {
            first += begin;
            rows.start(a, n, first, parts * W * R);
        }
        rows.end = end;
        used = parts_used(a, end - begin, W * R);
        return part < used;
    }
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address in the cluster's CTA `rank` of what has address p here.
__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return at;
}
__device__ __forceinline__ void push(float4* p, uint32_t rank, float4 x) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_address(p, rank)), "f"(x.x), "f"(x.y),
                 "f"(x.z), "f"(x.w)
                 : "memory");
}
__device__ __forceinline__ void push(float2* p, uint32_t rank, float2 x) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_address(p, rank)), "f"(x.x), "f"(x.y) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void add_scaled(float4& x, const float4& y, float f) {
    x.x = fmaf(y.x, f, x.x);
    x.y = fmaf(y.y, f, x.y);
    x.z = fmaf(y.z, f, x.z);
    x.w = fmaf(y.w, f, x.w);
}
// Channels d .. d + 3 of a query head's result.
template <typename TI> __device__ __forceinline__ void write_result(const AttendArgs& a, int64_t at, int V, int d, float m,
                                                                    float l, float4 x) {
    const float f = l == 0.f ? 0.f : 1.f / l;  // nothing attended: x is 0
    TI* o = (TI*)a.o + at * V + d;
    if constexpr (sizeof(TI) == 2) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * f, x.y * f), hi = __floats2bfloat162_rn(x.z * f, x.w * f);
        *(uint2*)o = make_uint2(*(const uint32_t*)&lo, *(const uint32_t*)&hi);
    } else {
        *(float4*)o = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    }
    if (d == 0 && a.lse) a.lse[at] = (finite_base(m) + log2f(l)) * kLn2;
}

// The results of a CTA's warps for HT heads: maxima m, sums of weights l, and weighted sums acc relative to m. In a
// cluster: what its CTAs send of the channels that this one joins, and of every head their m and l.
template <int W, int HT, int V> struct Partial {
    float m[W][HT], l[W][HT];
    float4 acc[W][HT][V / 4 + 1];
    float4 in_acc[HT * V / 4 + kMaxCluster];
    float2 in_ml[kMaxCluster][HT];
};

// Joins the warps of a CTA and, where the parts of a sequence are a cluster, its CTAs, and writes the result for the
// heads: the operator's, or, where a second kernel is to join the parts, this part's. The order of the sums is fixed.
template <typename TI, int V, int W, int HT, typename Wk>
__device__ __forceinline__ void join(const AttendArgs& a, const Wk& wk, Partial<W, HT, V>& p) {
    const int units = wk.heads * (V / 4), share = (units + a.parts - 1) / a.parts;  // of a CTA of the cluster
    if (a.cluster) cluster_wait();  // for the others to have started
    __syncthreads();
    for (int i = threadIdx.x; i < units; i += W * 32) {
        const int h = i / (V / 4), u = i % (V / 4);
        float m = p.m[0][h];
#pragma unroll
        for (int w = 1; w < W; ++w) m = fmaxf(m, p.m[w][h]);
        const float base = finite_base(m);
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2(p.m[w][h] - base);
            l = fmaf(p.l[w][h], f, l);
            add_scaled(x, p.acc[w][h][u], f);
        }
        const int64_t at = wk.n * a.HQ + wk.h0 + h;
        if (a.cluster) {
            push(&p.in_acc[wk.part * share + i % share], i / share, x);
            if (u < a.parts) push(&p.in_ml[wk.part][h], u, make_float2(m, l));
        } else if (wk.used == 1) {
            write_result<TI>(a, at, V, 4 * u, m, l, x);
        } else {
            ((float4*)a.part_acc)[(at * a.parts + wk.part) * (V / 4) + u] = x;
            if (u == 0) a.part_ml[at * a.parts + wk.part] = make_float2(m, l);
        }
    }
    if (!a.cluster) return;
    cluster_arrive();
    cluster_wait();
    for (int j = threadIdx.x; j < share && wk.part * share + j < units; j += W * 32) {
        const int i = wk.part * share + j, h = i / (V / 4), u = i % (V / 4);
        float m = p.in_ml[0][h].x;
        for (int c = 1; c < a.parts; ++c) m = fmaxf(m, p.in_ml[c][h].x);
        const float base = finite_base(m);
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < a.parts; ++c) {
            const float f = ex2(p.in_ml[c][h].x - base);
            l = fmaf(p.in_ml[c][h].y, f, l);
            add_scaled(x, p.in_acc[c * share + j], f);
        }
        write_result<TI>(a, wk.n * a.HQ + wk.h0 + h, V, 4 * u, m, l, x);
    }
}

// The parts of one query head, joined in an order that goes by their number alone: group g of the threads takes parts
// g, g + G, .., eight of them at a time, and the groups are joined in shared memory. The length, which says how many
// parts there are to join, is on its way together with the first of them.
constexpr int kJoinThreads = 512, kJoinBatch = 8;
template <typename TI, int V>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a) {
    constexpr int U = V / 4, G = kJoinThreads / U;
    __shared__ float4 sx[G][U];
    __shared__ float2 sml[G];
    const unsigned at = blockIdx.x, n = at / a.HQ;
    const int g = threadIdx.x / U, u = threadIdx.x % U;
    after_previous();
    const float2* ml = a.part_ml + (int64_t)at * a.parts;
    const float4* acc = (const float4*)a.part_acc + (int64_t)at * a.parts * U + u;
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    int used = a.parts, s = g;
    do {
        float2 e[kJoinBatch];
        float4 y[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const bool in = s + i * G < used;
            e[i] = in ? ml[s + i * G] : make_float2(-INFINITY, 0.f);
            y[i] = in ? acc[(s + i * G) * U] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (s == g) {
            int begin, end;
            kv_range(a, n, begin, end);
            used = parts_used(a, end - begin, a.turn);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (s + i * G >= used) {  // what lies there was not written
                e[i] = make_float2(-INFINITY, 0.f);
                y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            top = fmaxf(top, e[i].x);
        }
        const float base = finite_base(top), keep = ex2(m - base);
        l *= keep;
        x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
        m = top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const float f = ex2(e[i].x - base);
            l = fmaf(e[i].y, f, l);
            add_scaled(x, y[i], f);
        }
        s += G * kJoinBatch;
    } while (s < used);
    if (used == 1) return;  // the one part has written the result
    sx[g][u] = x;
    if (u == 0) sml[g] = make_float2(m, l);
    __syncthreads();
    if (g > 0) return;
    for (int i = 1; i < G; ++i) m = fmaxf(m, sml[i].x);
    const float base = finite_base(m);
    l = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const float f = ex2(sml[i].x - base);
        l = fmaf(sml[i].y, f, l);
        add_scaled(x, sx[i][u], f);
    }
    write_result<TI>(a, at, V, 4 * u, m, l, x);
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
template <int K, int V, int NT, int W>
__global__ void __launch_bounds__(W * 32, W == 8 ? 1 : NT == 1 ? 3 : 2) k_attend_mma(AttendArgs a) {
    using TI = __nv_bfloat16;
    constexpr int KI = K / 32, VC = V / 64, VJ = V / 16, HT = 8 * NT;
    __shared__ Partial<W, HT, V> sm;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    Work<W, 16, HT> wk;
    if (a.cluster) cluster_arrive();
    after_previous();
    if (!wk.start(a) && !a.cluster) return;
    const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
    Rows<16>& rows = wk.rows;
    uint4 q[NT][KI];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < KI; ++i)
            q[j][i] = load16((const TI*)a.q + wk.n * a.q_stride + (h0 + 8 * j + g) * K + (4 * i + t) * 8, 8 * j + g < heads);
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
    for (int first = wk.first; first < wk.end; first += rows.step) {
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
            float* row = (float*)sm.acc[warp][h] + 8 * g;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < VJ; i += 4)
                    *(float4*)(row + (VC == 2 ? 64 : 4) * r + i) =
                        make_float4(acc[j][i][e + 2 * r], acc[j][i + 1][e + 2 * r], acc[j][i + 2][e + 2 * r],
                                    acc[j][i + 3][e + 2 * r]);
        }
    join<TI>(a, wk, sm);
}

// ------------------------------------------------------------------ fp32

// FFMA kernel: one CTA per (part, up to HT query heads of one cache head, sequence), each warp R rows at a time, a
// lane holding K / 32 and V / 32 channels of each row and of every head. The R HT scores are sums over the lanes: a
// butterfly that halves the values with the lanes leaves value i, summed, in the lanes l with l % (R HT) == i.
template <int K, int V, int HT, int R, int W>
__global__ void __launch_bounds__(W * 32) k_attend_simt(AttendArgs a) {
    constexpr int KL = K / 32, VL = V / 32, NV = R * HT;
    __shared__ Partial<W, HT, V> sm;
    const int lane = threadIdx.x % 32;
    Work<W, R, HT> wk;
    if (a.cluster) cluster_arrive();
    after_previous();
    if (!wk.start(a) && !a.cluster) return;
    const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
    Rows<R>& rows = wk.rows;
    float q[HT][KL], acc[HT][VL];
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
        for (int i = 0; i < KL; ++i)
            q[h][i] = h < heads ? ((const float*)a.q)[wk.n * a.q_stride + (h0 + h) * K + lane * KL + i] : 0.f;
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
    for (int first = wk.first; first < wk.end; first += rows.step) {
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
        for (int i = 0; i < VL; ++i) ((float*)sm.acc[warp][h])[lane * VL + i] = acc[h][i];
    join<float>(a, wk, sm);
}

// ------------------------------------------------------------------ launch

// Query heads that a CTA takes together.
int head_tile(const kda_cache* c, int HQ) {
    const int group = HQ / c->HKV;
    if (c->dtype == KDA_DTYPE_BF16) return group <= 8 ? 8 : 16;
    return group == 1 ? 1 : group <= 4 ? 4 : 8;
}

// The split of each sequence's rows: warps to a CTA, CTAs.
struct Plan {
    int warps, parts, cluster, turn;
};
Plan plan_of(const kda_cache* c, int HQ, int N, int max_pages, int window) {
    const int group = HQ / c->HKV, ht = head_tile(c, HQ);
    const int64_t units = (int64_t)(N > 0 ? N : 1) * c->HKV * ((group + ht - 1) / ht);
    int64_t rows = (int64_t)max_pages * c->page_size;
    if (window > 0 && window < rows) rows = window;
    const int tile = c->dtype == KDA_DTYPE_BF16 ? 16 : ht == 8 ? 4 : 8;
    Plan p{4, (int)((152 * 3 + units - 1) / units), 0, 4 * tile};
#ifdef TUNE
    p.warps = atoi(getenv("KW")); p.parts = atoi(getenv("KS")); p.cluster = atoi(getenv("KC")); p.turn = p.warps * tile;
#endif
    return p;
}

typedef void (*Kernel)(AttendArgs);

template <int K, int V> Kernel kernel_of(bool bf16, int ht, int warps) {
    if (bf16 && warps == 8) return k_attend_mma<K, V, 1, 8>;
    if (bf16) return ht == 8 ? k_attend_mma<K, V, 1, 4> : k_attend_mma<K, V, 2, 4>;
    return ht == 1 ? k_attend_simt<K, V, 1, 8, 4> : ht == 4 ? k_attend_simt<K, V, 4, 8, 4> : k_attend_simt<K, V, 8, 4, 4>;
}

cudaError_t launch_attend(const AttendArgs& a, int warps, cudaStream_t st) {
    const bool bf16 = a.c.dtype == KDA_DTYPE_BF16;
    const int ht = head_tile(&a.c, a.HQ), group = a.HQ / a.c.HKV, K = a.c.K, V = a.c.V;
    const unsigned grid = (unsigned)((int64_t)a.N * a.c.HKV * ((group + ht - 1) / ht) * a.parts);
    const Kernel kernel = K == 128 ? (V == 128 ? kernel_of<128, 128>(bf16, ht, warps) : kernel_of<128, 64>(bf16, ht, warps))
                                   : (V == 128 ? kernel_of<64, 128>(bf16, ht, warps) : kernel_of<64, 64>(bf16, ht, warps));
    cudaError_t e = launch_after(kernel, a, grid, warps * 32, st, a.cluster ? a.parts : 1);
    if (e != cudaSuccess) return e;
    note_launch("cache_attend", st);
    if (a.parts == 1 || a.cluster) return cudaSuccess;
    const Kernel join = bf16 ? (V == 128 ? k_attend_join<__nv_bfloat16, 128> : k_attend_join<__nv_bfloat16, 64>)
                             : (V == 128 ? k_attend_join<float, 128> : k_attend_join<float, 64>);
    if ((e = launch_after(join, a, (unsigned)((int64_t)a.N * a.HQ), kJoinThreads, st)) != cudaSuccess) return e;
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
    const Plan plan = plan_of(c, HQ, N, max_pages, window);
    const int64_t parts = plan.cluster ? 1 : plan.parts;
    return parts == 1 ? 256 : 256 + (size_t)N * HQ * parts * ((size_t)c->V * sizeof(float) + sizeof(float2));
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
                 status, plan.parts, plan.cluster, plan.turn, nullptr, nullptr};
    a.part_acc = (float*)ws;
    a.part_ml = (float2*)(a.part_acc + (int64_t)N * HQ * a.parts * c->V);
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const cudaError_t e = launch_attend(a, plan.warps, st);
    if (e != cudaSuccess) return cuda_fail(e);
    return KDA_OK;
}
