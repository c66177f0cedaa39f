// Attention of one new token per sequence over a paged cache: what its kernels have in common. How the rows are given to
// CTAs, where a tile's rows are, how partial results join, and the plan. (Kernels: kda_attend_kernels.cuh, kda_attend8.cu.)
#pragma once
#include "../../include/kda_selftest.h"
#include "kda_cache.cuh"

namespace kda {
namespace attend {

// How the rows are given to CTAs (see Work).
enum Split { kWhole, kCluster, kParts, kShares };

struct AttendArgs {
    kda_cache c;
    const void* q;
    int64_t q_stride, table_stride;
    int HQ, N, max_pages, window, sinks;
    const int32_t *table, *kv_lens;
    float scale_log2;
    void* o;
    float* lse;
    int32_t* status;
    int group, tiles, units;      // query heads of a cache head, in tiles of HT; units of a sequence (HKV tiles)
    Divisor page;                 // by c.page_size
    // a cache in 8 bits: the scales of its blocks, and division by their rows
    const float *k_scale, *v_scale;
    int64_t ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    Divisor block;
    int step, step_pg, step_off;  // rows from a warp's tile to its next, in pages and rows
    int split, parts;  // parts: kCluster, kParts: CTAs of a unit; kShares: CTAs in all; kWhole: 1
    Divisor by_parts;
    int turn;  // rows that a CTA takes at a time
    int together;  // kShares: units that have a share together, a CTA each
    // What a CTA has of a unit that it does not have whole, head by head: the weighted sum relative to its maximum, and
    // its maximum (log2 units) and sum of weights. kParts: [units, parts, HT, V] and [units, parts, HT]; kShares: of the
    // unit that it ends (0) and of the one that it begins (1), [parts, 2, HT, V] and [parts, 2, HT], and of each unit the
    // first and last CTA that have some of it.
    float4* part_acc;
    float2* part_ml;
    int2* unit_parts;
};

// The rows that sequence n attends, by their numbers [begin, end). Those from `border` on, the window's, have their
// positions for numbers; the first rows, which stay visible beside a window (SINKS), have the numbers just below: row
// number r < border is at position r - begin.
template <bool SINKS>
__device__ __forceinline__ void kv_range(const AttendArgs& a, int64_t n, int& begin, int& end, int& border) {
    const int64_t len = a.kv_lens[n], room = (int64_t)a.max_pages * a.c.page_size;
    if (len > room && a.status && threadIdx.x == 0) *a.status = KDA_ERR_INVALID_ARG;
    end = (int)max(min(len, room), (int64_t)0);
    begin = border = a.window > 0 && len > a.window ? (int)min(len - a.window, (int64_t)end) : 0;
    if constexpr (SINKS) begin -= min(a.sinks, begin);
}
template <bool SINKS> __device__ __forceinline__ void kv_range(const AttendArgs& a, int64_t n, int& begin, int& end) {
    int border;
    kv_range<SINKS>(a, n, begin, end, border);
}

// How far above the running maximum a score may lie (log2 units) before acc and l are rescaled, so that most tiles only
// ask whether any score is higher. Weights, and sums of them, are held as 2^-8 of what they are relative to the maximum:
// none is above one, so sums over large values overflow no earlier than relative to the true maximum. (A power of two
// rounds nothing.)
constexpr float kSlack = 8.f, kAtMostOne = 0x1p-8f;

// The value that exponents are taken relative to: the maximum, or 0 where no score is above -inf, so that a
// weight there is 2^-inf = 0 and a NaN score stays a NaN.
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ rows of a tile
//
// R rows in a warp's tile: lane l looks up row l % R. Pages may be of any size, so every row has its own; the lookup
// of the next tile's pages is in flight while a tile is computed.
template <int R, bool SINKS> struct Rows {
    const int32_t* table;
    int left;           // rows from the next tile's row of this lane to the end
    int pg, off, page;  // that row's place
    int skip, to_window;   // SINKS: positions between the first rows and the window; rows from that row to the window
    int64_t at, k_off, v_off;  // this tile's row of this lane: its page, and where it begins
    int at_off;                // and its row in the page
    unsigned valid;        // bit r: row r is in range and its page exists

    // Rows from number `first` on, of a warp whose tiles are a.step rows apart.
    __device__ __forceinline__ void start(const AttendArgs& a, int64_t n, int first, int begin = 0, int border = 0) {
        int row = first + threadIdx.x % 32 % R;
        if constexpr (SINKS) {
            skip = begin;
            to_window = border - row;
            if (to_window > 0) row -= skip;
        }
        table = a.table + n * a.table_stride;
        pg = a.page(row);
        off = row - pg * a.c.page_size;
        page = pg < a.max_pages ? table[pg] : -1;
    }
    // The end of the rows, which may be known later than their beginning.
    __device__ __forceinline__ void until(int first, int end) { left = end - first - (int)(threadIdx.x % 32 % R); }
    __device__ __forceinline__ void next(const AttendArgs& a) {
        const bool in = left > 0, ok = in && (unsigned)page < (unsigned)a.c.num_pages;
        if (in && !ok && a.status) *a.status = KDA_ERR_INVALID_ARG;
        valid = __ballot_sync(0xffffffffu, ok);
        const int64_t p = ok ? page : 0;
        at = p;
        at_off = off;
        k_off = p * a.c.k_page + off * a.c.k_row;
        v_off = p * a.c.v_page + off * a.c.v_row;
        left -= a.step;
        pg += a.step_pg;
        off += a.step_off;
        if (off >= a.c.page_size) {
            off -= a.c.page_size;
            ++pg;
        }
        if constexpr (SINKS) {
            if (to_window > 0) {
                to_window -= a.step;
                if (to_window <= 0) {  // the row is the first of the window's
                    const int pages = a.page(skip);
                    pg += pages;
                    off += skip - pages * a.c.page_size;
                    if (off >= a.c.page_size) {
                        off -= a.c.page_size;
                        ++pg;
                    }
                }
            }
        }
        page = left > 0 ? table[pg] : -1;
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

// ------------------------------------------------------------------ split
//
// A unit is a sequence, a cache head and up to HT of its query heads. A CTA takes W R rows at a time, R for each of its
// W warps: a turn. The host knows the sizes but not the lengths, which lie on the device. It chooses between
//   kWhole    a CTA per unit: for units of few turns, or very many units;
//   kCluster  a cluster of CTAs per unit, which take its turns one after the other (so the first rows of a CTA do not
//             depend on the length, and their pages are looked up while it is on its way) and join their results in
//             shared memory: for few units of some turns, where latency counts;
//   kParts    the same with more CTAs than a cluster has, joined by a second kernel: for few units of many turns, and
//             over a cache in fp32 (k_attend_simt) for all of many rows;
//   kShares   (the tensor-core kernels: a cache in bf16, or in 8 bits with queries of either type) as many CTAs as the GPU
//             holds at once, each with an equal share of all turns in the order of the units, whatever the lengths are: every CTA adds up the lengths to find its share. A unit counts for
//             kUnitTurns more than it has, about what it costs to begin and end one; else the CTAs with many short units
//             would be the last (64 sequences of U[1,8192] rows, 32 heads on 8: 160 -> 154 us; 11 of U[1,4240], 256
//             heads on 16: 42 -> 28 us). A unit that falls to several CTAs is joined by a second kernel.
//             Over a cache in 8 bits, and with first rows beside a window, the units of a sequence have a share together, as
//             many of them as divide them all and leave few places empty: they read the same pages at the same time
//             (64 sequences of U[1,8192] rows in 8 bits, 32 heads on 8: 93 -> 87 us; of U[1,16384] in 16 bits that see
//             4160 of them: 138 -> 136).
constexpr int kUnitTurns = 2;
constexpr int kWarps = 4;
constexpr int kMaxCluster = 16;

template <int R, int HT, bool SHARES, bool SINKS, bool TOGETHER = false> struct Work {
    static constexpr int W = kWarps, kTurn = W * R;
    int n, hkv, h0, heads, warp;
    int left;  // rows from the warp's first one to the end
    int odd;  // kShares: which of the share's two states is the next
    Rows<R, SINKS> rows;

    // What a CTA keeps in shared memory (a barrier lies between two units).
    struct Share {
        // the unit, for the join: whole, if the CTA or its cluster has all of it; part: kCluster: the CTA's rank;
        // kParts, kShares: where it leaves its part
        int64_t head;
        int heads, whole, part;
        // kShares: the unit's number, if it begins here, and its last turn
        int64_t unit;
        int last_turn;
        // kShares: the turns [at, stop) of `total` are still to be done, from sequence n on, whose first turn is `seq`
        int sums[W], stop, total;
        struct {
            int at, n, seq;
        } state[2];
    };

    __device__ __forceinline__ static int turns_of(int begin, int end) {
        return max(1, (end - begin + kTurn - 1) / kTurn);  // one at least, which writes the result of no rows
    }
    // Unit u of sequence n.
    __device__ __forceinline__ void set_unit(const AttendArgs& a, unsigned u, bool whole, int part, Share& share) {
        unsigned qt = 0;
        hkv = u;
        if (a.tiles > 1) {
            hkv = u / (unsigned)a.tiles;
            qt = u - hkv * a.tiles;
        }
        h0 = hkv * a.group + qt * HT;
        heads = min(HT, (int)(a.group - qt * HT));
        if (threadIdx.x == 0) {
            share.head = (int64_t)n * a.HQ + h0;
            share.heads = heads;
            share.whole = whole;
            share.part = part;
        }
    }
    // The CTA's first unit; false if it has none.
    __device__ __forceinline__ bool start(const AttendArgs& a, Share& share) {
        warp = threadIdx.x / 32;
        odd = 0;
        if constexpr (SHARES) {
            find_share(a, share);
            return next(a, share);
        }
        // (the units of a sequence, which share its pages, come one after the other)
        const int unit = a.by_parts(blockIdx.x), part = blockIdx.x - unit * a.parts;
        n = blockIdx.y;
        int first = (part * W + warp) * R, begin, end, border;
        rows.start(a, n, first);
        kv_range<SINKS>(a, n, begin, end, border);
        if (a.window > 0) {
            first += begin;
            rows.start(a, n, first, begin, border);
        }
        left = end - first;
        rows.until(first, end);
        const bool alone = a.split != kParts || end - begin <= a.turn;
        set_unit(a, unit, alone, a.split == kParts ? (n * a.units + unit) * a.parts + part : part, share);
        return a.split != kParts || part < turns_of(begin, end);
    }
    // kShares: turns are dealt out evenly, one more to each of the first total % ctas CTAs: the first turn of CTA x, and
    // the CTA that has turn y.
    __device__ __forceinline__ static int first_turn(int x, int total, int ctas) {
        return x * (total / ctas) + min(x, total % ctas);
    }
    __device__ __forceinline__ static int cta_of(int y, int total, int ctas) {
        const int each = total / ctas, more = total % ctas, both = more * (each + 1);
        return y < both ? y / (each + 1) : more + (y - both) / each;
    }
    // kShares: the CTA's share, and the sequence that it begins in. Units are counted in bundles of `together`.
    __device__ __forceinline__ static int together(const AttendArgs& a) { return TOGETHER ? a.together : 1; }
    __device__ __forceinline__ static int my_share(const AttendArgs& a) {
        return TOGETHER ? (int)(blockIdx.x / (unsigned)a.together) : (int)blockIdx.x;
    }
    __device__ __forceinline__ void find_share(const AttendArgs& a, Share& share) {
        const int units = TOGETHER ? a.units / a.together : a.units, mine_is = my_share(a);
        const int per = (a.N + W * 32 - 1) / (W * 32), lane = threadIdx.x % 32;
        const int n0 = min((int)threadIdx.x * per, a.N), n1 = min(n0 + per, a.N);
        int mine = 0, begin, last;
        for (int i = n0; i < n1; ++i) {
            kv_range<SINKS>(a, i, begin, last);
            mine += (turns_of(begin, last) + kUnitTurns) * units;
        }
        int before = mine;
#pragma unroll
        for (int w = 1; w < 32; w *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, before, w);
            if (lane >= w) before += y;
        }
        if (lane == 31) share.sums[warp] = before;
        __syncthreads();
        before -= mine;
        int total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += share.sums[w];
            total += share.sums[w];
        }
        const int ctas = min(a.parts, total);  // with fewer turns than CTAs, those that have one
        const int at = first_turn(min(mine_is, ctas), total, ctas);
        if (mine_is >= ctas && threadIdx.x == 0) share.state[0].at = share.stop = 0;
        if (at >= before && at < before + mine) {
            int i = n0;
            for (;; ++i) {
                kv_range<SINKS>(a, i, begin, last);
                const int turns = (turns_of(begin, last) + kUnitTurns) * units;
                if (at < before + turns) break;
                before += turns;
            }
            share.stop = first_turn(mine_is + 1, total, ctas);
            share.total = total;
            share.state[0] = {at, i, before};
        }
        __syncthreads();
    }
    // kShares: the next unit, or part of one, of the CTA's share; false if there is none.
    __device__ __forceinline__ bool next(const AttendArgs& a, Share& share) {
        const int stop = share.stop, units = TOGETHER ? a.units / a.together : a.units;
        int at = share.state[odd].at, begin, last, border, turns, each, t0, seq = share.state[odd].seq;
        unsigned u;
        n = share.state[odd].n;
        for (;; at += each - t0) {  // (a share may begin behind a unit's rows)
            if (at >= stop) return false;
            for (;; ++n) {
                kv_range<SINKS>(a, n, begin, last, border);
                turns = turns_of(begin, last);
                each = turns + kUnitTurns;
                if (at < seq + each * units) break;
                seq += each * units;
            }
            u = (unsigned)(at - seq) / (unsigned)each;
            t0 = at - seq - u * each;
            if (t0 < turns) break;
        }
        const int t1 = min(turns, t0 + stop - at);
        int part = 2 * my_share(a) + (t0 == 0);
        if constexpr (TOGETHER) {
            const unsigned member = blockIdx.x % (unsigned)a.together;
            u = u * a.together + member;
            part = part * a.together + member;
        }
        set_unit(a, u, t0 == 0 && t1 == turns, part, share);
        odd ^= 1;
        if (threadIdx.x == 0) {
            share.state[odd] = {at + (t1 < turns ? t1 : each) - t0, n, seq};
            share.unit = t0 == 0 ? (int64_t)n * a.units + u : -1;
            share.last_turn = at + turns - 1;
        }
        const int first = begin + (t0 * W + warp) * R, end = min(last, begin + t1 * kTurn);
        rows.start(a, n, first, begin, border);
        left = end - first;
        rows.until(first, end);
        return true;
    }
};

// ------------------------------------------------------------------ joins

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_started() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
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
__device__ __forceinline__ void add_scaled(float4& x, const float4& y, float f) {
    x.x = fmaf(y.x, f, x.x);
    x.y = fmaf(y.y, f, x.y);
    x.z = fmaf(y.z, f, x.z);
    x.w = fmaf(y.w, f, x.w);
}
// Channels d .. d + 3 of the result of query head `at`.
template <typename TI>
__device__ __forceinline__ void write_result(const AttendArgs& a, int64_t at, int V, int d, float m, float l, float4 x) {
    if (l == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);  // nothing attended
    const float f = l == 0.f ? 0.f : 1.f / l;
    TI* o = (TI*)a.o + at * V + d;
    if constexpr (sizeof(TI) == 2) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * f, x.y * f), hi = __floats2bfloat162_rn(x.z * f, x.w * f);
        *(uint2*)o = make_uint2(*(const uint32_t*)&lo, *(const uint32_t*)&hi);
    } else {
        *(float4*)o = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    }
    if (d == 0 && a.lse) a.lse[at] = (finite_base(m) + log2f(l / kAtMostOne)) * kLn2;
}

// The results of a CTA's warps for HT heads: maxima m, sums of weights l, and weighted sums acc relative to m.
template <int HT, int V> struct Partial {
    float m[kWarps][HT], l[kWarps][HT];
    float4 acc[kWarps][HT][V / 4 + 1];
};
// In a cluster: what its CTAs send of the channels that this one joins, and of every head their m and l. They may do so
// while this one still has rows to attend.
template <int HT, int V> struct Inbox {
    float4 acc[HT * V / 4 + kMaxCluster];
    float2 ml[kMaxCluster][HT];
};

// Joins the warps of a CTA and, in a cluster, its CTAs, and writes the unit's result, or, where the CTA does not have
// all of the unit, its part. The order of the sums is fixed.
template <typename TI, int V, int HT, bool SHARES, typename Wk>
__device__ __forceinline__ void join(const AttendArgs& a, const typename Wk::Share& unit, Partial<HT, V>& p,
                                     Inbox<HT, V>& in) {
    const bool cluster = !SHARES && a.split == kCluster;
    if (cluster) cluster_wait();  // for the others to have started
    __syncthreads();
    const int items = unit.heads * (V / 4), share = (items + a.parts - 1) / a.parts;  // share: of a CTA of the cluster
    const int part = unit.part;
    const int64_t head = unit.head;
    if constexpr (SHARES) {
        if (threadIdx.x == kWarps * 32 - 1 && unit.unit >= 0)
            a.unit_parts[unit.unit] =
                make_int2(Wk::my_share(a), Wk::cta_of(unit.last_turn, unit.total, min(a.parts, unit.total)));
    }
    for (int i = threadIdx.x; i < items; i += kWarps * 32) {
        const int h = i / (V / 4), u = i % (V / 4);
        float m = p.m[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, p.m[w][h]);
        const float base = finite_base(m);
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(p.m[w][h] - base);
            l = fmaf(p.l[w][h], f, l);
            add_scaled(x, p.acc[w][h][u], f);
        }
        if (cluster) {
            push(&in.acc[part * share + i % share], i / share, x);
            if (u < a.parts) push(&in.ml[part][h], u, make_float2(m, l));
        } else if (unit.whole) {
            write_result<TI>(a, head + h, V, 4 * u, m, l, x);
        } else {
            const int64_t to = (int64_t)part * HT + h;
            a.part_acc[to * (V / 4) + u] = x;
            if (u == 0) a.part_ml[to] = make_float2(m, l);
        }
    }
    if (!cluster) return;
    cluster_arrive();
    cluster_wait();
    for (int j = threadIdx.x; j < share && part * share + j < items; j += kWarps * 32) {
        const int i = part * share + j, h = i / (V / 4), u = i % (V / 4);
        float m = in.ml[0][h].x;
        for (int c = 1; c < a.parts; ++c) m = fmaxf(m, in.ml[c][h].x);
        const float base = finite_base(m);
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < a.parts; ++c) {
            const float f = ex2(in.ml[c][h].x - base);
            l = fmaf(in.ml[c][h].y, f, l);
            add_scaled(x, in.acc[c * share + j], f);
        }
        write_result<TI>(a, head + h, V, 4 * u, m, l, x);
    }
}

// kParts, kShares: the parts of one query head and VS of its channels, joined in an order that goes by their number alone.
// Group g of G groups of VS / 4 threads takes parts g, g + G, .., a batch of them at a time; the groups are joined in
// shared memory.
constexpr int kJoinBatch = 8;
template <typename TI, int V, int HT, int VS, int G, int THREADS, bool SHARES, bool TOGETHER>
__global__ void __launch_bounds__(THREADS) k_attend_join(AttendArgs a) {
    constexpr int U = VS / 4, S = V / VS, HB = THREADS / (G * U);  // slices of a head; (head, slice) pairs of a CTA
    constexpr int GW = U < 32 && G > 1 ? 32 / U : 1;  // groups of a warp
    static_assert(G % GW == 0, "a warp has groups of one pair");
    __shared__ float4 sx[HB][G / GW][U];
    __shared__ float2 sml[HB][G / GW];
    const unsigned mine = threadIdx.x / (G * U), at = blockIdx.x * HB + mine, last = (unsigned)(a.N * a.HQ) * S - 1;
    const unsigned head = min(at, last) / S, u = min(at, last) % S * U + threadIdx.x % U;
    const int g = threadIdx.x / U % G;
    const unsigned n = head / a.HQ, hq = head % a.HQ, hkv = hq / a.group, qt = hq % a.group / HT, h = hq % a.group % HT;
    after_previous();
    // parts first .. first + count - 1 (with kParts the length says how many there are, and is on its way together with
    // the first of them)
    const int64_t unit = (int64_t)n * a.units + hkv * a.tiles + qt;
    int64_t first;
    int count;
    if constexpr (SHARES) {
        const int2 range = a.unit_parts[unit];
        first = 2 * (int64_t)range.x;
        if constexpr (TOGETHER) first = first * a.together + (hkv * a.tiles + qt) % (unsigned)a.together;
        count = range.y - range.x + 1;
    } else {
        first = unit * a.parts;
        count = a.parts;
    }
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    int s = g;
    if (count > 1) {
        do {
            float2 e[kJoinBatch];
            float4 y[kJoinBatch];
            float top = m;
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const int c = s + i * G;
                const int64_t part = SHARES ? 2 * c + (c == 0) : c, from = (first + (TOGETHER ? part * a.together : part)) * HT + h;
                e[i] = c < count ? a.part_ml[from] : make_float2(-INFINITY, 0.f);
                y[i] = c < count ? a.part_acc[from * (V / 4) + u] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (!SHARES && s == g) {
                int begin, end;
                kv_range<true>(a, n, begin, end);
                count = max(1, min(count, (end - begin + a.turn - 1) / a.turn));
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i) {
                    if (s + i * G >= count) {  // what lies there was not written
                        e[i] = make_float2(-INFINITY, 0.f);
                        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, e[i].x);
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
        } while (s < count);
    }
    if constexpr (G > 1) {
        // the groups of a warp, then the warps
#pragma unroll
        for (int w = U; w < 32; w *= 2) {
            const float m1 = __shfl_xor_sync(0xffffffffu, m, w), l1 = __shfl_xor_sync(0xffffffffu, l, w);
            const float4 x1 = make_float4(__shfl_xor_sync(0xffffffffu, x.x, w), __shfl_xor_sync(0xffffffffu, x.y, w),
                                          __shfl_xor_sync(0xffffffffu, x.z, w), __shfl_xor_sync(0xffffffffu, x.w, w));
            const float top = fmaxf(m, m1), base = finite_base(top), f = ex2(m - base), f1 = ex2(m1 - base);
            m = top;
            l = l * f + l1 * f1;
            x = make_float4(x.x * f + x1.x * f1, x.y * f + x1.y * f1, x.z * f + x1.z * f1, x.w * f + x1.w * f1);
        }
        if (threadIdx.x % 32 < U) {
            sx[mine][g / GW][threadIdx.x % U] = x;
            if (threadIdx.x % U == 0) sml[mine][g / GW] = make_float2(m, l);
        }
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int i = 1; i < G / GW; ++i) m = fmaxf(m, sml[mine][i].x);
        const float base = finite_base(m);
        l = 0.f;
        x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < G / GW; ++i) {
            const float f = ex2(sml[mine][i].x - base);
            l = fmaf(sml[mine][i].y, f, l);
            add_scaled(x, sx[mine][i][threadIdx.x % U], f);
        }
    }
    // (one part alone has written the result; the last CTA's spare threads have the last pair once more)
    if (count > 1 && at <= last) write_result<TI>(a, head, V, 4 * u, m, l, x);
}

// An 8 x 8 matrix of 16-bit values (lane 4 i + j holds columns 2 j, 2 j + 1 of row i), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ------------------------------------------------------------------ launch

typedef void (*Kernel)(AttendArgs);

// What the plan goes by, of a kernel.
struct Form {
    int ht;    // query heads of a unit
    int tile;  // rows of a warp's tile
    int ctas;  // CTAs to an SM
    bool even; // it has kShares
    size_t shared = 0;  // bytes of shared memory that a launch asks for
    bool together = false;  // units have a share together
    // what the joins cost, in turns of a CTA: of clusters of 2, 4 and 8, of parts, and of shares with their start
    double join2 = 1.2, join4 = 1.2, join8 = 1.7, join_parts = 3.6, join_shares = 6.0;
};
// Of a device: its SMs, and the largest cluster that the kernel can be placed in.
struct Gpu {
    int sms = 0, cluster = 0;
};
struct Plan {
    Split split;
    int parts, ht, units, turn;
    dim3 grid;
    size_t acc_bytes, ml_bytes, ws_bytes;  // of the workspace
    size_t shared;
    int together;
};
Plan plan_of(const kda_cache* c, int HQ, int N, int max_pages, int window, int sinks, const Form& form, const Gpu& gpu);

// The plan of a call on a cache in 8 bits (gpu.sms 0: on the present device).
kda_status plan_for8(const kda_cache8* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks, Gpu gpu,
                     Plan& plan);

// The sizes that all forms of the operator refuse.
kda_status check_sizes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks);

// What a call is given besides the cache.
struct Call {
    const void* q;
    int64_t q_stride;
    int32_t HQ, N;
    const int32_t* page_table;
    int64_t table_stride;
    int32_t max_pages;
    const int32_t* kv_lens;
    int32_t window, sinks;
    float scale;
    void* o;
    float* lse;
    int32_t* status;
    void* ws;
    size_t ws_bytes;
    cudaStream_t stream;
};
// Checks the call's arguments (`unit`: elements of 16 bytes of q).
kda_status check_call(const kda_cache* c, const Call& x, int64_t unit);
// The kernel's arguments, and the launch of it and, where the plan says so, of the join (`bf16`: the type of o). `names`:
// the kernel's, by the split.
AttendArgs args_of(const kda_cache* c, const Call& x, const Plan& plan);
kda_status launch(const AttendArgs& a, const Plan& plan, Kernel kernel, bool bf16, const char* const (&names)[4],
                  cudaStream_t stream);

// The kernels of a cache in 16 or 32 bits (kda_attend.cu; with first rows beside a window: kda_attend_sinks.cu).
Kernel kernel_without_sinks(const kda_cache& c, int ht, Split split);
Kernel kernel_with_sinks(const kda_cache& c, int ht, Split split);

}  // namespace attend
}  // namespace kda
