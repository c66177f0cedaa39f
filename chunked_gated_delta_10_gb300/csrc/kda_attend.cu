// kda_cache_attend: attention of one new token per sequence over a paged
// cache. Declared in include/kda_serve.h.
//
// One pass over the cached rows with the running maximum m and sum l of the
// softmax (in log2 units): a row's score s raises m to m' = max(m, s), and
//   l <- l 2^(m - m') + 2^(s - m'),   acc <- acc 2^(m - m') + 2^(s - m') V.
// Partial results over disjoint rows join by the same rule.
//
// Bound: the cached keys and values are read once. Measured on one GB300 (time of
// a call among others; GB/s of the cached rows), bf16, K = V = 128:
//   64 sequences of U[1,8192] rows, 32 query heads on 8: 154.5 to 157.4 us,
//     6.8 to 6.9 TB/s, a little above a plain copy's rate;
//   one of 65536 rows, 16 heads on 2: 17.0 us (9.9 at that rate): the length, the
//     pages and the first rows are read one after the other before the stream is
//     full (1.5 us), 410 CTAs of five turns each are three to some SMs and two to
//     others, and the second kernel takes 2 us;
//   one of 2048 rows, 32 heads on 8: 5.8 us in a graph, all of it latency (1.2 us of
//     rows).
// What was tried and is slower (measured with weights of two parts): two tiles under
// way in a warp's registers (two CTAs an SM instead of three: 180 us for the first of
// these); the tile after the next asked into L2 (166 us; fp32 with eight heads alone
// gains, 48 -> 44 us); joins of the parts by reading the other CTAs' shared memory
// instead of pushing to it (1.5 us more); clusters for large batches (169 to 180 us: a
// cluster waits for room for all of its CTAs); shares of the rows alone, without a
// weight for a unit's ends (160 us for the first of these); the sequences of a batch
// side by side instead of a sequence's heads, which share its pages (fp32, 12
// sequences: 15.7 against 13.6).
#include "../../include/kda_selftest.h"
#include "kda_cache.cuh"

namespace kda {
namespace {

// Division of numbers below 2^31 by an invariant d (Granlund and Montgomery, 1994): with 2^s >= d, floor(n / d) =
// floor(n ceil(2^(31 + s) / d) / 2^(31 + s)).
struct Divisor {
    unsigned factor, shift;
    Divisor() = default;
    __host__ explicit Divisor(unsigned d) : shift(31) {
        while (1ull << (shift - 31) < d) ++shift;
        factor = (unsigned)(((1ull << shift) + d - 1) / d);
    }
    __device__ __forceinline__ unsigned operator()(unsigned n) const {
        return (unsigned)((uint64_t)n * factor >> shift);
    }
};

// How the rows are given to CTAs (see Work).
enum Split { kWhole, kCluster, kParts, kShares };

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
    int group, tiles, units;      // query heads of a cache head, in tiles of HT; units of a sequence (HKV tiles)
    Divisor page;                 // by c.page_size
    int step, step_pg, step_off;  // rows from a warp's tile to its next, in pages and rows
    int split, parts;  // parts: kCluster, kParts: CTAs of a unit; kShares: CTAs in all; kWhole: 1
    Divisor by_parts;
    int turn;  // rows that a CTA takes at a time
    // What a CTA has of a unit that it does not have whole, head by head: the weighted sum relative to its maximum, and
    // its maximum (log2 units) and sum of weights. kParts: [units, parts, HT, V] and [units, parts, HT]; kShares: of the
    // unit that it ends (0) and of the one that it begins (1), [parts, 2, HT, V] and [parts, 2, HT], and of each unit the
    // first and last CTA that have some of it.
    float4* part_acc;
    float2* part_ml;
    int2* unit_parts;
};

// The rows [begin, end) that sequence n attends.
__device__ __forceinline__ void kv_range(const AttendArgs& a, int64_t n, int& begin, int& end) {
    const int64_t len = a.kv_lens[n], room = (int64_t)a.max_pages * a.c.page_size;
    if (len > room && a.status && threadIdx.x == 0) *a.status = KDA_ERR_INVALID_ARG;
    end = (int)max(min(len, room), (int64_t)0);
    begin = a.window > 0 && len > a.window ? (int)min(len - a.window, (int64_t)end) : 0;
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
template <int R> struct Rows {
    const int32_t* table;
    int left;           // rows from the next tile's row of this lane to the end
    int pg, off, page;  // that row's place
    int64_t k_off, v_off;  // this tile's row of this lane
    unsigned valid;        // bit r: row r is in range and its page exists

    // Rows from `first` on, of a warp whose tiles are a.step rows apart.
    __device__ __forceinline__ void start(const AttendArgs& a, int64_t n, int first) {
        const int row = first + threadIdx.x % 32 % R;
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
        k_off = p * a.c.k_page + off * a.c.k_row;
        v_off = p * a.c.v_page + off * a.c.v_row;
        left -= a.step;
        pg += a.step_pg;
        off += a.step_off;
        if (off >= a.c.page_size) {
            off -= a.c.page_size;
            ++pg;
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
//             with fp32 for all of many rows;
//   kShares   (bf16) as many CTAs as the GPU holds at once, each with an equal share of all turns in the order of the
//             units, whatever the lengths are: every CTA adds up the lengths to find its share. A unit counts for
//             kUnitTurns more than it has, about what it costs to begin and end one; else the CTAs with many short units
//             would be the last (64 sequences of U[1,8192] rows, 32 heads on 8: 160 -> 154 us; 11 of U[1,4240], 256
//             heads on 16: 42 -> 28 us). A unit that falls to several CTAs is joined by a second kernel.
constexpr int kUnitTurns = 2;
constexpr int kWarps = 4;
constexpr int kMaxCluster = 16;

template <int R, int HT, bool SHARES> struct Work {
    static constexpr int W = kWarps, kTurn = W * R;
    int n, hkv, h0, heads, warp;
    int left;  // rows from the warp's first one to the end
    int odd;  // kShares: which of the share's two states is the next
    Rows<R> rows;

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
        int first = (part * W + warp) * R, begin, end;
        rows.start(a, n, first);
        kv_range(a, n, begin, end);
        if (a.window > 0) {
            first += begin;
            rows.start(a, n, first);
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
    // kShares: the CTA's share, and the sequence that it begins in.
    __device__ __forceinline__ void find_share(const AttendArgs& a, Share& share) {
        const int units = a.units;
        const int per = (a.N + W * 32 - 1) / (W * 32), lane = threadIdx.x % 32;
        const int n0 = min((int)threadIdx.x * per, a.N), n1 = min(n0 + per, a.N);
        int mine = 0, begin, last;
        for (int i = n0; i < n1; ++i) {
            kv_range(a, i, begin, last);
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
        const int at = first_turn(min((int)blockIdx.x, ctas), total, ctas);
        if (blockIdx.x >= ctas && threadIdx.x == 0) share.state[0].at = share.stop = 0;
        if (at >= before && at < before + mine) {
            int i = n0;
            for (;; ++i) {
                kv_range(a, i, begin, last);
                const int turns = (turns_of(begin, last) + kUnitTurns) * units;
                if (at < before + turns) break;
                before += turns;
            }
            share.stop = first_turn(blockIdx.x + 1, total, ctas);
            share.total = total;
            share.state[0] = {at, i, before};
        }
        __syncthreads();
    }
    // kShares: the next unit, or part of one, of the CTA's share; false if there is none.
    __device__ __forceinline__ bool next(const AttendArgs& a, Share& share) {
        const int stop = share.stop, units = a.units;
        int at = share.state[odd].at, begin, last, turns, each, t0, seq = share.state[odd].seq;
        unsigned u;
        n = share.state[odd].n;
        for (;; at += each - t0) {  // (a share may begin behind a unit's rows)
            if (at >= stop) return false;
            for (;; ++n) {
                kv_range(a, n, begin, last);
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
        set_unit(a, u, t0 == 0 && t1 == turns, 2 * blockIdx.x + (t0 == 0), share);
        odd ^= 1;
        if (threadIdx.x == 0) {
            share.state[odd] = {at + (t1 < turns ? t1 : each) - t0, n, seq};
            share.unit = t0 == 0 ? (int64_t)n * units + u : -1;
            share.last_turn = at + turns - 1;
        }
        const int first = begin + (t0 * W + warp) * R, end = min(last, begin + t1 * kTurn);
        rows.start(a, n, first);
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

// The results of a CTA's warps for HT heads: maxima m, sums of weights l, and weighted sums acc relative to m. In a
// cluster: what its CTAs send of the channels that this one joins, and of every head their m and l.
template <int HT, int V> struct Partial {
    float m[kWarps][HT], l[kWarps][HT];
    float4 acc[kWarps][HT][V / 4 + 1];
    float4 in_acc[HT * V / 4 + kMaxCluster];
    float2 in_ml[kMaxCluster][HT];
};

// Joins the warps of a CTA and, in a cluster, its CTAs, and writes the unit's result, or, where the CTA does not have
// all of the unit, its part. The order of the sums is fixed.
template <typename TI, int V, int HT, bool SHARES, typename Wk>
__device__ __forceinline__ void join(const AttendArgs& a, const typename Wk::Share& unit, Partial<HT, V>& p) {
    const bool cluster = !SHARES && a.split == kCluster;
    if (cluster) cluster_wait();  // for the others to have started
    __syncthreads();
    const int items = unit.heads * (V / 4), share = (items + a.parts - 1) / a.parts;  // share: of a CTA of the cluster
    const int part = unit.part;
    const int64_t head = unit.head;
    if constexpr (SHARES) {
        if (threadIdx.x == kWarps * 32 - 1 && unit.unit >= 0)
            a.unit_parts[unit.unit] =
                make_int2(blockIdx.x, Wk::cta_of(unit.last_turn, unit.total, min(a.parts, unit.total)));
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
            push(&p.in_acc[part * share + i % share], i / share, x);
            if (u < a.parts) push(&p.in_ml[part][h], u, make_float2(m, l));
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
        write_result<TI>(a, head + h, V, 4 * u, m, l, x);
    }
}

// kParts, kShares: the parts of one query head and VS of its channels, joined in an order that goes by their number alone.
// Group g of G groups of VS / 4 threads takes parts g, g + G, .., a batch of them at a time; the groups are joined in
// shared memory.
constexpr int kJoinBatch = 8;
template <typename TI, int V, int HT, int VS, int G, int THREADS, bool SHARES>
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
                const int64_t from = (first + (SHARES ? 2 * c + (c == 0) : c)) * HT + h;
                e[i] = c < count ? a.part_ml[from] : make_float2(-INFINITY, 0.f);
                y[i] = c < count ? a.part_acc[from * (V / 4) + u] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (!SHARES && s == g) {
                int begin, end;
                kv_range(a, n, begin, end);
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
template <int K, int V, int NT, bool SHARES>
__global__ void __launch_bounds__(kWarps * 32, mma_ctas(NT, K, V)) k_attend_mma(AttendArgs a) {
    using TI = __nv_bfloat16;
    constexpr int KI = K / 32, VC = V / 64, VJ = V / 16, HT = 8 * NT;
    __shared__ Partial<HT, V> sm;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    if (!SHARES && a.split == kCluster) cluster_started();
    after_previous();
    Work<16, HT, SHARES> wk;
    __shared__ typename Work<16, HT, SHARES>::Share share;
#pragma unroll 1
    for (bool more = wk.start(a, share); more; more = wk.next(a, share)) {
        const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
        Rows<16>& rows = wk.rows;
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
        join<TI, V, HT, SHARES, Work<16, HT, SHARES>>(a, share, sm);
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
template <int K, int V, int HT, int R>
__global__ void __launch_bounds__(kWarps * 32, simt_ctas(HT, K, V)) k_attend_simt(AttendArgs a) {
    constexpr int KL = K / 32, VL = V / 32, NV = R * HT;
    __shared__ Partial<HT, V> sm;
    const int lane = threadIdx.x % 32;
    if (a.split == kCluster) cluster_started();
    after_previous();
    typedef Work<R, HT, false> Wk;
    Wk wk;
    __shared__ typename Wk::Share share;
    if (!wk.start(a, share)) return;
    const int h0 = wk.h0, heads = wk.heads, warp = wk.warp;
    Rows<R>& rows = wk.rows;
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
    join<float, V, HT, false, Wk>(a, share, sm);
}

// ------------------------------------------------------------------ launch

// Query heads that a CTA takes together.
int head_tile(const kda_cache* c, int HQ) {
    const int group = HQ / c->HKV;
    if (c->dtype == KDA_DTYPE_BF16) return group <= 8 ? 8 : 16;
    return group == 1 ? 1 : group <= 4 ? 4 : 8;
}

struct Plan {
    Split split;
    int parts, ht, units, turn;
    dim3 grid;
    size_t acc_bytes, ml_bytes, ws_bytes;  // of the workspace
};
// What a plan goes by besides the sizes: the device's SMs, and the largest cluster that the kernel can be placed in.
struct Gpu {
    int sms, cluster;
};
Plan plan_of(const kda_cache* c, int HQ, int N, int max_pages, int window, const Gpu& gpu) {
    const bool bf16 = c->dtype == KDA_DTYPE_BF16;
    const int group = HQ / c->HKV, ht = head_tile(c, HQ), units = c->HKV * ((group + ht - 1) / ht);
    const int turn = kWarps * (bf16 ? 16 : simt_rows(ht));
    int64_t rows = (int64_t)max_pages * c->page_size;
    if (window > 0 && window < rows) rows = window;
    const int64_t turns = rows > turn ? (rows + turn - 1) / turn : 1;  // of a unit
    const int64_t all = (int64_t)(N > 0 ? N : 1) * units;              // units
    const int slots = gpu.sms * (bf16 ? mma_ctas(ht / 8, c->K, c->V) : simt_ctas(ht, c->K, c->V));
    Plan p{kWhole, 1, ht, units, turn};
    // What each split costs, in turns (0.6 to 0.9 us) of a CTA that takes all of its rows in turn: fitted to 1600 times
    // of all splits. The CTAs of an SM start one after the other. Those that do not fit take the places of others that
    // end: with lengths that differ, the sequences of a batch have about 0.7 of the rows of all as long as the longest
    // that fits; with equal lengths the last wave takes almost as long as a full one. The cost is the mean of the two.
    const double mean = N > 1 ? 0.7 : 1.0;
    const auto begin = [&](int64_t ctas) { return (double)(ctas < slots ? ctas : slots) / gpu.sms; };
    const auto queue = [&](int64_t ctas) {
        const double x = (double)ctas / slots;
        return x > 1 ? (1 + mean) / 2 * x + (1 - mean) / 2 + 0.4 * (ceil(x) - x) : 1.0;
    };
    double least = turns * queue(all) + begin(all);
    // Clusters need room for all of their CTAs in one part of the GPU: of the SMs' room, clusters of 16 find 74 % (21 of
    // 28 clusters; the next one waits for the others' end, 7.0 -> 11.3 us), of 8 89 %, of 4 96 % (109 clusters in 456
    // places; 110 take 26.0 instead of 22.9 us, 111 31.5, where parts take 24.1. In 608 and 760 places 97 % are found).
    // None is to wait: that gains up to a quarter where lengths differ, and costs as much where they are equal (192
    // units, fp32, K = V = 64, of U[1,1500] and of 1500 rows with a window of 1024: 14.5 and 24.6 us; parts 16.4, 19.2).
    constexpr struct {
        int ctas, room;
        double join;
    } clusters[] = {{2, 100, 1.2}, {4, 96, 1.2}, {8, 89, 1.7}, {16, 73, 2.4}};
    for (const auto& x : clusters) {
        if (all * x.ctas * 100 > (int64_t)slots * x.room || x.ctas >= 2 * turns || x.ctas > gpu.cluster) continue;
        const double cost = x.join + (turns + x.ctas - 1) / x.ctas + begin(all * x.ctas);
        if (cost >= least) continue;
        least = cost;
        p.split = kCluster;
        p.parts = x.ctas;
    }
    // Parts, and the second kernel: as many as fit. fp32, sequences of several lengths: `times` as many, so that others
    // take the places of those that end early, which evens them out: T turns of a CTA become T (mean + (1 - mean) /
    // times), and each time costs a start of 0.9. (152 sequences of U[1,16000], K = V = 128, five heads: 414 -> 266 us;
    // of 16000: 465 -> 480.)
    const double each_fit = (double)turns * all / slots;
    const int times = bf16 || N <= 1 || each_fit < 12 ? 1 : each_fit > 192 ? 8 : (int)sqrt(each_fit / 3);
    int64_t parts = (int64_t)slots * times / all;
    if (parts > turns) parts = turns;
    if (parts > 1) {
        const int64_t each = (turns + parts - 1) / parts;
        parts = (turns + each - 1) / each;
        const double cost = 3.6 + each * queue(all * parts) + begin(all * parts);
        if (cost < least) {
            least = cost;
            p.split = kParts;
            p.parts = (int)parts;
        }
    }
    // Shares add up the lengths first, and have the ends of units within them. With fp32 the loop over units costs
    // registers, and 20 to 50 % of the time.
    const double shares = 6.0 + mean * (turns + kUnitTurns) * all / slots + begin(slots);
    if (bf16 && (turns + kUnitTurns) * all < INT32_MAX && shares < least) {
        p.split = kShares;
        p.parts = slots;
    }
    p.grid = p.split == kShares ? dim3(p.parts) : dim3(units * p.parts, N);
    p.ws_bytes = KDA_ATTEND_WORKSPACE_MIN;
    if (p.split >= kParts) {
        const size_t held = p.split == kParts ? (size_t)all * p.parts : (size_t)p.parts * 2;
        p.acc_bytes = held * ht * c->V * sizeof(float);
        p.ml_bytes = held * ht * sizeof(float2);
        p.ws_bytes += p.acc_bytes + p.ml_bytes + (size_t)all * sizeof(int2);
    }
    return p;
}

typedef void (*Kernel)(AttendArgs);

template <int K, int V> Kernel kernel_of(bool bf16, int ht, Split split) {
    if (bf16 && split == kShares) return ht == 8 ? k_attend_mma<K, V, 1, true> : k_attend_mma<K, V, 2, true>;
    if (bf16) return ht == 8 ? k_attend_mma<K, V, 1, false> : k_attend_mma<K, V, 2, false>;
    return ht == 1   ? k_attend_simt<K, V, 1, simt_rows(1)>
           : ht == 4 ? k_attend_simt<K, V, 4, simt_rows(4)>
                     : k_attend_simt<K, V, 8, simt_rows(8)>;
}
Kernel kernel_of(const kda_cache& c, int ht, Split split) {
    const bool bf16 = c.dtype == KDA_DTYPE_BF16;
    return c.K == 128 ? (c.V == 128 ? kernel_of<128, 128>(bf16, ht, split) : kernel_of<128, 64>(bf16, ht, split))
                      : (c.V == 128 ? kernel_of<64, 128>(bf16, ht, split) : kernel_of<64, 64>(bf16, ht, split));
}
// The present device and what it can do with the kernel for these sizes; without a device, what a GB300 can. A part of
// a GPU may have fewer SMs, and none of its processing clusters 16 of them.
Gpu gpu_for(const kda_cache* c, int HQ) {
    static std::atomic<int> known[5][2][2][kDevices];
    const int ht = head_tile(c, HQ);
    const int tile = c->dtype == KDA_DTYPE_BF16 ? ht / 16 : ht == 1 ? 2 : ht == 4 ? 3 : 4;
    const int device = present_device();
    return {sm_count(device), largest_cluster(device, (const void*)kernel_of(*c, ht, kCluster), kWarps * 32, kMaxCluster,
                                              known[tile][c->K / 128][c->V / 128])};
}

template <typename TI, int V, int HT, int VS, int G, int THREADS>
cudaError_t launch_join(const AttendArgs& a, cudaStream_t st) {
    const int64_t threads = (int64_t)a.N * a.HQ * (V / 4) * G;
    const unsigned grid = (unsigned)((threads + THREADS - 1) / THREADS);
    if constexpr (sizeof(TI) == 2)
        if (a.split == kShares) return launch_after(k_attend_join<TI, V, HT, VS, G, THREADS, true>, a, grid, THREADS, st);
    return launch_after(k_attend_join<TI, V, HT, VS, G, THREADS, false>, a, grid, THREADS, st);
}
// `parts`: of a unit, with equal lengths. A batch of loads is to cover them.
int join_groups(int64_t parts) { return parts <= kJoinBatch ? 1 : parts <= 4 * kJoinBatch ? 4 : 32; }
template <typename TI, int V, int HT> cudaError_t launch_join(const AttendArgs& a, int64_t parts, cudaStream_t st) {
    const int groups = join_groups(parts);
    if (groups == 1) return launch_join<TI, V, HT, V, 1, 128>(a, st);
    if (groups == 4) return launch_join<TI, V, HT, V, 4, 128>(a, st);
    return launch_join<TI, V, HT, 32, 32, 256>(a, st);
}
template <int V> cudaError_t launch_join(const AttendArgs& a, bool bf16, int ht, int64_t parts, cudaStream_t st) {
    if (bf16)
        return ht == 8 ? launch_join<__nv_bfloat16, V, 8>(a, parts, st) : launch_join<__nv_bfloat16, V, 16>(a, parts, st);
    return ht == 1   ? launch_join<float, V, 1>(a, parts, st)
           : ht == 4 ? launch_join<float, V, 4>(a, parts, st)
                     : launch_join<float, V, 8>(a, parts, st);
}

// Parts of a unit, with equal lengths (kParts, kShares).
int64_t unit_parts(const Plan& p, int N) {
    return p.split == kParts ? p.parts : p.parts / ((int64_t)(N > 0 ? N : 1) * p.units) + 2;
}

cudaError_t launch_attend(const AttendArgs& a, const Plan& p, cudaStream_t st) {
    const bool bf16 = a.c.dtype == KDA_DTYPE_BF16;
    const int V = a.c.V;
    cudaError_t e = launch_after(kernel_of(a.c, p.ht, p.split), a, p.grid, kWarps * 32, st, p.split == kCluster ? p.parts : 1);
    if (e != cudaSuccess) return e;
    static const char* const names[] = {"cache_attend", "cache_attend_cluster", "cache_attend_parts",
                                        "cache_attend_shares"};
    note_launch(names[p.split], st);
    if (p.split < kParts) return cudaSuccess;
    const int64_t parts = unit_parts(p, a.N);
    e = V == 128 ? launch_join<128>(a, bf16, p.ht, parts, st) : launch_join<64>(a, bf16, p.ht, parts, st);
    if (e != cudaSuccess) return e;
    note_launch("cache_attend_join", st);
    return cudaSuccess;
}

kda_status check_sizes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window) {
    const kda_status s = check_cache(c);
    if (s != KDA_OK) return s;
    if (N < 0 || HQ < 1 || HQ % c->HKV != 0 || max_pages < 0 || window < 0) return KDA_ERR_INVALID_ARG;
    if (N > 65535 || HQ > 65535 || (int64_t)N * HQ > (1 << 24) || (int64_t)max_pages * c->page_size > (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_cache_attend_workspace_bytes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                   int32_t window) {
    if (check_sizes(c, HQ, N, max_pages, window) != KDA_OK) return 0;
    return plan_of(c, HQ, N, max_pages, window, gpu_for(c, HQ)).ws_bytes;
}

extern "C" kda_status kda_debug_attend_plan(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window,
                                            int32_t sms, int32_t cluster, int32_t* plan) {
    const kda_status s = check_sizes(c, HQ, N, max_pages, window);
    if (s != KDA_OK) return s;
    if (!plan) return KDA_ERR_INVALID_ARG;
    const Gpu gpu = sms > 0 ? Gpu{sms, cluster} : gpu_for(c, HQ);
    const Plan p = plan_of(c, HQ, N, max_pages, window, gpu);
    plan[0] = p.split;
    plan[1] = p.parts;
    plan[2] = p.split < kParts ? 0 : join_groups(unit_parts(p, N));
    plan[3] = p.units * (N > 0 ? N : 1);
    return KDA_OK;
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
    const Plan plan = plan_of(c, HQ, N, max_pages, window, gpu_for(c, HQ));
    if (!ws || !aligned16(ws) || ws_bytes < plan.ws_bytes) return KDA_ERR_WORKSPACE;
    char* w = (char*)ws;
    const int step = plan.turn * (plan.split == kShares ? 1 : plan.parts);
    AttendArgs a;
    a.c = *c;
    a.q = q;
    a.q_stride = q_stride;
    a.table_stride = table_stride;
    a.HQ = HQ;
    a.N = N;
    a.max_pages = max_pages;
    a.window = window;
    a.table = page_table;
    a.kv_lens = kv_lens;
    a.scale_log2 = scale * kLog2e;
    a.o = o;
    a.lse = lse;
    a.status = status;
    a.group = HQ / c->HKV;
    a.tiles = plan.units / c->HKV;
    a.units = plan.units;
    a.page = Divisor(c->page_size);
    a.step = step;
    a.step_pg = step / c->page_size;
    a.step_off = step % c->page_size;
    a.split = plan.split;
    a.parts = plan.parts;
    a.by_parts = Divisor(plan.parts);
    a.turn = plan.turn;
    a.part_acc = (float4*)w;
    a.part_ml = (float2*)(w + plan.acc_bytes);
    a.unit_parts = (int2*)(w + plan.acc_bytes + plan.ml_bytes);
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const cudaError_t e = launch_attend(a, plan, st);
    if (e != cudaSuccess) return cuda_fail(e);
    return KDA_OK;
}
