// kda_cache8_append: new keys and values into a paged cache in 8 bits, keys and queries rotated by their position on the
// way. Declared in include/kda_serve.h.
//
// Of a block of rows of a page and head, with x its values in fp32 and s its scale,
//   s = 2^e, the smallest with max |x| <= 448 s,   c = e4m3(x / s),
// and where the block has rows c_old in units of s_old already: s = max(s_old, what the new rows want), and, if that is
// more than s_old, c_old <- e4m3(c_old s_old / s). A power of two divides without rounding, so a value is rounded once, and
// again only where it comes to lie below e4m3's normal values.
//
// Bound: every new row is read once and written once in half or a quarter of its bytes, every query read and written.
//   Several rows of each sequence: tiles of 16 rows or more in whole blocks, eight threads to a row, one head after the
//     other. A thread keeps its angles for all heads; rows come in ahead of their use through shared memory (cp.async: without
//     it 4 us more); the largest value of a block is an atomicMax in shared memory, whose order does not matter. 16 packed
//     prompts of U[1,4096] tokens, 32 query and 8 cache heads of 128, bf16, blocks of 16 (760 MB): 120 us, 6.3 TB/s. The tiles
//     alone (202 MB) take 40, bound by issue slots (72 %, 245 instructions for 16 values of a thread), the queries alone 83,
//     bound by the memory: a launch has them side by side, one CTA in four a tile (one after the other: 124). A warp to a
//     block of one head, which reads the rows twice and angles for each head: 163 us.
//   Few rows of each sequence (less than 8 on average) or blocks longer than 128: a warp has a block of one head to itself.
//     One token of each of 128 sequences 3.5 us in a graph, of one 2.4 (tiles, most of whose threads have no row: 5.2 to 13
//     and 2.5; from 8 rows on they are faster: 16 x 16 rows 4.4 and 8.1 us). Queries go with the same launch where that is
//     small, as CTAs of their own, and otherwise to a launch of 64 threads a CTA, 16 to an SM.
#include <cfloat>

#include "kda_cache.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kTileThreads = 1024;  // at most

// Lengths up to which rows are appended. Without any, 2^31 more than each sequence has, which no row reaches: the load goes
// beside that of the length (to ask whether there are any takes 0.1 us of a token's 2.5).
struct Granted {
    const int32_t* lens;
    unsigned more;
    Granted(const int32_t* granted, const int32_t* kv_lens) : lens(granted ? granted : kv_lens), more(granted ? 0u : 1u << 31) {}
    __device__ __forceinline__ unsigned limit(unsigned n) const { return (unsigned)max(lens[n], 0) + more; }
};

struct Append8Args {
    kda_cache8 c;
    const void *k, *v, *q;
    void* q_out;
    int64_t k_stride, v_stride, q_stride, table_stride;
    int HQ, N;
    unsigned R, per;  // new rows; of a sequence, where there is no cu
    const int64_t* cu;
    const float* rope;
    int rope_len, rope_dim, interleaved;
    const int32_t *table, *kv_lens;
    Granted granted;
    int max_pages;
    int32_t* status;
    int unit;                  // rows of an item: of a block, or of a tile of blocks
    unsigned items, splits;    // items, at most; CTAs of each
    unsigned most;             // items of a sequence, where there is no cu
    unsigned q_lanes, q_rows;  // query rows: threads of a row, rows of a CTA
    unsigned mix;              // CTAs of which one has a tile, the others queries
    Divisor by_unit, by_most, by_per, by_block, by_page;
};
// The page of a position. (Divisor is for numbers below 2^31.)
__device__ __forceinline__ unsigned page_of(const Append8Args& a, unsigned pos) {
    return pos < 1u << 31 ? a.by_page(pos) : pos / (unsigned)a.c.cache.page_size;
}

// C channels of a row (4 or 8) as they are.
template <typename TI, int C> struct Run {
    static constexpr int kBytes = C * sizeof(TI);
    uint32_t w[kBytes / 4];
    __device__ __forceinline__ void load(const TI* p) {
        if constexpr (kBytes == 8) {
            const uint2 x = *(const uint2*)p;
            w[0] = x.x, w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 x = ((const uint4*)p)[i];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void store(TI* p) const {
        if constexpr (kBytes == 8) {
            *(uint2*)p = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) ((uint4*)p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void values(float* x) const {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
            if constexpr (sizeof(TI) == 2) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
            if constexpr (sizeof(TI) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *(const uint32_t*)&b;
            } else {
                w[i] = __float_as_uint(x[i]);
            }
        }
    }
};

// A lane's share of a row: C channels from `a` on and C from `b` on. Where they turn, channel a + i turns with b + i, or, in
// pairs, with its neighbour. (rope_dim is a multiple of 16.)
template <int C> struct Share {
    int a, b;
    bool turns;
    __device__ __forceinline__ Share(int u, int rope_dim, int interleaved) {
        const int apart = interleaved ? 0 : rope_dim / (2 * C);
        turns = u < rope_dim / (2 * C);
        a = u < apart ? C * u : 2 * C * u;
        b = u < apart ? C * u + rope_dim / 2 : 2 * C * u + C;
    }
};
// The cosines and sines of a lane's share at a position.
template <int C> struct Angles {
    float co[C], si[C];
    __device__ __forceinline__ void load(const Share<C>& s, const float* rope, int64_t pos, int rope_dim, int interleaved) {
        const float* p = rope + pos * rope_dim + (interleaved ? s.a / 2 : s.a);
        Run<float, C> x, y;
        x.load(p);
        y.load(p + rope_dim / 2);
        x.values(co);
        y.values(si);
    }
    __device__ __forceinline__ void pair(float& p, float& q, int i) const {
        const float u = __fsub_rn(__fmul_rn(p, co[i]), __fmul_rn(q, si[i]));
        q = __fadd_rn(__fmul_rn(q, co[i]), __fmul_rn(p, si[i]));
        p = u;
    }
    // The rotation, each product and each sum rounded by itself, so that the scales, which go by the largest value, do not
    // depend on how a compiler joins them. (Instructions for two values at once are joined even where they say .rn.)
    __device__ __forceinline__ void turn(float (&x)[2 * C], int interleaved) const {
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < C; ++i) pair(x[2 * i], x[2 * i + 1], i);
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) pair(x[i], x[C + i], i);
        }
    }
};

// 4 values times f as e4m3 (a NaN as one; an infinite value would become the largest).
__device__ __forceinline__ uint32_t to_e4m3(const float* x, float f) {
    uint32_t w;
    asm("{.reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;"
        " mov.b32 %0, {lo, hi};}"
        : "=r"(w)
        : "f"(x[0] * f), "f"(x[1] * f), "f"(x[2] * f), "f"(x[3] * f));
    return w;
}
template <int C> __device__ __forceinline__ void store_e4m3(unsigned char* p, const float* x, float f) {
    if constexpr (C == 8)
        *(uint2*)p = make_uint2(to_e4m3(x, f), to_e4m3(x + 4, f));
    else
        *(uint32_t*)p = to_e4m3(x, f);
}
// 4 e4m3 values in fp32.
__device__ __forceinline__ void from_e4m3(uint32_t x, float* y) {
    asm("{.reg .b16 lo, hi, a, b; .reg .b32 p; mov.b32 {lo, hi}, %4; cvt.rn.f16x2.e4m3x2 p, lo; mov.b32 {a, b}, p;"
        " cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; cvt.rn.f16x2.e4m3x2 p, hi; mov.b32 {a, b}, p; cvt.f32.f16 %2, a;"
        " cvt.f32.f16 %3, b;}"
        : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3])
        : "r"(x));
}

// The exponent field of the smallest power of two, 2^-126 at least, by which values of this magnitude (finite) come to
// 448 = 1.75 2^8 at most.
__device__ __forceinline__ int least_scale(float top) { return max(((__float_as_int(top) + 0x1fffff) >> 23) - 8, 1); }
// And of the smallest that is not below a scale's magnitude (0 where it is 0 or not finite; 2^126, the largest whose
// reciprocal is a normal number, for what is above it).
__device__ __forceinline__ int held_scale(float s) {
    const int bits = __float_as_int(fabsf(s));
    return bits >= 0x7f800000 || bits == 0 ? 0 : min(max((bits + 0x7fffff) >> 23, 1), 253);
}

// N old values in the units of another scale (ratio: old to new; of one that is not finite they are NaNs).
template <int N> __device__ __forceinline__ void again(unsigned char* p, float ratio) {
    uint32_t* w = (uint32_t*)p;
    if (!(fabsf(ratio) <= FLT_MAX)) ratio = NAN;
    uint32_t old[N / 4];
    if constexpr (N == 16) {
        const uint4 x = *(const uint4*)p;
        old[0] = x.x, old[1] = x.y, old[2] = x.z, old[3] = x.w;
    } else {
        const uint2 x = *(const uint2*)p;
        old[0] = x.x, old[1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        float y[4];
        from_e4m3(old[i], y);
        if (fabsf(ratio) > 1.f) {  // (a scale above 2^126: what it makes larger than 448 2^126 is not held)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (fabsf(y[e] * ratio) > 448.f) y[e] = NAN;
        }
        w[i] = to_e4m3(y, ratio);
    }
}
// The largest finite magnitude; infinite values become NaNs.
template <int N> __device__ __forceinline__ float largest(float (&x)[N]) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(x[e]));  // (not of a NaN)
    if (top == INFINITY) {
        top = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (fabsf(x[e]) == INFINITY) x[e] = NAN;
            top = fmaxf(top, fabsf(x[e]));
        }
    }
    return top;
}

// Rows [first, last) of the positions of a block that begins at `start`, of one head: D channels each of `x`, whose row of
// position `first` is at `from` (rows `stride` apart), into `to`, position `start`'s row of the cache, rows `step` apart.
template <typename TI, int D>
__device__ __forceinline__ void write_block(const Append8Args& a, const TI* from, int64_t stride, unsigned char* to,
                                            int64_t step, float* scale, unsigned start, unsigned old_end, unsigned first,
                                            unsigned last, bool rotated) {
    constexpr int L = D / 16, P = 32 / L;  // lanes of a row, rows of a turn
    const int lane = threadIdx.x % 32, in = lane / L;
    const Share<8> s(lane % L, rotated ? a.rope_dim : 0, a.interleaved);
    const float before = start < old_end ? *scale : 0.f;
    const unsigned rows = last - first;
    float x[16], top = 0.f;
    const auto load = [&](unsigned row) {
        const TI* p = from + (int64_t)row * stride;
        Run<TI, 8> lo, hi;
        Angles<8> angles;
        lo.load(p + s.a);
        hi.load(p + s.b);
        if (s.turns) angles.load(s, a.rope, first + row, a.rope_dim, a.interleaved);
        lo.values(x);
        hi.values(x + 8);
        if (s.turns) angles.turn(x, a.interleaved);
    };
#pragma unroll 1
    for (unsigned row = in; row < rows; row += P) {
        load(row);
        top = fmaxf(top, largest(x));
    }
#pragma unroll
    for (int w = 1; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    const int field = max(least_scale(top), held_scale(before));
    const float now = __int_as_float(field << 23), f = __int_as_float((254 - field) << 23);
    if (start < old_end && before != now)  // the block's rows in the new units
#pragma unroll 2
        for (unsigned row = in; row < old_end - start; row += P) again<16>(to + row * step + (lane % L) * 16, before * f);
    if (lane == 0 && before != now) *scale = now;
#pragma unroll 1
    for (unsigned row = in; row < rows; row += P) {
        if (rows > P) {
            load(row);
            largest(x);
        }
        unsigned char* p = to + (first - start + row) * step;
        store_e4m3<8>(p + s.a, x, f);
        store_e4m3<8>(p + s.b, x + 8, f);
    }
}

// Where sequence n begins, of the rows that there are.
__device__ __forceinline__ int64_t row_at(const int64_t* cu, int n, unsigned R) { return min(max(cu[n], (int64_t)0), (int64_t)R); }
// The sequence that new row r or, with `unit`, item r of the launch's belongs to: the last n that begins at or before it. A
// sequence whose first row is cu[n] has items of so many rows from cu[n] / unit + 2 n on: two more than its rows fill, as
// many as it may begin and end in.
__device__ __forceinline__ int seq_of(const int64_t* cu, int N, int64_t r, unsigned R, const Divisor* unit) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((unit ? (*unit)((unsigned)row_at(cu, mid, R)) + 2 * (int64_t)mid : cu[mid]) <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void flag(const Append8Args& a) {
    if (a.status) *a.status = KDA_ERR_INVALID_ARG;
}

// The positions that item `item` of the launch appends, a.unit of them at most, from a multiple of it on:
// [max(start, len), stop) of sequence n, whose first new row is `begin`. False if there are none. (Rows that were not granted
// are dropped like those of an inactive sequence.)
struct Item {
    int n, len;
    int64_t begin, start, stop;
};
__device__ __forceinline__ bool find_item(const Append8Args& a, unsigned item, Item& x) {
    int n;
    unsigned j;
    int64_t begin, end;
    if (a.cu) {
        n = seq_of(a.cu, a.N, item, a.R, &a.by_unit);
        begin = a.cu[n];
        end = a.cu[n + 1];
        if (item == 0 && threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.N] != a.R)) flag(a);  // rows of no sequence
        if (begin < 0 || end < begin || end > a.R) {
            if (threadIdx.x == 0) flag(a);
            end = min(end, (int64_t)a.R);  // (rows that are there are appended)
            if (begin < 0 || end < begin) return false;
        }
        j = item - (a.by_unit((unsigned)begin) + 2 * n);
    } else {
        n = a.by_most(item);
        j = item - n * a.most;
        begin = (int64_t)n * a.per;
        end = begin + a.per;
    }
    const int len = a.kv_lens[n];
    const unsigned limit = a.granted.limit(n);
    if (len < 0 || begin == end) return false;
    const int64_t start = ((int64_t)a.by_unit(len) + j) * a.unit, stop = min(len + (end - begin), (int64_t)limit);
    x = {n, len, begin, start, min(stop, start + a.unit)};
    return start < stop && len < stop;
}

// A block of rows, the CTA's share of its heads.
template <typename TI> __device__ __forceinline__ void append_block(const Append8Args& a, unsigned item, unsigned split) {
    const kda_cache& c = a.c.cache;
    Item it;
    if (!find_item(a, item, it)) return;
    const int n = it.n, len = it.len;
    const unsigned from = (unsigned)it.start, first = max(from, (unsigned)len);
    unsigned last = (unsigned)it.stop;
    const unsigned pg = page_of(a, from), row = from - pg * c.page_size;
    int64_t page = -1;
    if (pg < (unsigned)a.max_pages) page = a.table[n * a.table_stride + pg];
    if (page < 0 || page >= c.num_pages || (a.rope && last > (unsigned)a.rope_len)) {
        if (threadIdx.x == 0) flag(a);
        if (page < 0 || page >= c.num_pages) return;
        last = min(last, (unsigned)a.rope_len);
        if (first >= last) return;
    }
    const int64_t r = it.begin + (first - (unsigned)len), b = a.by_block(row);
    const unsigned slabs = 2 * (unsigned)c.HKV;
    for (unsigned i = split * kWarps + threadIdx.x / 32; i < slabs; i += a.splits * kWarps) {
        const bool keys = i < (unsigned)c.HKV;
        const int h = keys ? i : i - c.HKV, D = keys ? c.K : c.V;
        const TI* x = keys ? (const TI*)a.k + r * a.k_stride : (const TI*)a.v + r * a.v_stride;
        const int64_t stride = keys ? a.k_stride : a.v_stride, step = keys ? c.k_row : c.v_row;
        unsigned char* to = keys ? (unsigned char*)c.k + page * c.k_page + h * c.k_head
                                 : (unsigned char*)c.v + page * c.v_page + h * c.v_head;
        float* scale = keys ? a.c.k_scale + page * a.c.k_scale_page + b * a.c.k_scale_block + h * a.c.k_scale_head
                            : a.c.v_scale + page * a.c.v_scale_page + b * a.c.v_scale_block + h * a.c.v_scale_head;
        to += row * step;
        x += (int64_t)h * D;
        if (D == 128)
            write_block<TI, 128>(a, x, stride, to, step, scale, from, (unsigned)len, first, last, keys && a.rope);
        else
            write_block<TI, 64>(a, x, stride, to, step, scale, from, (unsigned)len, first, last, keys && a.rope);
    }
}

// A thread's share of a row on its way to shared memory, of the heads ahead: C channels, twice, in pieces of 16 bytes or 8,
// the threads' pieces side by side.
template <typename TI, int C> struct Ahead {
    static constexpr int kHeads = sizeof(TI) == 2 ? 4 : 3;  // under way or in use
    static constexpr int kPiece = C * sizeof(TI) < 16 ? 8 : 16, kOfRun = C * sizeof(TI) / kPiece;
    static constexpr size_t bytes(int threads) { return (size_t)kHeads * threads * 2 * C * sizeof(TI); }
    uint32_t at, stage = 0, stages;
    __device__ __forceinline__ explicit Ahead(const void* shared) {
        at = (uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * kPiece;
        stages = blockDim.x * 2 * C * sizeof(TI);
    }
    // Piece i of the head that is `ahead` of the present one.
    __device__ __forceinline__ uint32_t piece(int ahead, int i) const {
        const uint32_t k = stage + ahead;
        return at + (k < kHeads ? k : k - kHeads) * stages + i * blockDim.x * kPiece;
    }
    __device__ __forceinline__ void fetch(int ahead, const TI* a, const TI* b) const {
#pragma unroll
        for (int i = 0; i < 2 * kOfRun; ++i) {
            const char* p = (const char*)(i < kOfRun ? a : b) + i % kOfRun * kPiece;
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(piece(ahead, i)), "l"(p), "n"(kPiece) : "memory");
        }
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // The present head's, once all groups but the newest kHeads - 1 are there.
    __device__ __forceinline__ void take(Run<TI, C>& a, Run<TI, C>& b) const {
#pragma unroll
        for (int i = 0; i < 2 * kOfRun; ++i) {
            uint32_t* w = (i < kOfRun ? a : b).w + i % kOfRun * (kPiece / 4);
            if constexpr (kPiece == 8)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(piece(0, i)) : "memory");
            else
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(piece(0, i))
                             : "memory");
        }
    }
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kHeads - 1) : "memory"); }
    __device__ __forceinline__ void next() { stage = stage + 1 == kHeads ? 0 : stage + 1; }
};

// A tile of rows, a.unit of them at most, in whole blocks, of some heads of keys or of values: eight threads to a row, each
// with the angles of its channels in registers, one head after the other, the next ones' rows on their way meanwhile.
template <typename TI, int D, bool KEYS>
__device__ __forceinline__ void append_tile(const Append8Args& a, unsigned item, int head, int heads) {
    constexpr int C = D / 16;
    __shared__ unsigned tops[3][kTileThreads / 8];  // of each block, of a head, of the next one, and of the one after
    extern __shared__ uint4 shared[];
    const kda_cache& c = a.c.cache;
    const int block = a.c.block, row = threadIdx.x / 8, u = threadIdx.x % 8, mine = a.by_block(row);
    Item it;
    if (!find_item(a, item, it)) return;
    const int len = it.len;
    const int64_t pos = it.start + row, first = it.start + mine * block;  // the row's, and its block's first
    const int64_t first_new = max(first, (int64_t)len);
    const bool rotated = KEYS && a.rope;
    bool live = row < a.unit && first + block > len && first_new < it.stop;  // the block has a new row
    int64_t page = -1;
    unsigned in = 0;
    if (live) {
        const unsigned pg = page_of(a, (unsigned)pos);
        in = (unsigned)pos - pg * c.page_size;
        if (pg < (unsigned)a.max_pages) page = a.table[it.n * a.table_stride + pg];
        const bool no_page = page < 0 || page >= c.num_pages, no_angle = a.rope && pos < it.stop && pos >= a.rope_len;
        if (u == 0 && (no_page || no_angle)) flag(a);
        live = !no_page && !(a.rope && first_new >= a.rope_len);
    }
    const bool fresh = live && pos >= len && pos < it.stop && !(a.rope && pos >= a.rope_len);
    const bool old = live && pos < len, held = live && first < len;
    const Share<C> s(u, rotated ? a.rope_dim : 0, a.interleaved);
    Angles<C> angles;
    const bool turns = fresh && s.turns;
    if (turns) angles.load(s, a.rope, pos, a.rope_dim, a.interleaved);
    const TI* from = (KEYS ? (const TI*)a.k : (const TI*)a.v) + head * D;
    unsigned char* to = KEYS ? (unsigned char*)c.k + head * c.k_head : (unsigned char*)c.v + head * c.v_head;
    float* scale = KEYS ? a.c.k_scale + head * a.c.k_scale_head : a.c.v_scale + head * a.c.v_scale_head;
    if (live) {
        from += (it.begin + (pos - len)) * (KEYS ? a.k_stride : a.v_stride);
        to += page * (KEYS ? c.k_page : c.v_page) + in * (KEYS ? c.k_row : c.v_row);
        scale += page * (KEYS ? a.c.k_scale_page : a.c.v_scale_page) + a.by_block(in) * (KEYS ? a.c.k_scale_block : a.c.v_scale_block);
    }
    for (int i = threadIdx.x; i < 3 * (kTileThreads / 8); i += blockDim.x) ((unsigned*)tops)[i] = 0;
    Ahead<TI, C> ahead(shared);
#pragma unroll
    for (int i = 0; i < ahead.kHeads - 1; ++i) {
        if (fresh && i < heads) ahead.fetch(i, from + i * D + s.a, from + i * D + s.b);
        ahead.commit();
    }
    from += (ahead.kHeads - 1) * D;
    __syncthreads();
    for (int h = 0, now_top = 0; h < heads; ++h) {
        float x[2 * C], top = 0.f, before = 0.f;
        if (held) before = *scale;
        if (fresh && h + ahead.kHeads - 1 < heads) ahead.fetch(ahead.kHeads - 1, from + s.a, from + s.b);
        ahead.commit();
        from += D;
        ahead.wait();
        if (fresh) {
            Run<TI, C> lo, hi;
            ahead.take(lo, hi);
            lo.values(x);
            hi.values(x + C);
            if (turns) angles.turn(x, a.interleaved);
            top = largest(x);
        }
#pragma unroll
        for (int w = 1; w < 8; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        if (u == 0 && fresh) atomicMax(&tops[now_top][mine], __float_as_uint(top));  // (the order does not matter)
        __syncthreads();
        const int field = max(least_scale(__uint_as_float(tops[now_top][mine])), held_scale(before));
        const float now = __int_as_float(field << 23), f = __int_as_float((254 - field) << 23);
        now_top = now_top == 2 ? 0 : now_top + 1;
        if (u == 0) tops[now_top == 2 ? 0 : now_top + 1][mine] = 0;  // (of the head after the next; last read before the barrier)
        if (fresh) {
            store_e4m3<C>(to + s.a, x, f);
            store_e4m3<C>(to + s.b, x + C, f);
            if (u == 0 && pos == first_new && before != now) *scale = now;
        } else if (old && before != now) {
            again<2 * C>(to + u * 2 * C, before * f);
        }
        ahead.next();
        to += KEYS ? c.k_head : c.v_head;
        scale += KEYS ? a.c.k_scale_head : a.c.v_scale_head;
    }
}

// Query rows: rotated, in their own type; 0 where the token's row is dropped or inactive.
template <typename TI> __device__ __forceinline__ void turn_queries(const Append8Args& a, unsigned cta) {
    const kda_cache& c = a.c.cache;
    unsigned lane = threadIdx.x;
    const unsigned in = lane / a.q_lanes;
    const int64_t r = (int64_t)cta * a.q_rows + in;
    lane -= in * a.q_lanes;
    if (in >= a.q_rows || r >= a.R) return;
    int n;
    unsigned idx;
    bool ok = true;
    if (a.cu) {
        n = seq_of(a.cu, a.N, r, a.R, nullptr);
        const int64_t begin = a.cu[n];
        ok = begin >= 0 && begin <= r && r < a.cu[n + 1];
        idx = (unsigned)(r - begin);
    } else {
        n = a.by_per((unsigned)r);
        idx = (unsigned)r - n * a.per;
    }
    const int len = a.kv_lens[n];
    const unsigned limit = a.granted.limit(n);
    const unsigned pos = (unsigned)len + idx, pg = page_of(a, pos);
    int64_t page = -1;
    if (len >= 0 && (pos < limit || !ok)) {
        ok = ok && pg < (unsigned)a.max_pages && (!a.rope || pos < (unsigned)a.rope_len);
        if (ok) page = a.table[n * a.table_stride + pg];
        if (page < 0 || page >= c.num_pages) {
            page = -1;
            if (lane == 0) flag(a);
        }
    }
    // (a thread has the same channels of several heads, so it reads its angles once)
    const unsigned L = c.K / 16, u = lane % L, step = a.q_lanes / L;
    const Share<8> s(u, a.rope_dim, a.interleaved);
    const bool turns = s.turns && page >= 0;
    Angles<8> angles;
    if (turns) angles.load(s, a.rope, pos, a.rope_dim, a.interleaved);
    const TI* from = (const TI*)a.q + r * a.q_stride;
    TI* to = (TI*)a.q_out + r * a.HQ * c.K;
    for (unsigned h = lane / L; h < (unsigned)a.HQ; h += step) {
        const int64_t at = (int64_t)h * c.K;
        Run<TI, 8> lo{}, hi{};
        if (page >= 0) {
            lo.load(from + at + s.a);
            hi.load(from + at + s.b);
        }
        if (turns) {
            float x[16];
            lo.values(x);
            hi.values(x + 8);
            angles.turn(x, a.interleaved);
            lo.set(x);
            hi.set(x + 8);
        }
        lo.store(to + at + s.a);
        hi.store(to + at + s.b);
    }
}

// A warp to a block. Queries in the same launch where that has no more than so many CTAs to an SM; else in their own.
constexpr int kFew = 32;
template <typename TI> __global__ void __launch_bounds__(kThreads, 4) k_append8(Append8Args a) {
    after_previous();
    const unsigned blocks = a.items * a.splits;
    if (blockIdx.x < blocks)
        append_block<TI>(a, blockIdx.x / a.splits, blockIdx.x % a.splits);
    else
        turn_queries<TI>(a, blockIdx.x - blocks);
}
constexpr int kQueryThreads = 64;
template <typename TI> __global__ void __launch_bounds__(kQueryThreads, 16) k_append8_queries(Append8Args a) {
    after_previous();
    turn_queries<TI>(a, blockIdx.x);
}
template <typename TI, int K, int V> __global__ void __launch_bounds__(kTileThreads) k_append8_tiles(Append8Args a) {
    after_previous();
    // (one CTA of a.mix has a tile, the others queries, so that what binds the ones leaves room for the others)
    const unsigned tiles = a.items * a.splits, at = blockIdx.x / a.mix, tile = min(at, tiles);
    if (at >= tiles || blockIdx.x != at * a.mix) {
        turn_queries<TI>(a, blockIdx.x - min(at + 1, tiles));
        return;
    }
    // (keys, then values, their heads in a.splits / 2 parts)
    const unsigned item = tile / a.splits, split = tile - item * a.splits, parts = a.splits / 2;
    const unsigned part = split < parts ? split : split - parts;
    const int head = (int)((uint64_t)part * a.c.cache.HKV / parts), end = (int)((uint64_t)(part + 1) * a.c.cache.HKV / parts);
    if (split < parts)
        append_tile<TI, K, true>(a, item, head, end - head);
    else
        append_tile<TI, V, false>(a, item, head, end - head);
}
template <typename TI, int K, int V>
cudaError_t launch_tiles(const Append8Args& a, unsigned ctas, int threads, cudaStream_t st) {
    // (the most that a kernel may ask for is set once on each device)
    static std::atomic<bool> known[kDevices];
    constexpr int C = (K > V ? K : V) / 16;
    const size_t shared = Ahead<TI, C>::bytes(threads);
    const int device = present_device();
    if (shared > 32 << 10 && (device < 0 || device >= kDevices || !known[device].load(std::memory_order_relaxed))) {
        const cudaError_t e = cudaFuncSetAttribute(k_append8_tiles<TI, K, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Ahead<TI, C>::bytes(kTileThreads));
        if (e != cudaSuccess) return e;
        if (device >= 0 && device < kDevices) known[device].store(true, std::memory_order_relaxed);
    }
    return launch_after(k_append8_tiles<TI, K, V>, a, ctas, threads, st, 1, shared);
}
template <typename TI> cudaError_t launch_tiles(const Append8Args& a, unsigned ctas, int threads, cudaStream_t st) {
    const int K = a.c.cache.K, V = a.c.cache.V;
    if (K == 128) return V == 128 ? launch_tiles<TI, 128, 128>(a, ctas, threads, st) : launch_tiles<TI, 128, 64>(a, ctas, threads, st);
    return V == 128 ? launch_tiles<TI, 64, 128>(a, ctas, threads, st) : launch_tiles<TI, 64, 64>(a, ctas, threads, st);
}
// Rows of a tile of whole blocks, and the threads for them: the fewest, from 16 rows on, of which most have a row. 0 where a
// block is longer than a CTA.
int tile_of(int block, int& threads) {
    int best = 0;
    threads = 0;
    for (int rows = 16; rows <= kTileThreads / 8; rows *= 2) {
        const int tile = rows / block * block;
        if (tile == 0 || (best > 0 && tile * (threads / 8) <= best * rows)) continue;  // no larger part of the threads
        best = tile;
        threads = 8 * rows;
        if (10 * tile >= 8 * rows) break;
    }
    return best;
}
// CTAs that append in units of so many rows, at most.
int64_t items_of(int64_t R, int64_t N, bool packed, int64_t unit) {
    const int64_t per = R / N;
    return packed ? R / unit + 2 * N : N * (per > 0 ? (per + unit - 2) / unit + 1 : 0);
}
// Query rows of a CTA of so many threads, and threads of a row.
constexpr unsigned kRowThreads = 64;
unsigned queries_of(Append8Args& a, int threads) {
    const unsigned tasks = a.HQ * (a.c.cache.K / 16), most = threads < kRowThreads ? threads : kRowThreads;
    if (tasks == 0) return 0;
    a.q_lanes = tasks < most ? tasks : most;
    a.q_rows = threads / a.q_lanes;
    return (a.R + a.q_rows - 1) / a.q_rows;
}
template <typename TI> cudaError_t launch(Append8Args a, bool tiles, int threads, cudaStream_t st) {
    const unsigned blocks = a.items * a.splits;
    if (tiles) {
        const unsigned queries = queries_of(a, threads);
        a.mix = queries / blocks + 1;
        return launch_tiles<TI>(a, blocks + queries, threads, st);
    }
    unsigned queries = queries_of(a, kThreads);
    const bool both = (int64_t)blocks + queries <= kFew * (int64_t)sm_count();
    const cudaError_t e = launch_after(k_append8<TI>, a, both ? blocks + queries : blocks, kThreads, st);
    if (e != cudaSuccess || both) return e;
    queries = queries_of(a, kQueryThreads);
    return queries ? launch_after(k_append8_queries<TI>, a, queries, kQueryThreads, st) : cudaSuccess;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_cache8_append(const kda_cache8* c8, const void* k, int64_t k_stride, const void* v,
                                        int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ,
                                        int32_t N, int64_t R, const int64_t* cu_seqlens, const float* rope,
                                        int32_t rope_len, int32_t rope_dim, int32_t interleaved,
                                        const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                        const int32_t* kv_lens, int32_t* status, kda_stream_t stream) {
    return kda_cache8_append_granted(c8, k, k_stride, v, v_stride, q, q_stride, q_out, HQ, N, R, cu_seqlens, rope, rope_len,
                                     rope_dim, interleaved, page_table, table_stride, max_pages, kv_lens, nullptr, status,
                                     stream);
}

extern "C" kda_status kda_cache8_append_granted(const kda_cache8* c8, const void* k, int64_t k_stride, const void* v,
                                                int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int32_t HQ,
                                                int32_t N, int64_t R, const int64_t* cu_seqlens, const float* rope,
                                                int32_t rope_len, int32_t rope_dim, int32_t interleaved,
                                                const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                                const int32_t* kv_lens, const int32_t* granted, int32_t* status,
                                                kda_stream_t stream) {
    const kda_status s = check_cache(c8);
    if (s != KDA_OK) return s;
    const kda_cache* c = &c8->cache;
    const bool bf16 = c8->dtype == KDA_DTYPE_BF16;
    // (scales that several blocks share are for reading)
    for (const int64_t* x : {&c8->k_scale_page, &c8->v_scale_page})
        if ((c->num_pages > 1 && x[0] == 0) || (c->page_size > c8->block && x[1] == 0) || (c->HKV > 1 && x[2] == 0))
            return KDA_ERR_INVALID_ARG;
    const AppendCall x{k, k_stride, v, v_stride, q, q_stride, q_out, HQ, N, R, cu_seqlens, rope, rope_len, rope_dim,
                       page_table, table_stride, max_pages, kv_lens, granted, status};
    const kda_status checked = check_append(c, x, bf16 ? 8 : 4);
    if (checked != KDA_OK || R == 0) return checked;
    // many rows of each sequence: tiles
    int threads;
    const int tile = tile_of(c8->block, threads);
    const bool tiles = tile > 0 && R / N >= 8;
    const int unit = tiles ? tile : c8->block;
    const int64_t items = items_of(R, N, cu_seqlens != nullptr, unit);
    // few blocks: as many CTAs of each as leave every warp one head
    const int64_t slabs = 2 * (int64_t)c->HKV, all = (slabs + kWarps - 1) / kWarps;
    int64_t splits = 8 * (int64_t)sm_count() / (items > 0 ? items : 1);
    if (splits > (tiles ? slabs : all)) splits = tiles ? slabs : all;
    if (splits < 1) splits = 1;
    if (tiles) splits = splits < 2 ? 2 : splits / 2 * 2;
    if (items * splits + (tiles && HQ > 0 ? R : 0) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const int64_t most = cu_seqlens ? 0 : items / N;
    const Append8Args a{*c8, k, v, q, q_out, k_stride, v_stride, q_stride, table_stride, HQ, N, (unsigned)R, (unsigned)(R / N),
                        cu_seqlens, rope, rope_len, rope_dim, interleaved, page_table, kv_lens,
                        Granted(granted, kv_lens), max_pages, status,
                        unit, (unsigned)items, (unsigned)splits, (unsigned)most, 1, 1, 1,
                        Divisor(unit), Divisor(most > 0 ? most : 1), Divisor(R / N > 0 ? R / N : 1), Divisor(c8->block),
                        Divisor(c->page_size)};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const cudaError_t e = bf16 ? launch<__nv_bfloat16>(a, tiles, threads, st) : launch<float>(a, tiles, threads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache8_append", st);
    return KDA_OK;
}
