// kda_cache8_append: new keys and values into a paged cache in 8 bits, keys and queries rotated by their position on the
// way. Declared in include/kda_serve.h.
//
// Of a block of rows of a page and head, with x its values in fp32 and s its scale,
//   s = 2^e, the smallest with max |x| <= 448 s,   c = e4m3(x / s),
// and where the block has rows c_old in units of s_old already: s = max(s_old, what the new rows want), and, if that is
// more than s_old, c_old <- e4m3(c_old s_old / s). A power of two divides without rounding, so a value is rounded once, and
// again only where it comes to lie below e4m3's normal values.
//
// A warp has a block of one head, of keys or of values, to itself, so that nothing is shared: it finds the largest value,
// then writes. Queries, which go on in their own type, are rows of other CTAs of the same launch.
#include <cfloat>

#include "kda_cache.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kHeld = 4;  // turns of a block's rows that a warp holds in registers

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
    int max_pages;
    int32_t* status;
    unsigned items, splits;  // blocks of rows, at most; CTAs of each
    unsigned most;           // blocks of a sequence, where there is no cu
    unsigned q_lanes, q_rows;  // query rows: threads of a row, rows of a CTA
};

// 8 channels of a row in fp32, and back.
__device__ __forceinline__ void load_8(const __nv_bfloat16* p, float* x) {
    Unit<__nv_bfloat16>::load(p, *(float(*)[8])x);
}
__device__ __forceinline__ void load_8(const float* p, float* x) {
    Unit<float>::load(p, *(float(*)[4])x);
    Unit<float>::load(p + 4, *(float(*)[4])(x + 4));
}
__device__ __forceinline__ void store_8(__nv_bfloat16* p, const float* x) {
    Unit<__nv_bfloat16>::store(p, *(const float(*)[8])x);
}
__device__ __forceinline__ void store_8(float* p, const float* x) {
    Unit<float>::store(p, *(const float(*)[4])x);
    Unit<float>::store(p + 4, *(const float(*)[4])(x + 4));
}

// A lane's share of a row: 8 channels from `a` on and 8 from `b` on. Where they turn, channel a + i turns with b + i, or,
// in pairs, with its neighbour.
struct Share {
    int a, b;
    bool turns;
    __device__ __forceinline__ Share(int u, int rope_dim, int interleaved) {
        const int pairs = interleaved ? 0 : rope_dim / 16;
        turns = u < (interleaved ? rope_dim / 16 : pairs);
        a = u < pairs ? 8 * u : 16 * u;
        b = u < pairs ? 8 * u + rope_dim / 2 : 16 * u + 8;
    }
};

// The rotation, each product and each sum rounded by itself (so that the scales, which go by the largest value, do not
// depend on how a compiler joins them). cs: the position's cosines and sines.
__device__ __forceinline__ void turn(float (&x)[16], const Share& s, const float* cs, int rope_dim, int interleaved) {
    const int half = rope_dim / 2;
    if (interleaved) {
        float co[8], si[8];
        load_8(cs + s.a / 2, co);
        load_8(cs + half + s.a / 2, si);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(p, co[i]), __fmul_rn(q, si[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(q, co[i]), __fmul_rn(p, si[i]));
        }
    } else {
        float co[8], si[8];
        load_8(cs + s.a, co);
        load_8(cs + half + s.a, si);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = x[i], q = x[8 + i];
            x[i] = __fsub_rn(__fmul_rn(p, co[i]), __fmul_rn(q, si[i]));
            x[8 + i] = __fadd_rn(__fmul_rn(q, co[i]), __fmul_rn(p, si[i]));
        }
    }
}

// 8 values times f as e4m3; what is not finite becomes a NaN (x 0 + x), which rounding alone would make the largest value.
__device__ __forceinline__ uint2 to_e4m3(const float* x, float f) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = x[4 * i + e] * f;
            y[e] = fmaf(y[e], 0.f, y[e]);
        }
        asm("{.reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;"
            " mov.b32 %0, {lo, hi};}"
            : "=r"(w[i])
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    }
    return make_uint2(w[0], w[1]);
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

// Rows [first, last) of the positions of a block that begins at `start`, of one head: D channels each of `x`, whose row of
// position `first` is at `from` (rows `stride` apart), into `to`, position `start`'s row of the cache, rows `step` apart.
template <typename TI, int D>
__device__ __forceinline__ void write_block(const Append8Args& a, const TI* from, int64_t stride, unsigned char* to,
                                            int64_t step, float* scale, unsigned start, unsigned old_end, unsigned first,
                                            unsigned last, bool rotated) {
    constexpr int L = D / 16, P = 32 / L;  // lanes of a row, rows of a turn
    const int lane = threadIdx.x % 32, in = lane / L;
    const Share s(lane % L, rotated ? a.rope_dim : 0, rotated ? a.interleaved : 1);
    const float before = start < old_end ? *scale : 0.f;
    const unsigned rows = last - first;
    float x[kHeld][16], top = 0.f;
    const auto load = [&](unsigned row, float (&y)[16]) {
        const TI* p = from + (int64_t)row * stride;
        load_8(p + s.a, y);
        load_8(p + s.b, y + 8);
        if (s.turns) turn(y, s, a.rope + (int64_t)(first + row) * a.rope_dim, a.rope_dim, a.interleaved);
    };
    for (unsigned at = 0; at < rows; at += kHeld * P) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const unsigned row = at + i * P + in;
            if (row >= rows) continue;
            load(row, x[i]);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float m = fabsf(x[i][e]);
                if (m <= FLT_MAX) top = fmaxf(top, m);
            }
        }
    }
#pragma unroll
    for (int w = 1; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    const int field = max(least_scale(top), held_scale(before));
    const float now = __int_as_float(field << 23), f = __int_as_float((254 - field) << 23);
    if (start < old_end && before != now) {  // the block's rows in the new units
        const float ratio = before * f;
        for (unsigned row = in; row < old_end - start; row += P) {
            uint4* p = (uint4*)(to + row * step + (lane % L) * 16);
            const uint4 old = *p;
            float y[16];
            from_e4m3(old.x, y), from_e4m3(old.y, y + 4), from_e4m3(old.z, y + 8), from_e4m3(old.w, y + 12);
            if (fabsf(ratio) > 1.f) {  // (a scale above 2^126: what it makes larger than 448 2^126 is not held)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (fabsf(y[e] * ratio) > 448.f) y[e] = INFINITY;
            }
            const uint2 lo = to_e4m3(y, ratio), hi = to_e4m3(y + 8, ratio);
            *p = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
    if (lane == 0 && before != now) *scale = now;
    for (unsigned at = 0; at < rows; at += kHeld * P) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const unsigned row = at + i * P + in;
            if (row >= rows) continue;
            if (rows > kHeld * P) load(row, x[i]);
            unsigned char* p = to + (first - start + row) * step;
            *(uint2*)(p + s.a) = to_e4m3(x[i], f);
            *(uint2*)(p + s.b) = to_e4m3(x[i] + 8, f);
        }
    }
}

// The sequence that new row r or, with `block`, block r of the launch's belongs to: the last n that begins at or before it.
// A sequence whose first row is cu[n] has blocks from cu[n] / block + 2 n on: two more than its rows fill, as many as it may
// begin and end in.
__device__ __forceinline__ int seq_of(const int64_t* cu, int N, int64_t r, int block) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((block ? cu[mid] / block + 2 * mid : cu[mid]) <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void flag(const Append8Args& a) {
    if (a.status) *a.status = KDA_ERR_INVALID_ARG;
}

// Block `item` of the launch's, the CTA's share of its heads.
template <typename TI> __device__ __forceinline__ void append_block(const Append8Args& a, unsigned item, unsigned split) {
    const int block = a.c.block;
    const kda_cache& c = a.c.cache;
    int n;
    unsigned j;
    int64_t begin, end;
    if (a.cu) {
        n = seq_of(a.cu, a.N, item, block);
        begin = a.cu[n];
        end = a.cu[n + 1];
        if (item == 0 && threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.N] != a.R)) flag(a);  // rows of no sequence
        if (begin < 0 || end < begin || end > a.R) {
            if (threadIdx.x == 0) flag(a);
            return;
        }
        j = (unsigned)(item - (begin / block + 2 * n));
    } else {
        n = item / a.most;
        j = item - n * a.most;
        begin = (int64_t)n * a.per;
        end = begin + a.per;
    }
    const int len = a.kv_lens[n];
    if (len < 0 || begin == end) return;
    const int64_t start = ((int64_t)(len / block) + j) * block, stop = len + (end - begin);
    if (start >= stop) return;
    const unsigned from = (unsigned)start, first = max(from, (unsigned)len);
    unsigned last = (unsigned)min(stop, start + block);
    const unsigned pg = from / (unsigned)c.page_size, row = from - pg * c.page_size;
    int64_t page = -1;
    if (pg < (unsigned)a.max_pages) page = a.table[n * a.table_stride + pg];
    if (page < 0 || page >= c.num_pages || (a.rope && last > (unsigned)a.rope_len)) {
        if (threadIdx.x == 0) flag(a);
        if (page < 0 || page >= c.num_pages) return;
        last = min(last, (unsigned)a.rope_len);
        if (first >= last) return;
    }
    const int64_t r = begin + (first - (unsigned)len), b = row / (unsigned)block;
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
        n = seq_of(a.cu, a.N, r, 0);
        const int64_t begin = a.cu[n];
        ok = begin <= r && r < a.cu[n + 1];
        idx = (unsigned)(r - begin);
    } else {
        n = (unsigned)r / a.per;
        idx = (unsigned)r - n * a.per;
    }
    const int len = a.kv_lens[n];
    const unsigned pos = (unsigned)len + idx, pg = pos / (unsigned)c.page_size;
    int64_t page = -1;
    if (len >= 0) {
        ok = ok && pg < (unsigned)a.max_pages && (!a.rope || pos < (unsigned)a.rope_len);
        if (ok) page = a.table[n * a.table_stride + pg];
        if (page < 0 || page >= c.num_pages) {
            page = -1;
            if (lane == 0) flag(a);
        }
    }
    const unsigned L = c.K / 16, tasks = a.HQ * L;
    for (unsigned i = lane; i < tasks; i += a.q_lanes) {
        const unsigned h = i / L;
        const Share s(i - h * L, a.rope_dim, a.interleaved);
        float x[16];
        if (page >= 0) {
            const TI* p = (const TI*)a.q + r * a.q_stride + (int64_t)h * c.K;
            load_8(p + s.a, x);
            load_8(p + s.b, x + 8);
            if (s.turns) turn(x, s, a.rope + (int64_t)pos * a.rope_dim, a.rope_dim, a.interleaved);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        TI* p = (TI*)a.q_out + (r * a.HQ + h) * c.K;
        store_8(p + s.a, x);
        store_8(p + s.b, x + 8);
    }
}

template <typename TI> __global__ void __launch_bounds__(kThreads) k_append8(Append8Args a) {
    after_previous();
    const unsigned blocks = a.items * a.splits;
    if (blockIdx.x < blocks)
        append_block<TI>(a, blockIdx.x / a.splits, blockIdx.x % a.splits);
    else
        turn_queries<TI>(a, blockIdx.x - blocks);
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
    const kda_status s = check_cache(c8);
    if (s != KDA_OK) return s;
    const kda_cache* c = &c8->cache;
    const bool bf16 = c8->dtype == KDA_DTYPE_BF16;
    // (scales that several blocks share are for reading)
    for (const int64_t* x : {&c8->k_scale_page, &c8->v_scale_page})
        if ((c->num_pages > 1 && x[0] == 0) || (c->page_size > c8->block && x[1] == 0) || (c->HKV > 1 && x[2] == 0))
            return KDA_ERR_INVALID_ARG;
    const AppendCall x{k, k_stride, v, v_stride, q, q_stride, q_out, HQ, N, R, cu_seqlens, rope, rope_len, rope_dim,
                       page_table, table_stride, max_pages, kv_lens, status};
    const kda_status checked = check_append(c, x, bf16 ? 8 : 4);
    if (checked != KDA_OK || R == 0) return checked;
    const int64_t per = R / N, block = c8->block;
    const int64_t most = per > 0 ? (per + block - 2) / block + 1 : 0;
    const int64_t items = cu_seqlens ? R / block + 2 * (int64_t)N : N * most;
    // few blocks: as many CTAs of each as leave every warp one head
    const int64_t slabs = 2 * (int64_t)c->HKV, all = (slabs + kWarps - 1) / kWarps;
    int64_t splits = 8 * (int64_t)sm_count() / (items > 0 ? items : 1);
    if (splits > all) splits = all;
    if (splits < 1) splits = 1;
    const int64_t tasks = (int64_t)HQ * (c->K / 16);
    const int64_t lanes = tasks == 0 ? kThreads : tasks < kThreads ? tasks : kThreads, rows = kThreads / lanes;
    const int64_t grid = items * splits + (HQ > 0 ? (R + rows - 1) / rows : 0);
    if (grid > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const Append8Args a{*c8, k, v, q, q_out, k_stride, v_stride, q_stride, table_stride, HQ, N, (unsigned)R, (unsigned)per,
                        cu_seqlens, rope, rope_len, rope_dim, interleaved, page_table, kv_lens, max_pages, status,
                        (unsigned)items, (unsigned)splits, (unsigned)most, (unsigned)lanes, (unsigned)rows};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const cudaError_t e = launch_after(bf16 ? k_append8<__nv_bfloat16> : k_append8<float>, a, (unsigned)grid, kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache8_append", st);
    return KDA_OK;
}
