// kda_cache_resize: pages for new lengths. Declared in include/kda_serve.h.
//
// With has = ceil(len / P), need = ceil(new / P), back = max(0, has - need) and take = max(0, need - has) of each
// sequence, everything follows from prefix sums over the sequences:
//   page i of those that sequence n gives back goes to free[count + B(n) + i], B the sum of `back` before n;
//   with count' = count + B(N), page i of those it takes is free[count' - 1 - T(n) - i], T the sum of `take` before n;
//   it is served if T(n) + take(n) <= count'; its new rows begin at the sum of new - len before it.
// So every CTA adds up the lengths before its sequences by itself (they are few numbers, read from L2), and no CTA waits
// for another. Pages are taken behind those that come back, so the second step is a launch of its own; where all is little
// work one CTA does both.
#include "../../include/kda_serve.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "serve_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kAlone = 1024;  // threads of the CTA that does both steps
constexpr int kRows = 2048;   // new rows of a CTA in the second step

struct ResizeArgs {
    int32_t* table;
    int64_t table_stride;
    int max_pages, N, page_size;
    Divisor page;
    const int32_t *lens, *wanted;
    int32_t* free;
    int num_pages;
    int32_t* count;
    int64_t *cu, *slots;
    int64_t rows;
    int32_t *granted, *status;
    int64_t* ends;   // [N]: T(n) + take(n); then count', and pages taken in all
    int64_t* begin;  // [N + 1]: where each sequence's new rows begin (cu_seqlens, if it is wanted)
    int seqs;           // of a CTA in the first step
    unsigned page_ctas;  // that take pages, in the second
};

__device__ __forceinline__ void flag(const ResizeArgs& a) {
    if (a.status) *a.status = KDA_ERR_INVALID_ARG;
}

struct Sums {
    int64_t back, take, rows;
    __device__ __forceinline__ Sums& operator+=(const Sums& x) {
        back += x.back, take += x.take, rows += x.rows;
        return *this;
    }
};

// What sequence n has and needs, in pages.
struct Change {
    int len, wanted, has, need;
    __device__ __forceinline__ Change(const ResizeArgs& a, int n) {
        len = a.lens[n], wanted = a.wanted[n];
        has = pages(a, len), need = pages(a, wanted);
    }
    __device__ __forceinline__ static int pages(const ResizeArgs& a, int len) {
        return len > 0 ? (int)a.page((unsigned)len - 1) + 1 : 0;
    }
    __device__ __forceinline__ bool fits(const ResizeArgs& a) const { return need <= a.max_pages; }
    // pages to give back (entries of the table alone) and to take
    __device__ __forceinline__ int back(const ResizeArgs& a) const { return max(0, min(has, a.max_pages) - need); }
    __device__ __forceinline__ int take(const ResizeArgs& a) const { return fits(a) ? max(0, need - has) : 0; }
    __device__ __forceinline__ int rows() const { return max(0, max(wanted, 0) - max(len, 0)); }
    __device__ __forceinline__ Sums sums(const ResizeArgs& a) const { return {back(a), take(a), rows()}; }
};

__device__ __forceinline__ int64_t free_count(const ResizeArgs& a) {
    return min(max((int64_t)*a.count, (int64_t)0), (int64_t)a.num_pages);
}

// The sum over all threads of the CTA, and, with `before`, over the threads before this one.
template <int THREADS> __device__ __forceinline__ Sums add_up(Sums x, Sums* before) {
    __shared__ Sums of_warp[THREADS / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Sums upto = x;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
        const Sums y{__shfl_up_sync(0xffffffffu, upto.back, w), __shfl_up_sync(0xffffffffu, upto.take, w),
                     __shfl_up_sync(0xffffffffu, upto.rows, w)};
        if (lane >= w) upto += y;
    }
    __syncthreads();
    if (lane == 31) of_warp[warp] = upto;
    __syncthreads();
    Sums all{0, 0, 0}, first{0, 0, 0};
#pragma unroll 8
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w == warp) first = all;
        all += of_warp[w];
    }
    if (before) {
        *before = first;
        *before += {upto.back - x.back, upto.take - x.take, upto.rows - x.rows};
    }
    return all;
}

// The first step, for sequences [begin, stop), THREADS of them at most: pages go back; what the second step has to know is
// written.
template <int THREADS> __device__ __forceinline__ void give_back(const ResizeArgs& a, int begin, int stop) {
    __shared__ int from[THREADS], upto[THREADS];  // first entry to go back; entries of the CTA's sequences so far
    Sums earlier{0, 0, 0}, later{0, 0, 0};
    for (int n = threadIdx.x; n < a.N; n += THREADS) {
        if (n >= begin && n < stop) continue;
        (n < begin ? earlier : later) += Change(a, n).sums(a);
    }
    const int n = begin + threadIdx.x;
    Sums mine{0, 0, 0}, before;
    int need = 0;
    const int64_t count = free_count(a);
    if (n < stop) {
        const Change x(a, n);
        mine = x.sums(a);
        need = x.need;
        if (x.need > x.has ? !x.fits(a) : x.has > a.max_pages) flag(a);
    }
    earlier = add_up<THREADS>(earlier, nullptr);
    Sums all = add_up<THREADS>(mine, &before);
    later = add_up<THREADS>(later, nullptr);
    const int entries = (int)all.back;
    from[threadIdx.x] = need;
    upto[threadIdx.x] = (int)(before.back + mine.back);
    before += earlier;
    all += earlier;
    all += later;
    const int64_t room = min(count + all.back, (int64_t)a.num_pages);
    if (n < stop) {
        const int64_t end = before.take + mine.take;
        a.ends[n] = end;
        a.begin[n] = before.rows;
        const Change x(a, n);
        const bool served = x.fits(a) && (x.need <= x.has || end <= room);
        if (a.granted) a.granted[n] = served ? x.wanted : x.len;
        if (!served) flag(a);
        // (the ends rise: the last that is served says how many pages are taken)
        const int64_t next = n + 1 < a.N ? end + Change(a, n + 1).take(a) : INT64_MAX;
        if (end <= room && next > room) a.ends[a.N + 1] = end;
        if (n == 0 && end > room) a.ends[a.N + 1] = 0;
    }
    if (begin == 0 && threadIdx.x == 0) {
        a.ends[a.N] = room;
        if (a.N == 0) a.ends[a.N + 1] = 0;
        a.begin[a.N] = all.rows;
        if (*a.count != count || count + all.back > room || (a.slots && all.rows > a.rows)) flag(a);
    }
    __syncthreads();
    const int64_t to = count + earlier.back;
#pragma unroll 4
    for (int e = threadIdx.x; e < entries; e += THREADS) {
        int i = 0;  // the sequence: the first with more than e entries so far
        for (int hi = stop - begin - 1; i < hi;) {
            const int mid = (i + hi) / 2;
            if (upto[mid] > e)
                hi = mid;
            else
                i = mid + 1;
        }
        int32_t* entry = a.table + (begin + i) * a.table_stride + from[i] + (e - (i > 0 ? upto[i - 1] : 0));
        const int page = *entry;
        if ((unsigned)page >= (unsigned)a.num_pages) flag(a);
        if (to + e < a.num_pages) a.free[to + e] = page;
        *entry = -1;
    }
}

// Page number i of all that are taken.
__device__ __forceinline__ int taken(const ResizeArgs& a, int64_t room, int64_t i) {
    const int page = a.free[room - 1 - i];
    if ((unsigned)page < (unsigned)a.num_pages) return page;
    flag(a);
    return -1;
}

// The second step: the pages that are taken, dealt out to `threads` threads, this one being `thread`.
__device__ __forceinline__ void take_pages(const ResizeArgs& a, int64_t thread, int64_t threads) {
    const int64_t room = a.ends[a.N], all = a.ends[a.N + 1];
    for (int64_t i = thread; i < all; i += threads) {
        int n = 0;  // the sequence: the first that ends behind it
        for (int hi = a.N - 1; n < hi;) {
            const int mid = (n + hi) / 2;
            if (a.ends[mid] > i)
                hi = mid;
            else
                n = mid + 1;
        }
        const Change x(a, n);
        a.table[n * a.table_stride + x.need - (a.ends[n] - i)] = taken(a, room, i);
    }
}

// The last of sequences [lo, hi] that begins at or before row r.
__device__ __forceinline__ int seq_of(const int64_t* begin, int lo, int hi, int64_t r) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (begin[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The second step, rows [r0, r0 + count): their slots.
template <int THREADS> __device__ __forceinline__ void find_slots(const ResizeArgs& a, int64_t r0, int count) {
    __shared__ int range[2];
    const int64_t rows = a.begin[a.N], room = a.ends[a.N];
    if (threadIdx.x < 64 && threadIdx.x % 32 == 0)
        range[threadIdx.x / 32] = a.N > 0 ? seq_of(a.begin, 0, a.N - 1, threadIdx.x ? r0 + count - 1 : r0) : 0;
    __syncthreads();
    const int lo = range[0], hi = range[1];
    for (int i = threadIdx.x; i < count; i += THREADS) {
        const int64_t r = r0 + i;
        int64_t slot = -1;
        if (r < rows) {
            const int n = seq_of(a.begin, lo, hi, r);
            const Change x(a, n);
            const int64_t end = a.ends[n];
            const unsigned pos = (unsigned)max(x.len, 0) + (unsigned)(r - a.begin[n]);
            const int pg = (int)a.page(pos);
            if (x.fits(a) && (x.need <= x.has || end <= room)) {
                int page;
                if (pg < x.has) {
                    page = a.table[n * a.table_stride + pg];
                    if ((unsigned)page >= (unsigned)a.num_pages) {
                        flag(a);
                        page = -1;
                    }
                } else {
                    page = taken(a, room, end - (x.need - pg));
                }
                if (page >= 0) slot = (int64_t)page * a.page_size + (pos - (unsigned)pg * a.page_size);
            }
        }
        a.slots[r] = slot;
    }
}

__global__ void __launch_bounds__(kThreads) k_resize_back(ResizeArgs a) {
    after_previous();
    const int begin = blockIdx.x * a.seqs;
    give_back<kThreads>(a, begin, min(begin + a.seqs, a.N));
}

__global__ void __launch_bounds__(kThreads) k_resize_take(ResizeArgs a) {
    after_previous();
    if (blockIdx.x < a.page_ctas) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = (int)(a.ends[a.N] - a.ends[a.N + 1]);
        take_pages(a, blockIdx.x * kThreads + threadIdx.x, a.page_ctas * kThreads);
    } else {
        const int64_t r0 = (int64_t)(blockIdx.x - a.page_ctas) * kRows;
        find_slots<kThreads>(a, r0, (int)min((int64_t)kRows, a.rows - r0));
    }
}

__global__ void __launch_bounds__(kAlone) k_resize_alone(ResizeArgs a) {
    __shared__ int64_t ends[kAlone + 2], begin[kAlone + 1];
    after_previous();
    int64_t* cu = a.begin;
    a.ends = ends;
    a.begin = begin;
    give_back<kAlone>(a, 0, a.N);
    __syncthreads();
    if (threadIdx.x == 0) *a.count = (int)(ends[a.N] - ends[a.N + 1]);
    if (cu)
        for (int n = threadIdx.x; n <= a.N; n += kAlone) cu[n] = begin[n];
    take_pages(a, threadIdx.x, kAlone);
    if (a.slots && a.rows > 0) find_slots<kAlone>(a, 0, (int)a.rows);
}

// Whether one CTA does both steps.
bool alone(int32_t N, int32_t max_pages, int64_t rows) {
    return N <= kAlone && (int64_t)N * max_pages <= 1 << 17 && rows <= 4 * kAlone;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_cache_resize_workspace_bytes(int32_t N, int32_t max_pages, int64_t rows) {
    if (N < 0 || max_pages < 0 || rows < 0 || alone(N, max_pages, rows)) return 0;
    return ((size_t)N + 2 + (size_t)N + 1) * sizeof(int64_t);
}

extern "C" kda_status kda_cache_resize(int32_t* page_table, int64_t table_stride, int32_t max_pages, int32_t N,
                                       int32_t page_size, const int32_t* kv_lens, const int32_t* new_lens,
                                       int32_t* free_pages, int32_t num_pages, int32_t* free_count, int64_t* cu_seqlens,
                                       int64_t* slots, int64_t rows, int32_t* granted, int32_t* status, void* ws,
                                       size_t ws_bytes, kda_stream_t stream) {
    if (max_pages < 0 || N < 0 || page_size < 1 || num_pages < 0 || rows < 0 || table_stride < 0) return KDA_ERR_INVALID_ARG;
    if (N > 1 && table_stride < max_pages) return KDA_ERR_INVALID_ARG;
    if (N > 65535 || rows > INT32_MAX || (int64_t)N * max_pages > 1 << 30) return KDA_ERR_UNSUPPORTED;
    if ((N > 0 && (!kv_lens || !new_lens || (!page_table && max_pages > 0))) || (!free_pages && num_pages > 0) || !free_count)
        return KDA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)page_table, (const void*)kv_lens, (const void*)new_lens, (const void*)free_pages,
                          (const void*)free_count, (const void*)granted, (const void*)status})
        if ((uintptr_t)p & 3u) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)cu_seqlens & 7u) || ((uintptr_t)slots & 7u)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_cache_resize_workspace_bytes(N, max_pages, rows);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    ResizeArgs a{page_table, table_stride, max_pages, N, page_size, Divisor(page_size), kv_lens, new_lens, free_pages,
                 num_pages, free_count, cu_seqlens, slots, slots ? rows : 0, granted, status, nullptr, cu_seqlens, 0, 0};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    if (need == 0) {
        const cudaError_t e = launch_after(k_resize_alone, a, 1, kAlone, st);
        if (e != cudaSuccess) return cuda_fail(e);
        note_launch("cache_resize", st);
        return KDA_OK;
    }
    a.ends = (int64_t*)ws;
    if (!a.begin) a.begin = a.ends + N + 2;
    const int ctas = 4 * sm_count();
    a.seqs = N <= 8 * ctas ? 8 : (N + ctas - 1) / ctas;
    if (a.seqs > kThreads) a.seqs = kThreads;
    const int64_t pages = ((int64_t)N * max_pages + kThreads - 1) / kThreads;
    a.page_ctas = pages < ctas ? (unsigned)pages + (pages == 0) : (unsigned)ctas;
    cudaError_t e = launch_after(k_resize_back, a, (N + a.seqs - 1) / a.seqs + (N == 0), kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_resize_back", st);
    e = launch_after(k_resize_take, a, (unsigned)(a.page_ctas + (a.rows + kRows - 1) / kRows), kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_resize_take", st);
    return KDA_OK;
}
