// kda_cache_resize: pages for new lengths. Declared in include/kda_serve.h.
//
// With has = ceil(len / P), need = ceil(new / P), back = max(0, has - need) and take = max(0, need - has) of each
// sequence, everything follows from prefix sums over the sequences:
//   page i of those that sequence n gives back goes to free[count + B(n) + i], B the sum of `back` before n;
//   with count' = count + B(N), page i of those it takes is free[count' - 1 - T(n) - i], T the sum of `take` before n;
//   it is served if T(n) + take(n) <= count'; its new rows begin at the sum of new - len before it.
// So every CTA adds up the lengths before its sequences by itself (they are few numbers, read from L2), and no CTA waits
// for another. Pages are taken behind those that come back, so the second step is a launch of its own; for few sequences one
// CTA does both (see alone).
//
// Bound: latencies, one after the other: the lengths, their sums, entries of the list or the table, and again for the second
// step. 256 sequences of 4000 rows that get one more 4.4 us in a graph, one CTA; 1000 sequences that get U[1,4096] rows
// each (128,000 pages, 2 million slots) 11.7 us, and when they end 10 (8.6 and 8.6 MB of entries and slots: 2.5 us at a
// plain copy's rate; two launches that change nothing take 5.2, a fill of the slots alone 3.4). Searches by whole warps,
// four entries of a thread under way, a thread's four slots from one look-up, what is known of a CTA's sequences in shared
// memory: 16 -> 11.7 us; CTAs of 4096 rows instead of 1024 12.8, of 8192 18.
#include "../../include/kda_serve.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "serve_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 1024;       // new rows of a CTA in the second step

constexpr int kBatch = 4;          // entries that a thread has under way

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
    int64_t* begin;  // [N + 1]: where each sequence's new rows begin (cu_seqlens, if it is wanted)
    int* ends;       // [N]: T(n) + take(n); then count', and pages taken in all
    int seqs;           // of a CTA in the first step
    unsigned page_ctas;  // that take pages, in the second
};

__device__ __forceinline__ void flag(const ResizeArgs& a) {
    if (a.status) *a.status = KDA_ERR_INVALID_ARG;
}

// Pages that go back and pages that are taken, 32 bits each (no more than N max_pages, 2^30), and new rows.
struct Sums {
    uint64_t pages;
    int64_t rows;
    __device__ __forceinline__ int back() const { return (int)(unsigned)pages; }
    __device__ __forceinline__ int take() const { return (int)(pages >> 32); }
    __device__ __forceinline__ Sums& operator+=(const Sums& x) {
        pages += x.pages, rows += x.rows;
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
    __device__ __forceinline__ Sums sums(const ResizeArgs& a) const { return {(uint64_t)take(a) << 32 | (unsigned)back(a), rows()}; }
};

__device__ __forceinline__ int64_t free_count(const ResizeArgs& a) {
    return min(max((int64_t)*a.count, (int64_t)0), (int64_t)a.num_pages);
}

// The sum over all threads of the CTA, and over the threads before this one.
__device__ __forceinline__ Sums add_up(const Sums& x, Sums& before) {
    __shared__ Sums of_warp[kThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    before = x;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
        Sums y;
        y.pages = __shfl_up_sync(0xffffffffu, before.pages, w);
        y.rows = __shfl_up_sync(0xffffffffu, before.rows, w);
        if (lane >= w) before += y;
    }
    __syncthreads();
    if (lane == 31) of_warp[warp] = before;
    __syncthreads();
    before.pages -= x.pages;
    before.rows -= x.rows;
    Sums all{};
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before += all;
        all += of_warp[w];
    }
    return all;
}

// The first step, for sequences [begin, stop), kThreads of them at most: pages go back; what the second step has to know is
// written. ALONE: they are all there are.
template <bool ALONE> __device__ __forceinline__ void give_back(const ResizeArgs& a, int begin, int stop) {
    __shared__ int from[kThreads], upto[kThreads];  // first entry to go back; entries of the CTA's sequences so far
    const int n = begin + threadIdx.x;
    const int64_t count = free_count(a);
    const Change x(a, min(n, a.N - 1));
    const int next_take = n + 1 < a.N ? Change(a, n + 1).take(a) : 0;
    Sums mine{}, before, all, earlier{};
    if (n < stop) {
        mine = x.sums(a);
        if (x.need > x.has ? !x.fits(a) : x.has > a.max_pages) flag(a);
    }
    all = add_up(mine, before);
    const int entries = all.back();
    from[threadIdx.x] = x.need;
    upto[threadIdx.x] = before.back() + mine.back();
    // Entry e of those that go back, and its page: a few to a thread are read before the other sequences are added up.
    const auto entry_of = [&](int e) {
        int i = 0;  // the sequence: the first with more than e entries so far
        for (int hi = stop - begin - 1; i < hi;) {
            const int mid = (i + hi) / 2;
            if (upto[mid] > e)
                hi = mid;
            else
                i = mid + 1;
        }
        return a.table + (begin + i) * a.table_stride + from[i] + (e - (i > 0 ? upto[i - 1] : 0));
    };
    int32_t* entry[kBatch];
    int page[kBatch];
    const auto read = [&](int first) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int e = first + k * kThreads;
            entry[k] = e < entries ? entry_of(e) : nullptr;
            page[k] = entry[k] ? *entry[k] : -1;
        }
    };
    __syncthreads();
    read(threadIdx.x);
    if constexpr (!ALONE) {
        Sums later{}, unused;
        for (int i = threadIdx.x; i < a.N; i += kThreads) {
            if (i < begin)
                earlier += Change(a, i).sums(a);
            else if (i >= stop)
                later += Change(a, i).sums(a);
        }
        earlier = add_up(earlier, unused);
        before += earlier;
        all += earlier;
        all += add_up(later, unused);
    }
    const int64_t room = min(count + all.back(), (int64_t)a.num_pages);
    if (n < stop) {
        const int end = before.take() + mine.take();
        a.ends[n] = end;
        a.begin[n] = before.rows;
        const bool served = x.fits(a) && (x.need <= x.has || end <= room);
        if (a.granted) a.granted[n] = served ? x.wanted : x.len;
        if (!served) flag(a);
        // (the ends rise: the last that is served says how many pages are taken)
        if (end <= room && (n + 1 == a.N || end + next_take > room)) a.ends[a.N + 1] = end;
        if (n == 0 && end > room) a.ends[a.N + 1] = 0;
    }
    if (begin == 0 && threadIdx.x == 0) {
        a.ends[a.N] = (int)room;
        a.begin[a.N] = all.rows;
        if (*a.count != count || count + all.back() > room || (a.slots && all.rows > a.rows)) flag(a);
    }
    const int64_t to = count + earlier.back();
    for (int first = threadIdx.x; first < entries; first += kBatch * kThreads) {
        if (first >= kBatch * kThreads) read(first);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!entry[k]) continue;
            const int64_t at = to + first + k * kThreads;
            if ((unsigned)page[k] >= (unsigned)a.num_pages) flag(a);
            if (at < a.num_pages) a.free[at] = page[k];
            *entry[k] = -1;
        }
    }
}

// The first of [0, n) whose value is above x, n - 1 if none is: the values rise. By a whole warp, 32 at a time.
template <typename T> __device__ __forceinline__ int first_above(const T* values, int n, T x) {
    int lo = 0, hi = n - 1;  // it lies in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo) / 32 + 1, at = lo + (int)(threadIdx.x % 32 + 1) * step - 1;
        const unsigned above = __ballot_sync(0xffffffffu, at >= hi || values[at] > x);
        const int i = __ffs(above) - 1;
        lo += i * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}
template <typename T> __device__ __forceinline__ int first_above(const T* values, int lo, int hi, T x) {
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (values[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Page number i of all that are taken.
__device__ __forceinline__ int taken(const ResizeArgs& a, int room, int64_t i) {
    const int page = a.free[room - 1 - i];
    if ((unsigned)page < (unsigned)a.num_pages) return page;
    flag(a);
    return -1;
}

// The second step: the pages that are taken, as many for each of `ctas` CTAs.
__device__ __forceinline__ void take_pages(const ResizeArgs& a, int cta, int ctas) {
    __shared__ int range[2];
    const int room = a.ends[a.N], all = a.ends[a.N + 1], each = (all + ctas - 1) / ctas;
    const int begin = (int)min((int64_t)cta * each, (int64_t)all), end = min(begin + each, all);
    if (begin >= end) return;
    if (threadIdx.x < 64) {
        const int n = first_above(a.ends, a.N, threadIdx.x < 32 ? begin : end - 1);
        if (threadIdx.x % 32 == 0) range[threadIdx.x / 32] = n;
    }
    __syncthreads();
    for (int i = begin + threadIdx.x; i < end; i += kThreads) {
        const int n = first_above(a.ends, range[0], range[1], i);
        a.table[n * a.table_stride + Change(a, n).need - (a.ends[n] - i)] = taken(a, room, i);
    }
}

// What the slots of a sequence's rows go by.
struct Rows {
    int64_t begin, stop;  // its new rows
    int len, has;         // rows and pages that it has
    int base;             // page pg >= has is number base + pg of those that are taken
    bool served;
    Rows() = default;
    __device__ __forceinline__ Rows(const ResizeArgs& a, int n) {
        const Change x(a, n);
        const int end = a.ends[n];
        begin = a.begin[n], stop = a.begin[n + 1];
        len = max(x.len, 0), has = x.has, base = end - x.need;
        served = x.fits(a) && (x.need <= x.has || end <= a.ends[a.N]);
    }
};

// The second step, rows [r0, r0 + count): their slots, four to a thread. Where they are of few sequences, what is known of
// these lies in shared memory.
__device__ __forceinline__ void find_slots(const ResizeArgs& a, int64_t r0, int count) {
    constexpr int kFew = 64;
    __shared__ int range[2];
    __shared__ Rows few[kFew];
    const int64_t rows = a.begin[a.N];
    const int room = a.ends[a.N];
    if (r0 >= rows) {  // (as where the lengths have become shorter)
        for (int i = threadIdx.x; i < count; i += kThreads) a.slots[r0 + i] = -1;
        return;
    }
    if (threadIdx.x < 64) {  // sequences of the first and the last row: the first that ends behind it
        const int n = first_above(a.begin + 1, a.N, threadIdx.x < 32 ? r0 : r0 + count - 1);
        if (threadIdx.x % 32 == 0) range[threadIdx.x / 32] = n;
    }
    __syncthreads();
    const int lo = range[0], hi = range[1];
    const bool known = hi - lo < kFew;
    if (known && lo + (int)threadIdx.x <= hi) few[threadIdx.x] = Rows(a, lo + threadIdx.x);
    __syncthreads();
    for (int i = 4 * threadIdx.x; i < count; i += 4 * kThreads) {
        int64_t slot[4];
        int64_t stop = -1, add = -1;  // of the rows that lie in one page: the last, and what makes a slot of a row
        int n = -1;
        Rows x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + i + j;
            slot[j] = -1;
            if (r >= rows || i + j >= count) continue;
            if (r >= stop) {
                if (n < 0 || r >= x.stop) {
                    if (known) {
                        int to = hi - lo;
                        for (n = max(n, 0); n < to;) {
                            const int mid = (n + to) / 2;
                            if (few[mid].stop > r)
                                to = mid;
                            else
                                n = mid + 1;
                        }
                        x = few[n];
                    } else {
                        n = first_above(a.begin + 1, max(n, lo), hi, r);
                        x = Rows(a, n);
                    }
                }
                const unsigned pos = x.len + (unsigned)(r - x.begin);
                const int pg = (int)a.page(pos);
                stop = min(x.stop, x.begin + ((int64_t)(pg + 1) * a.page_size - x.len));
                int page = -1;
                if (x.served) {
                    if (pg >= x.has) {
                        page = taken(a, room, x.base + pg);
                    } else {
                        page = a.table[(known ? lo + n : n) * a.table_stride + pg];
                        if ((unsigned)page >= (unsigned)a.num_pages) {
                            flag(a);
                            page = -1;
                        }
                    }
                }
                add = page < 0 ? INT64_MIN : ((int64_t)page - pg) * a.page_size + x.len - x.begin;
            }
            if (add != INT64_MIN) slot[j] = r + add;
        }
        int64_t* to = a.slots + r0 + i;
        if (i + 3 < count && ((uintptr_t)to & 15) == 0) {
            ((longlong2*)to)[0] = make_longlong2(slot[0], slot[1]);
            ((longlong2*)to)[1] = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < count) to[j] = slot[j];
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_resize_back(ResizeArgs a) {
    after_previous();
    const int begin = blockIdx.x * a.seqs;
    give_back<false>(a, begin, min(begin + a.seqs, a.N));
}

__global__ void __launch_bounds__(kThreads) k_resize_take(ResizeArgs a) {
    after_previous();
    if (blockIdx.x < a.page_ctas) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = a.ends[a.N] - a.ends[a.N + 1];
        take_pages(a, blockIdx.x, a.page_ctas);
    } else {
        const int64_t r0 = (int64_t)(blockIdx.x - a.page_ctas) * kRows;
        find_slots(a, r0, (int)min((int64_t)kRows, a.rows - r0));
    }
}

__global__ void __launch_bounds__(kThreads, 1) k_resize_alone(ResizeArgs a) {
    __shared__ int ends[kThreads + 2];
    __shared__ int64_t begin[kThreads + 1];
    after_previous();
    int64_t* cu = a.begin;
    a.ends = ends;
    a.begin = begin;
    give_back<true>(a, 0, a.N);
    __syncthreads();
    if (threadIdx.x == 0) *a.count = ends[a.N] - ends[a.N + 1];
    if (cu)
        for (int n = threadIdx.x; n <= a.N; n += kThreads) cu[n] = begin[n];
    take_pages(a, 0, 1);
    if (a.rows > 0) find_slots(a, 0, (int)a.rows);
}

// No sequences: no row has a slot.
__global__ void __launch_bounds__(kThreads) k_resize_none(ResizeArgs a) {
    after_previous();
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at == 0 && a.begin) a.begin[0] = 0;
    if (at < a.rows) a.slots[at] = -1;
}

// Whether one CTA does both steps: the fastest where little changes, and the host does not know what does. One more token for
// each of 1 to 256 sequences 2.2 to 3.2 us (without slots), of two launches 3.7 to 4.7; but a page that goes or comes takes it 1.5 to 2.2 ns,
// two launches of many CTAs a tenth or less: 64 sequences of 64 pages that begin or end 10.3 and 4.9 us, 256 of 256 144 and
// 5.5, 16 of 8192 201 and 22. So with this many pages at most it is ahead where all sequences change in fewer than one of
// about 130 calls. (A CTA of 1024 threads for as many sequences took 7.3 to 8.9 us for a token where two launches take 5.1
// to 5.9, and 21 to 111 us for 16 to 131 pages of 1000 sequences where they take 6.4 to 6.7.)
bool alone(int32_t N, int32_t max_pages, int64_t rows) {
    return N <= kThreads && (int64_t)N * max_pages <= 1 << 17 && rows <= 4 * kRows;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_cache_resize_workspace_bytes(int32_t N, int32_t max_pages, int64_t rows) {
    if (N < 1 || max_pages < 0 || rows < 0 || alone(N, max_pages, rows)) return 0;
    return ((size_t)N + 1) * sizeof(int64_t) + ((size_t)N + 2) * sizeof(int);
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
                 num_pages, free_count, cu_seqlens, slots, slots ? rows : 0, granted, status, cu_seqlens, nullptr, 0, 0};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    cudaError_t e;
    if (need == 0) {
        e = N == 0 ? launch_after(k_resize_none, a, (unsigned)(a.rows / kThreads + 1), kThreads, st)
                   : launch_after(k_resize_alone, a, 1, kThreads, st);
        if (e != cudaSuccess) return cuda_fail(e);
        note_launch("cache_resize", st);
        return KDA_OK;
    }
    int64_t* begin = (int64_t*)ws;
    a.ends = (int*)(begin + N + 1);
    if (!a.begin) a.begin = begin;
    const int ctas = 4 * sm_count();
    a.seqs = N <= 2 * ctas ? 4 : 2 * ((N + ctas - 1) / ctas);
    if (a.seqs > kThreads) a.seqs = kThreads;
    const int64_t pages = (int64_t)N * max_pages / kThreads + 1;
    a.page_ctas = pages < ctas ? (unsigned)pages : (unsigned)ctas;
    e = launch_after(k_resize_back, a, (N + a.seqs - 1) / a.seqs, kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_resize_back", st);
    e = launch_after(k_resize_take, a, (unsigned)(a.page_ctas + (a.rows + kRows - 1) / kRows), kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_resize_take", st);
    return KDA_OK;
}
