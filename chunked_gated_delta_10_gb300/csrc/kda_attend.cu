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

constexpr int kWarps = 4;

// One CTA per (query head, sequence); its warps take the rows in turn, a lane
// holding K / 32 and V / 32 channels.
template <typename TI, int K, int V>
__global__ void __launch_bounds__(kWarps * 32) k_attend(AttendArgs a) {
    constexpr int KL = K / 32, VL = V / 32;
    __shared__ float sm[kWarps], sl[kWarps], sacc[kWarps][V];
    const int64_t n = blockIdx.x / a.HQ;
    const int hq = blockIdx.x % a.HQ, hkv = hq / (a.HQ / a.c.HKV);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int begin, end;
    kv_range(a, n, begin, end);
    float q[KL], acc[VL];
#pragma unroll
    for (int i = 0; i < KL; ++i)
        q[i] = a.scale_log2 * to_f(((const TI*)a.q)[n * a.q_stride + hq * K + lane * KL + i]);
#pragma unroll
    for (int i = 0; i < VL; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int t = begin + warp; t < end; t += kWarps) {
        const int64_t page = a.table[n * a.table_stride + t / a.c.page_size];
        if (page < 0 || page >= a.c.num_pages) {
            if (a.status && lane == 0) *a.status = KDA_ERR_INVALID_ARG;
            continue;
        }
        const int64_t row = t % a.c.page_size;
        const TI* kp = (const TI*)a.c.k + page * a.c.k_page + row * a.c.k_row + hkv * a.c.k_head + lane * KL;
        const TI* vp = (const TI*)a.c.v + page * a.c.v_page + row * a.c.v_row + hkv * a.c.v_head + lane * VL;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < KL; ++i) s = fmaf(q[i], to_f(kp[i]), s);
#pragma unroll
        for (int w = 16; w > 0; w /= 2) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float top = fmaxf(m, s), base = finite_base(top);
        const float keep = exp2f(m - base), p = exp2f(s - base);
        m = top;
        l = fmaf(l, keep, p);
#pragma unroll
        for (int i = 0; i < VL; ++i) acc[i] = fmaf(acc[i], keep, p * to_f(vp[i]));
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) sacc[warp][lane * VL + i] = acc[i];
    __syncthreads();
    float top = sm[0];
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    const float base = finite_base(top);
    float total = 0.f;
    for (int w = 0; w < kWarps; ++w) total = fmaf(sl[w], exp2f(sm[w] - base), total);
    for (int d = threadIdx.x; d < V; d += kWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x = fmaf(sacc[w][d], exp2f(sm[w] - base), x);
        ((TI*)a.o)[(n * a.HQ + hq) * V + d] = from_f<TI>(total == 0.f ? 0.f : x / total);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[n * a.HQ + hq] = (base + log2f(total)) * kLn2;
}

template <typename TI>
void launch_attend(const AttendArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.N * a.HQ);
    const int K = a.c.K, V = a.c.V;
    if (K == 128 && V == 128) k_attend<TI, 128, 128><<<grid, kWarps * 32, 0, st>>>(a);
    if (K == 128 && V == 64) k_attend<TI, 128, 64><<<grid, kWarps * 32, 0, st>>>(a);
    if (K == 64 && V == 128) k_attend<TI, 64, 128><<<grid, kWarps * 32, 0, st>>>(a);
    if (K == 64 && V == 64) k_attend<TI, 64, 64><<<grid, kWarps * 32, 0, st>>>(a);
}

kda_status check_sizes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window) {
    const kda_status s = check_cache(c);
    if (s != KDA_OK) return s;
    if (N < 0 || HQ < 1 || HQ % c->HKV != 0 || max_pages < 0 || window < 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)N * HQ > INT32_MAX || (int64_t)max_pages * c->page_size > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_cache_attend_workspace_bytes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                   int32_t window) {
    return check_sizes(c, HQ, N, max_pages, window) == KDA_OK ? 256 : 0;
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
    AttendArgs a{*c, q, q_stride, table_stride, HQ, N, max_pages, window, page_table, kv_lens, scale * kLog2e, o, lse,
                 status};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    if (c->dtype == KDA_DTYPE_BF16)
        launch_attend<__nv_bfloat16>(a, st);
    else
        launch_attend<float>(a, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_attend", st);
    return KDA_OK;
}
