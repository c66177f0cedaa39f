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
#include "kda_attend_kernels.cuh"

namespace kda {
namespace attend {

// ------------------------------------------------------------------ launch

namespace {

Form form_of(const kda_cache* c, int HQ) {
    const int group = HQ / c->HKV;
    if (c->dtype == KDA_DTYPE_BF16) {
        const int ht = group <= 8 ? 8 : 16;
        return {ht, 16, mma_ctas(ht / 8, c->K, c->V), true};
    }
    const int ht = group == 1 ? 1 : group <= 4 ? 4 : 8;
    return {ht, simt_rows(ht), simt_ctas(ht, c->K, c->V), false};
}

}  // namespace

Plan plan_of(const kda_cache* c, int HQ, int N, int max_pages, int window, int sinks, const Form& form, const Gpu& gpu) {
    const int group = HQ / c->HKV, ht = form.ht, units = c->HKV * ((group + ht - 1) / ht);
    const int turn = kWarps * form.tile;
    int64_t rows = (int64_t)max_pages * c->page_size;
    if (window > 0 && (int64_t)window + sinks < rows) rows = (int64_t)window + sinks;
    const int64_t turns = rows > turn ? (rows + turn - 1) / turn : 1;  // of a unit
    const int64_t all = (int64_t)(N > 0 ? N : 1) * units;              // units
    const int slots = gpu.sms * form.ctas;
    Plan p{kWhole, 1, ht, units, turn};
    p.together = 1;
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
    const struct {
        int ctas, room;
        double join;
    } clusters[] = {{2, 100, form.join2}, {4, 96, form.join4}, {8, 89, form.join8}, {16, 73, 2.4}};
    for (const auto& x : clusters) {
        if (all * x.ctas * 100 > (int64_t)slots * x.room || x.ctas >= 2 * turns || x.ctas > gpu.cluster) continue;
        const double cost = x.join + (turns + x.ctas - 1) / x.ctas + begin(all * x.ctas);
        if (cost >= least) continue;
        least = cost;
        p.split = kCluster;
        p.parts = x.ctas;
    }
    // Parts, and the second kernel: as many as fit. A cache in fp32, sequences of several lengths: `times` as many, so that others
    // take the places of those that end early, which evens them out: T turns of a CTA become T (mean + (1 - mean) /
    // times), and each time costs a start of 0.9. (152 sequences of U[1,16000], K = V = 128, five heads: 414 -> 266 us;
    // of 16000: 465 -> 480.)
    const double each_fit = (double)turns * all / slots;
    const int times = form.even || N <= 1 || each_fit < 12 ? 1 : each_fit > 192 ? 8 : (int)sqrt(each_fit / 3);
    int64_t parts = (int64_t)slots * times / all;
    if (parts > turns) parts = turns;
    if (parts > 1) {
        const int64_t each = (turns + parts - 1) / parts;
        parts = (turns + each - 1) / each;
        const double cost = form.join_parts + each * queue(all * parts) + begin(all * parts);
        if (cost < least) {
            least = cost;
            p.split = kParts;
            p.parts = (int)parts;
        }
    }
    // Shares add up the lengths first, and have the ends of units within them. In k_attend_simt (a cache in fp32) the loop
    // over units costs registers, and 20 to 50 % of the time, so it has none.
    const double shares = form.join_shares + mean * (turns + kUnitTurns) * all / slots + begin(slots);
    if (form.even && (turns + kUnitTurns) * all < INT32_MAX && shares < least) {
        p.split = kShares;
        p.parts = slots;
        // (as many units together as divide a sequence's and leave few places empty)
        if (form.together)
            for (int t = units; t > 1 && p.together == 1; --t)
                if (units % t == 0 && slots / t * t * 100 >= slots * 97) p.together = t;
        p.parts = slots / p.together;
    }
    p.grid = p.split == kShares ? dim3(p.parts * p.together) : dim3(units * p.parts, N);
    p.ws_bytes = KDA_ATTEND_WORKSPACE_MIN;
    p.shared = form.shared;
    if (p.split >= kParts) {
        const size_t held = p.split == kParts ? (size_t)all * p.parts : (size_t)p.parts * p.together * 2;
        p.acc_bytes = held * ht * c->V * sizeof(float);
        p.ml_bytes = held * ht * sizeof(float2);
        p.ws_bytes += p.acc_bytes + p.ml_bytes + (size_t)all * sizeof(int2);
    }
    return p;
}

namespace {

// The present device and what it can do with the kernel for these sizes; without a device, what a GB300 can. A part of
// a GPU may have fewer SMs, and none of its processing clusters 16 of them.
Gpu gpu_for(const kda_cache* c, const Form& form, bool sinks) {
    static std::atomic<int> known[2][5][2][2][kDevices];
    const int tile = form.even ? form.ht / 16 : form.ht == 1 ? 2 : form.ht == 4 ? 3 : 4;
    const int device = present_device();
    const Kernel kernel = sinks ? kernel_with_sinks(*c, form.ht, kCluster) : kernel_without_sinks(*c, form.ht, kCluster);
    return {sm_count(device), largest_cluster(device, (const void*)kernel, kWarps * 32, kMaxCluster,
                                              known[sinks][tile][c->K / 128][c->V / 128])};
}

template <typename TI, int V, int HT, int VS, int G, int THREADS>
cudaError_t launch_join(const AttendArgs& a, cudaStream_t st) {
    const int64_t threads = (int64_t)a.N * a.HQ * (V / 4) * G;
    const unsigned grid = (unsigned)((threads + THREADS - 1) / THREADS);
    if constexpr (sizeof(TI) == 2 || HT >= 8) {  // (fp32 with fewer heads has no shares)
        if (a.split == kShares && a.together > 1)
            return launch_after(k_attend_join<TI, V, HT, VS, G, THREADS, true, true>, a, grid, THREADS, st);
        if (a.split == kShares) return launch_after(k_attend_join<TI, V, HT, VS, G, THREADS, true, false>, a, grid, THREADS, st);
    }
    return launch_after(k_attend_join<TI, V, HT, VS, G, THREADS, false, false>, a, grid, THREADS, st);
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
           : ht == 8 ? launch_join<float, V, 8>(a, parts, st)
                     : launch_join<float, V, 16>(a, parts, st);
}

// Parts of a unit, with equal lengths (kParts, kShares).
int64_t unit_parts(const Plan& p, int N) {
    return p.split == kParts ? p.parts : (int64_t)p.parts * p.together / ((int64_t)(N > 0 ? N : 1) * p.units) + 2;
}

}  // namespace

Kernel kernel_without_sinks(const kda_cache& c, int ht, Split split) { return kernel_of<false>(c, ht, split); }

kda_status launch(const AttendArgs& a, const Plan& p, Kernel kernel, bool bf16, const char* const (&names)[4],
                  cudaStream_t st) {
    const int V = a.c.V;
    begin_launches(st);
    cudaError_t e = launch_after(kernel, a, p.grid, kWarps * 32, st, p.split == kCluster ? p.parts : 1, p.shared);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch(names[p.split], st);
    if (p.split < kParts) return KDA_OK;
    const int64_t parts = unit_parts(p, a.N);
    e = V == 128 ? launch_join<128>(a, bf16, p.ht, parts, st) : launch_join<64>(a, bf16, p.ht, parts, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("cache_attend_join", st);
    return KDA_OK;
}

kda_status check_sizes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks) {
    if (N < 0 || HQ < 1 || HQ % c->HKV != 0 || max_pages < 0 || window < 0 || sinks < 0) return KDA_ERR_INVALID_ARG;
    if (N > 65535 || HQ > 65535 || (int64_t)N * HQ > (1 << 24) || (int64_t)max_pages * c->page_size > (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_call(const kda_cache* c, const Call& x, int64_t unit) {
    if (x.q_stride < (int64_t)x.HQ * c->K || x.q_stride % unit || x.table_stride < 0) return KDA_ERR_INVALID_ARG;
    if (x.N == 0) return KDA_OK;
    if (!x.q || !x.o || !x.kv_lens || (!x.page_table && x.max_pages > 0)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x.q) || !aligned16(x.o) || ((uintptr_t)x.lse & 3u) || ((uintptr_t)x.page_table & 3u) ||
        ((uintptr_t)x.kv_lens & 3u) || ((uintptr_t)x.status & 3u))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

AttendArgs args_of(const kda_cache* c, const Call& x, const Plan& plan) {
    char* w = (char*)x.ws;
    const int step = plan.turn * (plan.split == kShares ? 1 : plan.parts);
    AttendArgs a{};
    a.c = *c;
    a.q = x.q;
    a.q_stride = x.q_stride;
    a.table_stride = x.table_stride;
    a.HQ = x.HQ;
    a.N = x.N;
    a.max_pages = x.max_pages;
    a.window = x.window;
    a.sinks = x.sinks;
    a.table = x.page_table;
    a.kv_lens = x.kv_lens;
    a.scale_log2 = x.scale * kLog2e;
    a.o = x.o;
    a.lse = x.lse;
    a.status = x.status;
    a.group = x.HQ / c->HKV;
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
    a.together = plan.together;
    a.part_acc = (float4*)w;
    a.part_ml = (float2*)(w + plan.acc_bytes);
    a.unit_parts = (int2*)(w + plan.acc_bytes + plan.ml_bytes);
    return a;
}

namespace {

// The plan of a call on a cache in 16 or 32 bits (first rows without a window are not apart).
kda_status plan_for(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window, int32_t sinks, Plan& plan) {
    kda_status s = check_cache(c);
    if (s == KDA_OK) s = check_sizes(c, HQ, N, max_pages, window, sinks);
    if (s != KDA_OK) return s;
    Form form = form_of(c, HQ);
    form.together = window > 0 && sinks > 0;
    plan = plan_of(c, HQ, N, max_pages, window, sinks, form, gpu_for(c, form, form.together));
    return KDA_OK;
}

}  // namespace
}  // namespace attend
}  // namespace kda

using namespace kda;
using namespace kda::attend;

extern "C" size_t kda_cache_attend_workspace_bytes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                   int32_t window) {
    return kda_cache_attend_sinks_workspace_bytes(c, HQ, N, max_pages, window, 0);
}

extern "C" size_t kda_cache_attend_sinks_workspace_bytes(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages,
                                                         int32_t window, int32_t sinks) {
    Plan plan;
    return plan_for(c, HQ, N, max_pages, window, sinks, plan) == KDA_OK ? plan.ws_bytes : 0;
}

extern "C" kda_status kda_debug_attend_plan(const kda_cache* c, int32_t HQ, int32_t N, int32_t max_pages, int32_t window,
                                            int32_t sms, int32_t cluster, int32_t* out) {
    Plan p;
    if (c && c->dtype == KDA_DTYPE_E4M3) {
        kda_cache8 c8{};
        c8.cache = *c;
        c8.dtype = KDA_DTYPE_BF16;
        c8.block = 1;
        c8.k_scale = c8.v_scale = (float*)c->k;  // (a plan does not go by them)
        const kda_status s = plan_for8(&c8, HQ, N, max_pages, window, 0, sms > 0 ? Gpu{sms, cluster} : Gpu{}, p);
        if (s != KDA_OK) return s;
    } else {
        const kda_status s = plan_for(c, HQ, N, max_pages, window, 0, p);
        if (s != KDA_OK) return s;
        if (sms > 0) p = plan_of(c, HQ, N, max_pages, window, 0, form_of(c, HQ), Gpu{sms, cluster});
    }
    if (!out) return KDA_ERR_INVALID_ARG;
    out[0] = p.split;
    out[1] = p.parts * p.together;
    out[2] = p.split < kParts ? 0 : join_groups(unit_parts(p, N));
    out[3] = p.units * (N > 0 ? N : 1);
    return KDA_OK;
}

extern "C" kda_status kda_cache_attend(const kda_cache* c, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                       const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                       const int32_t* kv_lens, int32_t window, float scale, void* o, float* lse,
                                       int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream) {
    return kda_cache_attend_sinks(c, q, q_stride, HQ, N, page_table, table_stride, max_pages, kv_lens, window, 0, scale, o,
                                  lse, status, ws, ws_bytes, stream);
}

extern "C" kda_status kda_cache_attend_sinks(const kda_cache* c, const void* q, int64_t q_stride, int32_t HQ, int32_t N,
                                             const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                             const int32_t* kv_lens, int32_t window, int32_t sinks, float scale, void* o,
                                             float* lse, int32_t* status, void* ws, size_t ws_bytes, kda_stream_t stream) {
    Plan plan;
    kda_status s = plan_for(c, HQ, N, max_pages, window, sinks, plan);
    if (s != KDA_OK) return s;
    const bool bf16 = c->dtype == KDA_DTYPE_BF16;
    const Call x{q, q_stride, HQ, N, page_table, table_stride, max_pages, kv_lens, window, sinks, scale, o, lse, status, ws,
                 ws_bytes, (cudaStream_t)stream};
    s = check_call(c, x, bf16 ? 8 : 4);
    if (s != KDA_OK || N == 0) return s;
    if (!ws || !aligned16(ws) || ws_bytes < plan.ws_bytes) return KDA_ERR_WORKSPACE;
    static const char* const names[] = {"cache_attend", "cache_attend_cluster", "cache_attend_parts",
                                        "cache_attend_shares"};
    const Kernel kernel = window > 0 && sinks > 0 ? kernel_with_sinks(*c, plan.ht, plan.split)
                                                  : kernel_without_sinks(*c, plan.ht, plan.split);
    return launch(args_of(c, x, plan), plan, kernel, bf16, names, x.stream);
}
