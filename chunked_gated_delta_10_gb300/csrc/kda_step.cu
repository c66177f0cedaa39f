// kda_step: the recurrent form of KDA on a few tokens per sequence, the fp32
// states updated in place. Declared in include/kda_serve.h.
//
// With S' = Diag(e^g) S the token needs the state twice, once for S'^T k (the
// delta) and once for the output after the update, but
//   o = scale (S' + k d^T)^T q = scale (S'^T q + (q . k) d),
// so both products come from one sweep over S', and the columns of S are
// independent of one another. A thread holds one column in registers for all T
// tokens: the state is read once and written once.
//
// Bound: 8 K V bytes of state traffic per (sequence, value head).
#include "../../include/kda_serve.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "serve_common.cuh"

namespace kda {
namespace {

struct StepArgs {
    const void *q, *k, *v, *beta;
    const float* g;
    float* state;
    const int32_t* slots;
    void* o;
    int32_t* status;
    int N, T, H, HV, num_slots;
    float scale;
};

template <typename TI, int K, int V>
__global__ void __launch_bounds__(V) k_step(StepArgs a) {
    __shared__ float4 sk[K / 4], sq[K / 4], se[K / 4];
    const int64_t n = blockIdx.x / a.HV;
    const int hv = blockIdx.x % a.HV, h = hv / (a.HV / a.H), col = threadIdx.x;
    after_previous();
    const int64_t slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) {
        for (int t = 0; t < a.T; ++t)
            ((TI*)a.o)[((n * a.T + t) * a.HV + hv) * V + col] = from_f<TI>(0.f);
        if (slot >= 0 && a.status && col == 0) *a.status = KDA_ERR_INVALID_ARG;
        return;
    }
    float* S = a.state + (slot * a.HV + hv) * K * V + col;
    float s[K];
#pragma unroll
    for (int j = 0; j < K; ++j) s[j] = S[j * V];
    for (int t = 0; t < a.T; ++t) {
        const int64_t row = n * a.T + t;
        __syncthreads();
        for (int j = col; j < K; j += V) {
            ((float*)sk)[j] = to_f(((const TI*)a.k)[(row * a.H + h) * K + j]);
            ((float*)sq)[j] = to_f(((const TI*)a.q)[(row * a.H + h) * K + j]);
            ((float*)se)[j] = exp2f(a.g[(row * a.HV + hv) * K + j] * kLog2e);
        }
        const float v = to_f(((const TI*)a.v)[(row * a.HV + hv) * V + col]);
        const float beta = to_f(((const TI*)a.beta)[row * a.HV + hv]);
        __syncthreads();
        float sum_k = 0.f, sum_q = 0.f, qk = 0.f;
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
            const float4 kk = sk[j], qq = sq[j], e = se[j];
            const float kv[4] = {kk.x, kk.y, kk.z, kk.w}, qv[4] = {qq.x, qq.y, qq.z, qq.w};
            const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[4 * j + i] *= ev[i];
                sum_k = fmaf(kv[i], s[4 * j + i], sum_k);
                sum_q = fmaf(qv[i], s[4 * j + i], sum_q);
                qk = fmaf(qv[i], kv[i], qk);
            }
        }
        const float d = beta * (v - sum_k);
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
            const float4 kk = sk[j];
            s[4 * j] = fmaf(kk.x, d, s[4 * j]);
            s[4 * j + 1] = fmaf(kk.y, d, s[4 * j + 1]);
            s[4 * j + 2] = fmaf(kk.z, d, s[4 * j + 2]);
            s[4 * j + 3] = fmaf(kk.w, d, s[4 * j + 3]);
        }
        ((TI*)a.o)[(row * a.HV + hv) * V + col] = from_f<TI>(a.scale * fmaf(qk, d, sum_q));
    }
#pragma unroll
    for (int j = 0; j < K; ++j) S[j * V] = s[j];
}

template <typename TI> void (*kernel_of(int K, int V))(StepArgs) {
    return K == 128 ? (V == 128 ? k_step<TI, 128, 128> : k_step<TI, 128, 64>)
                    : (V == 128 ? k_step<TI, 64, 128> : k_step<TI, 64, 64>);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_step(const kda_step_dims* d, const void* q, const void* k, const void* v, const float* g,
                               const void* beta, float* state, const int32_t* slots, void* o, int32_t* status,
                               kda_stream_t stream) {
    if (!d || d->N < 0 || d->T < 0 || d->H < 1 || d->HV < 1 || d->HV % d->H != 0 || d->num_slots < 0)
        return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_DTYPE_BF16 && d->dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARG;
    if (!((d->K == 64 || d->K == 128) && (d->V == 64 || d->V == 128))) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)d->N * d->HV > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!slots && d->num_slots < d->N) return KDA_ERR_INVALID_ARG;
    if (d->N == 0 || d->T == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !o || (!state && d->num_slots > 0)) return KDA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, (const void*)g, beta, (const void*)state, (const void*)o})
        if (!aligned16(x)) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)slots & 3u) || ((uintptr_t)status & 3u)) return KDA_ERR_INVALID_ARG;
    StepArgs a{q, k, v, beta, g, state, slots, o, status, d->N, d->T, d->H, d->HV, d->num_slots, d->scale};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const auto kernel = d->dtype == KDA_DTYPE_BF16 ? kernel_of<__nv_bfloat16>(d->K, d->V) : kernel_of<float>(d->K, d->V);
    const cudaError_t e = launch_after(kernel, a, (unsigned)(d->N * d->HV), d->V, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("step", st);
    return KDA_OK;
}
