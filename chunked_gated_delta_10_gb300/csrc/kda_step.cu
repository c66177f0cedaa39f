// kda_step: the recurrent form of KDA on a few tokens per sequence, the fp32
// states updated in place. Declared in include/kda_serve.h.
//
// With S' = Diag(e^g) S the token needs the state twice, once for S'^T k (the
// delta) and once for the output after the update, but
//   o = scale (S' + k d^T)^T q = scale (S'^T q + (q . k) d),
// so both products come from one sweep over S', and the columns of S are
// independent of one another. A CTA holds 32 columns of one state in registers
// for all T tokens: the state is read once and written once.
//
// Bound: 8 K V bytes of state traffic per (sequence, value head), 128 KB at
// K = V = 128. What the split is for: a CTA's loads, sums and stores follow one
// another, so an SM needs many of them at different points of their way. With
// 32 columns eight CTAs fit an SM, each with 16 KB under way. Measured at N = 256,
// HV = 32, K = V = 128, bf16: 159.5 us (6.81 TB/s, the rate of a plain copy);
// with 64 columns and four CTAs 158 us, but small batches take 0.3 to 0.5 us
// longer (N = 1: 2.0 -> 2.3 us); with 16 columns 187 us; with a column per
// thread, a whole state per CTA, 248 us.
// With several tokens the sums bound it (two barriers and about 200
// instructions a warp and token): N = 16, T = 4, HV = 32 takes 19.4 us where
// the states' traffic takes 10.3.
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

constexpr int kThreads = 128, kCols = 32;

// Two fp32 values in a 64-bit register: one instruction multiplies or adds both.
using Pair = uint64_t;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 values(Pair p) {
    float2 x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(p));
    return x;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
    return p;
}
__device__ __forceinline__ Pair shuffle_xor(Pair p, int w) { return __shfl_xor_sync(0xffffffffu, p, w); }

// A token's inputs as a thread reads them: one channel of k, q and g, its four columns of v, and beta.
template <typename TI> struct Token {
    TI k, q, v[4], beta;
    float g;
    template <int K, int V> __device__ __forceinline__ void load(const StepArgs& a, int64_t row, int h, int hv, int col) {
        if (threadIdx.x < K) {
            k = ((const TI*)a.k)[(row * a.H + h) * K + threadIdx.x];
            q = ((const TI*)a.q)[(row * a.H + h) * K + threadIdx.x];
            g = a.g[(row * a.HV + hv) * K + threadIdx.x];
        }
        const TI* p = (const TI*)a.v + (row * a.HV + hv) * V + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p[i];
        beta = ((const TI*)a.beta)[row * a.HV + hv];
    }
};

// One CTA per (sequence, value head, slice of kCols columns). A row of the slice is kCols / 4 threads with four columns
// each; a thread has every (4 kThreads / kCols)-th row. The next token's inputs are loaded while a token is computed.
template <typename TI, int K, int V, bool MANY>
__global__ void __launch_bounds__(kThreads, MANY ? 7 : 8) k_step(StepArgs a) {
    constexpr int LR = kCols / 4, RP = kThreads / LR, P = K / RP, W = kThreads / 32;  // threads of a row, rows of a pass, passes
    __shared__ float factors[MANY ? 2 : 1][3][K];  // k, q and e^g of a token; the next token has the other buffer
    __shared__ ulonglong2 sum_k[W][LR], sum_q[W][LR];
    __shared__ float sum_qk[W];
    after_previous();
    const unsigned slice = blockIdx.x % (V / kCols), nh = blockIdx.x / (V / kCols);
    const int64_t n = nh / (unsigned)a.HV;
    const int hv = nh % (unsigned)a.HV, h = hv / (a.HV / a.H);
    const int warp = threadIdx.x / 32, c = threadIdx.x % LR, r0 = threadIdx.x / LR, col = slice * kCols + 4 * c;
    const int64_t slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) {
        for (int t = 0; t < a.T; ++t)
            if (threadIdx.x < kCols)
                ((TI*)a.o)[((n * a.T + t) * a.HV + hv) * V + slice * kCols + threadIdx.x] = from_f<TI>(0.f);
        if (slot >= 0 && a.status && threadIdx.x == 0) *a.status = KDA_ERR_INVALID_ARG;
        return;
    }
    Token<TI> in;
    in.template load<K, V>(a, n * a.T, h, hv, col);
    float* S = a.state + (slot * a.HV + hv) * K * V + r0 * V + col;
    ulonglong2 s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = *(const ulonglong2*)(S + i * RP * V);
    for (int t = 0; t < (MANY ? a.T : 1); ++t) {
        const auto& f = factors[MANY ? t % 2 : 0];
        if (threadIdx.x < K) {
            float(*to)[K] = factors[MANY ? t % 2 : 0];
            to[0][threadIdx.x] = to_f(in.k);
            to[1][threadIdx.x] = to_f(in.q);
            to[2][threadIdx.x] = exp2f(in.g * kLog2e);
        }
        const Pair v0 = pair(to_f(in.v[0]), to_f(in.v[1])), v1 = pair(to_f(in.v[2]), to_f(in.v[3]));
        const float beta = to_f(in.beta);
        __syncthreads();
        if (MANY && t + 1 < a.T) in.template load<K, V>(a, n * a.T + t + 1, h, hv, col);
        Pair k0 = 0, k1 = 0, q0 = 0, q1 = 0;  // sums of k S' and q S' (0 is a pair of zeros)
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int j = i * RP + r0;
            const Pair k = pair(f[0][j], f[0][j]), q = pair(f[1][j], f[1][j]), e = pair(f[2][j], f[2][j]);
            s[i].x = mul(s[i].x, e);
            s[i].y = mul(s[i].y, e);
            k0 = fma(k, s[i].x, k0);
            k1 = fma(k, s[i].y, k1);
            q0 = fma(q, s[i].x, q0);
            q1 = fma(q, s[i].y, q1);
            qk = fmaf(f[1][j], f[0][j], qk);
        }
#pragma unroll
        for (int w = LR; w < 32; w *= 2) {
            k0 = add(k0, shuffle_xor(k0, w));
            k1 = add(k1, shuffle_xor(k1, w));
            q0 = add(q0, shuffle_xor(q0, w));
            q1 = add(q1, shuffle_xor(q1, w));
            qk += __shfl_xor_sync(0xffffffffu, qk, w);
        }
        if (threadIdx.x % 32 < LR) {
            sum_k[warp][c] = make_ulonglong2(k0, k1);
            sum_q[warp][c] = make_ulonglong2(q0, q1);
            if (c == 0) sum_qk[warp] = qk;
        }
        __syncthreads();
        k0 = sum_k[0][c].x;
        k1 = sum_k[0][c].y;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            k0 = add(k0, sum_k[w][c].x);
            k1 = add(k1, sum_k[w][c].y);
        }
        const Pair b = pair(beta, beta), minus = pair(-1.f, -1.f);
        const Pair d0 = mul(b, fma(minus, k0, v0)), d1 = mul(b, fma(minus, k1, v1));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const Pair k = pair(f[0][i * RP + r0], f[0][i * RP + r0]);
            s[i].x = fma(k, d0, s[i].x);
            s[i].y = fma(k, d1, s[i].y);
        }
        if (r0 == 0) {
            q0 = sum_q[0][c].x;
            q1 = sum_q[0][c].y;
            qk = sum_qk[0];
#pragma unroll
            for (int w = 1; w < W; ++w) {
                q0 = add(q0, sum_q[w][c].x);
                q1 = add(q1, sum_q[w][c].y);
                qk += sum_qk[w];
            }
            const Pair x = pair(qk, qk);
            const float2 lo = values(fma(x, d0, q0)), hi = values(fma(x, d1, q1));
            TI* op = (TI*)a.o + ((n * a.T + t) * a.HV + hv) * V + col;
            op[0] = from_f<TI>(a.scale * lo.x);
            op[1] = from_f<TI>(a.scale * lo.y);
            op[2] = from_f<TI>(a.scale * hi.x);
            op[3] = from_f<TI>(a.scale * hi.y);
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) *(ulonglong2*)(S + i * RP * V) = s[i];
}

template <typename TI, bool MANY> void (*kernel_of(int K, int V))(StepArgs) {
    return K == 128 ? (V == 128 ? k_step<TI, 128, 128, MANY> : k_step<TI, 128, 64, MANY>)
                    : (V == 128 ? k_step<TI, 64, 128, MANY> : k_step<TI, 64, 64, MANY>);
}
template <typename TI> void (*kernel_of(int K, int V, int T))(StepArgs) {
    return T > 1 ? kernel_of<TI, true>(K, V) : kernel_of<TI, false>(K, V);
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
    if ((int64_t)d->N * d->HV * 4 > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!slots && d->num_slots < d->N) return KDA_ERR_INVALID_ARG;
    if (d->N == 0 || d->T == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !o || (!state && d->num_slots > 0)) return KDA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, (const void*)g, beta, (const void*)state, (const void*)o})
        if (!aligned16(x)) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)slots & 3u) || ((uintptr_t)status & 3u)) return KDA_ERR_INVALID_ARG;
    StepArgs a{q, k, v, beta, g, state, slots, o, status, d->N, d->T, d->H, d->HV, d->num_slots, d->scale};
    cudaStream_t st = (cudaStream_t)stream;
    begin_launches(st);
    const auto kernel = d->dtype == KDA_DTYPE_BF16 ? kernel_of<__nv_bfloat16>(d->K, d->V, d->T)
                                                     : kernel_of<float>(d->K, d->V, d->T);
    const cudaError_t e = launch_after(kernel, a, (unsigned)(d->N * d->HV * (d->V / kCols)), kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("step", st);
    return KDA_OK;
}
