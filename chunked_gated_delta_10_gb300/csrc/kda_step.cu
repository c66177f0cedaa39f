// kda_step: the recurrent form of KDA on a few tokens per sequence, the fp32
// states updated in place. Declared in include/kda_serve.h.
//
// With S' = Diag(e^g) S the token needs the state twice, once for S'^T k (the
// delta) and once for the output after the update, but
//   o = scale (S' + k d^T)^T q = scale (S'^T q + (q . k) d),
// so both products come from one sweep over S', and the columns of S are
// independent of one another. A CTA holds 64 (or 32) columns of one state in
// registers for all T tokens: the state is read once and written once.
//
// Bound: 8 K V bytes of state traffic per (sequence, value head), 128 KB at
// K = V = 128. A CTA's loads, sums and stores follow one another, so an SM needs
// several at different points of their way: four CTAs of 32 KB (64 columns) fit.
// Measured, bf16, K = V = 128:
//   N = 256, HV = 32: 157.3 us, 6.91 TB/s, a little above the rate of a plain
//     copy; with 32 columns (seven CTAs) 159.4; a column of a whole state per
//     thread 248.
//   N = 1, HV = 16: 1.9 us with 32 columns, 2.2 with 64: where 64 would leave SMs
//     without a CTA, 32 are taken.
//   N = 16, T = 4, HV = 32: 17.1 us (the states' traffic alone: 10.3); N = 64,
//     T = 7: 73 us (42). Tokens after the first cost sums alone: four operations
//     for each element of a state, 3.6 us a token of the fp32 pipes for N = 64,
//     where a token takes 4.7. With one column a lane the shared memory's return
//     path came first (95 to 115 us): the factors of a row (k, q, e^g, and k
//     again) come back 32 times, for every lane, so a lane takes two columns.
//     Tried: four columns, two CTAs of 128 or 256 threads an SM, 87 and 118 us;
//     eight columns of all rows to a warp, without shared memory and barriers, 100
//     (each warp then forms the factors for itself); one barrier a token instead
//     of two, with three sets of factors, 77 (T = 2: 48 against 50).
// Two rows are a pair of fp32 values (one instruction for both); the rows of a
// column are summed in the same order whatever T and the split are, so several
// tokens at once give the bits of one after the other.
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

constexpr int kThreads = 128;

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

template <int C> __device__ __forceinline__ void load_columns(const float* p, float (&x)[C]) {
    if constexpr (C == 2) {
        const float2 y = *(const float2*)p;
        x[0] = y.x, x[1] = y.y;
    } else {
        x[0] = *p;
    }
}
template <int C> __device__ __forceinline__ void store_columns(float* p, const float (&x)[C]) {
    if constexpr (C == 2)
        *(float2*)p = make_float2(x[0], x[1]);
    else
        *p = x[0];
}

// A token's inputs as a thread reads them: one channel of k, q and g, its columns of v, and beta.
template <typename TI, int C> struct Token {
    TI k, q, v[C], beta;
    float g;
    template <int K, int V> __device__ __forceinline__ void load(const StepArgs& a, int64_t row, int h, int hv, int col) {
        if (threadIdx.x < K) {
            k = ((const TI*)a.k)[(row * a.H + h) * K + threadIdx.x];
            q = ((const TI*)a.q)[(row * a.H + h) * K + threadIdx.x];
            g = a.g[(row * a.HV + hv) * K + threadIdx.x];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = ((const TI*)a.v)[(row * a.HV + hv) * V + col + c];
        beta = ((const TI*)a.beta)[row * a.HV + hv];
    }
};

// One CTA per (sequence, value head, slice of 32 C columns): a lane has C columns, a warp K / 4 rows, two rows to a
// pair. The next token's inputs are loaded while a token is computed.
constexpr int ctas(bool many, int C) { return C == 2 ? 4 : many ? 5 : 7; }  // to an SM
template <typename TI, int K, int V, bool MANY, int C>
__global__ void __launch_bounds__(kThreads, ctas(MANY, C)) k_step(StepArgs a) {
    constexpr int W = kThreads / 32, P = K / W, COLS = 32 * C;  // warps, rows of a warp, columns
    __shared__ __align__(16) float factors[MANY ? 2 : 1][3][K];  // k, q and e^g of a token; the next token has the other
    __shared__ float sum_k[W][COLS], sum_q[W][COLS], sum_qk[W];
    after_previous();
    const unsigned slice = blockIdx.x % (V / COLS), nh = blockIdx.x / (V / COLS);
    const int64_t n = nh / (unsigned)a.HV;
    const int hv = nh % (unsigned)a.HV, h = hv / (a.HV / a.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r0 = warp * P, col = slice * COLS + lane * C;
    const int64_t slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) {
        for (int t = 0; t < a.T; ++t)
            if (warp == 0)
#pragma unroll
                for (int c = 0; c < C; ++c) ((TI*)a.o)[((n * a.T + t) * a.HV + hv) * V + col + c] = from_f<TI>(0.f);
        if (slot >= 0 && a.status && threadIdx.x == 0) *a.status = KDA_ERR_INVALID_ARG;
        return;
    }
    Token<TI, C> in;
    in.template load<K, V>(a, n * a.T, h, hv, col);
    float* S = a.state + (slot * a.HV + hv) * K * V + r0 * V + col;
    Pair s[P / 2][C];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        float x[C], y[C];
        load_columns(S + 2 * i * V, x);
        load_columns(S + (2 * i + 1) * V, y);
#pragma unroll
        for (int c = 0; c < C; ++c) s[i][c] = pair(x[c], y[c]);
    }
    for (int t = 0; t < (MANY ? a.T : 1); ++t) {
        float(*f)[K] = factors[MANY ? t % 2 : 0];
        if (threadIdx.x < K) {
            f[0][threadIdx.x] = to_f(in.k);
            f[1][threadIdx.x] = to_f(in.q);
            f[2][threadIdx.x] = exp2f(in.g * kLog2e);
        }
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = to_f(in.v[c]);
        const float beta = to_f(in.beta);
        __syncthreads();
        if (MANY && t + 1 < a.T) in.template load<K, V>(a, n * a.T + t + 1, h, hv, col);
        float qk = lane < P ? f[0][r0 + lane] * f[1][r0 + lane] : 0.f;
        Pair xk[2][C], xq[2][C];  // sums of k S' and q S'
#pragma unroll
        for (int c = 0; c < C; ++c) xk[0][c] = xk[1][c] = xq[0][c] = xq[1][c] = 0;  // a pair of zeros
#pragma unroll
        for (int i = 0; i < P; i += 4) {
            const ulonglong2 k = *(const ulonglong2*)&f[0][r0 + i], q = *(const ulonglong2*)&f[1][r0 + i];
            const ulonglong2 e = *(const ulonglong2*)&f[2][r0 + i];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                s[i / 2][c] = mul(s[i / 2][c], e.x);
                s[i / 2 + 1][c] = mul(s[i / 2 + 1][c], e.y);
                xk[0][c] = fma(k.x, s[i / 2][c], xk[0][c]);
                xk[1][c] = fma(k.y, s[i / 2 + 1][c], xk[1][c]);
                xq[0][c] = fma(q.x, s[i / 2][c], xq[0][c]);
                xq[1][c] = fma(q.y, s[i / 2 + 1][c], xq[1][c]);
            }
        }
#pragma unroll
        for (int w = 16; w > 0; w /= 2) qk += __shfl_xor_sync(0xffffffffu, qk, w);
        float zk[C], zq[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float2 yk = values(add(xk[0][c], xk[1][c])), yq = values(add(xq[0][c], xq[1][c]));
            zk[c] = yk.x + yk.y;
            zq[c] = yq.x + yq.y;
        }
        store_columns(&sum_k[warp][lane * C], zk);
        store_columns(&sum_q[warp][lane * C], zq);
        if (lane == 0) sum_qk[warp] = qk;
        __syncthreads();
        float d[C];
        load_columns(&sum_k[0][lane * C], zk);
#pragma unroll
        for (int w = 1; w < W; ++w) {
            float y[C];
            load_columns(&sum_k[w][lane * C], y);
#pragma unroll
            for (int c = 0; c < C; ++c) zk[c] += y[c];
        }
        Pair dd[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            d[c] = beta * (v[c] - zk[c]);
            dd[c] = pair(d[c], d[c]);
        }
#pragma unroll
        for (int i = 0; i < P; i += 4) {
            const ulonglong2 k = *(const ulonglong2*)&f[0][r0 + i];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                s[i / 2][c] = fma(k.x, dd[c], s[i / 2][c]);
                s[i / 2 + 1][c] = fma(k.y, dd[c], s[i / 2 + 1][c]);
            }
        }
        if (warp == 0) {
            float z = sum_qk[0];
            load_columns(&sum_q[0][lane * C], zq);
#pragma unroll
            for (int w = 1; w < W; ++w) {
                float y[C];
                load_columns(&sum_q[w][lane * C], y);
#pragma unroll
                for (int c = 0; c < C; ++c) zq[c] += y[c];
                z += sum_qk[w];
            }
            TI* o = (TI*)a.o + ((n * a.T + t) * a.HV + hv) * V + col;
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] = from_f<TI>(a.scale * fmaf(z, d[c], zq[c]));
        }
    }
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        float x[C], y[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float2 z = values(s[i][c]);
            x[c] = z.x;
            y[c] = z.y;
        }
        store_columns(S + 2 * i * V, x);
        store_columns(S + (2 * i + 1) * V, y);
    }
}

template <typename TI, bool MANY, int C> void (*kernel_of(int K, int V))(StepArgs) {
    return K == 128 ? (V == 128 ? k_step<TI, 128, 128, MANY, C> : k_step<TI, 128, 64, MANY, C>)
                    : (V == 128 ? k_step<TI, 64, 128, MANY, C> : k_step<TI, 64, 64, MANY, C>);
}
template <typename TI> void (*kernel_of(int K, int V, int T, int C))(StepArgs) {
    return T > 1 ? (C == 2 ? kernel_of<TI, true, 2>(K, V) : kernel_of<TI, true, 1>(K, V))
                 : (C == 2 ? kernel_of<TI, false, 2>(K, V) : kernel_of<TI, false, 1>(K, V));
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
    const int C = (int64_t)d->N * d->HV * (d->V / 64) >= sm_count() ? 2 : 1;
    const auto kernel = d->dtype == KDA_DTYPE_BF16 ? kernel_of<__nv_bfloat16>(d->K, d->V, d->T, C)
                                                   : kernel_of<float>(d->K, d->V, d->T, C);
    const cudaError_t e = launch_after(kernel, a, (unsigned)(d->N * d->HV * (d->V / (32 * C))), kThreads, st);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch("step", st);
    return KDA_OK;
}
