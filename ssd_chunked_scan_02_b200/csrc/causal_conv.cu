// causal_conv.cu -- the short causal depthwise convolution in front of the
// layer, its gradients and its single-token form:
//
//     p_t = bias + sum_k w[k] x_{t-W+1+k},     y_t = silu(p_t)
//     g_t = dy_t silu'(p_t),   dx_s = sum_k w[k] g_{s+W-1-k},
//     dw[k] = sum_t g_t x_{t-W+1+k},   dbias = sum_t g_t
//
// Every channel is on its own and a token touches its W - 1 neighbours, so the
// operator is a stream: x is read and y written once (2 bytes an element each
// in bf16).  A thread owns a few neighbouring channels (one wide load a token)
// and walks a run of tokens with the last W inputs in registers; only the W - 1
// rows before a run are read twice, and those come from L2.
#include <cuda_bf16.h>

#include "common.cuh"
#include "layer_ops.h"
#include "vec_io.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t own_length(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : (n > L ? L : n);
}

// w[k][i], bias[i] of the V channels from c on (weights are (D, W) fp32).
template <int V, int W>
__device__ __forceinline__ void load_params(const float* w, const float* bias, int64_t c,
                                            float (&wk)[W][V], float (&bv)[V]) {
    float flat[V * W];
    if constexpr (V * W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * W; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(w + c * W + i));
            flat[i] = q.x; flat[i + 1] = q.y; flat[i + 2] = q.z; flat[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) flat[i] = __ldg(w + c * W + i);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) wk[k][i] = flat[i * W + k];
        bv[i] = bias ? __ldg(bias + c + i) : 0.f;
    }
}

// The inputs before token 0 come from the entering state (row W-1+t holds
// token t < 0), or are zero.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_row(const T* x, int64_t token_stride, const T* init,
                                              int64_t D, int W, int64_t t) {
    if (t >= 0) return raw_load<T, V>(x + t * token_stride);
    return init ? raw_load<T, V>(init + (W - 1 + t) * D) : raw_zero<T, V>();
}

// ------------------------------------------------------------------ forward
// One thread: V channels, `run` tokens of one sequence.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const T* __restrict__ x, Stride xs, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ init,
                const int32_t* __restrict__ lens, int silu, T* __restrict__ y,
                T* __restrict__ final_state, int64_t b, int64_t L, int64_t D, int64_t run,
                int64_t nrun) {
    const int64_t nvec = D / V;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= nvec * nrun * b) return;
    const int64_t c = item % nvec * V, r = item / nvec % nrun, bb = item / nvec / nrun;
    const int64_t len = own_length(lens, bb, L);
    x += bb * xs.batch + c;
    if (init) init += bb * (W - 1) * D + c;
    y += bb * L * D + c;

    float wk[W][V], bv[V];
    load_params<V, W>(w, bias, c, wk, bv);

    if (final_state && r == 0) {
        T* f = final_state + bb * (W - 1) * D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            raw_store<T, V>(f + j * D,
                            load_row<T, V>(x, xs.token, init, D, W, len - (W - 1) + j));
    }

    const int64_t t0 = r * run, t1 = t0 + run < L ? t0 + run : L;
    const int64_t te = t1 < len ? t1 : len;          // tokens of the sequence itself
    int64_t t = t0;
    if (t < te) {
        float win[W][V];                             // win[k]: token t - W + 1 + k
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            raw_to_f32(load_row<T, V>(x, xs.token, init, D, W, t0 - (W - 1) + j), win[j + 1]);
        constexpr int U = 8;                         // rows in flight
        for (; t < te; t += U) {
            Raw<T, V> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < te) raw[u] = raw_load<T, V>(x + (t + u) * xs.token);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < te) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
                    raw_to_f32(raw[u], win[W - 1]);
                    float p[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        p[i] = bv[i];
#pragma unroll
                        for (int k = 0; k < W; ++k) p[i] = fmaf(wk[k][i], win[k][i], p[i]);
                        if (silu) p[i] *= sigmoid_f32(p[i]);
                    }
                    raw_store<T, V>(y + (t + u) * D, raw_from_f32<T, V>(p));
                }
            }
        }
        t = te;
    }
    for (; t < t1; ++t) raw_store<T, V>(y + t * D, raw_zero<T, V>());
}

// ------------------------------------------------------------------ backward
// A block of 32 x 8 threads: 32 channel vectors, 8 runs of kRun tokens.  A
// thread walks its run and the W - 1 tokens behind it (whose g its last dx
// need); at token t the gradient of token t - W + 1 is complete.  Each block
// adds its eight runs' dw and dbias and writes one partial row a channel; a
// second kernel adds the partial rows in a fixed order.
constexpr int kRun = 32, kSlots = 8;
constexpr int64_t kTile = (int64_t)kRun * kSlots;

template <typename T, typename TG, int V, int W>
__global__ void __launch_bounds__(32 * kSlots)
conv_bwd_kernel(const T* __restrict__ x, Stride xs, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ init,
                const int32_t* __restrict__ lens, int silu, const TG* __restrict__ dy,
                const T* __restrict__ dfinal, T* __restrict__ dx, T* __restrict__ dinit,
                float* __restrict__ part, int64_t L, int64_t D, int64_t ncb, int64_t ntile) {
    const int lane = threadIdx.x, slot = threadIdx.y;
    const int64_t cb = blockIdx.x % ncb, tile = blockIdx.x / ncb % ntile,
                  bb = blockIdx.x / ncb / ntile;
    const int64_t c = (cb * 32 + lane) * V;
    const bool mine = c < D;
    const int64_t len = own_length(lens, bb, L);
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0.f;
    }
    if (mine) {
        x += bb * xs.batch + c;
        dy += bb * L * D + c;
        dx += bb * L * D + c;
        if (init) init += bb * (W - 1) * D + c;
        if (dfinal) dfinal += bb * (W - 1) * D + c;
        if (dinit) dinit += bb * (W - 1) * D + c;
        float wk[W][V], bv[V];
        load_params<V, W>(w, bias, c, wk, bv);

        // dL/dx of token s < len, or of the entering state's row W-1+s for s < 0
        auto emit = [&](int64_t s, float (&v)[V]) {
            const int64_t j = s - (len - (W - 1));      // its row in the final state
            if (dfinal && j >= 0 && j < W - 1) {
                float f[V];
                raw_to_f32(raw_load<T, V>(dfinal + j * D), f);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += f[i];
            }
            if (s >= 0) raw_store<T, V>(dx + s * D, raw_from_f32<T, V>(v));
            else if (dinit) raw_store<T, V>(dinit + (W - 1 + s) * D, raw_from_f32<T, V>(v));
        };

        const int64_t t0 = tile * kTile + slot * kRun;
        const int64_t t1 = t0 + kRun < L ? t0 + kRun : L;
        // the first run also gives the entering state's gradient: tokens -(W-1) .. -1
        const int64_t s0 = t0 == 0 ? -(int64_t)(W - 1) : t0;
        const int64_t s1 = t1 < len ? t1 : len;         // dx of tokens s0 .. s1-1
        if (t0 <= t1 && s0 < s1) {
            float win[W][V], g[W][V];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                raw_to_f32(load_row<T, V>(x, xs.token, init, D, W, t0 - (W - 1) + j), win[j + 1]);
#pragma unroll
                for (int i = 0; i < V; ++i) g[j + 1][i] = 0.f;
            }
            // g of the tokens before t0 only reaches inputs that belong to the
            // run before (or, at t0 == 0, does not exist), so it starts at zero
            constexpr int U = 4;
            const int64_t te = s1 + W - 1;              // last token walked, exclusive
            for (int64_t t = t0; t < te; t += U) {
                Raw<T, V> rx[U];
                Raw<TG, V> rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = t + u < te && t + u < len;
                    rx[u] = in ? raw_load<T, V>(x + (t + u) * xs.token) : raw_zero<T, V>();
                    rg[u] = in ? raw_load<TG, V>(dy + (t + u) * D) : raw_zero<TG, V>();
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u >= te) break;
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            win[k][i] = win[k + 1][i];
                            g[k][i] = g[k + 1][i];
                        }
                    raw_to_f32(rx[u], win[W - 1]);
                    raw_to_f32(rg[u], g[W - 1]);
                    if (silu) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float p = bv[i];
#pragma unroll
                            for (int k = 0; k < W; ++k) p = fmaf(wk[k][i], win[k][i], p);
                            const float sg = sigmoid_f32(p);
                            g[W - 1][i] *= sg * fmaf(p, 1.f - sg, 1.f);
                        }
                    }
                    if (t + u >= len) {                 // behind the sequence: no gradient
#pragma unroll
                        for (int i = 0; i < V; ++i) g[W - 1][i] = 0.f;
                    }
                    if (t + u < s1) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            db[i] += g[W - 1][i];
#pragma unroll
                            for (int k = 0; k < W; ++k)
                                dw[k][i] = fmaf(g[W - 1][i], win[k][i], dw[k][i]);
                        }
                    }
                    const int64_t s = t + u - (W - 1);
                    if (s >= s0) {
                        float v[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            v[i] = 0.f;
#pragma unroll
                            for (int k = 0; k < W; ++k) v[i] = fmaf(wk[W - 1 - k][i], g[k][i], v[i]);
                        }
                        emit(s, v);
                    }
                }
            }
        }
        for (int64_t t = s1 > t0 ? s1 : t0; t < t1; ++t)
            raw_store<T, V>(dx + t * D, raw_zero<T, V>());
    }

    // the block's partial row: per channel W weights, then the bias
    __shared__ float red[kSlots][(W + 1) * V][32];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) red[slot][i * (W + 1) + k][lane] = dw[k][i];
        red[slot][i * (W + 1) + W][lane] = db[i];
    }
    __syncthreads();
    for (int j = slot; j < (W + 1) * V; j += kSlots) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) v += red[q][j][lane];
        if (mine) part[((bb * ntile + tile) * D + c) * (W + 1) + j] = v;
    }
}

// dweight, dbias: the sum of the partial rows.  32 columns x 8 row groups a
// block; column j of a row is weight k = j % (W+1) of channel j / (W+1).
template <int W>
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float* __restrict__ part, int64_t rows, int64_t D,
                   float* __restrict__ dw, float* __restrict__ dbias) {
    const int64_t cols = D * (W + 1);
    const int64_t j = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (j < cols)
        for (int64_t r = threadIdx.y; r < rows; r += 8) v += part[r * cols + j];
    __shared__ float red[8][32];
    red[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y || j >= cols) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) v += red[q][threadIdx.x];
    const int64_t c = j / (W + 1);
    const int k = (int)(j % (W + 1));
    if (k < W) dw[c * W + k] = v;
    else dbias[c] = v;
}

// ------------------------------------------------------------------ one token
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(T* __restrict__ state, const T* __restrict__ x, int64_t x_batch,
                 const float* __restrict__ w, const float* __restrict__ bias, int silu,
                 T* __restrict__ y, int64_t b, int64_t D) {
    const int64_t nvec = D / V;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= nvec * b) return;
    const int64_t c = item % nvec * V, bb = item / nvec;
    T* st = state + bb * (W - 1) * D + c;
    Raw<T, V> row[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row[k] = *reinterpret_cast<const Raw<T, V>*>(st + k * D);
    row[W - 1] = raw_load<T, V>(x + bb * x_batch + c);
    float wk[W][V], p[V];
    load_params<V, W>(w, bias, c, wk, p);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float v[V];
        raw_to_f32(row[k], v);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = fmaf(wk[k][i], v[i], p[i]);
        if (k > 0) raw_store<T, V>(st + (k - 1) * D, row[k]);
    }
    if (silu) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] *= sigmoid_f32(p[i]);
    }
    raw_store<T, V>(y + bb * D + c, raw_from_f32<T, V>(p));
}

// Whether x's rows can be read V elements at a time (D % V == 0 and every
// row's first element aligned; the other tensors are dense and 16-byte aligned,
// so that D % V == 0 is enough for them).
template <typename T>
bool rows_aligned(const void* x, Stride xs, int64_t D, int V) {
    return D % V == 0 && reinterpret_cast<uintptr_t>(x) % (V * sizeof(T)) == 0 &&
           xs.batch % V == 0 && xs.token % V == 0;
}

template <typename T, int V, int W>
void fwd_v(const void* x, Stride xs, const float* w, const float* bias, const void* init,
           const int32_t* lens, bool silu, void* y, void* fin, const ConvDims& d,
           cudaStream_t s) {
    // 32-token runs read 9% of the rows twice at W = 4; where those are too few
    // threads for 148 SMs, shorter runs spread the tokens over more of them
    const int64_t nvec = d.D / V;
    int64_t run = 32;
    while (run > 8 && d.b * nvec * ((d.L + run - 1) / run) < 148 * 1024) run /= 2;
    const int64_t nrun = d.L > 0 ? (d.L + run - 1) / run : 1;
    const int64_t items = d.b * nvec * nrun;
    conv_fwd_kernel<T, V, W><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(
        static_cast<const T*>(x), xs, w, bias, static_cast<const T*>(init), lens, silu,
        static_cast<T*>(y), static_cast<T*>(fin), d.b, d.L, d.D, run, nrun);
}

template <typename T, int V, int W>
void step_v(void* state, const void* x, int64_t x_batch, const float* w, const float* bias,
            bool silu, void* y, const ConvDims& d, cudaStream_t s) {
    const int64_t items = d.b * (d.D / V);
    conv_step_kernel<T, V, W><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(
        static_cast<T*>(state), static_cast<const T*>(x), x_batch, w, bias, silu,
        static_cast<T*>(y), d.b, d.D);
}

int64_t bwd_tiles(const ConvDims& d) { return d.L > 0 ? (d.L + kTile - 1) / kTile : 1; }

template <typename T, typename TG, int V, int W>
void bwd_v(const void* x, Stride xs, const float* w, const float* bias, const void* init,
           const int32_t* lens, bool silu, const void* dy, const void* dfinal, void* dx,
           float* dw, float* dbias, void* dinit, float* ws, const ConvDims& d, cudaStream_t s) {
    const int64_t ncb = (d.D / V + 31) / 32, nt = bwd_tiles(d);
    if (d.b > 0)
        conv_bwd_kernel<T, TG, V, W><<<(unsigned)(ncb * nt * d.b), dim3(32, kSlots), 0, s>>>(
            static_cast<const T*>(x), xs, w, bias, static_cast<const T*>(init), lens, silu,
            static_cast<const TG*>(dy), static_cast<const T*>(dfinal), static_cast<T*>(dx),
            static_cast<T*>(dinit), ws, d.L, d.D, ncb, nt);
    conv_reduce_kernel<W><<<(unsigned)((d.D * (W + 1) + 31) / 32), dim3(32, 8), 0, s>>>(
        ws, d.b * nt, d.D, dw, dbias);
}

// Calls f with the element type, the vector width and the taps as types.
template <int N> struct Int { static constexpr int value = N; };
template <typename T> struct Type { using type = T; };

template <typename F>
void with_width(int W, F f) {
    if (W == 2) f(Int<2>{});
    else if (W == 3) f(Int<3>{});
    else f(Int<4>{});
}
template <typename F>
void with_type(Elt t, F f) {
    if (t == Elt::F32) f(Type<float>{});
    else f(Type<__nv_bfloat16>{});
}

}  // namespace

cudaError_t launch_conv_fwd(const void* x, Stride xs, const float* w, const float* bias,
                            const void* init, const int32_t* lens, bool silu, void* y,
                            void* final_state, const ConvDims& d, Elt t, cudaStream_t s) {
    with_type(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        constexpr int V = 16 / sizeof(T);
        with_width(d.W, [&](auto wi) {
            constexpr int W = decltype(wi)::value;
            if (rows_aligned<T>(x, xs, d.D, V))
                fwd_v<T, V, W>(x, xs, w, bias, init, lens, silu, y, final_state, d, s);
            else
                fwd_v<T, 1, W>(x, xs, w, bias, init, lens, silu, y, final_state, d, s);
        });
    });
    return cudaGetLastError();
}

size_t conv_bwd_workspace_bytes(const ConvDims& d) {
    return (size_t)(d.b * bwd_tiles(d) * d.D * (d.W + 1)) * 4;
}

cudaError_t launch_conv_bwd(const void* x, Stride xs, const float* w, const float* bias,
                            const void* init, const int32_t* lens, bool silu, const void* dy,
                            bool dy_f32, const void* dfinal, void* dx, float* dw, float* dbias,
                            void* dinit, float* ws, const ConvDims& d, Elt t, cudaStream_t s) {
    with_type(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_width(d.W, [&](auto wi) {
            constexpr int W = decltype(wi)::value;
            auto go = [&](auto tg) {
                using TG = typename decltype(tg)::type;
                if (rows_aligned<T>(x, xs, d.D, 4))
                    bwd_v<T, TG, 4, W>(x, xs, w, bias, init, lens, silu, dy, dfinal, dx, dw,
                                       dbias, dinit, ws, d, s);
                else
                    bwd_v<T, TG, 1, W>(x, xs, w, bias, init, lens, silu, dy, dfinal, dx, dw,
                                       dbias, dinit, ws, d, s);
            };
            if (dy_f32) go(Type<float>{});
            else go(Type<T>{});
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_conv_step(void* state, const void* x, int64_t x_batch, const float* w,
                             const float* bias, bool silu, void* y, const ConvDims& d, Elt t,
                             cudaStream_t s) {
    with_type(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        constexpr int V = 16 / sizeof(T);
        with_width(d.W, [&](auto wi) {
            constexpr int W = decltype(wi)::value;
            if (rows_aligned<T>(x, Stride{x_batch, 0}, d.D, V))
                step_v<T, V, W>(state, x, x_batch, w, bias, silu, y, d, s);
            else
                step_v<T, 1, W>(state, x, x_batch, w, bias, silu, y, d, s);
        });
    });
    return cudaGetLastError();
}

}  // namespace ssd
