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
// rows before a run are read twice, and those come from L2.  What keeps the
// memory busy is the number of rows under way: asynchronous copies into a ring in
// shared memory, each thread its own rows (no barrier), run 12 rows ahead
// without a register.
//
// 4 x 8192 x 5376 in bf16 (W = 4, SiLU): forward 126 us, 704 MB at 5.6 TB/s (85%
// of a plain copy's rate); gradients 228 us, 1057 MB at 4.6 TB/s, and 6 us for the
// sum of the partial rows.  Loads held in registers instead of the ring took 156
// and 465 us (too few rows under way, then too many registers).
#include <cuda_bf16.h>

#include "common.cuh"
#include "layer_ops.h"
#include "vec_io.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

template <int N> struct Int { static constexpr int value = N; };
template <typename T> struct Type { using type = T; };

// V fp32 values: pairs in 64-bit registers, one instruction for both (V even).
template <int V>
struct Vals {
    F2 v[V / 2];
    __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 q = unpack2(v[i]);
            f[2 * i] = q.x;
            f[2 * i + 1] = q.y;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = 0;
    }
};
template <>
struct Vals<1> {
    float v[1];
    __device__ __forceinline__ void set(const float (&f)[1]) { v[0] = f[0]; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v[0]; }
    __device__ __forceinline__ void zero() { v[0] = 0.f; }
};
__device__ __forceinline__ F2 mad(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
// a * b + c
template <int V>
__device__ __forceinline__ Vals<V> mad(const Vals<V>& a, const Vals<V>& b, const Vals<V>& c) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i) r.v[i] = mad(a.v[i], b.v[i], c.v[i]);
    return r;
}
__device__ __forceinline__ F2 times(F2 a, F2 b) { return mul2(a, b); }
__device__ __forceinline__ float times(float a, float b) { return a * b; }
__device__ __forceinline__ F2 plus(F2 a, F2 b) { return add2(a, b); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ void both(F2& v, float f) { v = pack2(f, f); }
__device__ __forceinline__ void both(float& v, float f) { v = f; }
// silu(p) = p sigmoid(p)
template <int V>
__device__ __forceinline__ Vals<V> silu_of(const Vals<V>& p) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i)
        r.v[i] = times(p.v[i], sigmoid_fast(p.v[i]));
    return r;
}
// dy silu'(p) = dy s (1 + p (1 - s)), s = sigmoid(p)
template <int V>
__device__ __forceinline__ Vals<V> silu_slope(const Vals<V>& p, const Vals<V>& dy) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i) {
        auto s = sigmoid_fast(p.v[i]), one = s, minus = s;
        both(one, 1.f);
        both(minus, -1.f);
        r.v[i] = times(times(dy.v[i], s), mad(p.v[i], mad(s, minus, one), one));
    }
    return r;
}
template <int V>
__device__ __forceinline__ Vals<V> operator+(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i) r.v[i] = plus(a.v[i], b.v[i]);
    return r;
}
template <int V>
__device__ __forceinline__ Vals<V> operator*(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i) r.v[i] = times(a.v[i], b.v[i]);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> vals_of(const Raw<T, V>& r) {
    float f[V];
    raw_to_f32(r, f);
    Vals<V> o;
    o.set(f);
    return o;
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_of(const Vals<V>& a) {
    float f[V];
    a.get(f);
    return raw_from_f32<T, V>(f);
}

// w[k][i], bias[i] of the V channels from c on (weights are (D, W) fp32), as
// operands of the arithmetic below.
template <int V, int W>
__device__ __forceinline__ void load_params(const float* w, const float* bias, int64_t c,
                                            Vals<V> (&wk)[W], Vals<V>& bv) {
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
    float f[V];
#pragma unroll
    for (int k = 0; k < W; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = flat[i * W + k];
        wk[k].set(f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = bias ? __ldg(bias + c + i) : 0.f;
    bv.set(f);
}

// The inputs before token 0 come from the entering state (row W-1+t holds
// token t < 0), or are zero.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_row(const T* x, int64_t token_stride, const T* init,
                                              int64_t D, int W, int64_t t) {
    if (t >= 0) return raw_load<T, V>(x + t * token_stride);
    return init ? raw_load<T, V>(init + (W - 1 + t) * D) : raw_zero<T, V>();
}

// A thread's rows on their way through shared memory, in groups of kGroup: a group
// is asked for kAhead groups before it is taken.  Rows of two bytes a thread (bf16 of
// odd width or view) are too small for an asynchronous copy: the gradients hold a
// group in registers until the next is asked for (6 x 2048 x 1001: 89 -> 69 us for
// both), the forward, with more threads an SM, loads them as they are needed (18 us;
// 22 with held groups).
constexpr int kGroup = 4, kAhead = 3, kRing = kGroup * (kAhead + 1);

template <typename T, int V, int THREADS, bool HOLD>
struct Rows {
    static constexpr bool kAsync = sizeof(T) * V >= 4, kRinged = kAsync || HOLD;
    static constexpr int kBytes = kRinged ? kRing * THREADS * V * (int)sizeof(T) : 0;
    Raw<T, V>* ring;                  // [kRing][THREADS], this thread's column
    const T* p;                       // the next row to ask for
    int64_t step;
    Raw<T, V> held[kGroup];           // HOLD, not kAsync: the group asked for last
    __device__ __forceinline__ Rows(unsigned char* smem, int tid, const T* from, int64_t stride)
        : ring(reinterpret_cast<Raw<T, V>*>(smem) + tid), p(from), step(stride) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) held[u] = raw_zero<T, V>();
    }
    __device__ __forceinline__ Raw<T, V>* place(int r) { return ring + r % kRing * THREADS; }
    // asks for the rows of group g (0, 1, ... in turn) that are below n
    __device__ __forceinline__ void ask(int g, int n) {
        if constexpr (kRinged) {
            if (!kAsync && g > 0) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u) *place((g - 1) * kGroup + u) = held[u];
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                if (g * kGroup + u < n) {
                    if constexpr (kAsync) copy_async(place(g * kGroup + u), p, true);
                    else held[u] = raw_load<T, V>(p);
                }
                p += step;
            }
        }
    }
    // row r, whose group has arrived (or is loaded now)
    __device__ __forceinline__ Raw<T, V> take(int r) {
        if constexpr (kRinged) {
            return *place(r);
        } else {
            const Raw<T, V> v = raw_load<T, V>(p);
            p += step;
            return v;
        }
    }
};

// ------------------------------------------------------------------ forward
// One thread: V channels, `run` tokens of one sequence.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 5)
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

    const int64_t t0 = r * run, t1 = t0 + run < L ? t0 + run : L;
    const int64_t te = t1 < len ? t1 : len;          // tokens of the sequence itself
    y += t0 * D;
    int left = (int)(t1 - t0), live = (int)(te - t0);
    __shared__ __align__(16) unsigned char ring[Rows<T, V, kThreads, false>::kBytes + 16];
    Rows<T, V, kThreads, false> rows(ring, threadIdx.x, x + t0 * xs.token, xs.token);
    for (int g = 0; g < kAhead; ++g) {
        rows.ask(g, live);
        copies_commit();
    }
    Vals<V> wk[W], bv;
    load_params<V, W>(w, bias, c, wk, bv);

    if (final_state && r == 0) {
        T* f = final_state + bb * (W - 1) * D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            raw_store<T, V>(f + j * D,
                            load_row<T, V>(x, xs.token, init, D, W, len - (W - 1) + j));
    }

    if (live > 0) {
        // p[j]: what the inputs up to here give to the output j tokens ahead
        Vals<V> p[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p[j] = bv;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {            // token t0 - (W-1) + i
            const Vals<V> v = vals_of(load_row<T, V>(x, xs.token, init, D, W, t0 - (W - 1) + i));
#pragma unroll
            for (int j = 0; j <= i; ++j) p[j] = mad(wk[i - j], v, p[j]);
        }
        auto step = [&](const Raw<T, V>& row) {
            const Vals<V> v = vals_of(row);
            const Vals<V> out = mad(wk[W - 1], v, p[0]);
#pragma unroll
            for (int j = 0; j < W - 2; ++j) p[j] = mad(wk[W - 2 - j], v, p[j + 1]);
            p[W - 2] = mad(wk[0], v, bv);
            raw_store<T, V>(y, raw_of<T, V>(silu ? silu_of(out) : out));
            y += D;
        };
        left -= live;
        const int groups = (live + kGroup - 1) / kGroup;
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            copies_pending<kAhead - 1>();
            if ((g + 1) * kGroup <= live) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u) step(rows.take(g * kGroup + u));
            } else {
                for (int u = g * kGroup; u < live; ++u) step(rows.take(u));
            }
            rows.ask(g + kAhead, live);
            copies_commit();
        }
    }
    for (; left > 0; --left, y += D) raw_store<T, V>(y, raw_zero<T, V>());
}

// ------------------------------------------------------------------ backward
// A block of 32 x 4 threads: 32 channel vectors, 4 runs of kRun tokens.  A
// thread walks its run and the W - 1 tokens behind it (whose g its last dx
// need); at token t the gradient of token t - W + 1 is complete.  Each block
// adds its four runs' dw and dbias and writes one partial row a channel; a
// second kernel adds the partial rows in a fixed order.
constexpr int kRun = 64, kSlots = 4;
constexpr int64_t kTile = (int64_t)kRun * kSlots;

// g = dy silu'(p)
template <int V, int W>
__device__ __forceinline__ Vals<V> slope(const Vals<V> (&wk)[W], const Vals<V>& bv,
                                         const Vals<V> (&win)[W], const Vals<V>& dy, bool silu) {
    if (!silu) return dy;
    Vals<V> p = bv;
#pragma unroll
    for (int k = 0; k < W; ++k) p = mad(wk[k], win[k], p);
    return silu_slope(p, dy);
}

template <typename T, typename TG, int V, int W>
__global__ void __launch_bounds__(32 * kSlots, 4)
conv_bwd_kernel(const T* __restrict__ x, Stride xs, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ init,
                const int32_t* __restrict__ lens, int silu, const TG* __restrict__ dy,
                const T* __restrict__ dfinal, T* __restrict__ dx, float* __restrict__ part,
                int64_t L, int64_t D, int64_t ncb, int64_t ntile) {
    extern __shared__ __align__(16) unsigned char ring[];
    const int lane = threadIdx.x, slot = threadIdx.y;
    const int64_t cb = blockIdx.x % ncb, tile = blockIdx.x / ncb % ntile,
                  bb = blockIdx.x / ncb / ntile;
    const int64_t c = (cb * 32 + lane) * V;
    const bool mine = c < D;
    const int64_t len = own_length(lens, bb, L);
    Vals<V> dw[W], db;
    db.zero();
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k].zero();
    const int64_t t0 = tile * kTile + slot * kRun;
    if (mine && t0 < L) {
        const int64_t t1 = t0 + kRun < L ? t0 + kRun : L;
        const int64_t s1 = t1 < len ? t1 : len;         // dx of tokens t0 .. s1-1
        x += bb * xs.batch + c;
        dy += (bb * L + t0) * D + c;
        dx += (bb * L + t0) * D + c;
        if (init) init += bb * (W - 1) * D + c;
        if (dfinal) dfinal += bb * (W - 1) * D + c;
        int todo = s1 > t0 ? (int)(s1 - t0) : 0;        // tokens of the run with a gradient
        const int zeros = (int)(t1 - t0) - todo;
        if (todo > 0) {
            const int ahead = (int)(len - s1 < W - 1 ? len - s1 : W - 1);   // tokens behind with a g
            const int rows = todo + ahead;
            constexpr int kAll = 32 * kSlots;
            Rows<T, V, kAll, true> rx(ring, slot * 32 + lane, x + t0 * xs.token, xs.token);
            Rows<TG, V, kAll, true> rg(ring + Rows<T, V, kAll, true>::kBytes, slot * 32 + lane, dy, D);
            auto ask = [&](int g) {
                rx.ask(g, rows);
                rg.ask(g, rows);
                copies_commit();
            };
            for (int g = 0; g < kAhead; ++g) ask(g);
            Vals<V> wk[W], bv, win[W], q[W];
            load_params<V, W>(w, bias, c, wk, bv);
            // win[k]: token t - W + 1 + k; q[j]: what the g so far give to the
            // gradient of token t - (W-1) + j.  (g before t0 only reaches tokens
            // of the run before.)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                win[j + 1] = vals_of(load_row<T, V>(x, xs.token, init, D, W, t0 - (W - 1) + j));
                q[j].zero();
            }
            // token t: its g, what it gives to dw and dbias (own), and dx of token
            // t - (W-1), which it completes
            auto walk = [&](const Raw<T, V>& rx, const Raw<TG, V>& rg, bool own) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
                win[W - 1] = vals_of(rx);
                const Vals<V> g = slope<V, W>(wk, bv, win, vals_of(rg), silu != 0);
                if (own) {
                    db = db + g;
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k] = mad(g, win[k], dw[k]);
                }
                const Vals<V> done = mad(wk[0], g, q[0]);
#pragma unroll
                for (int j = 0; j < W - 2; ++j) q[j] = mad(wk[j + 1], g, q[j + 1]);
                q[W - 2] = wk[W - 1] * g;
                return done;
            };
            if (todo == kRun && ahead == W - 1) {
                // a whole run, and none of its rows is in the final state
                auto group = [&](int g, auto first, auto own, auto n) {
                    copies_pending<kAhead - 1>();
#pragma unroll
                    for (int u = 0; u < decltype(n)::value; ++u) {
                        const Vals<V> v = walk(rx.take(g * kGroup + u), rg.take(g * kGroup + u),
                                               decltype(own)::value);
                        if (!decltype(first)::value || u >= W - 1) {
                            raw_store<T, V>(dx, raw_of<T, V>(v));
                            dx += D;
                        }
                    }
                    ask(g + kAhead);
                };
                group(0, Int<1>{}, Int<1>{}, Int<kGroup>{});
#pragma unroll 1
                for (int g = 1; g < kRun / kGroup; ++g) group(g, Int<0>{}, Int<1>{}, Int<kGroup>{});
                group(kRun / kGroup, Int<0>{}, Int<0>{}, Int<W - 1>{});
            } else {
                int kept = (int)(t0 - (len - (W - 1)));     // row of the final state of the next dx
                auto emit = [&](const Vals<V>& v) {
                    float f[V];
                    v.get(f);
                    if (dfinal && kept >= 0) {              // a row that the final state keeps
                        float h[V];
                        raw_to_f32(raw_load<T, V>(dfinal + (int64_t)kept * D), h);
#pragma unroll
                        for (int i = 0; i < V; ++i) f[i] += h[i];
                    }
                    raw_store<T, V>(dx, raw_from_f32<T, V>(f));
                    dx += D;
                    ++kept;
                };
#pragma unroll 1
                for (int i = 0; i < todo + W - 1; ++i) {
                    Vals<V> v = q[0];
                    if (i < rows) {
                        if (i % kGroup == 0) copies_pending<kAhead - 1>();
                        v = walk(rx.take(i), rg.take(i), i < todo);
                        if (i % kGroup == kGroup - 1) ask(i / kGroup + kAhead);
                    } else {                                // behind the sequence g is zero
#pragma unroll
                        for (int j = 0; j < W - 2; ++j) q[j] = q[j + 1];
                        q[W - 2].zero();
                    }
                    if (i >= W - 1) emit(v);
                }
            }
        }
        for (int i = 0; i < zeros; ++i, dx += D) raw_store<T, V>(dx, raw_zero<T, V>());
    }

    // the block's partial row: per channel W weights, then the bias
    float(*red)[(W + 1) * V][32] = reinterpret_cast<float(*)[(W + 1) * V][32]>(ring);
    copies_pending<0>();
    __syncthreads();                                    // the rows are done with
    {
        float f[V];
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            if (k < W) dw[k < W ? k : 0].get(f);
            else db.get(f);
#pragma unroll
            for (int i = 0; i < V; ++i) red[slot][i * (W + 1) + k][lane] = f[i];
        }
    }
    __syncthreads();
    for (int j = slot; j < (W + 1) * V; j += kSlots) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) v += red[q][j][lane];
        if (mine) part[((bb * ntile + tile) * D + c) * (W + 1) + j] = v;
    }
}

// dL/d(entering state): row j is the input W - 1 - j tokens before the first, and
// reaches p of the tokens 0 .. j, and (where the sequence is shorter than W - 1)
// the final state's row j - len.
template <typename T, typename TG, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_dinit_kernel(const T* __restrict__ x, Stride xs, const float* __restrict__ w,
                  const float* __restrict__ bias, const T* __restrict__ init,
                  const int32_t* __restrict__ lens, int silu, const TG* __restrict__ dy,
                  const T* __restrict__ dfinal, T* __restrict__ dinit, int64_t b, int64_t L,
                  int64_t D) {
    const int64_t nvec = D / V, item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= nvec * b) return;
    const int64_t c = item % nvec * V, bb = item / nvec;
    const int64_t len = own_length(lens, bb, L);
    x += bb * xs.batch + c;
    if (init) init += bb * (W - 1) * D + c;
    Vals<V> wk[W], bv, win[W], out[W - 1];
    load_params<V, W>(w, bias, c, wk, bv);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        win[j + 1] = vals_of(load_row<T, V>(x, xs.token, init, D, W, j - (W - 1)));
        out[j].zero();
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= len) break;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
        win[W - 1] = vals_of(raw_load<T, V>(x + t * xs.token));
        const Vals<V> g = slope<V, W>(wk, bv, win,
                                      vals_of(raw_load<TG, V>(dy + (bb * L + t) * D + c)), silu != 0);
#pragma unroll
        for (int j = t; j < W - 1; ++j) out[j] = mad(wk[j - t], g, out[j]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float f[V];
        out[j].get(f);
        if (dfinal && j >= len) {
            float h[V];
            raw_to_f32(raw_load<T, V>(dfinal + (bb * (W - 1) + j - len) * D + c), h);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] += h[i];
        }
        raw_store<T, V>(dinit + (bb * (W - 1) + j) * D + c, raw_from_f32<T, V>(f));
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
    Vals<V> wk[W], p;
    load_params<V, W>(w, bias, c, wk, p);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        p = mad(wk[k], vals_of(row[k]), p);
        if (k > 0) raw_store<T, V>(st + (k - 1) * D, row[k]);
    }
    raw_store<T, V>(y + bb * D + c, raw_of<T, V>(silu ? silu_of(p) : p));
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
    // 64-token runs read 5% of the rows twice at W = 4 (runs of 32: 358 instead of
    // 353 us for the convolution and its gradients at 4 x 8192 x 5376); where those
    // are too few threads for 148 SMs, shorter runs spread the tokens over more
    const int64_t nvec = d.D / V;
    int64_t run = 64;
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

int64_t bwd_tiles(const ConvDims& d) { return (d.L + kTile - 1) / kTile; }

template <typename T, typename TG, int V, int W>
cudaError_t bwd_v(const void* x, Stride xs, const float* w, const float* bias, const void* init,
           const int32_t* lens, bool silu, const void* dy, const void* dfinal, void* dx,
           float* dw, float* dbias, void* dinit, float* ws, const ConvDims& d, cudaStream_t s) {
    const int64_t ncb = (d.D / V + 31) / 32, nt = bwd_tiles(d);
    if (d.b > 0 && d.L > 0) {
        constexpr int rows = Rows<T, V, 32 * kSlots, true>::kBytes + Rows<TG, V, 32 * kSlots, true>::kBytes,
                      sums = kSlots * (W + 1) * V * 32 * 4, smem = rows > sums ? rows : sums;
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(
                conv_bwd_kernel<T, TG, V, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        conv_bwd_kernel<T, TG, V, W><<<(unsigned)(ncb * nt * d.b), dim3(32, kSlots), smem, s>>>(
            static_cast<const T*>(x), xs, w, bias, static_cast<const T*>(init), lens, silu,
            static_cast<const TG*>(dy), static_cast<const T*>(dfinal), static_cast<T*>(dx), ws,
            d.L, d.D, ncb, nt);
    }
    if (d.b > 0 && dinit)
        conv_dinit_kernel<T, TG, V, W>
            <<<(unsigned)((d.b * (d.D / V) + kThreads - 1) / kThreads), kThreads, 0, s>>>(
                static_cast<const T*>(x), xs, w, bias, static_cast<const T*>(init), lens, silu,
                static_cast<const TG*>(dy), static_cast<const T*>(dfinal),
                static_cast<T*>(dinit), d.b, d.L, d.D);
    conv_reduce_kernel<W><<<(unsigned)((d.D * (W + 1) + 31) / 32), dim3(32, 8), 0, s>>>(
        ws, d.b * nt, d.D, dw, dbias);
    return cudaGetLastError();
}

// Calls f with the element type, the vector width and the taps as types.
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
        constexpr int V = 4;     // 8-byte bf16 loads: half the registers of 16, twice the threads
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
    cudaError_t err = cudaSuccess;
    with_type(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_width(d.W, [&](auto wi) {
            constexpr int W = decltype(wi)::value;
            auto go = [&](auto tg) {
                using TG = typename decltype(tg)::type;
                if (rows_aligned<T>(x, xs, d.D, 4))
                    err = bwd_v<T, TG, 4, W>(x, xs, w, bias, init, lens, silu, dy, dfinal, dx, dw,
                                             dbias, dinit, ws, d, s);
                else
                    err = bwd_v<T, TG, 1, W>(x, xs, w, bias, init, lens, silu, dy, dfinal, dx, dw,
                                             dbias, dinit, ws, d, s);
            };
            if (dy_f32) go(Type<float>{});
            else go(Type<T>{});
        });
    });
    return err;
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
