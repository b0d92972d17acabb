// selective_scan_bwd.cu -- gradients of the selective scan.  With
// dyg = dy silu(z) and the reverse recurrence
//
//     g_t = C_t dyg_t + a_{t+1} g_{t+1}                (dL/dh_t)
//
// and q_t = g_t a_t h_{t-1}, the chain rule on h_t = a_t h_{t-1} + dt x B_t gives
//
//     dC_t[n] = sum_d dyg h,      dB_t[n] = sum_d dt x g,     du = sum_n B g,
//     dx = dt du + D dyg,         ddt = x du + sum_n A q,     dA = sum_t dt q,
//     dz = dy (C h + D x) silu'(z),   dD = sum dyg x,
//     d dt_raw = ddt sigmoid(dt_raw + bias),   ddt_bias = sum d dt_raw.
//
// Two walks: the first, in token order, leaves the states at every TS-th token
// in the workspace; the second takes the tokens in reverse, TS at a time: it
// computes their TS states again from the state before them, in registers, and
// then walks them backwards.  What the exponentials of the first walk cost is
// what keeping every state would cost in memory several times over.
//
// Sums over a group's channels (dB, dC) go over the channels of a warp by
// shuffles, over a block's warps in shared memory, and over the blocks through
// partial rows in the workspace that a last kernel adds in a fixed order; sums
// over tokens (dA, dD, ddt_bias) stay with their thread and go over the batch
// the same way.
#include "selective.cuh"

namespace ssd {

template <typename T>
bool selective_vec(const SelectiveArgs& a, const SelectiveDims& d, int w);

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 128, kWarps = kThreads / 32;

template <typename Lay>
struct Bwd {
    static constexpr int TS = 32 / Lay::SPL;                     // tokens in registers
    static constexpr int TT = Lay::NP <= 32 ? 32 : (Lay::NP == 64 ? 16 : 8);
    static constexpr int SMEM = TT * Lay::CH * 6 * 4 + TT * Lay::NP * 2 * 4 * (1 + kWarps);
};

// dt (after bias and softplus) of token t, channel c of the block.
template <typename T>
__device__ __forceinline__ float step_of(T raw, const SelectiveArgs& a, int64_t c) {
    const float v = to_f32(raw) + (a.dt_bias ? a.dt_bias[c] : 0.f);
    return a.softplus ? softplus_f32(v) : v;
}

// ------------------------------------------------------------------ states at every TS-th token
// ckpt (b, ceil(L / TS), D, NP): the state before token TS * j.
template <typename T, typename Lay>
__global__ void __launch_bounds__(kThreads)
checkpoint_kernel(const SelectiveArgs a, float* __restrict__ ckpt, const SelectiveDims d, bool vec) {
    constexpr int SPL = Lay::SPL, LPC = Lay::LPC, NP = Lay::NP, CH = Lay::CH, TT = Lay::TT;
    constexpr int TS = Bwd<Lay>::TS, VW = load_width<T, CH>();
    __shared__ float2 s_du[TT][CH];
    __shared__ __align__(16) float s_B[TT][NP];
    const Place pl = place_of<CH>(blockIdx.x, d);
    const int tid = threadIdx.x, lane = tid % LPC, ch = tid / LPC;
    const int64_t len = own_length(a.lens, pl.b, d.L), nck = (d.L + TS - 1) / TS;
    const T* x = static_cast<const T*>(a.x) + pl.b * a.xs.batch + pl.c0;
    const T* dt = static_cast<const T*>(a.dt) + pl.b * a.dts.batch + pl.c0;
    const T* Bp = static_cast<const T*>(a.B) + pl.b * a.Bs.batch + pl.g * d.N;
    float A[SPL], h[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const int n = lane * SPL + i;
        const bool on = ch < pl.count && n < d.N;
        A[i] = on ? a.A[(pl.c0 + ch) * d.N + n] : 0.f;
        h[i] = on && a.init ? a.init[(pl.b * d.D + pl.c0 + ch) * d.N + n] : 0.f;
    }
    for (int64_t t0 = 0; t0 < d.L; t0 += TT) {
        __syncthreads();
        for (int i = tid; i < TT * CH / VW; i += kThreads) {
            const int t = i / (CH / VW), c = i % (CH / VW) * VW;
            const int n = t0 + t < len ? pl.count - c : 0;
            const auto rx = load_channels<T, VW>(x + (t0 + t) * a.xs.token + c, n, vec);
            const auto rdt = load_channels<T, VW>(dt + (t0 + t) * a.dts.token + c, n, vec);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float v = j < n ? step_of(rdt.v[j], a, pl.c0 + c + j) : 0.f;
                s_du[t][c + j] = make_float2(v * kLog2E, v * to_f32(rx.v[j]));
            }
        }
        for (int i = tid; i < TT * NP; i += kThreads) {
            const int t = i / NP, n = i % NP;
            s_B[t][n] = n < d.N && t0 + t < len ? to_f32(Bp[(t0 + t) * a.Bs.token + n]) : 0.f;
        }
        __syncthreads();
#pragma unroll 1
        for (int tt = 0; tt < TT; tt += TS) {
            if (t0 + tt >= d.L) break;
            if (ch < pl.count) {
                float* q = ckpt + ((pl.b * nck + (t0 + tt) / TS) * d.D + pl.c0 + ch) * NP + lane * SPL;
#pragma unroll
                for (int i = 0; i < SPL; i += 4)
                    *reinterpret_cast<float4*>(q + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
            }
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                const float2 du = s_du[tt + k][ch];
#pragma unroll
                for (int i = 0; i < SPL; ++i)
                    h[i] = fmaf(ex2(du.x * A[i]), h[i], du.y * s_B[tt + k][lane * SPL + i]);
            }
        }
    }
}

// ------------------------------------------------------------------ the reverse walk
template <typename T, typename Lay>
__global__ void __launch_bounds__(kThreads)
scan_bwd_kernel(const SelectiveArgs a, const SelectiveGrads gr, const float* __restrict__ ckpt,
                float* __restrict__ part_bc, float* __restrict__ part_a,
                float* __restrict__ part_d, const SelectiveDims d, bool vec) {
    constexpr int SPL = Lay::SPL, LPC = Lay::LPC, NP = Lay::NP, CH = Lay::CH;
    constexpr int TS = Bwd<Lay>::TS, TT = Bwd<Lay>::TT, VW = load_width<T, CH>();
    constexpr int CPW = 32 / LPC;                               // channels of a warp
    constexpr int IT = (TT * CH / VW + kThreads - 1) / kThreads;
    extern __shared__ __align__(16) float smem[];
    float* s_dt = smem;                                         // [TT][CH] each; dt log2(e)
    float* s_u = s_dt + TT * CH;
    float* s_g = s_u + TT * CH;
    float* s_y = s_g + TT * CH;
    float* s_du = s_y + TT * CH;
    float* s_q = s_du + TT * CH;
    float* s_B = s_q + TT * CH;                                 // [TT][NP]
    float* s_C = s_B + TT * NP;
    float* s_red = s_C + TT * NP;                               // [warps][TT][2][NP]

    const Place pl = place_of<CH>(blockIdx.x, d);
    const int tid = threadIdx.x, lane = tid % LPC, ch = tid / LPC, warp = tid / 32;
    const int64_t len = own_length(a.lens, pl.b, d.L), nck = (d.L + TS - 1) / TS;
    const T* x = static_cast<const T*>(a.x) + pl.b * a.xs.batch + pl.c0;
    const T* dt = static_cast<const T*>(a.dt) + pl.b * a.dts.batch + pl.c0;
    const T* z = a.z ? static_cast<const T*>(a.z) + pl.b * a.zs.batch + pl.c0 : nullptr;
    const T* Bp = static_cast<const T*>(a.B) + pl.b * a.Bs.batch + pl.g * d.N;
    const T* Cp = static_cast<const T*>(a.C) + pl.b * a.Cs.batch + pl.g * d.N;
    const int64_t dense = pl.b * d.L * d.D + pl.c0;
    const T* dy = static_cast<const T*>(gr.dy) + dense;
    T* dx = static_cast<T*>(gr.dx) + dense;
    T* ddt = static_cast<T*>(gr.ddt) + dense;
    T* dz = z ? static_cast<T*>(gr.dz) + dense : nullptr;
    const int64_t cb = blockIdx.x % (gridDim.x / d.b);          // channel block over all groups

    float A[SPL], g[SPL], dA[SPL];
    const int64_t row = pl.b * d.D + pl.c0 + ch;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const int n = lane * SPL + i;
        const bool on = ch < pl.count && n < d.N;
        A[i] = on ? a.A[(pl.c0 + ch) * d.N + n] : 0.f;
        g[i] = on && gr.dfinal ? gr.dfinal[row * d.N + n] : 0.f;
        dA[i] = 0.f;
    }
    float sumD[IT][VW], sumB[IT][VW];
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < VW; ++j) sumD[k][j] = sumB[k][j] = 0.f;

    const int64_t ntile = (d.L + TT - 1) / TT;
    for (int64_t tile = ntile - 1; tile >= 0; --tile) {
        const int64_t t0 = tile * TT;
        Raw<T, VW> rx[IT], rdt[IT], rz[IT], rdy[IT];
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
            if (t >= TT) continue;
            const int n = t0 + t < len ? pl.count - c : 0;
            rx[k] = load_channels<T, VW>(x + (t0 + t) * a.xs.token + c, n, vec);
            rdt[k] = load_channels<T, VW>(dt + (t0 + t) * a.dts.token + c, n, vec);
            rdy[k] = load_channels<T, VW>(dy + (t0 + t) * d.D + c, n, vec);
            if (z) rz[k] = load_channels<T, VW>(z + (t0 + t) * a.zs.token + c, n, vec);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float v = j < n ? step_of(rdt[k].v[j], a, pl.c0 + c + j) : 0.f;
                float gy = j < n ? to_f32(rdy[k].v[j]) : 0.f;
                if (z && j < n) {
                    const float zv = to_f32(rz[k].v[j]);
                    gy *= zv * sigmoid_f32(zv);
                }
                s_dt[t * CH + c + j] = v * kLog2E;
                s_u[t * CH + c + j] = v * to_f32(rx[k].v[j]);
                s_g[t * CH + c + j] = gy;
            }
        }
        for (int i = tid; i < TT * NP; i += kThreads) {
            const int t = i / NP, n = i % NP;
            const bool on = n < d.N && t0 + t < len;
            s_B[i] = on ? to_f32(Bp[(t0 + t) * a.Bs.token + n]) : 0.f;
            s_C[i] = on ? to_f32(Cp[(t0 + t) * a.Cs.token + n]) : 0.f;
        }
        __syncthreads();

#pragma unroll 1
        for (int tt = TT - TS; tt >= 0; tt -= TS) {
            // the states of TS tokens: a_t and a_t h_{t-1} (h_t is that plus u B)
            float e[TS][SPL], eh[TS][SPL], h[SPL];
#pragma unroll
            for (int i = 0; i < SPL; ++i) h[i] = 0.f;
            if (ch < pl.count && t0 + tt < d.L) {
                const float* q = ckpt + ((pl.b * nck + (t0 + tt) / TS) * d.D + pl.c0 + ch) * NP + lane * SPL;
#pragma unroll
                for (int i = 0; i < SPL; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(q + i);
                    h[i] = f.x; h[i + 1] = f.y; h[i + 2] = f.z; h[i + 3] = f.w;
                }
            }
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                const float v = s_dt[(tt + k) * CH + ch], u = s_u[(tt + k) * CH + ch];
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    e[k][i] = ex2(v * A[i]);
                    eh[k][i] = e[k][i] * h[i];
                    h[i] = fmaf(u, s_B[(tt + k) * NP + lane * SPL + i], eh[k][i]);
                }
            }
            float py[TS], pu[TS], pq[TS], pB[TS * SPL], pC[TS * SPL], at[SPL];
#pragma unroll
            for (int i = 0; i < SPL; ++i) at[i] = 0.f;
#pragma unroll
            for (int k = TS - 1; k >= 0; --k) {
                const float v = s_dt[(tt + k) * CH + ch], u = s_u[(tt + k) * CH + ch];
                const float gy = s_g[(tt + k) * CH + ch];
                py[k] = pu[k] = pq[k] = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const float Bv = s_B[(tt + k) * NP + lane * SPL + i];
                    const float Cv = s_C[(tt + k) * NP + lane * SPL + i];
                    const float ht = fmaf(u, Bv, eh[k][i]);
                    g[i] = fmaf(gy, Cv, g[i]);
                    py[k] = fmaf(Cv, ht, py[k]);
                    pC[k * SPL + i] = gy * ht;
                    pu[k] = fmaf(Bv, g[i], pu[k]);
                    pB[k * SPL + i] = u * g[i];
                    const float qv = g[i] * eh[k][i];
                    pq[k] = fmaf(A[i], qv, pq[k]);
                    at[i] = fmaf(v, qv, at[i]);
                    g[i] *= e[k][i];
                }
            }
#pragma unroll
            for (int i = 0; i < SPL; ++i) dA[i] += at[i];
            // over a channel's lanes: lane l holds token l * TS / LPC of y, du and A q
            fold<TS, LPC>(py, lane);
            fold<TS, LPC>(pu, lane);
            fold<TS, LPC>(pq, lane);
            constexpr int NT = TS >= LPC ? TS / LPC : 1, SH = TS >= LPC ? 1 : LPC / TS;
            if (lane % SH == 0) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int t = tt + lane / SH * NT + i;
                    s_y[t * CH + ch] = py[i];
                    s_du[t * CH + ch] = pu[i];
                    s_q[t * CH + ch] = pq[i];
                }
            }
            // over a warp's channels: the lanes of one place in the channel differ by LPC
            fold<TS * SPL, CPW, LPC>(pB, tid % 32 / LPC);
            fold<TS * SPL, CPW, LPC>(pC, tid % 32 / LPC);
            constexpr int NV = TS * SPL / CPW;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = tid % 32 / LPC * NV + i, t = tt + v / SPL, n = lane * SPL + v % SPL;
                s_red[((warp * TT + t) * 2 + 0) * NP + n] = pB[i];
                s_red[((warp * TT + t) * 2 + 1) * NP + n] = pC[i];
            }
        }
        __syncthreads();

        for (int i = tid; i < TT * 2 * NP; i += kThreads) {
            const int t = i / (2 * NP), n = i % NP, which = i / NP % 2;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s_red[w * TT * 2 * NP + i];
            if (t0 + t < d.L && n < d.N)
                part_bc[(((cb * d.b + pl.b) * d.L + t0 + t) * 2 + which) * d.N + n] = v;
        }
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
            if (t >= TT || t0 + t >= d.L) continue;
            const int n = t0 + t < len ? pl.count - c : 0;
            float ox[VW], ot[VW], oz[VW];
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                ox[j] = ot[j] = oz[j] = 0.f;
                if (j >= n) continue;
                const int q = t * CH + c + j;
                const float xv = to_f32(rx[k].v[j]), gy = s_g[q], du = s_du[q];
                const float Dv = a.D ? a.D[pl.c0 + c + j] : 0.f;
                ox[j] = fmaf(s_dt[q] * kLn2, du, Dv * gy);
                ot[j] = fmaf(du, xv, s_q[q]);
                if (a.softplus) {
                    const float v = to_f32(rdt[k].v[j]) + (a.dt_bias ? a.dt_bias[pl.c0 + c + j] : 0.f);
                    ot[j] *= sigmoid_f32(v);
                }
                if (z) {
                    const float zv = to_f32(rz[k].v[j]), sg = sigmoid_f32(zv);
                    oz[j] = to_f32(rdy[k].v[j]) * fmaf(Dv, xv, s_y[q]) * sg * fmaf(zv, 1.f - sg, 1.f);
                }
                sumD[k][j] = fmaf(gy, xv, sumD[k][j]);
                sumB[k][j] += ot[j];
            }
            const int left = pl.count - c;
            store_channels<T, VW>(dx + (t0 + t) * d.D + c, raw_from_f32<T, VW>(ox), left, vec);
            store_channels<T, VW>(ddt + (t0 + t) * d.D + c, raw_from_f32<T, VW>(ot), left, vec);
            if (z) store_channels<T, VW>(dz + (t0 + t) * d.D + c, raw_from_f32<T, VW>(oz), left, vec);
        }
        __syncthreads();
    }

    // sums over the tokens: dA by lane; dD and ddt_bias over the threads of a channel
    if (ch < pl.count) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const int n = lane * SPL + i;
            if (n < d.N) {
                part_a[row * d.N + n] = dA[i] * kLn2;
                if (gr.dinit) gr.dinit[row * d.N + n] = g[i];
            }
        }
    }
    float* s_sum = smem;                                        // [2][TT][CH]
    __syncthreads();
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
        if (t >= TT) continue;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            s_sum[t * CH + c + j] = sumD[k][j];
            s_sum[(TT + t) * CH + c + j] = sumB[k][j];
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * CH; i += kThreads) {
        const int c = i % CH, which = i / CH;
        if (c >= pl.count) continue;
        float v = 0.f;
        for (int t = 0; t < TT; ++t) v += s_sum[(which * TT + t) * CH + c];
        part_d[((int64_t)which * d.b + pl.b) * d.D + pl.c0 + c] = v;
    }
}

// dB, dC (b,L,G,N): the sum of a group's channel blocks' partial rows.
template <typename T>
__global__ void __launch_bounds__(256)
reduce_bc_kernel(const float* __restrict__ part, T* __restrict__ dB, T* __restrict__ dC,
                 const SelectiveDims d, int64_t per_group) {
    const int64_t tokens = d.b * d.L, total = tokens * d.G * 2 * d.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i % d.N, which = i / d.N % 2, tok = i / (2 * d.N) % tokens,
                      g = i / (2 * d.N * tokens);
        float v = 0.f;
        for (int64_t k = 0; k < per_group; ++k)
            v += part[(((g * per_group + k) * tokens + tok) * 2 + which) * d.N + n];
        (which ? dC : dB)[(tok * d.G + g) * d.N + n] = from_f32<T>(v);
    }
}

// out[i] = sum over the batch of part[b][i]
__global__ void __launch_bounds__(256)
reduce_batch_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t b, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int64_t k = 0; k < b; ++k) v += part[k * n + i];
    out[i] = v;
}

struct Work {
    size_t ckpt, bc, a, d, total;       // floats
};
Work work_of(const SelectiveDims& d) {
    Work w{};
    with_layout(d.N, [&](auto lay) {
        using Lay = decltype(lay);
        const int64_t TS = Bwd<Lay>::TS;
        w.ckpt = 0;
        w.bc = w.ckpt + (size_t)(d.b * ((d.L + TS - 1) / TS) * d.D * Lay::NP);
        w.a = w.bc + (size_t)(channel_blocks<Lay::CH>(d) * d.b * d.L * 2 * d.N);
        w.d = w.a + (size_t)(d.b * d.D * d.N);
        w.total = w.d + (size_t)(2 * d.b * d.D);
    });
    return w;
}

}  // namespace

size_t selective_bwd_workspace_bytes(const SelectiveDims& d) { return work_of(d).total * 4; }

cudaError_t launch_selective_bwd(const SelectiveArgs& a, const SelectiveGrads& g, float* ws,
                                 const SelectiveDims& d, Elt t, cudaStream_t s) {
    const Work w = work_of(d);
    cudaError_t err = cudaSuccess;
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_layout(d.N, [&](auto lay) {
            using Lay = decltype(lay);
            const int64_t nb = channel_blocks<Lay::CH>(d), blocks = d.b * nb;
            const bool vec = selective_vec<T>(a, d, load_width<T, Lay::CH>());
            if (blocks > 0) {
                constexpr int smem = Bwd<Lay>::SMEM;
                err = cudaFuncSetAttribute(scan_bwd_kernel<T, Lay>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
                if (err != cudaSuccess) return;
                if (d.L > 0)
                    checkpoint_kernel<T, Lay><<<(unsigned)blocks, kThreads, 0, s>>>(a, ws + w.ckpt, d, vec);
                scan_bwd_kernel<T, Lay><<<(unsigned)blocks, kThreads, smem, s>>>(
                    a, g, ws + w.ckpt, ws + w.bc, ws + w.a, ws + w.d, d, vec);
                if (d.L > 0) {
                    const int64_t total = d.b * d.L * d.G * 2 * d.N, nblk = (total + 255) / 256;
                    reduce_bc_kernel<T><<<(unsigned)(nblk < 148 * 16 ? nblk : 148 * 16), 256, 0, s>>>(
                        ws + w.bc, static_cast<T*>(g.dB), static_cast<T*>(g.dC), d, nb / d.G);
                }
            }
        });
    });
    if (err != cudaSuccess) return err;
    auto over_batch = [&](size_t from, float* out, int64_t n) {
        if (out)
            reduce_batch_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(ws + from, out, d.b, n);
    };
    over_batch(w.a, g.dA, d.D * d.N);
    over_batch(w.d, g.dD, d.D);
    over_batch(w.d + (size_t)(d.b * d.D), g.ddt_bias, d.D);
    return cudaGetLastError();
}

}  // namespace ssd
