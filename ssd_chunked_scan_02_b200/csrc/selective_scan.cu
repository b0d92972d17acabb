// selective_scan.cu -- the selective scan with a decay of its own for every
// (channel, state), forward and single token:
//
//     a = exp(dt A[d,n]),  h[d,n] = a h[d,n] + dt x B[n],
//     y[d] = (sum_n C[n] h[d,n] + D[d] x) silu(z[d])
//
// A token and channel brings 8 bytes (x, dt, z, y in bf16) and N exponentials,
// all different, so that the exponentials bound the operator, not the memory.
// The recurrence is walked in token order with the states in registers: a
// channel's states lie over a few lanes, the terms dt A and the exponentials
// do not depend on the state and run ahead of it.
//
// A block takes tiles of 32 tokens: its threads first load the tile with wide
// loads and put dt, dt x, B and C as fp32 into shared memory, then every lane
// walks the tile, then the threads that loaded x and z finish y (skip, gate)
// and write it.  The next tile's loads are in flight meanwhile.
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

template <typename T, typename Lay>
__global__ void __launch_bounds__(kThreads)
scan_fwd_kernel(const SelectiveArgs a, T* __restrict__ y, float* __restrict__ final_states,
                const SelectiveDims d, bool vec) {
    constexpr int SPL = Lay::SPL, LPC = Lay::LPC, NP = Lay::NP, CH = Lay::CH, TT = Lay::TT;
    constexpr int VW = load_width<T, CH>();
    constexpr int NI = (TT * CH / VW + kThreads - 1) / kThreads;    // loads a thread and tile
    constexpr int TG = LPC < 8 ? LPC : 8;                           // tokens summed at once
    __shared__ float2 s_du[TT][CH];                                 // dt, dt x
    __shared__ float s_y[TT][CH];
    __shared__ __align__(16) float s_B[TT][NP], s_C[TT][NP];

    const Place pl = place_of<CH>(blockIdx.x, d);
    const int tid = threadIdx.x, lane = tid % LPC, ch = tid / LPC;
    const int64_t len = own_length(a.lens, pl.b, d.L);
    const T* x = static_cast<const T*>(a.x) + pl.b * a.xs.batch + pl.c0;
    const T* dt = static_cast<const T*>(a.dt) + pl.b * a.dts.batch + pl.c0;
    const T* z = a.z ? static_cast<const T*>(a.z) + pl.b * a.zs.batch + pl.c0 : nullptr;
    const T* Bp = static_cast<const T*>(a.B) + pl.b * a.Bs.batch + pl.g * d.N;
    const T* Cp = static_cast<const T*>(a.C) + pl.b * a.Cs.batch + pl.g * d.N;
    y += pl.b * d.L * d.D + pl.c0;

    float A2[SPL], h[SPL];
    const int64_t row = pl.b * d.D + pl.c0 + ch;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const int n = lane * SPL + i;
        const bool on = ch < pl.count && n < d.N;
        A2[i] = on ? a.A[(pl.c0 + ch) * d.N + n] * kLog2E : 0.f;
        h[i] = on && a.init ? a.init[row * d.N + n] : 0.f;
    }

    Raw<T, VW> rx[NI], rdt[NI], rz[NI], nx[NI], ndt[NI], nz[NI];
    auto load = [&](int64_t t0, Raw<T, VW>* px, Raw<T, VW>* pdt, Raw<T, VW>* pz) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
            const int n = t < TT && t0 + t < len ? pl.count - c : 0;
            px[k] = load_channels<T, VW>(x + (t0 + t) * a.xs.token + c, n, vec);
            pdt[k] = load_channels<T, VW>(dt + (t0 + t) * a.dts.token + c, n, vec);
            if (z) pz[k] = load_channels<T, VW>(z + (t0 + t) * a.zs.token + c, n, vec);
        }
    };
    load(0, rx, rdt, rz);

    for (int64_t t0 = 0; t0 < d.L; t0 += TT) {
        // the tile into shared memory; rows behind the sequence: dt = 0, no input
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
            if (t < TT) {
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    float v = 0.f;
                    if (t0 + t < len && c + j < pl.count) {
                        v = to_f32(rdt[k].v[j]) + (a.dt_bias ? a.dt_bias[pl.c0 + c + j] : 0.f);
                        if (a.softplus) v = softplus_f32(v);
                    }
                    s_du[t][c + j] = make_float2(v, v * to_f32(rx[k].v[j]));
                }
            }
        }
        for (int i = tid; i < TT * NP; i += kThreads) {
            const int t = i / NP, n = i % NP;
            const bool on = n < d.N && t0 + t < len;
            s_B[t][n] = on ? to_f32(Bp[(t0 + t) * a.Bs.token + n]) : 0.f;
            s_C[t][n] = on ? to_f32(Cp[(t0 + t) * a.Cs.token + n]) : 0.f;
        }
        __syncthreads();
        if (t0 + TT < d.L) load(t0 + TT, nx, ndt, nz);

#pragma unroll 1
        for (int tt = 0; tt < TT; tt += TG) {
            float ys[TG];
#pragma unroll
            for (int k = 0; k < TG; ++k) {
                const float2 du = s_du[tt + k][ch];
                ys[k] = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const float e = ex2(du.x * A2[i]);
                    h[i] = fmaf(e, h[i], du.y * s_B[tt + k][lane * SPL + i]);
                    ys[k] = fmaf(s_C[tt + k][lane * SPL + i], h[i], ys[k]);
                }
            }
            fold<TG, LPC>(ys, lane);
            if (lane % (LPC / TG) == 0) s_y[tt + lane / (LPC / TG)][ch] = ys[0];
        }
        __syncthreads();

#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int i = k * kThreads + tid, t = i / (CH / VW), c = i % (CH / VW) * VW;
            if (t < TT && t0 + t < d.L) {
                float o[VW];
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    o[j] = 0.f;
                    if (t0 + t < len && c + j < pl.count) {
                        const float Dv = a.D ? a.D[pl.c0 + c + j] : 0.f;
                        o[j] = fmaf(Dv, to_f32(rx[k].v[j]), s_y[t][c + j]);
                        if (z) {
                            const float zv = to_f32(rz[k].v[j]);
                            o[j] *= zv * sigmoid_f32(zv);
                        }
                    }
                }
                store_channels<T, VW>(y + (t0 + t) * d.D + c, raw_from_f32<T, VW>(o),
                                      pl.count - c, vec);
            }
            rx[k] = nx[k]; rdt[k] = ndt[k];
            if (z) rz[k] = nz[k];
        }
    }
    if (final_states && ch < pl.count) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (lane * SPL + i < d.N) final_states[row * d.N + lane * SPL + i] = h[i];
    }
}

// ------------------------------------------------------------------ one token
// Each state element is read and written once (8 bytes against one
// exponential): a stream.  Lanes of a channel as in decode: four neighbouring
// states each.
template <typename T, bool Vec>
__global__ void __launch_bounds__(256)
step_kernel(float* __restrict__ state, const SelectiveArgs a, T* __restrict__ y,
            const SelectiveDims d, int lanes) {
    const int per = 256 / lanes;
    const int lane = threadIdx.x % lanes;
    const int64_t item = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
    const bool on = item < d.b * d.D;
    const int64_t bb = on ? item / d.D : 0, c = on ? item - bb * d.D : 0;
    const int64_t g = c / (d.D / d.G);
    float v = 0.f, xv = 0.f;
    if (on) {
        xv = to_f32(static_cast<const T*>(a.x)[bb * a.xs.batch + c]);
        v = to_f32(static_cast<const T*>(a.dt)[bb * a.dts.batch + c]) +
            (a.dt_bias ? a.dt_bias[c] : 0.f);
        if (a.softplus) v = softplus_f32(v);
    }
    const float u = v * xv;
    const T* Bp = static_cast<const T*>(a.B) + bb * a.Bs.batch + g * d.N;
    const T* Cp = static_cast<const T*>(a.C) + bb * a.Cs.batch + g * d.N;
    float* st = state + (bb * d.D + c) * d.N;
    const float* Ar = a.A + c * d.N;
    float acc = 0.f;
    if (on) {
        for (int64_t n = lane * 4; n < d.N; n += lanes * 4) {
            float hs[4], As[4], Bs[4], Cs[4];
            if constexpr (Vec) {
                const float4 q = __ldcs(reinterpret_cast<const float4*>(st + n));
                const float4 r = __ldg(reinterpret_cast<const float4*>(Ar + n));
                hs[0] = q.x; hs[1] = q.y; hs[2] = q.z; hs[3] = q.w;
                As[0] = r.x; As[1] = r.y; As[2] = r.z; As[3] = r.w;
                raw_to_f32(raw_load<T, 4>(Bp + n), Bs);
                raw_to_f32(raw_load<T, 4>(Cp + n), Cs);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool in = n + i < d.N;
                    hs[i] = in ? st[n + i] : 0.f;
                    As[i] = in ? Ar[n + i] : 0.f;
                    Bs[i] = in ? to_f32(Bp[n + i]) : 0.f;
                    Cs[i] = in ? to_f32(Cp[n + i]) : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hs[i] = fmaf(ex2(v * (As[i] * kLog2E)), hs[i], u * Bs[i]);
                acc = fmaf(Cs[i], hs[i], acc);
            }
            if constexpr (Vec) {
                __stcs(reinterpret_cast<float4*>(st + n), make_float4(hs[0], hs[1], hs[2], hs[3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < d.N) st[n + i] = hs[i];
            }
        }
    }
    for (int o = lanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (on && lane == 0) {
        float o = fmaf(a.D ? a.D[c] : 0.f, xv, acc);
        if (a.z) {
            const float zv = to_f32(static_cast<const T*>(a.z)[bb * a.zs.batch + c]);
            o *= zv * sigmoid_f32(zv);
        }
        y[bb * d.D + c] = from_f32<T>(o);
    }
}

template <typename T>
bool rows_fit(const void* p, Stride s, int w) {
    return reinterpret_cast<uintptr_t>(p) % (w * sizeof(T)) == 0 && s.batch % w == 0 &&
           s.token % w == 0;
}

}  // namespace

// Whether every token's channels can be loaded w elements at a time: all rows
// aligned, and the groups' first channels too.
template <typename T>
bool selective_vec(const SelectiveArgs& a, const SelectiveDims& d, int w) {
    return (d.D / d.G) % w == 0 && rows_fit<T>(a.x, a.xs, w) && rows_fit<T>(a.dt, a.dts, w) &&
           (!a.z || rows_fit<T>(a.z, a.zs, w));
}
template bool selective_vec<float>(const SelectiveArgs&, const SelectiveDims&, int);
template bool selective_vec<__nv_bfloat16>(const SelectiveArgs&, const SelectiveDims&, int);

size_t selective_fwd_workspace_bytes(const SelectiveDims&) { return 0; }

cudaError_t launch_selective_fwd(const SelectiveArgs& a, void* y, float* final_states, float*,
                                 const SelectiveDims& d, Elt t, cudaStream_t s) {
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_layout(d.N, [&](auto lay) {
            using Lay = decltype(lay);
            const int64_t blocks = d.b * channel_blocks<Lay::CH>(d);
            scan_fwd_kernel<T, Lay><<<(unsigned)blocks, kThreads, 0, s>>>(
                a, static_cast<T*>(y), final_states, d,
                selective_vec<T>(a, d, load_width<T, Lay::CH>()));
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_selective_step(float* state, const SelectiveArgs& a, void* y,
                                  const SelectiveDims& d, Elt t, cudaStream_t s) {
    int lanes = 1;
    while (lanes < 32 && lanes * 4 < d.N) lanes *= 2;
    const int64_t per = 256 / lanes, blocks = (d.b * d.D + per - 1) / per;
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        const bool vec = d.N % 4 == 0 && rows_fit<T>(a.B, Stride{a.Bs.batch, 0}, 4) &&
                         rows_fit<T>(a.C, Stride{a.Cs.batch, 0}, 4);
        if (vec) step_kernel<T, true><<<(unsigned)blocks, 256, 0, s>>>(state, a, static_cast<T*>(y), d, lanes);
        else step_kernel<T, false><<<(unsigned)blocks, 256, 0, s>>>(state, a, static_cast<T*>(y), d, lanes);
    });
    return cudaGetLastError();
}

}  // namespace ssd
