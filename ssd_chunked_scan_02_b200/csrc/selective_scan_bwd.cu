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
// Two walks: the first, in token order, leaves the states at every kTS-th token
// in the workspace; the second takes the tokens in reverse, TS at a time: it
// computes their TS states again from the state before them, in registers, and
// then walks them backwards.  What the exponentials of the first walk cost is
// what keeping every state would cost in memory several times over.  a_t g_t is
// both the next g and, times h_{t-1}, q_t.
//
// Sums over a group's channels (dB, dC) go over the channels of a warp by
// shuffles, over a block's warps in shared memory, and over the blocks through
// partial rows in the workspace that a last kernel adds in a fixed order; sums
// over tokens (dA, dD, ddt_bias) stay with their thread and go over the batch
// the same way.
// 4 x 2048 x 5120, N = 16, bf16 with the gate: 1097 us for the reverse walk, 267 for
// the states (one launch of the forward's walk), 30 for the sums of dB and dC.  The
// reverse walk is bound by its instructions, about 140 for 32 lanes of four
// states (issue slots 64% busy, 640 blocks on 740 places): 44 are the recurrences
// and products in two-element form, 37 the sums over channels and states, the
// rest loads, softplus, gates and the results.  Four tokens in registers and five
// blocks an SM beat eight tokens and three (1494 us); the operands doubled in
// shared memory to save moves cost more in its bandwidth (+80 us).
#include "selective.cuh"

namespace ssd {

template <typename T>
bool selective_vec(const SelectiveArgs& a, const SelectiveDims& d, int w);

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 128, kWarps = kThreads / 32;

template <typename T, typename Lay>
struct Bwd {
    static constexpr int NP = Lay::NP, CH = Lay::CH;
    static constexpr int TT = NP <= 64 ? 16 : 8;                     // tokens of a tile
    // channels of a load: as many as keep every thread busy
    static constexpr int VW = TT * CH / kThreads < load_width<T, CH>()
                                  ? (TT * CH / kThreads < 4 ? 4 : TT * CH / kThreads)
                                  : load_width<T, CH>();
    static constexpr int PER = CH / VW;
    static constexpr int IT = (TT * PER + kThreads - 1) / kThreads;  // loads a thread and tile
    static constexpr int VB = 16 / sizeof(T);
    static constexpr int BCV = TT * NP * 2 / VB;                     // loads of B and C
    static constexpr int NB = (BCV + kThreads - 1) / kThreads;
    static constexpr int PY = CH + 8;                                // a row of results: no bank twice
    static constexpr int RAW = (kThreads * 4 * IT * VW + BCV * VB) * (int)sizeof(T);
    static constexpr int SMEM = 2 * RAW + TT * CH * 12 + 3 * TT * PY * 4 +
                                TT * NP * 8 * (1 + kWarps) + 2 * kThreads * VW * 4 + 2 * CH * 4;
    // blocks of an SM: five (102 registers a thread) hold the four states a lane of
    // the smaller layouts, three the eight of the larger
    static constexpr int BLOCKS = Lay::SPL == 4 && SMEM <= 45670 ? 5 : SMEM <= 75 * 1024 ? 3 : 2;
};

// ------------------------------------------------------------------ the reverse walk
// ckpt (b, ceil(L / TS), D, NP): the state before token TS * j.  blockIdx.y: the span
// of the sequence.  Carry: only what a span's tokens send to the token before its
// first, from nothing behind its last, and its sum of dt; the walk for the
// gradients then finds the g that enters a span from those of the spans behind.
template <typename T, typename Lay, bool Vec, bool Carry>
__global__ void __launch_bounds__(kThreads, (Bwd<T, Lay>::BLOCKS))
scan_bwd_kernel(const SelectiveArgs a, const SelectiveGrads gr, const float* __restrict__ ckpt,
                float* __restrict__ part_bc, float* __restrict__ part_a,
                float* __restrict__ part_d, const Spans sp, const SelectiveDims d) {
    using S = Bwd<T, Lay>;
    constexpr int SPL = Lay::SPL, LPC = Lay::LPC, NP = Lay::NP, CH = Lay::CH, TS = kTS;
    constexpr int TT = S::TT, VW = S::VW, PER = S::PER, IT = S::IT, VB = S::VB, NB = S::NB;
    constexpr int PY = S::PY;
    constexpr bool Each = !Vec && sizeof(T) == 4;               // copied element by element
    constexpr int CPW = 32 / LPC;                               // channels of a warp
    constexpr int FG = 2;                                       // tokens of a sum over channels
    constexpr int NG = 4;                                       // tokens of a sum over states
    using RV = Raw<T, VW>;
    using RB = Raw<T, VB>;
    extern __shared__ __align__(16) unsigned char smem[];
    // two tiles as they come: a thread copies and reads its own elements
    RB* r_bc = reinterpret_cast<RB*>(smem);                     // [2][BCV]
    RV* r_x = reinterpret_cast<RV*>(r_bc + 2 * S::BCV);  // [2][IT][threads] each
    RV* r_dt = r_x + 2 * IT * kThreads;
    RV* r_z = r_dt + 2 * IT * kThreads;
    RV* r_dy = r_z + 2 * IT * kThreads;
    float2* s_du = reinterpret_cast<float2*>(r_dy + 2 * IT * kThreads);   // [TT][CH]: dt log2(e), u
    float* s_g = reinterpret_cast<float*>(s_du + TT * CH);      // [TT][CH]: dyg
    float* s_B = s_g + TT * CH;                                 // [TT][NP] each
    float* s_C = s_B + TT * NP;
    float* s_red = s_C + TT * NP;                               // [warps][TT][2][NP]
    float* s_sum = s_red + kWarps * TT * 2 * NP;                // [2][VW][threads]: dD, ddt_bias
    float* s_y = s_sum + 2 * kThreads * VW;                     // [TT][PY] each
    float* s_dtg = s_y + TT * PY;                               // du = sum B g
    float* s_q = s_dtg + TT * PY;
    float* s_bias = s_q + TT * PY;                              // [CH] each
    float* s_skip = s_bias + CH;

    const Place pl = place_of<CH>(blockIdx.x, d);
    const int tid = threadIdx.x, lane = tid % LPC, ch = tid / LPC, warp = tid / 32;
    const int64_t len = own_length(a.lens, pl.b, d.L), nck = (d.L + TS - 1) / TS;
    const int span = Carry ? blockIdx.y + 1 : blockIdx.y;
    const int first = (int)(span * sp.tokens), own = (int)len;
    const int L = span + 1 == sp.count ? (int)d.L : first + (int)sp.tokens;     // the span's end
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
    const int64_t row = pl.b * d.D + pl.c0 + ch;

    for (int i = tid; i < 2 * TT * NP; i += kThreads) s_B[i] = 0.f;       // states beyond N
    for (int i = tid; i < 2 * kThreads * VW; i += kThreads) s_sum[i] = 0.f;
    for (int c = tid; c < CH; c += kThreads) {
        s_bias[c] = a.dt_bias && c < pl.count ? a.dt_bias[pl.c0 + c] : 0.f;
        s_skip[c] = a.D && c < pl.count ? a.D[pl.c0 + c] : 0.f;
    }

    F2 A[SPL / 2], g[SPL / 2], dA[SPL / 2];
    {
        float av[SPL], gv[SPL];
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const int n = lane * SPL + i;
            const bool on = ch < pl.count && n < d.N;
            av[i] = on ? decay_rate(a.A[(pl.c0 + ch) * d.N + n]) : 0.f;
            gv[i] = on && !Carry && gr.dfinal ? gr.dfinal[row * d.N + n] : 0.f;
        }
        if (!Carry && ch < pl.count) {
            for (int k = sp.count - 1; k > span; --k) {         // the spans behind this one
                const int64_t at = (pl.b * (sp.count - 1) + k - 1) * d.D + pl.c0 + ch;
                const float sum = sp.sum[at];
                const float* G = sp.state + at * NP + lane * SPL;
#pragma unroll
                for (int i = 0; i < SPL; ++i) gv[i] = over_span(sum * av[i], gv[i], G[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < SPL / 2; ++i) {
            A[i] = pack2(av[2 * i], av[2 * i + 1]);
            g[i] = pack2(gv[2 * i], gv[2 * i + 1]);
            dA[i] = 0;
        }
    }

    const int nvb = Vec ? (int)d.N / VB : 1;
    // token strides below 2^31: one wide multiply-add an address
    const int xt = (int)a.xs.token, dtt = (int)a.dts.token, zt = (int)a.zs.token,
              Bt_ = (int)a.Bs.token, Ct_ = (int)a.Cs.token, Dt = (int)d.D;
    auto load = [&](int t0, int w) {
        if constexpr (Vec) {
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const int i = k * kThreads + tid, t = t0 + i / PER, c = i % PER * VW;
                const int o = (w * IT + k) * kThreads + tid;
                const bool in = i / PER < TT && t < own && c < pl.count;
                const int r = in ? t : 0, cc = in ? c : 0;
                copy_async(r_x + o, x + (int64_t)r * xt + cc, in);
                copy_async(r_dt + o, dt + (int64_t)r * dtt + cc, in);
                copy_async(r_dy + o, dy + (int64_t)r * Dt + cc, in);
                if (z) copy_async(r_z + o, z + (int64_t)r * zt + cc, in);
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int i = k * kThreads + tid, t = t0 + i / (2 * nvb), v = i % (2 * nvb);
                const bool in = i / (2 * nvb) < TT && t < own;
                const int r = in ? t : 0;
                if (i < S::BCV)
                    copy_async(r_bc + w * S::BCV + i,
                               v < nvb ? Bp + (int64_t)r * Bt_ + v * VB
                                       : Cp + (int64_t)r * Ct_ + (v - nvb) * VB, in);
            }
            copies_commit();
        } else if constexpr (Each) {
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const int i = k * kThreads + tid, t = t0 + i / PER, c = i % PER * VW;
                const int o = (w * IT + k) * kThreads + tid;
                const int n = i / PER < TT && t < own ? pl.count - c : 0;
                const int r = n > 0 ? t : 0, cc = n > 0 ? c : 0;
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const int e = j < n ? cc + j : 0;
                    copy_async(&r_x[o].v[j], x + (int64_t)r * xt + e, j < n);
                    copy_async(&r_dt[o].v[j], dt + (int64_t)r * dtt + e, j < n);
                    copy_async(&r_dy[o].v[j], dy + (int64_t)r * Dt + e, j < n);
                    if (z) copy_async(&r_z[o].v[j], z + (int64_t)r * zt + e, j < n);
                }
            }
            copies_commit();
        }
    };
    auto stage = [&](int t0, int w) {
        if constexpr (Vec || Each) copies_pending<0>();
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int i = k * kThreads + tid, tl = i / PER, t = t0 + tl, c = i % PER * VW;
            const int o = (w * IT + k) * kThreads + tid;
            if (tl >= TT) continue;
            const int n = t < own ? pl.count - c : 0;
            if constexpr (!Vec && !Each) {
                r_x[o] = load_channels<T, VW>(x + (int64_t)t * a.xs.token + c, n, false);
                r_dt[o] = load_channels<T, VW>(dt + (int64_t)t * a.dts.token + c, n, false);
                r_dy[o] = load_channels<T, VW>(dy + (int64_t)t * Dt + c, n, false);
                if (z) r_z[o] = load_channels<T, VW>(z + (int64_t)t * a.zs.token + c, n, false);
            }
            const RV rx = r_x[o], rdt = r_dt[o], rdy = r_dy[o];
            RV rz;
            if (z) rz = r_z[o];
            float dl[VW], u[VW], gy[VW];
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                float v = to_f32(rdt.v[j]) + s_bias[c + j];
                gy[j] = to_f32(rdy.v[j]);
                if (a.softplus) v = softplus_f32(v);
                if (z) {
                    const float zv = to_f32(rz.v[j]);
                    gy[j] *= zv * sigmoid_fast(zv);
                }
                u[j] = v * to_f32(rx.v[j]);
                if (j >= n) v = u[j] = gy[j] = 0.f;
                dl[j] = v * kLog2E;
                if (Carry) s_sum[j * kThreads + tid] += dl[j];
            }
#pragma unroll
            for (int j = 0; j < VW; j += 4) {
                float4* q = reinterpret_cast<float4*>(s_du + tl * CH + c + j);
                q[0] = make_float4(dl[j], u[j], dl[j + 1], u[j + 1]);
                q[1] = make_float4(dl[j + 2], u[j + 2], dl[j + 3], u[j + 3]);
                *reinterpret_cast<float4*>(s_g + tl * CH + c + j) =
                    make_float4(gy[j], gy[j + 1], gy[j + 2], gy[j + 3]);
            }
        }
        if constexpr (Vec) {
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int i = k * kThreads + tid, tl = i / (2 * nvb), v = i % (2 * nvb);
                if (tl < TT) {
                    float f[VB];
                    raw_to_f32(t0 + tl < own ? r_bc[w * S::BCV + i] : raw_zero<T, VB>(), f);
                    float* q = v < nvb ? s_B + tl * NP + v * VB : s_C + tl * NP + (v - nvb) * VB;
#pragma unroll
                    for (int j = 0; j < VB; j += 4)
                        *reinterpret_cast<float4*>(q + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                }
            }
        } else {
            for (int i = tid; i < TT * NP; i += kThreads) {
                const int t = t0 + i / NP, n = i % NP;
                const bool on = n < d.N && t < own;
                s_B[i] = on ? to_f32(Bp[(int64_t)t * a.Bs.token + n]) : 0.f;
                s_C[i] = on ? to_f32(Cp[(int64_t)t * a.Cs.token + n]) : 0.f;
            }
        }
    };
    // the states before token t0 (a multiple of TS), a step ahead of their use
    Raw<float, 4> hn[SPL / 4];
    const float* ck = ckpt + (pl.b * nck * d.D + pl.c0 + (ch < pl.count ? ch : 0)) * NP + lane * SPL;
    auto fetch = [&](int t0) {
        const int64_t j = t0 <= 0 ? 0 : t0 / TS < nck ? t0 / TS : nck - 1;
#pragma unroll
        for (int i = 0; i < SPL / 4; ++i) hn[i] = raw_load<float, 4>(ck + j * d.D * NP + 4 * i);
    };

    const int tile0 = first / TT, ntile = (L + TT - 1) / TT;
    if (ntile > tile0) {
        load((ntile - 1) * TT, (ntile - 1) & 1);
        if (!Carry) fetch(ntile * TT - TS);
        __syncthreads();                                        // s_B's zeros, s_bias
    }
    for (int tile = ntile - 1; tile >= tile0; --tile) {
        const int t0 = tile * TT, w = tile & 1;
        stage(t0, w);
        __syncthreads();
        if (tile > tile0) load(t0 - TT, w ^ 1);
        if constexpr (Carry) {
#pragma unroll 1
            for (int tt = TT - TS; tt >= 0; tt -= TS) {
#pragma unroll
                for (int k = TS - 1; k >= 0; --k) {
                    const float dl = s_du[(tt + k) * CH + ch].x, gy = s_g[(tt + k) * CH + ch];
                    const F2 dd = pack2(dl, dl), gg = pack2(gy, gy);
                    const float* Ct = s_C + (tt + k) * NP + lane * SPL;
#pragma unroll
                    for (int i = 0; i < SPL / 2; ++i) {
                        const float2 c2 = *reinterpret_cast<const float2*>(Ct + 2 * i);
                        g[i] = mul2(fma2(gg, pack2(c2.x, c2.y), g[i]), decay2(dd, A[i]));
                    }
                }
            }
        } else {

            // (two rounds unrolled: the sums of one overlap the states of the next;
            // 1120 -> 1060 us at 4 x 2048 x 5120 x 16, four rounds spill)
#pragma unroll 2
            for (int tt = TT - TS; tt >= 0; tt -= TS) {
                // a_t and h_t of TS tokens; h[0] is the state before them.  (Behind the
                // last token dt = 0 keeps the state, and u, dyg, B and C are zero.)
                F2 e[TS][SPL / 2], h[TS + 1][SPL / 2];
#pragma unroll
                for (int i = 0; i < SPL / 2; ++i) h[0][i] = pack2(hn[i / 2].v[i % 2 * 2], hn[i / 2].v[i % 2 * 2 + 1]);
                fetch(t0 + tt - TS);
#pragma unroll
                for (int k = 0; k < TS; ++k) {
                    const float2 q = s_du[(tt + k) * CH + ch];
                    const F2 dd = pack2(q.x, q.x), uu = pack2(q.y, q.y);
                    const float* Bt = s_B + (tt + k) * NP + lane * SPL;
#pragma unroll
                    for (int i = 0; i < SPL / 2; i += 2) {
                        const float4 bv = *reinterpret_cast<const float4*>(Bt + 2 * i);
                        e[k][i] = decay2(dd, A[i]);
                        e[k][i + 1] = decay2(dd, A[i + 1]);
                        h[k + 1][i] = fma2(e[k][i], h[k][i], mul2(uu, pack2(bv.x, bv.y)));
                        h[k + 1][i + 1] = fma2(e[k][i + 1], h[k][i + 1], mul2(uu, pack2(bv.z, bv.w)));
                    }
                }
                F2 at[SPL / 2];
#pragma unroll
                for (int i = 0; i < SPL / 2; ++i) at[i] = 0;
                float py[NG], pu[NG], pq[NG], pB[FG * SPL], pC[FG * SPL];
#pragma unroll
                for (int k = TS - 1; k >= 0; --k) {
                    const float2 q = s_du[(tt + k) * CH + ch];
                    const float gy = s_g[(tt + k) * CH + ch];
                    const F2 dd = pack2(q.x, q.x), uu = pack2(q.y, q.y), gg = pack2(gy, gy);
                    const float* Bt = s_B + (tt + k) * NP + lane * SPL;
                    const float* Ct = s_C + (tt + k) * NP + lane * SPL;
                    F2 sy = 0, su = 0, sq = 0;
#pragma unroll
                    for (int i4 = 0; i4 < SPL; i4 += 4) {
                        const float4 b4 = *reinterpret_cast<const float4*>(Bt + i4);
                        const float4 c4 = *reinterpret_cast<const float4*>(Ct + i4);
                        const F2 Bv[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
                        const F2 Cv[2] = {pack2(c4.x, c4.y), pack2(c4.z, c4.w)};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int i = i4 / 2 + j;
                            g[i] = fma2(gg, Cv[j], g[i]);
                            sy = i == 0 ? mul2(Cv[j], h[k + 1][i]) : fma2(Cv[j], h[k + 1][i], sy);
                            su = i == 0 ? mul2(Bv[j], g[i]) : fma2(Bv[j], g[i], su);
                            const float2 dc = unpack2(mul2(gg, h[k + 1][i])), db = unpack2(mul2(uu, g[i]));
                            pC[k % FG * SPL + 2 * i] = dc.x;
                            pC[k % FG * SPL + 2 * i + 1] = dc.y;
                            pB[k % FG * SPL + 2 * i] = db.x;
                            pB[k % FG * SPL + 2 * i + 1] = db.y;
                            g[i] = mul2(g[i], e[k][i]);
                            const F2 qv = mul2(g[i], h[k][i]);
                            sq = i == 0 ? mul2(A[i], qv) : fma2(A[i], qv, sq);
                            at[i] = fma2(dd, qv, at[i]);
                        }
                    }
                    const float2 fy = unpack2(sy), fu = unpack2(su), fq = unpack2(sq);
                    py[k % NG] = fy.x + fy.y;
                    pu[k % NG] = fu.x + fu.y;
                    pq[k % NG] = fq.x + fq.y;
                    if (k % FG == 0) {
                        // over a warp's channels: the lanes of one place in the channel lie LPC apart
                        const int place = tid % 32 / LPC;
                        constexpr int ALL = FG * SPL, NV = ALL >= CPW ? ALL / CPW : 1;
                        constexpr int SH = ALL >= CPW ? 1 : CPW / ALL;
                        fold<ALL, CPW, LPC>(pB, place);
                        fold<ALL, CPW, LPC>(pC, place);
                        if (place % SH == 0) {
#pragma unroll
                            for (int i = 0; i < NV; ++i) {
                                const int v = place / SH * NV + i, t = tt + k + v / SPL, n = lane * SPL + v % SPL;
                                float* q = s_red + (warp * TT + t) * 2 * NP + n;
                                q[(t & 1) * NP] = pB[i];            // odd tokens: dC first, so that
                                q[(t & 1 ^ 1) * NP] = pC[i];        // two tokens meet no bank twice
                            }
                        }
                    }
                    if (k % NG == 0) {
                        // over a channel's lanes
                        fold<NG, LPC>(py, lane);
                        fold<NG, LPC>(pu, lane);
                        fold<NG, LPC>(pq, lane);
                        constexpr int NT = NG >= LPC ? NG / LPC : 1, SH = NG >= LPC ? 1 : LPC / NG;
                        if (lane % SH == 0) {
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                const int o = (tt + k + lane / SH * NT + i) * PY + ch;
                                s_y[o] = py[i];
                                s_dtg[o] = pu[i];
                                s_q[o] = pq[i];
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < SPL / 2; ++i) dA[i] = add2(dA[i], at[i]);
            }
            __syncthreads();

            for (int i = tid * 4; i < TT * 2 * NP; i += 4 * kThreads) {
                const int t = t0 + i / (2 * NP), col = i % (2 * NP);
                if (t < L) {
                    float4 v = *reinterpret_cast<const float4*>(s_red + i);
#pragma unroll
                    for (int k = 1; k < kWarps; ++k) {
                        const float4 o = *reinterpret_cast<const float4*>(s_red + k * TT * 2 * NP + i);
                        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                    }
                    *reinterpret_cast<float4*>(part_bc + ((cb * d.b + pl.b) * d.L + t) * 2 * NP +
                                               (col ^ (t & 1) * NP)) = v;
                }
            }
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const int i = k * kThreads + tid, tl = i / PER, t = t0 + tl, c = i % PER * VW;
                if (tl >= TT || t >= L) continue;
                const int n = t < own ? pl.count - c : 0, o = (w * IT + k) * kThreads + tid;
                const RV rx = r_x[o], rdt = r_dt[o], rdy = r_dy[o];
                RV rz;
                if (z) rz = r_z[o];
                float ox[VW], ot[VW], oz[VW];
#pragma unroll
                for (int j4 = 0; j4 < VW; j4 += 4) {
                    const float4 du4 = *reinterpret_cast<const float4*>(s_dtg + tl * PY + c + j4);
                    const float4 q4 = *reinterpret_cast<const float4*>(s_q + tl * PY + c + j4);
                    const float4 y4 = *reinterpret_cast<const float4*>(s_y + tl * PY + c + j4);
                    const float4 g4 = *reinterpret_cast<const float4*>(s_g + tl * CH + c + j4);
                    const float4 d0 = reinterpret_cast<const float4*>(s_du + tl * CH + c + j4)[0];
                    const float4 d1 = reinterpret_cast<const float4*>(s_du + tl * CH + c + j4)[1];
                    const float du[4] = {du4.x, du4.y, du4.z, du4.w}, q[4] = {q4.x, q4.y, q4.z, q4.w};
                    const float gy[4] = {g4.x, g4.y, g4.z, g4.w}, yv[4] = {y4.x, y4.y, y4.z, y4.w};
                    const float dl[4] = {d0.x, d0.z, d1.x, d1.z};
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        const int j = j4 + jj;
                        const float xv = to_f32(rx.v[j]), Dv = s_skip[c + j];
                        ox[j] = fmaf(dl[jj] * kLn2, du[jj], Dv * gy[jj]);
                        ot[j] = fmaf(du[jj], xv, q[jj]);
                        if (a.softplus) ot[j] *= sigmoid_fast(to_f32(rdt.v[j]) + s_bias[c + j]);
                        oz[j] = 0.f;
                        if (z) {
                            const float zv = to_f32(rz.v[j]), sg = sigmoid_fast(zv);
                            oz[j] = to_f32(rdy.v[j]) * fmaf(Dv, xv, yv[jj]) * sg * fmaf(zv, 1.f - sg, 1.f);
                        }
                        float gx = gy[jj] * xv;
                        if (j >= n) ox[j] = ot[j] = oz[j] = gx = 0.f;
                        s_sum[j * kThreads + tid] += gx;
                        s_sum[(VW + j) * kThreads + tid] += ot[j];
                    }
                }
                const int left = pl.count - c;
                const int64_t at = (int64_t)t * Dt + c;
                store_channels<T, VW>(dx + at, raw_from_f32<T, VW>(ox), left, Vec);
                store_channels<T, VW>(ddt + at, raw_from_f32<T, VW>(ot), left, Vec);
                if (z) store_channels<T, VW>(dz + at, raw_from_f32<T, VW>(oz), left, Vec);
            }
        }
        __syncthreads();
    }

    if constexpr (Carry) {
        const int64_t at = (pl.b * (sp.count - 1) + span - 1) * d.D + pl.c0;
        if (ch < pl.count) {
#pragma unroll
            for (int i = 0; i < SPL / 2; ++i) {
                const float2 gv = unpack2(g[i]);
                *reinterpret_cast<float2*>(sp.state + (at + ch) * NP + lane * SPL + 2 * i) = gv;
            }
        }
        __syncthreads();
        for (int c = tid; c < pl.count; c += kThreads) {
            float v = 0.f;
            for (int q = c / VW; q < kThreads; q += PER) v += s_sum[c % VW * kThreads + q];
            sp.sum[at + c] = v;
        }
        return;
    }
    // sums over the span's tokens: dA by lane; dD and ddt_bias over the threads of a channel
    const int64_t part = span * d.b + pl.b;
    if (ch < pl.count) {
#pragma unroll
        for (int i = 0; i < SPL / 2; ++i) {
            const float2 da = unpack2(dA[i]), gv = unpack2(g[i]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = lane * SPL + 2 * i + j;
                if (n >= d.N) continue;
                // (nothing from an empty sequence: steps of zero times an infinite or
                // NaN entering state would be NaN)
                part_a[(part * d.D + pl.c0 + ch) * d.N + n] = own > 0 ? (j ? da.y : da.x) * kLn2 : 0.f;
                if (gr.dinit && span == 0) gr.dinit[row * d.N + n] = j ? gv.y : gv.x;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * CH; i += kThreads) {
        const int c = i % CH, which = i / CH;
        if (c >= pl.count) continue;
        float v = 0.f;
        for (int q = c / VW; q < kThreads; q += PER) v += s_sum[(which * VW + c % VW) * kThreads + q];
        part_d[((int64_t)which * sp.count * d.b + part) * d.D + pl.c0 + c] = v;
    }
}

// dB, dC (b,L,G,N): the sum of a group's channel blocks' partial rows
// (blocks, b, L, 2, NP); zero behind a sequence, where an infinite or NaN state, times a
// dyg of zero, is NaN.  64 columns of four states x 4 shares of the blocks a
// thread block, eight rows of a share in flight.
template <typename T>
__global__ void __launch_bounds__(256)
reduce_bc_kernel(const float* __restrict__ part, const int32_t* __restrict__ lens,
                 T* __restrict__ dB, T* __restrict__ dC, const SelectiveDims d, int per_group,
                 int NP) {
    const int64_t tokens = d.b * d.L, row = 2 * NP, total = tokens * d.G * row / 4;
    __shared__ float4 red[4][64];
    for (int64_t i0 = (int64_t)blockIdx.x * 64; i0 < total; i0 += (int64_t)gridDim.x * 64) {
        const int64_t i = i0 + threadIdx.x;
        const int64_t at = i * 4 % (tokens * row), g = i * 4 / (tokens * row);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < total) {
            const float4* p = reinterpret_cast<const float4*>(part + g * per_group * tokens * row + at);
            const int64_t step = tokens * row / 4;
#pragma unroll 8
            for (int k = threadIdx.y; k < per_group; k += 4) {
                const float4 o = __ldcs(p + k * step);
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
        }
        __syncthreads();
        red[threadIdx.y][threadIdx.x] = v;
        __syncthreads();
        if (threadIdx.y || i >= total) continue;
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const float4 o = red[k][threadIdx.x];
            v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
        }
        const int64_t tok = at / row, n = at % NP;
        if (lens && tok % d.L >= own_length(lens, tok / d.L, d.L)) v = make_float4(0.f, 0.f, 0.f, 0.f);
        T* out = (at % row >= NP ? dC : dB) + (tok * d.G + g) * d.N + n;
        if (n < d.N) out[0] = from_f32<T>(v.x);
        if (n + 1 < d.N) out[1] = from_f32<T>(v.y);
        if (n + 2 < d.N) out[2] = from_f32<T>(v.z);
        if (n + 3 < d.N) out[3] = from_f32<T>(v.w);
    }
}

// out[i] = sum over the rows (spans and batch) of part[b][i]
__global__ void __launch_bounds__(256)
reduce_batch_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t b, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int64_t k = 0; k < b; ++k) v += part[k * n + i];
    out[i] = v;
}

struct Work {
    size_t ckpt, bc, a, d, fwd, total;       // floats; fwd: the spans, of either walk
};
Work work_of(const SelectiveDims& d, Elt t) {
    Work w{};
    with_layout(d.N, [&](auto lay) {
        using Lay = decltype(lay);
        const int64_t TS = kTS;
        w.ckpt = 0;
        w.bc = w.ckpt + (size_t)(d.b * ((d.L + TS - 1) / TS) * d.D * Lay::NP);
        w.a = w.bc + (size_t)(channel_blocks<Lay::CH>(d) * d.b * d.L * 2 * Lay::NP);
        const int64_t rows = d.b * selective_spans(d, t, nullptr).count;
        w.d = w.a + (size_t)(rows * d.D * d.N);
        w.fwd = (w.d + (size_t)(2 * rows * d.D) + 3) / 4 * 4;
        w.total = w.fwd + selective_fwd_workspace_bytes(d, t) / 4;
    });
    return w;
}

}  // namespace

size_t selective_bwd_workspace_bytes(const SelectiveDims& d, Elt t) { return work_of(d, t).total * 4; }

cudaError_t launch_selective_bwd(const SelectiveArgs& a, const SelectiveGrads& g, float* ws,
                                 const SelectiveDims& d, Elt t, cudaStream_t s) {
    const Work w = work_of(d, t);
    const Spans sp = selective_spans(d, t, ws + w.fwd);
    cudaError_t err = cudaSuccess;
    if (d.b > 0 && d.L > 0) err = launch_selective_checkpoints(a, ws + w.ckpt, ws + w.fwd, d, t, s);
    if (err != cudaSuccess) return err;
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_layout(d.N, [&](auto lay) {
            using Lay = decltype(lay);
            using S = Bwd<T, Lay>;
            const int64_t nb = channel_blocks<Lay::CH>(d), blocks = d.b * nb;
            if (blocks == 0) return;
            auto go = [&](auto kernel, unsigned spans) {
                if (err == cudaSuccess)
                    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::SMEM);
                if (err == cudaSuccess)
                    kernel<<<dim3((unsigned)blocks, spans), kThreads, S::SMEM, s>>>(
                        a, g, ws + w.ckpt, ws + w.bc, ws + w.a, ws + w.d, sp, d);
            };
            auto both = [&](auto carry, auto whole) {
                if (sp.count > 1) go(carry, (unsigned)sp.count - 1);
                go(whole, (unsigned)sp.count);
            };
            if (selective_vec<T>(a, d, S::VW) && d.N % S::VB == 0 && rows_fit<T>(a.B, a.Bs, S::VB) &&
                rows_fit<T>(a.C, a.Cs, S::VB))
                both(scan_bwd_kernel<T, Lay, true, true>, scan_bwd_kernel<T, Lay, true, false>);
            else
                both(scan_bwd_kernel<T, Lay, false, true>, scan_bwd_kernel<T, Lay, false, false>);
            if (err == cudaSuccess && d.L > 0) {
                const int64_t nblk = (d.b * d.L * d.G * 2 * Lay::NP / 4 + 63) / 64;
                reduce_bc_kernel<T><<<(unsigned)(nblk < 148 * 8 ? nblk : 148 * 8), dim3(64, 4), 0, s>>>(
                    ws + w.bc, a.lens, static_cast<T*>(g.dB), static_cast<T*>(g.dC), d,
                    (int)(nb / d.G), Lay::NP);
            }
        });
    });
    if (err != cudaSuccess) return err;
    const int64_t rows = d.b * sp.count;
    auto add_rows = [&](size_t from, float* out, int64_t n) {
        if (out)
            reduce_batch_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(ws + from, out, rows, n);
    };
    add_rows(w.a, g.dA, d.D * d.N);
    add_rows(w.d, g.dD, d.D);
    add_rows(w.d + (size_t)(rows * d.D), g.ddt_bias, d.D);
    return cudaGetLastError();
}

}  // namespace ssd
