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
// A block has two kinds of warps.  Four carriers load a tile of 32 tokens with
// wide loads, put dt, dt x, B and C as fp32 into shared memory, and finish y (skip, gate)
// from the x and z that they still hold.  Four walkers do nothing but the
// recurrence and the sum over states.  While the walkers are on one tile, the
// carriers finish the one before and put down the one behind, with the loads
// of the next in flight: one barrier a tile, and the exponential units are fed
// while the rest of the work goes on beside them.
//
// 8 x 2048 x 1536, N = 16, bf16 with the gate: 203 us; its 403 million exponentials
// alone take 90 us at 16 a clock and SM, 104 with three blocks on some SMs and two
// on others.  The units are 60% busy; what is left is latency: the walkers by
// themselves take 158 us, the carriers by themselves 128.  Holding the loads in
// registers (220 us), both jobs in one kind of warp (259 us; with half the registers
// and more blocks no faster than this either, 361 against 360 us at 4 x 2048 x
// 5120), exponentials computed a step ahead of the recurrence (no change) and eight
// or sixteen states a lane with two or one walking warps (210 and 272 us) were tried.
//
// Where batch and channels are too few blocks for the GPU, a sequence is cut
// into spans (blockIdx.y).  A first launch walks all spans but the last from a
// zero state and leaves the state S each one reaches and its sum of dt; the
// decay over a span is exp(A sum dt), so the second launch finds the state that
// enters span s by h <- exp(A sum dt_k) h + S_k over the spans k before it, and
// walks it for y.  That doubles the exponentials.
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kWalkers = 128;      // threads of the walking warps

enum class What { SpanState, Output, Checkpoints };

template <typename T, typename Lay>
struct Fwd {
    static constexpr int TT = Lay::TT, CH = Lay::CH, NP = Lay::NP;
    static constexpr int PY = CH + 4;                               // s_y's row: no bank twice
    static constexpr int KC = 128;                                  // threads of the carriers
    static constexpr int THREADS = kWalkers + KC;
    static constexpr int VW = load_width<T, CH>();
    static constexpr int NI = (TT * CH / VW + KC - 1) / KC;               // loads a thread and tile
    static constexpr int VB = 16 / sizeof(T);
    static constexpr int NB = (TT * NP * 2 / VB + KC - 1) / KC;
    static constexpr int RAW = KC * (3 * NI * VW + NB * VB) * (int)sizeof(T);   // a tile as it comes
    static constexpr int SMEM = 4 * RAW + 2 * (TT * CH * 8 + TT * PY * 4 + TT * NP * 8) + 2 * CH * 4;
    static constexpr int BLOCKS = SMEM <= 75 * 1024 ? 3 : 2;   // of an SM
};

// What: the state a span reaches from zero; y and the final states; or the
// states before every kTS-th token, for the gradients.  Vec: x, dt and z can be
// copied VW channels, B and C VB states at a time.
template <typename T, typename Lay, What W, bool Vec>
__global__ void __launch_bounds__((Fwd<T, Lay>::THREADS), (Fwd<T, Lay>::BLOCKS))
scan_fwd_kernel(const SelectiveArgs a, T* __restrict__ y, float* __restrict__ final_states,
                const Spans sp, const SelectiveDims d) {
    using F = Fwd<T, Lay>;
    constexpr bool Output = W == What::Output, Sum = W == What::SpanState;
    constexpr int SPL = Lay::SPL, LPC = Lay::LPC, NP = Lay::NP, CH = Lay::CH, TT = Lay::TT;
    constexpr int VW = F::VW, NI = F::NI, VB = F::VB, NB = F::NB, PY = F::PY, KC = F::KC;
    // s_du's columns are permuted by the number of the load that brings them, so
    // that neither the eight lanes that store side by side nor those that read
    // meet a bank twice
    // fp32 rows of odd widths or views are copied element by element (3 x 1825 x 1365,
    // N = 16: 213 -> 123 us); bf16's two bytes cannot be, and are loaded in place
    // (155 us; 170 with the loads held in registers)
    constexpr bool Each = !Vec && sizeof(T) == 4;
    constexpr int SWZ = (CH < 8 ? CH : 8) - 1, PER = CH / VW;       // PER: loads of a token
    static_assert(8 * PER % (SWZ + 1) == 0, "the permutation repeats after eight tokens");
    extern __shared__ __align__(16) unsigned char smem[];
    using RV = Raw<T, VW>;
    using RB = Raw<T, VB>;
    // four tiles as they come: every carrier copies and reads its own elements
    RB* r_bc = reinterpret_cast<RB*>(smem);                         // [4][NB][KC]
    RV* r_x = reinterpret_cast<RV*>(r_bc + 4 * NB * KC);            // [4][NI][KC] each
    RV* r_dt = r_x + 4 * NI * KC;
    RV* r_z = r_dt + 4 * NI * KC;
    float2* s_du = reinterpret_cast<float2*>(r_z + 4 * NI * KC);    // [2][TT][CH]: dt, u
    float* s_B = reinterpret_cast<float*>(s_du + 2 * TT * CH);      // [2][TT][NP]
    float* s_C = s_B + 2 * TT * NP;
    float* s_y = s_C + 2 * TT * NP;                                 // [2][TT][PY]
    float* s_bias = s_y + 2 * TT * PY;                              // [CH] each
    float* s_skip = s_bias + CH;

    const Place pl = place_of<CH>(blockIdx.x, d);
    const bool walker = threadIdx.x < kWalkers;
    const int tid = walker ? threadIdx.x : threadIdx.x - kWalkers;
    const int64_t own = own_length(a.lens, pl.b, d.L);
    const int span = blockIdx.y;
    const int64_t first = span * sp.tokens;
    const int64_t last = span + 1 == sp.count ? d.L : first + sp.tokens;
    const int64_t len = own < last ? own : last;                    // rows read: [first, len)
    const int rows = (int)(last - first);                           // of y
    const T* x = static_cast<const T*>(a.x) + pl.b * a.xs.batch + pl.c0;
    const T* dt = static_cast<const T*>(a.dt) + pl.b * a.dts.batch + pl.c0;
    const T* z = Output && a.z ? static_cast<const T*>(a.z) + pl.b * a.zs.batch + pl.c0 : nullptr;
    const T* Bp = static_cast<const T*>(a.B) + pl.b * a.Bs.batch + pl.g * d.N;
    const T* Cp = static_cast<const T*>(a.C) + pl.b * a.Cs.batch + pl.g * d.N;
    if (Output) y += pl.b * d.L * d.D + pl.c0;

    for (int i = threadIdx.x; i < 4 * TT * NP; i += F::THREADS) s_B[i] = 0.f;   // states beyond N
    for (int c = threadIdx.x; c < CH; c += F::THREADS) {
        s_bias[c] = a.dt_bias && c < pl.count ? a.dt_bias[pl.c0 + c] : 0.f;
        s_skip[c] = Output && a.D && c < pl.count ? a.D[pl.c0 + c] : 0.f;
    }
    __syncthreads();

    if (walker) {
        const int lane = tid % LPC, ch = tid / LPC;
        F2 A[SPL / 2], h[SPL / 2];
        const int64_t row = pl.b * d.D + pl.c0 + ch;
        {
            float av[SPL], hv[SPL];
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                const int n = lane * SPL + i;
                const bool on = ch < pl.count && n < d.N;
                av[i] = on ? decay_rate(a.A[(pl.c0 + ch) * d.N + n]) : 0.f;
                hv[i] = on && !Sum && a.init ? a.init[row * d.N + n] : 0.f;
            }
            if (!Sum && ch < pl.count) {
                for (int k = 0; k < span; ++k) {                        // the spans before this one
                    const int64_t at = (pl.b * (sp.count - 1) + k) * d.D + pl.c0 + ch;
                    const float sum = sp.sum[at];
                    const float* S = sp.state + at * NP + lane * SPL;
#pragma unroll
                    for (int i = 0; i < SPL; ++i) hv[i] = over_span(sum * av[i], hv[i], S[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < SPL / 2; ++i) {
                A[i] = pack2(av[2 * i], av[2 * i + 1]);
                h[i] = pack2(hv[2 * i], hv[2 * i + 1]);
            }
        }
        constexpr int TS = kTS;
        const int64_t nck = (d.L + TS - 1) / TS;
        float* ck = W == What::Checkpoints
                        ? final_states + ((pl.b * nck + first / TS) * d.D + pl.c0 + ch) * NP + lane * SPL
                        : nullptr;
        int ck_left = (rows + TS - 1) / TS;
        auto walk = [&](int w) {
            const float2* du = s_du + w * TT * CH;
            const float* Bt = s_B + w * TT * NP + lane * SPL;
            const float* Ct = s_C + w * TT * NP + lane * SPL;
#pragma unroll 1
            for (int tt = 0; tt < TT; tt += 8) {
                float ys[8];                    // of eight tokens, summed over the lanes at once
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (W == What::Checkpoints && k % TS == 0) {
                        if (ch < pl.count && ck_left > 0) {
#pragma unroll
                            for (int i = 0; i < SPL; i += 4) {
                                const float2 lo = unpack2(h[i / 2]), hi = unpack2(h[i / 2 + 1]);
                                *reinterpret_cast<float4*>(ck + i) = make_float4(lo.x, lo.y, hi.x, hi.y);
                            }
                        }
                        ck += d.D * NP;
                        --ck_left;
                    }
                    const float2 q = du[(tt + k) * CH + (ch ^ ((k * PER + ch / VW) & SWZ))];
                    const F2 dd = pack2(q.x, q.x), uu = pack2(q.y, q.y);
                    F2 yy = 0;
#pragma unroll
                    for (int i = 0; i < SPL; i += 4) {
                        const float4 bv = *reinterpret_cast<const float4*>(Bt + (tt + k) * NP + i);
                        const F2 e0 = decay2(dd, A[i / 2]), e1 = decay2(dd, A[i / 2 + 1]);
                        h[i / 2] = fma2(e0, h[i / 2], mul2(uu, pack2(bv.x, bv.y)));
                        h[i / 2 + 1] = fma2(e1, h[i / 2 + 1], mul2(uu, pack2(bv.z, bv.w)));
                        if (Output) {
                            const float4 cv = *reinterpret_cast<const float4*>(Ct + (tt + k) * NP + i);
                            yy = i == 0 ? mul2(pack2(cv.x, cv.y), h[0])
                                        : fma2(pack2(cv.x, cv.y), h[i / 2], yy);
                            yy = fma2(pack2(cv.z, cv.w), h[i / 2 + 1], yy);
                        }
                    }
                    const float2 f = unpack2(yy);
                    ys[k] = f.x + f.y;
                }
                if (Output) {
                    fold<8, LPC>(ys, lane);
                    constexpr int NT = LPC < 8 ? 8 / LPC : 1, SH = LPC < 8 ? 1 : LPC / 8;
                    if (lane % SH == 0) {
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            s_y[(w * TT + tt + lane / SH * NT + i) * PY + ch] = ys[i];
                    }
                }
            }
        };
        __syncthreads();                                             // the first tile is down
        for (int at = 0; at < rows; at += 2 * TT) {
            walk(0);
            __syncthreads();
            if (at + TT < rows) {
                walk(1);
                __syncthreads();
            }
        }
        float hv[SPL];
#pragma unroll
        for (int i = 0; i < SPL / 2; ++i) {
            const float2 f = unpack2(h[i]);
            hv[2 * i] = f.x;
            hv[2 * i + 1] = f.y;
        }
        if (Output) {
            if (final_states && span + 1 == sp.count && ch < pl.count) {
#pragma unroll
                for (int i = 0; i < SPL; ++i)
                    if (lane * SPL + i < d.N) final_states[row * d.N + lane * SPL + i] = hv[i];
            }
        } else if (Sum) {
            const int64_t at = (pl.b * (sp.count - 1) + span) * d.D + pl.c0;
            if (ch < pl.count) {
#pragma unroll
                for (int i = 0; i < SPL; ++i) sp.state[(at + ch) * NP + lane * SPL + i] = hv[i];
            }
        }
    } else {
        // where this thread's loads of a tile come from and go to; positions `at`
        // of a tile are tokens from the span's first on
        const int own_rows = (int)(len - first > 0 ? len - first : 0);
        const T *px[NI], *pdt[NI], *pz[NI], *pbc[NB];
        int bc_token[NB], bc_to[NB];
        bool is_b[NB];
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int i = k * KC + tid, t = i / PER, c = i % PER * VW < pl.count ? i % PER * VW : 0;
            px[k] = x + (first + t) * a.xs.token + c;
            pdt[k] = dt + (first + t) * a.dts.token + c;
            pz[k] = z ? z + (first + t) * a.zs.token + c : px[k];
        }
        const int nvb = Vec ? (int)d.N / VB : 1;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = k * KC + tid, t = i / (2 * nvb), v = i % (2 * nvb);
            is_b[k] = v < nvb;
            bc_token[k] = t;
            bc_to[k] = (is_b[k] ? v * VB : 2 * TT * NP + (v - nvb) * VB) + t * NP;
            pbc[k] = is_b[k] ? Bp + (first + t) * a.Bs.token + v * VB
                             : Cp + (first + t) * a.Cs.token + (v - nvb) * VB;
        }
        const int64_t x_step = TT * a.xs.token, dt_step = TT * a.dts.token,
                      z_step = TT * (z ? a.zs.token : a.xs.token);
        auto load = [&](int at) {                                   // into ring place at / TT % 4
            const int ring = at / TT & 3;
            if (at < own_rows) {
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const int i = k * KC + tid, t = i / PER, c = i % PER * VW, o = (ring * NI + k) * KC + tid;
                    if constexpr (Vec) {
                        const bool in = t < TT && at + t < own_rows && c < pl.count;
                        copy_async(r_x + o, px[k], in);
                        copy_async(r_dt + o, pdt[k], in);
                        if (z) copy_async(r_z + o, pz[k], in);
                    } else if constexpr (Each) {
                        const int n = t < TT && at + t < own_rows ? pl.count - c : 0;
#pragma unroll
                        for (int j = 0; j < VW; ++j) {
                            copy_async(&r_x[o].v[j], px[k] + j, j < n);
                            copy_async(&r_dt[o].v[j], pdt[k] + j, j < n);
                            if (z) copy_async(&r_z[o].v[j], pz[k] + j, j < n);
                        }
                    } else {
                        const int n = t < TT && at + t < own_rows ? pl.count - c : 0;
                        r_x[o] = load_channels<T, VW>(px[k], n, false);
                        r_dt[o] = load_channels<T, VW>(pdt[k], n, false);
                        if (z) r_z[o] = load_channels<T, VW>(pz[k], n, false);
                    }
                    px[k] += x_step;
                    pdt[k] += dt_step;
                    pz[k] += z_step;
                }
                if constexpr (Vec) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        copy_async(r_bc + (ring * NB + k) * KC + tid, pbc[k],
                                   bc_token[k] < TT && at + bc_token[k] < own_rows);
                        pbc[k] += TT * (is_b[k] ? a.Bs.token : a.Cs.token);
                    }
                }
            }
            if constexpr (Vec || Each) copies_commit();
        };
        float sum_dt[NI][VW];
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < VW; ++j) sum_dt[k][j] = 0.f;
        // the loaded tile into buffer w; rows behind the sequence: dt = 0, no input
        auto stage = [&](int at, int w) {
            float2* du = s_du + w * TT * CH;
            const int ring = at / TT & 3;
            if constexpr (Vec || Each) copies_pending<1>();         // the tile behind may be under way
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int i = k * KC + tid, t = i / PER, c = i % PER * VW, o = (ring * NI + k) * KC + tid;
                if (t < TT) {
                    const int n = at + t < own_rows ? pl.count - c : 0;
                    const RV rx = r_x[o], rdt = r_dt[o];
#pragma unroll
                    for (int j = 0; j < VW; ++j) {
                        float v = to_f32(rdt.v[j]) + s_bias[c + j];
                        if (a.softplus) v = softplus_f32(v);
                        float u = v * to_f32(rx.v[j]);
                        if (j >= n) v = u = 0.f;
                        v *= kLog2E;                      // the decays are powers of two
                        if (Sum) sum_dt[k][j] += v;
                        du[t * CH + ((c + j) ^ (i & SWZ))] = make_float2(v, u);
                    }
                }
            }
            if constexpr (Vec) {
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    if (bc_token[k] < TT) {
                        float f[VB];
                        raw_to_f32(at + bc_token[k] < own_rows ? r_bc[(ring * NB + k) * KC + tid]
                                                               : raw_zero<T, VB>(), f);
                        float* q = s_B + w * TT * NP + bc_to[k];
#pragma unroll
                        for (int j = 0; j < VB; j += 4)
                            *reinterpret_cast<float4*>(q + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                    }
                }
            } else {
                for (int i = tid; i < TT * NP; i += KC) {
                    const int t = i / NP, n = i % NP;
                    const bool on = n < d.N && at + t < own_rows;
                    s_B[w * TT * NP + i] = on ? to_f32(Bp[(first + at + t) * a.Bs.token + n]) : 0.f;
                    if (Output)
                        s_C[w * TT * NP + i] = on ? to_f32(Cp[(first + at + t) * a.Cs.token + n]) : 0.f;
                }
            }
        };
        T* py = y + first * d.D;
        auto finish = [&](int at, int w) {
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int i = k * KC + tid, t = i / PER, c = i % PER * VW;
                if (t < TT && at + t < rows) {
                    const int n = at + t < own_rows ? pl.count - c : 0;
                    const int q = ((at / TT & 3) * NI + k) * KC + tid;
                    const RV kx = r_x[q];
                    RV kz;
                    if (z) kz = r_z[q];
                    float o[VW];
#pragma unroll
                    for (int j = 0; j < VW; ++j) {
                        o[j] = fmaf(s_skip[c + j], to_f32(kx.v[j]), s_y[(w * TT + t) * PY + c + j]);
                        if (z) {
                            const float zv = to_f32(kz.v[j]);
                            o[j] *= zv * sigmoid_fast(zv);
                        }
                        if (j >= n) o[j] = 0.f;
                    }
                    store_channels<T, VW>(py + (int64_t)(at + t) * d.D + c, raw_from_f32<T, VW>(o),
                                          pl.count - c, Vec);
                }
            }
        };

        load(0);
        load(TT);
        if (rows > 0) stage(0, 0);
        load(2 * TT);
        __syncthreads();                                             // the first tile is down
        auto tile = [&](int at, int w) {
            if (Output && at > 0) finish(at - TT, w ^ 1);
            if (at + TT < rows) {
                stage(at + TT, w ^ 1);
                load(at + 3 * TT);
            }
            __syncthreads();
            if (Output && at + TT >= rows) finish(at, w);
        };
        for (int at = 0; at < rows; at += 2 * TT) {
            tile(at, 0);
            if (at + TT < rows) tile(at + TT, 1);
        }
        if (Sum) {
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int i = k * KC + tid, t = i / PER, c = i % PER * VW;
                if (t < TT) {
#pragma unroll
                    for (int j = 0; j < VW; ++j) s_y[t * PY + c + j] = sum_dt[k][j];
                }
            }
        }
    }
    if (Sum) {
        // sums of dt: the threads of a channel, in order
        __syncthreads();
        const int64_t at = (pl.b * (sp.count - 1) + span) * d.D + pl.c0;
        for (int c = threadIdx.x; c < pl.count; c += F::THREADS) {
            float v = 0.f;
            for (int t = 0; t < TT; ++t) v += s_y[t * PY + c];
            sp.sum[at + c] = v;
        }
    }
}

// ------------------------------------------------------------------ one token
// Each state element is read and written once (8 bytes against one
// exponential): a stream.  Four neighbouring states a lane, as in decode.  A
// thread takes its channel of kStepBatch sequences, whose states are all under
// way before the first is used (256 x 5120 x 16: 43 us, 179 MB at 4.1 TB/s, 63% of a
// plain copy's rate; one sequence a thread 65, two 49, eight 57), and reads A once for them; what a channel and
// sequence needs once (softplus, gate) is shared out over the channel's lanes.
constexpr int kStepBatch = 4;

template <typename T, int LANES, bool Vec>
__global__ void __launch_bounds__(256, 3)
step_kernel(float* __restrict__ state, const SelectiveArgs a, T* __restrict__ y, int64_t b, int D,
            int count, int N, int per_group, unsigned across) {
    constexpr int KB = kStepBatch, PER = 256 / LANES;
    constexpr int OWN = LANES >= KB ? 1 : KB / LANES;      // sequences a lane is in charge of
    constexpr int SPAN = LANES >= KB ? LANES / KB : 1;     // lanes in charge of one
    const int lane = threadIdx.x % LANES;
    const unsigned group = blockIdx.x / across;            // `across` blocks hold a sequence's channels
    const unsigned at = (blockIdx.x - group * across) * PER + threadIdx.x / LANES;
    const bool on = at < (unsigned)count;
    const int c = on ? (int)at : 0, g = c / per_group;
    const int64_t b0 = (int64_t)group * KB;
    const int nb = b - b0 < KB ? (int)(b - b0) : KB;
    const float* Ar = a.A + (int64_t)c * N;
    float* st = state + (b0 * D + c) * N;
    const int64_t next = (int64_t)D * N;                   // the same channel of the next sequence
    const T* Bp = static_cast<const T*>(a.B) + b0 * a.Bs.batch + g * N;
    const T* Cp = static_cast<const T*>(a.C) + b0 * a.Cs.batch + g * N;

    // one round for up to 4 LANES states, two for 129 to 256
    float hs[KB][4], As[4], acc[KB];
    Raw<T, 4> rB[KB], rC[KB];
    auto load = [&](int n) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int kk = k < nb ? k : 0, m = n < N ? n : 0;      // what does not exist reads what does
            if constexpr (Vec) {
                const float4 q = __ldcs(reinterpret_cast<const float4*>(st + kk * next + m));
                hs[k][0] = q.x; hs[k][1] = q.y; hs[k][2] = q.z; hs[k][3] = q.w;
                rB[k] = raw_load<T, 4>(Bp + kk * a.Bs.batch + m);
                rC[k] = raw_load<T, 4>(Cp + kk * a.Cs.batch + m);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool in = n + i < N;
                    hs[k][i] = in ? st[kk * next + n + i] : 0.f;
                    rB[k].v[i] = in ? Bp[kk * a.Bs.batch + n + i] : from_f32<T>(0.f);
                    rC[k].v[i] = in ? Cp[kk * a.Cs.batch + n + i] : from_f32<T>(0.f);
                }
            }
        }
        if constexpr (Vec) {
            const float4 r = __ldg(reinterpret_cast<const float4*>(Ar + (n < N ? n : 0)));
            As[0] = r.x; As[1] = r.y; As[2] = r.z; As[3] = r.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) As[i] = n + i < N ? Ar[n + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) As[i] = decay_rate(As[i]);
    };
    load(lane * 4);

    float v[OWN], u[OWN], skip[OWN], gate[OWN];
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int k = lane / SPAN * OWN + j;
        v[j] = u[j] = skip[j] = 0.f;
        gate[j] = 1.f;
        if (k >= nb) continue;
        const float xv = to_f32(static_cast<const T*>(a.x)[(b0 + k) * a.xs.batch + c]);
        v[j] = to_f32(static_cast<const T*>(a.dt)[(b0 + k) * a.dts.batch + c]) +
               (a.dt_bias ? __ldg(a.dt_bias + c) : 0.f);
        if (a.softplus) v[j] = softplus_f32(v[j]);
        u[j] = v[j] * xv;
        v[j] *= kLog2E;
        if (a.D) skip[j] = __ldg(a.D + c) * xv;
        if (a.z) {
            const float zv = to_f32(static_cast<const T*>(a.z)[(b0 + k) * a.zs.batch + c]);
            gate[j] = zv * sigmoid_fast(zv);
        }
    }
#pragma unroll
    for (int k = 0; k < KB; ++k) acc[k] = 0.f;
    for (int n0 = 0; n0 < N; n0 += 4 * LANES) {
        const int n = n0 + lane * 4;
        if (n0 > 0) load(n);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const float vk = __shfl_sync(0xffffffffu, v[k % OWN], k / OWN * SPAN, LANES);
            const float uk = __shfl_sync(0xffffffffu, u[k % OWN], k / OWN * SPAN, LANES);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hs[k][i] = fmaf(decay(vk, As[i]), hs[k][i], uk * to_f32(rB[k].v[i]));
                if (n < N) acc[k] = fmaf(to_f32(rC[k].v[i]), hs[k][i], acc[k]);
            }
            if (k < nb && on && n < N) {
                if constexpr (Vec) {
                    __stcs(reinterpret_cast<float4*>(st + k * next + n),
                           make_float4(hs[k][0], hs[k][1], hs[k][2], hs[k][3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < N) st[k * next + n + i] = hs[k][i];
                }
            }
        }
    }
    fold<KB, LANES>(acc, lane);
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int k = lane / SPAN * OWN + j;
        if (on && k < nb && lane % SPAN == 0)
            y[(b0 + k) * D + c] = from_f32<T>((acc[j] + skip[j]) * gate[j]);
    }
}

// A launch takes groups whose states' elements together stay below 2^31, which is
// all of them but for millions of groups: a thread's offset into B and C then fits 32
// bits (64-bit ones spill without Vec: 256 x 5120 x 33 took 162 us instead of 140).
template <typename T, bool Vec>
void step_lanes(float* state, const SelectiveArgs& a, void* y, const SelectiveDims& d, cudaStream_t s) {
    auto go = [&](auto kernel, int lanes) {
        const int64_t per = d.D / d.G, most = 0x7fffffff / d.N;
        for (int64_t g0 = 0; g0 < d.G; g0 += most) {
            const int64_t c0 = g0 * per, count = (d.G - g0 < most ? d.G - g0 : most) * per;
            const int64_t across = (count + 256 / lanes - 1) / (256 / lanes);
            const int64_t blocks = across * ((d.b + kStepBatch - 1) / kStepBatch);
            SelectiveArgs q = a;                           // from group g0 on
            q.x = static_cast<const T*>(a.x) + c0;
            q.dt = static_cast<const T*>(a.dt) + c0;
            if (a.z) q.z = static_cast<const T*>(a.z) + c0;
            q.B = static_cast<const T*>(a.B) + g0 * d.N;
            q.C = static_cast<const T*>(a.C) + g0 * d.N;
            q.A = a.A + c0 * d.N;
            if (a.D) q.D = a.D + c0;
            if (a.dt_bias) q.dt_bias = a.dt_bias + c0;
            kernel<<<(unsigned)blocks, 256, 0, s>>>(state + c0 * d.N, q, static_cast<T*>(y) + c0, d.b,
                                                    (int)d.D, (int)count, (int)d.N, (int)per,
                                                    (unsigned)across);
        }
    };
    if (d.N <= 4) go(step_kernel<T, 1, Vec>, 1);
    else if (d.N <= 8) go(step_kernel<T, 2, Vec>, 2);
    else if (d.N <= 16) go(step_kernel<T, 4, Vec>, 4);
    else if (d.N <= 32) go(step_kernel<T, 8, Vec>, 8);
    else if (d.N <= 64) go(step_kernel<T, 16, Vec>, 16);
    else go(step_kernel<T, 32, Vec>, 32);
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

// Spans of a sequence: one where the blocks of (batch, channels) are two for each
// of 148 SMs or more; else as many as give every SM what it holds (three blocks in
// bf16, two in fp32), of at least two tiles.  Below three spans the second walk
// over the tokens costs what the first gains.  (1 x 32768 x 1536, 9 spans: 608 us;
// 6 spans 631, 12 spans 630, 18 spans 602, one 1471.)
Spans selective_spans(const SelectiveDims& d, Elt t, float* ws) {
    Spans sp{1, d.L, nullptr, nullptr};
    with_layout(d.N, [&](auto lay) {
        using Lay = decltype(lay);
        const int64_t blocks = d.b * channel_blocks<Lay::CH>(d), tiles = (d.L + Lay::TT - 1) / Lay::TT;
        if (blocks == 0 || blocks >= 148 * 2) return;
        int64_t want = 148 * (t == Elt::F32 ? 2 : 3) / blocks;
        if (want > tiles / 2) want = tiles / 2;
        if (want < 3) return;
        const int64_t per = (tiles + want - 1) / want;
        sp.tokens = per * Lay::TT;
        sp.count = (int)((tiles + per - 1) / per);
        sp.state = ws;
        sp.sum = ws + d.b * (sp.count - 1) * d.D * Lay::NP;
    });
    return sp;
}

size_t selective_fwd_workspace_bytes(const SelectiveDims& d, Elt t) {
    const Spans sp = selective_spans(d, t, nullptr);
    return (size_t)(d.b * (sp.count - 1) * d.D * (padded_states(d.N) + 1)) * 4;
}

// The span states where there are several spans, then the walk for `W`.
template <What W>
cudaError_t run_fwd(const SelectiveArgs& a, void* y, float* out, float* ws, const SelectiveDims& d,
                    Elt t, cudaStream_t s) {
    const Spans sp = selective_spans(d, t, ws);
    cudaError_t err = cudaSuccess;
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        with_layout(d.N, [&](auto lay) {
            using Lay = decltype(lay);
            using F = Fwd<T, Lay>;
            const unsigned blocks = (unsigned)(d.b * channel_blocks<Lay::CH>(d));
            const bool vec = selective_vec<T>(a, d, F::VW) && d.N % F::VB == 0 &&
                             rows_fit<T>(a.B, a.Bs, F::VB) && rows_fit<T>(a.C, a.Cs, F::VB);
            auto go = [&](auto kernel, unsigned spans) {
                err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           F::SMEM);
                if (err == cudaSuccess)
                    kernel<<<dim3(blocks, spans), F::THREADS, F::SMEM, s>>>(
                        a, static_cast<T*>(y), out, sp, d);
            };
            auto both = [&](auto state_only, auto whole) {
                if (sp.count > 1) go(state_only, (unsigned)sp.count - 1);
                if (err == cudaSuccess) go(whole, (unsigned)sp.count);
            };
            if (vec)
                both(scan_fwd_kernel<T, Lay, What::SpanState, true>, scan_fwd_kernel<T, Lay, W, true>);
            else
                both(scan_fwd_kernel<T, Lay, What::SpanState, false>, scan_fwd_kernel<T, Lay, W, false>);
        });
    });
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_selective_fwd(const SelectiveArgs& a, void* y, float* final_states, float* ws,
                                 const SelectiveDims& d, Elt t, cudaStream_t s) {
    return run_fwd<What::Output>(a, y, final_states, ws, d, t, s);
}

cudaError_t launch_selective_checkpoints(const SelectiveArgs& a, float* ckpt, float* ws,
                                         const SelectiveDims& d, Elt t, cudaStream_t s) {
    return run_fwd<What::Checkpoints>(a, nullptr, ckpt, ws, d, t, s);
}

cudaError_t launch_selective_step(float* state, const SelectiveArgs& a, void* y,
                                  const SelectiveDims& d, Elt t, cudaStream_t s) {
    with_elt(t, [&](auto ty) {
        using T = typename decltype(ty)::type;
        const bool vec = d.N % 4 == 0 && rows_fit<T>(a.B, Stride{a.Bs.batch, 0}, 4) &&
                         rows_fit<T>(a.C, Stride{a.Cs.batch, 0}, 4);
        if (vec) step_lanes<T, true>(state, a, y, d, s);
        else step_lanes<T, false>(state, a, y, d, s);
    });
    return cudaGetLastError();
}

}  // namespace ssd
