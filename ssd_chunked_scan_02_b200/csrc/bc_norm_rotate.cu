// bc_norm_rotate.cu -- root-mean-square norm and position rotation of B and C
// in one pass, and their gradients:
//
//     r = 1 / sqrt(mean(v^2) + eps),  u = v r w,  out = R(pos) u
//     du = R(-pos) dout,  dw = sum du v r,  dv = r (du w - v r^2 mean(du w v))
//
// Every element is read once and written once; the rows are short (N <= 256),
// so a row stays in the registers of a few neighbouring lanes and its sum of
// squares is a handful of shuffles.  A lane holds four pairs, as two runs of
// four elements, so that both halves of a pair are in one lane in either
// order of pairs.
//
// The angles depend on (token, pair) alone, and B and C of every group share
// them.  A block first writes the cosines and sines of a tile of tokens into
// shared memory, then its lane groups ("units") walk the tile's rows.  A unit
// keeps to one row index (B or C, one group), so that the weights, and in the
// backward their gradients' sums, stay in registers over all its tokens.
//
// 4 x 8192 tokens of 8 groups, N = 128, 64 elements turned, bf16: 53 us, 269 MB at
// 5.0 TB/s (77% of a plain copy's rate), the issue slots 67% busy: conversions,
// norm and turn are about 130 instructions a lane and eight elements.  Gradients
// (8 x 2048 tokens, fp32 in, all turned): 61 us, and 6 us for the weights' sums.
//
// Far positions: pos * freq is wanted modulo 2 pi, where the product's integer
// part is useless.  freq / (2 pi) is taken as a 64-bit fixed-point fraction of
// a turn, and pos times it modulo 2^64 is one exact integer product: what the
// fraction's last place leaves out, 2^-64 of a turn, times pos is its error (7e-10
// radians at 2^31, less than the sines' own; 4e-7 at 2^40).  freq / (2 pi) has to be
// known to as many places for that (a product in fp64 is off by 5e-7 radians at 2^33).
#include <cuda_bf16.h>

#include "common.cuh"
#include "layer_ops.h"
#include "vec_io.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

struct Args {
    const void *B, *C, *gB, *gC;      // gB, gC: dL/dout (backward)
    Stride bs, cs;
    const float *wB, *wC;
    int per_group;                    // weights (G, N) instead of (N)
    const int64_t* pos;
    const float* freq;
    float eps;
    int interleaved;
    void *oB, *oC;                    // out, or dL/dB and dL/dC
    float* part;                      // (blocks, 2 G, N): partial sums of dweight
    int64_t L;
    int G, N, R;
    int lanes;                        // lanes of a unit: a power of two
    int tile;                         // tokens of a block's tile, all of one sequence
    int table_bytes;                  // of the tile's cosines and sines
    int64_t tiles, ntile;             // of a sequence, and of all
};

// The fraction of a turn that a position makes, freq / (2 pi), as a signed 64-bit
// fixed-point number less than 2^-64 off; kNoStep where freq is infinite or NaN.
// 1 / (2 pi) is the sum of two fp64 numbers, and the product keeps its rounding error.
constexpr int64_t kNoStep = -0x7fffffffffffffffLL - 1;
__device__ __forceinline__ int64_t turn_step(float freq) {
    const double f = freq, hi = 0.15915494309189533577, lo = -9.8393383375912434770e-18;
    const double turns = f * hi, rest = fma(f, hi, -turns) + f * lo;
    // (whole turns of one step drop out, and the sum is modulo a turn)
    const uint64_t step = (uint64_t)__double2ll_rn((turns - rint(turns)) * 18446744073709551616.0) +
                          (uint64_t)__double2ll_rn((rest - rint(rest)) * 18446744073709551616.0);
    if (!isfinite(freq)) return kNoStep;
    return (int64_t)step == kNoStep ? kNoStep + 1 : (int64_t)step;
}

// Cosine and sine of pos * freq: the turn modulo 2^64, its upper 32 bits to the
// nearest quarter and a rest of at most an eighth of a turn (exact), and there the
// Taylor series, to x^9 and x^10 (below 2e-9 at pi / 4).
__device__ __forceinline__ float2 cos_sin(int64_t pos, int64_t step) {
    const uint32_t turn = (uint32_t)(((uint64_t)pos * (uint64_t)step) >> 32);
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float x2 = x * x;
    float s = 2.7557319e-6f, c = -2.7557319e-7f;        // 1 / 9!, -1 / 10!
    s = fmaf(s, x2, -1.9841270e-4f);
    s = fmaf(s, x2, 8.3333333e-3f);
    s = fmaf(s, x2, -1.6666667e-1f);
    s = fmaf(s * x2, x, x);
    c = fmaf(c, x2, 2.4801587e-5f);
    c = fmaf(c, x2, -1.3888889e-3f);
    c = fmaf(c, x2, 4.1666667e-2f);
    c = fmaf(c, x2, -0.5f);
    c = fmaf(c, x2, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// Element e (0..7) of the lane's four pairs: pairs p0 .. p0+3 sit at runs of
// four elements from o0 and from o1.  In registers, v[0..3] and v[4..7] are the
// runs; pair q is (v[q], v[4+q]) where the runs are the halves, else neighbours.
template <bool Halves>
__device__ __forceinline__ void turn_pairs(float (&v)[8], const float2 (&cs)[4], float sign) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int i = Halves ? q : 2 * q, j = Halves ? 4 + q : 2 * q + 1;
        const float a = v[i], b = v[j], sn = cs[q].y * sign;
        v[i] = a * cs[q].x - b * sn;
        v[j] = a * sn + b * cs[q].x;
    }
}

// Over a unit's lanes (LANES, or `lanes` where that is 0).
template <int LANES>
__device__ __forceinline__ float unit_sum(float v, int lanes) {
    if constexpr (LANES > 0) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// A lane's part of the rows to come.  Vec: the runs of four are whole, aligned
// copies of 8 or 16 bytes, kAhead rows ahead through a ring in shared memory (a
// lane copies and reads its own elements: no barrier); otherwise each element is
// loaded on its own, where it exists, as its row is taken.
constexpr int kRing = 4, kAhead = kRing - 1;

template <typename T, bool Vec>
struct Rows {
    static constexpr int kBytes = Vec ? kRing * kThreads * 8 * (int)sizeof(T) : 0;
    Raw<T, 4>* ring;                  // [kRing][2][threads], this thread's column
    const T* ask_at;
    const T* take_at;
    int64_t step;
    __device__ __forceinline__ Rows(unsigned char* smem)
        : ring(reinterpret_cast<Raw<T, 4>*>(smem) + threadIdx.x), ask_at(nullptr), take_at(nullptr),
          step(0) {}
    __device__ __forceinline__ void start(const T* p, int64_t stride) {
        ask_at = take_at = p;
        step = stride;
    }
    __device__ __forceinline__ void ask(int i, bool exists, const int (&at)[8]) {
        if constexpr (Vec) {
            if (exists) {
                copy_async(ring + (i % kRing * 2) * kThreads, ask_at + at[0], true);
                copy_async(ring + (i % kRing * 2 + 1) * kThreads, ask_at + at[4], true);
            }
            ask_at += step;
        }
    }
    __device__ __forceinline__ void take(int i, bool exists, const int (&at)[8], int N, float (&v)[8]) {
        if constexpr (Vec) {
            const Raw<T, 4> lo = ring[(i % kRing * 2) * kThreads], hi = ring[(i % kRing * 2 + 1) * kThreads];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = exists ? to_f32(lo.v[k]) : 0.f;
                v[4 + k] = exists ? to_f32(hi.v[k]) : 0.f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = exists && at[k] < N ? to_f32(take_at[at[k]]) : 0.f;
            take_at += step;
        }
    }
};
template <typename T, bool Vec>
__device__ __forceinline__ void store8(T* row, const int (&at)[8], int N, const float (&v)[8]) {
    if constexpr (Vec) {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        raw_store<T, 4>(row + at[0], raw_from_f32<T, 4>(a));
        raw_store<T, 4>(row + at[4], raw_from_f32<T, 4>(b));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at[i] < N) row[at[i]] = from_f32<T>(v[i]);
    }
}

// The eight elements of a lane: pairs 4 q .. 4 q + 3 of the row, R / 2 turned
// pairs first, then the unturned elements two by two.  Elements that do not
// exist get index N.
__device__ __forceinline__ void lane_elements(int lane, int N, int R, bool interleaved,
                                              int (&at)[8]) {
    const int half = R / 2;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int p = lane * 4 + q;
        int i, j;
        if (p < half) {
            i = interleaved ? 2 * p : p;
            j = interleaved ? 2 * p + 1 : p + half;
        } else {
            i = R + 2 * (p - half);
            j = i + 1;
        }
        if (interleaved || p >= half) {      // neighbours: the runs are 8 elements in a row
            at[2 * q] = i < N ? i : N;
            at[2 * q + 1] = j < N ? j : N;
        } else {
            at[q] = i;
            at[4 + q] = j;
        }
    }
}

// Lanes whose four pairs are partly turned halves and partly neighbours exist
// only where R / 2 is no multiple of 4; they take the scalar path, on pairs
// (v[q], v[4+q]) throughout.
__device__ __forceinline__ void lane_pairs(int lane, int N, int R, bool interleaved,
                                           int (&at)[8]) {
    const int half = R / 2;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int p = lane * 4 + q;
        int i, j;
        if (p < half) {
            i = interleaved ? 2 * p : p;
            j = interleaved ? 2 * p + 1 : p + half;
        } else {
            i = R + 2 * (p - half);
            j = i + 1;
        }
        at[q] = i < N ? i : N;
        at[4 + q] = j < N ? j : N;
    }
}

// Halves: pairs (p, p + R / 2).  LANES: lanes of a unit where that is known (16
// and 8: dstate 128 and 64), so that the sums over them are straight code.
template <typename T, typename TG, bool Vec, bool Halves, int LANES, bool Bwd>
__global__ void __launch_bounds__(kThreads)
norm_rotate_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char smem[];
    float* table = reinterpret_cast<float*>(smem);     // (tile, 2, R / 2): cosines, sines
    Rows<T, Vec> xr(smem + a.table_bytes);
    Rows<TG, Vec> gr(smem + a.table_bytes + Rows<T, Vec>::kBytes);
    const int half = a.R / 2, rows = 2 * a.G, lanes = LANES > 0 ? LANES : a.lanes;
    const int units = kThreads / lanes;
    const int unit = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    // rows of a token a block walks at once, and the tokens side by side
    const int wide = rows < units ? rows : units, slots = units / wide;
    const int slot = unit / wide;
    const float inv_n = 1.f / (float)a.N;
    // the pair whose angles this thread computes, and the tokens it does so for
    int pairs = 1;
    while (pairs < half) pairs *= 2;
    const int pair = threadIdx.x % pairs, pair_from = threadIdx.x / pairs, pair_step = kThreads / pairs;
    const int64_t turn = pair < half ? turn_step(a.freq[pair]) : 0;

    // (elements that no pair turns follow the same order: lane_elements)
    int at[8];
    if constexpr (Vec) lane_elements(lane, a.N, a.R, !Halves, at);
    else lane_pairs(lane, a.N, a.R, !Halves, at);
    const bool on = Vec ? lane * 8 < a.N : true;    // spare lanes of a row hold zeros
    const bool turned = lane * 4 < half;            // Vec: all of the lane's pairs or none
    constexpr bool kHalves = Vec ? Halves : true;   // lane_pairs puts pair q at (q, 4 + q)

    for (int first = 0; first < rows; first += wide) {
        const int row = first + unit % wide;
        const bool mine = slot < slots && row < rows;
        const bool isB = row < a.G;
        const int g = isB ? row : row - a.G;
        F2 w2[4], dw2[4];
        {
            float w[8];
            const float* wp = (isB ? a.wB : a.wC) + (a.per_group ? (int64_t)g * a.N : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = mine && on && at[i] < a.N ? wp[at[i]] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w2[i] = pack2(w[2 * i], w[2 * i + 1]);
                dw2[i] = 0;
            }
        }
        for (int64_t tl = blockIdx.x; tl < a.ntile; tl += gridDim.x) {
            const int64_t bb = tl / a.tiles, t0 = (tl - bb * a.tiles) * a.tile;
            const int nt = (int)(a.L - t0 < a.tile ? a.L - t0 : a.tile);
            // this unit's rows of the tile, kAhead of them on their way
            const Stride st = isB ? a.bs : a.cs;
            const int64_t dense = ((bb * a.L + t0 + slot) * a.G + g) * a.N, step = (int64_t)slots * a.G * a.N;
            T* dst = static_cast<T*>(isB ? a.oB : a.oC) + dense;
            xr.start(static_cast<const T*>(isB ? a.B : a.C) + bb * st.batch + (t0 + slot) * st.token +
                     (int64_t)g * a.N, slots * st.token);
            if (Bwd) gr.start(static_cast<const TG*>(isB ? a.gB : a.gC) + dense, step);
            auto ask = [&](int i) {
                const bool exists = mine && on && slot + i * slots < nt;
                xr.ask(i, exists, at);
                if (Bwd) gr.ask(i, exists, at);
                copies_commit();
            };
            for (int i = 0; i < kAhead; ++i) ask(i);
            __syncthreads();                        // the last tile's readers are done
            for (int t = pair_from; t < nt; t += pair_step)
                if (pair < half) {
                    const float2 q = cos_sin(a.pos[bb * a.L + t0 + t], turn);
                    table[2 * t * half + pair] = q.x;
                    table[(2 * t + 1) * half + pair] = q.y;
                }
            if (turn == kNoStep)
                for (int t = pair_from; t < nt; t += pair_step)
                    table[2 * t * half + pair] = table[(2 * t + 1) * half + pair] = __int_as_float(0x7fffffff);
            __syncthreads();
            for (int i = 0; i * slots < nt; ++i) {               // uniform in a block
                const int t = slot + i * slots;
                const bool live = mine && on && t < nt;
                float v[8], d[8];
                copies_pending<kAhead - 1>();
                xr.take(i, live, at, a.N, v);
                if (Bwd) gr.take(i, live, at, a.N, d);
                ask(i + kAhead);
                F2 v2[4], sq2 = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v2[k] = pack2(v[2 * k], v[2 * k + 1]);
                    sq2 = fma2(v2[k], v2[k], sq2);
                }
                const float2 sq = unpack2(sq2);
                // (a place without a row has no norm: eps may be 0, and 1 / 0 times its
                // zeros would reach the weights' gradients)
                const float mean = unit_sum<LANES>(sq.x + sq.y, lanes) * inv_n;
                const float r = !Bwd || live ? rsqrtf(mean + a.eps) : 0.f;
                const F2 rr = pack2(r, r);
                auto turn_by = [&](float (&u)[8], float sign) {
                    if (!turned || !live) return;
                    float2 cs[4];
                    const float* tc = table + 2 * t * half + lane * 4;
                    if constexpr (Vec) {
                        const float4 c4 = *reinterpret_cast<const float4*>(tc);
                        const float4 s4 = *reinterpret_cast<const float4*>(tc + half);
                        cs[0] = make_float2(c4.x, s4.x); cs[1] = make_float2(c4.y, s4.y);
                        cs[2] = make_float2(c4.z, s4.z); cs[3] = make_float2(c4.w, s4.w);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            cs[q] = lane * 4 + q < half ? make_float2(tc[q], tc[q + half])
                                                        : make_float2(1.f, 0.f);
                    }
                    turn_pairs<kHalves>(u, cs, sign);
                };
                if constexpr (!Bwd) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 u = unpack2(mul2(mul2(v2[k], rr), w2[k]));
                        v[2 * k] = u.x;
                        v[2 * k + 1] = u.y;
                    }
                    turn_by(v, 1.f);
                    if (live) store8<T, Vec>(dst, at, a.N, v);
                } else {
                    turn_by(d, -1.f);
                    F2 dot2 = 0, d2[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        d2[k] = pack2(d[2 * k], d[2 * k + 1]);
                        dw2[k] = fma2(d2[k], mul2(v2[k], rr), dw2[k]);
                        d2[k] = mul2(d2[k], w2[k]);
                        dot2 = fma2(d2[k], v2[k], dot2);
                    }
                    const float2 dot = unpack2(dot2);
                    const float m = -unit_sum<LANES>(dot.x + dot.y, lanes) * inv_n * r * r;
                    const F2 mm = pack2(m, m);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 o = unpack2(mul2(rr, fma2(v2[k], mm, d2[k])));
                        d[2 * k] = o.x;
                        d[2 * k + 1] = o.y;
                    }
                    if (live) store8<T, Vec>(dst, at, a.N, d);
                }
                dst += step;
            }
        }
        if constexpr (Bwd) {
            // the block's partial sums: its slots' in order
            float* acc = reinterpret_cast<float*>(smem);         // (slots, wide, N)
            copies_pending<0>();
            __syncthreads();
            if (mine && on) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 q = unpack2(dw2[i / 2]);
                    if (at[i] < a.N) acc[(slot * wide + unit % wide) * a.N + at[i]] = i % 2 ? q.y : q.x;
                }
            }
            __syncthreads();
            for (int j = threadIdx.x; j < wide * a.N; j += kThreads) {
                if (first + j / a.N >= rows) break;
                float v = 0.f;
                for (int q = 0; q < slots; ++q) v += acc[q * wide * a.N + j];
                a.part[((int64_t)blockIdx.x * rows + first) * a.N + j] = v;
            }
            __syncthreads();                        // before the next rows' copies land there
        }
    }
}

// dweight: the blocks' partial rows (and, for weights that all groups share,
// the groups') added in a fixed order.  32 columns x 32 row groups a block;
// blockIdx.y: B or C.
__global__ void __launch_bounds__(1024)
norm_reduce_kernel(const float* __restrict__ part, int64_t blocks, int G, int N, int per_group,
                   float* __restrict__ dwB, float* __restrict__ dwC) {
    const int which = blockIdx.y;
    const int cols = per_group ? G * N : N;
    const int j = blockIdx.x * 32 + threadIdx.x;
    // eight rows in flight; the groups of one block's partial rows lie N apart
    const int64_t rows = per_group ? blocks : blocks * G;
    float v = 0.f;
    if (j < cols) {
        const float* p = part + (int64_t)which * G * N + j;
        if (per_group) {
#pragma unroll 8
            for (int b = threadIdx.y; b < (int)rows; b += 32) v += __ldg(p + (int64_t)b * 2 * G * N);
        } else {
#pragma unroll 8
            for (int r = threadIdx.y; r < (int)rows; r += 32)
                v += __ldg(p + (int64_t)(r / G) * 2 * G * N + (r % G) * N);
        }
    }
    __shared__ float red[32][33];
    red[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y || j >= cols) return;
#pragma unroll 8
    for (int q = 1; q < 32; ++q) v += red[q][threadIdx.x];
    (which ? dwC : dwB)[j] = v;
}

int lanes_of(int N) {
    int lanes = 1;
    while (lanes * 8 < N) lanes *= 2;
    return lanes;
}

// 592 blocks, four for each of 148 SMs, each with the same number of tiles of at most
// kMaxTile tokens.  (Of the gradients' kernels, with up to 110 registers and 63 KB or
// more for bf16 rows and fp32 gradients, two or three fit an SM at a time.)
constexpr int kMaxTile = 32;
int tile_of(const RotateDims& d) {
    const int64_t per = (d.b * d.L + 591) / 592;         // tokens of a block
    const int64_t tiles = (per + kMaxTile - 1) / kMaxTile;
    const int64_t tile = tiles > 0 ? (per + tiles - 1) / tiles : 1;
    return (int)(tile < d.L ? tile : (d.L > 0 ? d.L : 1));
}

int64_t blocks_of(const RotateDims& d) {
    const int64_t n = d.b * ((d.L + tile_of(d) - 1) / tile_of(d));
    return n < 592 ? n : 592;
}

// Sequences that lie behind one another as their tokens do are one long sequence,
// of which tiles then hold whole (single tokens of many sequences above all).
RotateDims joined(RotateArgs& r, const RotateDims& d) {
    if (d.L == 1) {
        r.bs.token = r.bs.batch;
        r.cs.token = r.cs.batch;
    } else if (r.bs.batch != d.L * r.bs.token || r.cs.batch != d.L * r.cs.token) {
        return d;
    }
    RotateDims j = d;
    j.b = 1;
    j.L = d.b * d.L;
    return j;
}

template <typename T>
bool vec_rows(const void* p, Stride s) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && s.batch % 4 == 0 &&
           s.token % 4 == 0;
}

Args args_of(const RotateArgs& r, const RotateDims& d) {
    Args a{};
    a.B = r.B; a.C = r.C; a.bs = r.bs; a.cs = r.cs; a.wB = r.wB; a.wC = r.wC;
    a.per_group = r.per_group; a.pos = r.pos; a.freq = r.freq; a.eps = r.eps;
    a.interleaved = r.interleaved;
    a.L = d.L; a.G = (int)d.G; a.N = (int)d.N; a.R = (int)d.R;
    a.lanes = lanes_of(a.N);
    a.tile = tile_of(d);
    a.tiles = (d.L + a.tile - 1) / a.tile;
    a.ntile = d.b * a.tiles;
    return a;
}

template <typename T, typename TG, bool Bwd, bool Vec>
cudaError_t launch(Args& a, int64_t blocks, cudaStream_t s) {
    const int units = kThreads / a.lanes, rows = 2 * a.G, wide = rows < units ? rows : units;
    a.table_bytes = (a.tile * (a.R / 2) * (int)sizeof(float2) + 15) / 16 * 16;
    int smem = a.table_bytes + Rows<T, Vec>::kBytes + (Bwd ? Rows<TG, Vec>::kBytes : 0);
    const int acc = units / wide * wide * a.N * 4;
    if (Bwd && smem < acc) smem = acc;
    // The limit that a kernel instance is given is the largest that any call of it
    // needs, the same every time: other host threads launch it too.  (A block's sums,
    // at most 2048 floats, are less than the table.)
    constexpr int most = kMaxTile * (256 / 2) * (int)sizeof(float2) + Rows<T, Vec>::kBytes +
                         (Bwd ? Rows<TG, Vec>::kBytes : 0);
    auto go = [&](auto kernel) {
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            if (e != cudaSuccess) return e;
        }
        kernel<<<(unsigned)blocks, kThreads, smem, s>>>(a);
        return cudaGetLastError();
    };
    if (Vec && a.lanes == 16)
        return a.interleaved ? go(norm_rotate_kernel<T, TG, Vec, false, Vec ? 16 : 0, Bwd>)
                             : go(norm_rotate_kernel<T, TG, Vec, true, Vec ? 16 : 0, Bwd>);
    if (Vec && a.lanes == 8)
        return a.interleaved ? go(norm_rotate_kernel<T, TG, Vec, false, Vec ? 8 : 0, Bwd>)
                             : go(norm_rotate_kernel<T, TG, Vec, true, Vec ? 8 : 0, Bwd>);
    return a.interleaved ? go(norm_rotate_kernel<T, TG, Vec, false, 0, Bwd>)
                         : go(norm_rotate_kernel<T, TG, Vec, true, 0, Bwd>);
}

template <typename T, typename TG, bool Bwd>
cudaError_t run(Args& a, int64_t blocks, cudaStream_t s) {
    const bool vec = a.N % 8 == 0 && a.R / 2 % 4 == 0 && vec_rows<T>(a.B, a.bs) &&
                     vec_rows<T>(a.C, a.cs);
    return vec ? launch<T, TG, Bwd, true>(a, blocks, s) : launch<T, TG, Bwd, false>(a, blocks, s);
}

}  // namespace

cudaError_t launch_norm_rotate_fwd(const RotateArgs& args, void* oB, void* oC,
                                   const RotateDims& dims, Elt t, cudaStream_t s) {
    RotateArgs r = args;
    const RotateDims d = joined(r, dims);
    Args a = args_of(r, d);
    a.oB = oB; a.oC = oC;
    return t == Elt::F32 ? run<float, float, false>(a, blocks_of(d), s)
                         : run<__nv_bfloat16, __nv_bfloat16, false>(a, blocks_of(d), s);
}

// Partial rows for the sequences by themselves or joined, whichever are more (the
// workspace does not depend on the strides).
size_t norm_rotate_bwd_workspace_bytes(const RotateDims& d) {
    const RotateDims j{1, d.b * d.L, d.G, d.N, d.R};
    const int64_t n = blocks_of(d) > blocks_of(j) ? blocks_of(d) : blocks_of(j);
    return (size_t)(n * 2 * d.G * d.N) * 4;
}

cudaError_t launch_norm_rotate_bwd(const RotateArgs& args, const void* gB, const void* gC,
                                   bool grad_f32, void* dB, void* dC, float* dwB, float* dwC,
                                   float* ws, const RotateDims& dims, Elt t, cudaStream_t s) {
    RotateArgs r = args;
    const RotateDims d = joined(r, dims);
    Args a = args_of(r, d);
    a.gB = gB; a.gC = gC; a.oB = dB; a.oC = dC; a.part = ws;
    const int64_t n = blocks_of(d);
    if (n > 0) {
        cudaError_t e = t == Elt::F32 ? run<float, float, true>(a, n, s)
                        : grad_f32    ? run<__nv_bfloat16, float, true>(a, n, s)
                                      : run<__nv_bfloat16, __nv_bfloat16, true>(a, n, s);
        if (e != cudaSuccess) return e;
    }
    const int cols = a.per_group ? a.G * a.N : a.N;
    norm_reduce_kernel<<<dim3((unsigned)((cols + 31) / 32), 2), dim3(32, 32), 0, s>>>(
        ws, n, a.G, a.N, a.per_group, dwB, dwC);
    return cudaGetLastError();
}

}  // namespace ssd
