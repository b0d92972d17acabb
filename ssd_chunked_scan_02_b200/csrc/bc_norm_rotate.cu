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
// Far positions: pos * freq is wanted modulo 2 pi, where the product's integer
// part is useless.  freq / (2 pi) is taken as a 64-bit fixed-point fraction of
// a turn, and pos times it modulo 2^64 is one exact integer product: its error
// is pos * 2^-65 turns, and the error of freq / (2 pi) in fp64 (2^-53 of it)
// times pos.
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
    int64_t tiles, ntile;             // of a sequence, and of all
};

// The fraction of a turn that position `pos` makes at `step` = freq / (2 pi),
// as a signed 64-bit fixed-point number.
__device__ __forceinline__ int64_t turn_step(float freq) {
    const double turns = (double)freq * 0.15915494309189533577;
    const double frac = turns - rint(turns);                 // whole turns of one step drop out
    return __double2ll_rn(frac * 18446744073709551616.0);    // half a turn saturates: 2^-64 off
}

__device__ __forceinline__ float2 cos_sin(int64_t pos, int64_t step) {
    const int64_t turn = (int64_t)((uint64_t)pos * (uint64_t)step);
    // upper 32 bits, in half turns in [-1, 1)
    const float half = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;
    float2 q;
    sincospif(half, &q.y, &q.x);
    return q;
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

__device__ __forceinline__ float unit_sum(float v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row's eight elements of a lane as loaded.  Vec: the runs of four are whole,
// aligned loads; otherwise each element is loaded on its own where it exists.
template <typename T, bool Vec>
struct Row8 {
    Raw<T, 4> lo, hi;
    __device__ __forceinline__ void load(const T* row, const int (&at)[8], int N) {
        if constexpr (Vec) {
            lo = raw_load<T, 4>(row + at[0]);
            hi = raw_load<T, 4>(row + at[4]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo.v[i] = at[i] < N ? row[at[i]] : from_f32<T>(0.f);
                hi.v[i] = at[4 + i] < N ? row[at[4 + i]] : from_f32<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = to_f32(lo.v[i]);
            v[4 + i] = to_f32(hi.v[i]);
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

template <typename T, typename TG, bool Vec, bool Bwd>
__global__ void __launch_bounds__(kThreads)
norm_rotate_kernel(const Args a) {
    extern __shared__ float2 table[];               // (tile, R / 2): cosine, sine
    __shared__ int64_t steps[128];
    const int half = a.R / 2, rows = 2 * a.G;
    for (int k = threadIdx.x; k < half; k += kThreads) steps[k] = turn_step(a.freq[k]);
    const int units = kThreads / a.lanes;
    const int unit = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
    // rows of a token a block walks at once, and the tokens side by side
    const int wide = rows < units ? rows : units, slots = units / wide;
    const int slot = unit / wide;
    const float inv_n = 1.f / (float)a.N;

    // Vec: halves in lanes whose pairs are all turned, neighbours elsewhere
    int at[8];
    const bool halves = Vec ? (!a.interleaved && lane * 4 < half) : true;
    if constexpr (Vec) lane_elements(lane, a.N, a.R, a.interleaved, at);
    else lane_pairs(lane, a.N, a.R, a.interleaved, at);
    const bool on = Vec ? lane * 8 < a.N : true;    // spare lanes of a row hold zeros

    for (int first = 0; first < rows; first += wide) {
        const int row = first + unit % wide;
        const bool mine = slot < slots && row < rows;
        const bool isB = row < a.G;
        const int g = isB ? row : row - a.G;
        float w[8], dw[8];
        {
            const float* wp = (isB ? a.wB : a.wC) + (a.per_group ? (int64_t)g * a.N : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = mine && on && at[i] < a.N ? wp[at[i]] : 0.f;
                dw[i] = 0.f;
            }
        }
        for (int64_t tl = blockIdx.x; tl < a.ntile; tl += gridDim.x) {
            const int64_t bb = tl / a.tiles, t0 = (tl - bb * a.tiles) * a.tile;
            const int nt = (int)(a.L - t0 < a.tile ? a.L - t0 : a.tile);
            __syncthreads();                        // the last tile's readers are done
            for (int i = threadIdx.x; i < nt * half; i += kThreads) {
                const int t = i / half;
                table[i] = cos_sin(a.pos[bb * a.L + t0 + t], steps[i - t * half]);
            }
            // this unit's rows of the tile, the next one loaded a step ahead
            const Stride st = isB ? a.bs : a.cs;
            const T* src = static_cast<const T*>(isB ? a.B : a.C) + bb * st.batch +
                           (t0 + slot) * st.token + (int64_t)g * a.N;
            const int64_t dense = ((bb * a.L + t0 + slot) * a.G + g) * a.N, step = (int64_t)slots * a.G * a.N;
            T* dst = static_cast<T*>(isB ? a.oB : a.oC) + dense;
            const TG* grd = Bwd ? static_cast<const TG*>(isB ? a.gB : a.gC) + dense : nullptr;
            Row8<T, Vec> nv{};
            Row8<TG, Vec> nd{};
            if (mine && on && slot < nt) {
                nv.load(src, at, a.N);
                if (Bwd) nd.load(grd, at, a.N);
            }
            __syncthreads();
            for (int t = slot; t - slot < nt; t += slots) {      // uniform in a warp's units
                const bool live = mine && on && t < nt;
                float v[8], d[8];
                nv.get(v);
                if (Bwd) nd.get(d);
                src += slots * st.token;
                if (Bwd) grd += step;
                if (mine && on && t + slots < nt) {
                    nv.load(src, at, a.N);
                    if (Bwd) nd.load(grd, at, a.N);
                }
                float2 cs[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    cs[q] = live && lane * 4 + q < half ? table[t * half + lane * 4 + q]
                                                        : make_float2(1.f, 0.f);
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(v[i], v[i], sq);
                const float r = rsqrtf(unit_sum(sq, a.lanes) * inv_n + a.eps);
                if constexpr (!Bwd) {
                    float u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = v[i] * r * w[i];
                    if (halves) turn_pairs<true>(u, cs, 1.f);
                    else turn_pairs<false>(u, cs, 1.f);
                    if (live) store8<T, Vec>(dst, at, a.N, u);
                } else {
                    if (halves) turn_pairs<true>(d, cs, -1.f);
                    else turn_pairs<false>(d, cs, -1.f);
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (live) dw[i] = fmaf(d[i], v[i] * r, dw[i]);
                        d[i] *= w[i];
                        dot = fmaf(d[i], v[i], dot);
                    }
                    const float m = unit_sum(dot, a.lanes) * inv_n * r * r;
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = r * (d[i] - v[i] * m);
                    if (live) store8<T, Vec>(dst, at, a.N, d);
                }
                dst += step;
            }
        }
        if constexpr (Bwd) {
            // the block's partial sums: its slots' in order
            float* acc = reinterpret_cast<float*>(table);        // (slots, wide, N)
            __syncthreads();
            if (mine && on) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (at[i] < a.N) acc[(slot * wide + unit % wide) * a.N + at[i]] = dw[i];
            }
            __syncthreads();
            for (int j = threadIdx.x; j < wide * a.N; j += kThreads) {
                if (first + j / a.N >= rows) break;
                float v = 0.f;
                for (int q = 0; q < slots; ++q) v += acc[q * wide * a.N + j];
                a.part[((int64_t)blockIdx.x * rows + first) * a.N + j] = v;
            }
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
    const int64_t rows = per_group ? blocks : blocks * G;
    float v = 0.f;
    if (j < cols)
        for (int64_t r = threadIdx.y; r < rows; r += 32) {
            const int64_t block = per_group ? r : r / G;
            const int64_t off = per_group ? j : (r % G) * N + j;
            v += part[(block * 2 + which) * G * N + off];
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

// Tiles of 32 tokens, shorter where those are too few to give every SM four blocks.
int tile_of(const RotateDims& d) {
    int tile = 32;
    while (tile > 1 && d.b * ((d.L + tile - 1) / tile) < 592) tile /= 2;
    return tile;
}

int64_t blocks_of(const RotateDims& d) {
    const int64_t n = d.b * ((d.L + tile_of(d) - 1) / tile_of(d));
    return n < 592 ? n : 592;            // four blocks for each of 148 SMs
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

template <typename T, typename TG, bool Bwd>
cudaError_t run(const Args& a, int64_t nblocks, cudaStream_t s) {
    const int units = kThreads / a.lanes, rows = 2 * a.G, wide = rows < units ? rows : units;
    size_t smem = (size_t)a.tile * (a.R / 2) * sizeof(float2);
    if (Bwd) {
        const size_t acc = (size_t)(units / wide) * wide * a.N * 4;
        smem = smem > acc ? smem : acc;
    }
    const unsigned blocks = (unsigned)nblocks;
    const bool vec = a.N % 8 == 0 && a.R / 2 % 4 == 0 && vec_rows<T>(a.B, a.bs) &&
                     vec_rows<T>(a.C, a.cs);
    if (vec) norm_rotate_kernel<T, TG, true, Bwd><<<blocks, kThreads, smem, s>>>(a);
    else norm_rotate_kernel<T, TG, false, Bwd><<<blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
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
