// selective.cuh -- what the selective scan's kernels share: how channels and
// states lie over a warp's lanes, sums across lanes, and a tile's loads.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "layer_ops.h"
#include "vec_io.cuh"

namespace ssd {

// softplus(v) = max(v, 0) + log(1 + w), w = exp(-|v|) in (0, 1].  log(1 + w) =
// w P(w), P the degree-9 polynomial that interpolates log(1 + w) / w at the
// Chebyshev points of [0, 1]; the nearest singularity, w = -1, makes its error
// fall by 3 + sqrt(8) a degree, to 6e-9 relative, so that small steps (large
// negative v, where 1 + w would lose w) keep their accuracy but for the rounding
// of w's exponent, |v| 2^-24 relative.  One element at a time: the coefficients
// are then immediates and hold no registers.
__device__ __forceinline__ float softplus_f32(float v) {
    constexpr float kP[10] = {
        0.999999995f, -0.499998926f,
        0.333297105f, -0.249516163f,
        0.196632743f, -0.152696671f,
        0.105436238f, -0.0563736128f,
        0.0195425273f, -0.00317605702f,
    };
    const float w = ex2(-fabsf(v) * kLog2E);
    float p = kP[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) p = fmaf(p, w, kP[i]);
    return fmaf(w, p, fmaxf(v, 0.f));
}

// a = exp(dt A) = 2^(dl A), dl = dt log2(e).  ex2 comes out low: by 2e-8 of its value on
// average over the exponents of slowly decaying states, (-0.3, 0) (measured over
// 4 million of them; 3e-8 rms about that).  A state takes the product of as many
// factors as it remembers tokens, so that the shift would build up where the rest
// averages out; 2e-8 log2(e) added to the exponent takes it away, in the same
// instruction (the gradient of A over 2048 tokens: 1.9e-6 off without, 1.0e-6 with).  2^(the shift)
// alone is 1: a step of length zero leaves the state as it is.
constexpr float kDecayShift = 2.9e-8f;
// A parameter's A as the kernels hold it: -inf (a state that forgets at once) as the
// lowest finite value, whose product with the dt = 0 of rows behind a sequence is 0
// and not NaN, and with any dt above 1e-36 decays to 0 just the same.  NaN stays.
__device__ __forceinline__ float decay_rate(float A) { return A < -3.4028234e38f ? -3.4028234e38f : A; }
__device__ __forceinline__ float decay(float dl, float A) { return ex2(fmaf(dl, A, kDecayShift)); }
__device__ __forceinline__ F2 decay2(F2 dl, F2 A) {
    return ex2_2(fma2(dl, A, pack2(kDecayShift, kDecayShift)));
}
// What a span of tokens leaves of a state h that enters it, 2^e h (e = sum of dl A), and
// what it adds, S.  The factor goes in as two roots: a growth beyond fp32 (A > 0)
// takes a small state only as far as the tokens one by one would, and a decay
// below it a large one.  The roots stay finite (2^254 takes any normal number beyond
// fp32), so that zero stays zero.
__device__ __forceinline__ float over_span(float e, float h, float S) {
    const float root = ex2(fminf(0.5f * e, 127.f));
    return fmaf(root, root * h, S);
}

// Adds v[i] over LANES lanes that lie STRIDE apart, `lane` being this one's place
// among them, for all NV values at once: each step gives half of the values away and keeps the sums of the
// other half, so NV values cost NV - NV / LANES shuffles instead of
// NV * log2(LANES).  Lane l ends with values l * NV / LANES + i in v[i]
// (NV >= LANES), or with value l * NV / LANES in v[0] (NV < LANES).
template <int NV, int LANES, int STRIDE = 1>
__device__ __forceinline__ void fold(float* v, int lane) {
    int n = NV;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        if (n > 1) {
            n /= 2;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) {
                if (i < n) {
                    const float keep = up ? v[n + i] : v[i], give = up ? v[i] : v[n + i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * STRIDE);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STRIDE);
        }
    }
}

// Tokens whose states the backward holds in registers at once; the states before
// every kTS-th token are its checkpoints.
constexpr int kTS = 4;

// Layout of (channel, state) over a block of 128 threads: LPC lanes a channel,
// SPL neighbouring states a lane.  Few states a lane give more threads, many
// spare the work that every lane of a channel repeats (loads of dt and u, sums
// across lanes).
template <int SPL_, int LPC_>
struct Layout {
    static constexpr int SPL = SPL_, LPC = LPC_, NP = SPL_ * LPC_;   // NP: N rounded up
    static constexpr int CH = 128 / LPC_;                            // channels of a block
    static constexpr int TT = NP <= 64 ? 32 : (NP == 128 ? 16 : 8);  // tokens of a tile
};

inline int padded_states(int64_t N) {
    int n = 8;
    while (n < N) n *= 2;
    return n;
}

// Calls f with the layout for N states.
template <typename F>
void with_layout(int64_t N, F f) {
    switch (padded_states(N)) {
        case 8: f(Layout<4, 2>{}); break;
        case 16: f(Layout<4, 4>{}); break;
        case 32: f(Layout<8, 4>{}); break;
        case 64: f(Layout<8, 8>{}); break;
        case 128: f(Layout<8, 16>{}); break;
        default: f(Layout<8, 32>{}); break;
    }
}
template <typename T> struct TypeOf { using type = T; };
template <typename F>
void with_elt(Elt t, F f) {
    if (t == Elt::F32) f(TypeOf<float>{});
    else f(TypeOf<__nv_bfloat16>{});
}

// The block's place: 128 / LPC channels of one group, one sequence.
struct Place {
    int64_t b, c0;      // sequence, first channel
    int g, count;       // group, channels of the block that exist
};
template <int CH>
__device__ __forceinline__ Place place_of(int64_t index, const SelectiveDims& d) {
    const int64_t per = d.D / d.G, nb = (per + CH - 1) / CH;
    Place p;
    const int64_t k = index % nb, rest = index / nb;
    p.g = (int)(rest % d.G);
    p.b = rest / d.G;
    p.c0 = p.g * per + k * CH;
    const int64_t left = per - k * CH;
    p.count = left < CH ? (int)left : CH;
    return p;
}
template <int CH>
int64_t channel_blocks(const SelectiveDims& d) {
    return d.G * ((d.D / d.G + CH - 1) / CH);
}

// Where batch and channels are too few blocks, a sequence is cut into spans that
// run side by side; what each does to a state that enters it is in the workspace:
// state (b, spans - 1, D, NP), then sums of dt log2(e) (b, spans - 1, D).
struct Spans {
    int count;            // spans of a sequence
    int64_t tokens;       // tokens of a span, a multiple of the tile
    float *state, *sum;
};
Spans selective_spans(const SelectiveDims& d, Elt t, float* ws);

// VW neighbouring channels of one token: `n` of them exist; vec: one aligned
// load where all do.
template <typename T, int VW>
__device__ __forceinline__ Raw<T, VW> load_channels(const T* p, int n, bool vec) {
    if (vec && n >= VW) return raw_load<T, VW>(p);
    Raw<T, VW> r;
#pragma unroll
    for (int i = 0; i < VW; ++i) r.v[i] = i < n ? p[i] : from_f32<T>(0.f);
    return r;
}
template <typename T, int VW>
__device__ __forceinline__ void store_channels(T* p, const Raw<T, VW>& r, int n, bool vec) {
    if (vec && n >= VW) {
        raw_store<T, VW>(p, r);
    } else {
#pragma unroll
        for (int i = 0; i < VW; ++i)
            if (i < n) p[i] = r.v[i];
    }
}

// Whether all rows of a view can be read w elements at a time.
template <typename T>
bool rows_fit(const void* p, Stride s, int w) {
    return reinterpret_cast<uintptr_t>(p) % (w * sizeof(T)) == 0 && s.batch % w == 0 &&
           s.token % w == 0;
}

// Channels of one load: 16 bytes, or a block's channels where those are fewer.
template <typename T, int CH>
constexpr int load_width() {
    return CH < (int)(16 / sizeof(T)) ? CH : (int)(16 / sizeof(T));
}

}  // namespace ssd
