// layer_ops.h -- launchers of the operators around the SSD layer, shared
// between their C-ABI entry points (layer_api.cu) and their kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd_internal.h"

namespace ssd {

struct Stride {
    int64_t batch, token;    // elements
};

// ------------------------------------------------------------------ causal convolution
struct ConvDims {
    int64_t b, L, D;
    int W;                   // 2..4
};
cudaError_t launch_conv_fwd(const void* x, Stride xs, const float* w, const float* bias,
                            const void* init, const int32_t* lens, bool silu, void* y,
                            void* final_state, const ConvDims& d, Elt t, cudaStream_t s);
size_t conv_bwd_workspace_bytes(const ConvDims& d);
cudaError_t launch_conv_bwd(const void* x, Stride xs, const float* w, const float* bias,
                            const void* init, const int32_t* lens, bool silu, const void* dy,
                            bool dy_f32, const void* dfinal, void* dx, float* dw, float* dbias,
                            void* dinit, float* ws, const ConvDims& d, Elt t, cudaStream_t s);
cudaError_t launch_conv_step(void* state, const void* x, int64_t x_batch, const float* w,
                             const float* bias, bool silu, void* y, const ConvDims& d, Elt t,
                             cudaStream_t s);

// ------------------------------------------------------------------ selective scan
struct SelectiveDims {
    int64_t b, L, D, N, G;
};
struct SelectiveArgs {
    const void *x, *dt, *B, *C, *z;
    Stride xs, dts, Bs, Cs, zs;
    const float *A, *D, *dt_bias, *init;
    const int32_t* lens;
    bool softplus;
};
size_t selective_fwd_workspace_bytes(const SelectiveDims& d, Elt t);
cudaError_t launch_selective_fwd(const SelectiveArgs& a, void* y, float* final_states, float* ws,
                                 const SelectiveDims& d, Elt t, cudaStream_t s);
// The states before every kTS-th token, ckpt (b, ceil(L / TS), D, padded N) (ws: as
// the forward's).
cudaError_t launch_selective_checkpoints(const SelectiveArgs& a, float* ckpt, float* ws,
                                         const SelectiveDims& d, Elt t, cudaStream_t s);
struct SelectiveGrads {
    const void* dy;
    const float* dfinal;
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *ddt_bias, *dinit;
};
size_t selective_bwd_workspace_bytes(const SelectiveDims& d, Elt t);
cudaError_t launch_selective_bwd(const SelectiveArgs& a, const SelectiveGrads& g, float* ws,
                                 const SelectiveDims& d, Elt t, cudaStream_t s);
cudaError_t launch_selective_step(float* state, const SelectiveArgs& a, void* y,
                                  const SelectiveDims& d, Elt t, cudaStream_t s);

// ------------------------------------------------------------------ norm and rotation of B and C
struct RotateDims {
    int64_t b, L, G, N, R;
};
struct RotateArgs {
    const void *B, *C;
    Stride bs, cs;
    const float *wB, *wC;
    bool per_group;
    const int64_t* pos;
    const float* freq;
    float eps;
    bool interleaved;
};
cudaError_t launch_norm_rotate_fwd(const RotateArgs& r, void* oB, void* oC, const RotateDims& d,
                                   Elt t, cudaStream_t s);
size_t norm_rotate_bwd_workspace_bytes(const RotateDims& d);
cudaError_t launch_norm_rotate_bwd(const RotateArgs& r, const void* gB, const void* gC,
                                   bool grad_f32, void* dB, void* dC, float* dwB, float* dwC,
                                   float* ws, const RotateDims& d, Elt t, cudaStream_t s);

}  // namespace ssd
