// layer_api.cu -- C-ABI entry points of the operators around the SSD layer
// (include/ssd.h, "Operators around the layer"): host-side validation, then
// launches.  Nothing here allocates device memory or synchronises the device.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_checks.h"
#include "layer_ops.h"

namespace {

using ssd::cuda_fail;
using ssd::fail;

constexpr int64_t kMaxSize = 0x7fffffffLL;

ssd_status_t check_dtype(ssd_dtype_t dtype, ssd::Elt* t) {
    if (dtype != SSD_F32 && dtype != SSD_BF16)
        return fail(SSD_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    *t = dtype == SSD_F32 ? ssd::Elt::F32 : ssd::Elt::BF16;
    return SSD_OK;
}

// batch, seqlen >= 0 and every size below 2^31, so that their products fit 64 bits.
ssd_status_t check_tokens(int64_t batch, int64_t seqlen) {
    if (batch < 0 || seqlen < 0)
        return fail(SSD_ERR_INVALID_ARG, "batch (%lld) and seqlen (%lld) must be >= 0",
                    (long long)batch, (long long)seqlen);
    // (token indexes are 32 bits wide, with room for the tile behind the last token)
    if (batch > kMaxSize || seqlen > kMaxSize - 0xffff)
        return fail(SSD_ERR_UNSUPPORTED, "batch must be below 2^31 and seqlen below 2^31 - 2^16");
    return SSD_OK;
}

ssd_status_t conv_dims(const ssd_conv_dims_t* dims, ssd_dtype_t dtype, ssd::ConvDims* d,
                       ssd::Elt* t) {
    if (!dims) return fail(SSD_ERR_INVALID_ARG, "dims is NULL");
    ssd_status_t st = check_tokens(dims->batch, dims->seqlen);
    if (st != SSD_OK) return st;
    if (dims->channels < 1) return fail(SSD_ERR_INVALID_ARG, "channels must be >= 1");
    if (dims->width < 2 || dims->width > 4)
        return fail(SSD_ERR_UNSUPPORTED, "width must be in 2..4, got %lld",
                    (long long)dims->width);
    if (dims->channels > kMaxSize / 8)
        return fail(SSD_ERR_UNSUPPORTED, "channels must be below 2^28");
    // the finest split: a channel and 8 tokens a thread, 32 channels across a block
    // (the gradients' blocks; the forward's are 128 threads)
    if ((double)dims->batch * ((double)dims->seqlen / 8 + 1) * ((double)dims->channels / 32 + 1) >
        (double)kMaxSize)
        return fail(SSD_ERR_UNSUPPORTED, "batch * seqlen * channels exceeds the launch grid");
    *d = ssd::ConvDims{dims->batch, dims->seqlen, dims->channels, (int)dims->width};
    return check_dtype(dtype, t);
}

ssd_status_t selective_dims(const ssd_selective_dims_t* dims, ssd_dtype_t dtype,
                            ssd::SelectiveDims* d, ssd::Elt* t) {
    if (!dims) return fail(SSD_ERR_INVALID_ARG, "dims is NULL");
    ssd_status_t st = check_tokens(dims->batch, dims->seqlen);
    if (st != SSD_OK) return st;
    if (dims->channels < 1 || dims->dstate < 1 || dims->ngroups < 1)
        return fail(SSD_ERR_INVALID_ARG, "channels, dstate and ngroups must be >= 1");
    if (dims->channels % dims->ngroups != 0)
        return fail(SSD_ERR_INVALID_ARG, "channels (%lld) must be a multiple of ngroups (%lld)",
                    (long long)dims->channels, (long long)dims->ngroups);
    if (dims->dstate > 256) return fail(SSD_ERR_UNSUPPORTED, "dstate must be <= 256");
    if (dims->channels > kMaxSize)
        return fail(SSD_ERR_UNSUPPORTED, "channels must be below 2^31");
    // at most a block a channel and sequence
    if ((double)dims->batch * (double)dims->channels > (double)kMaxSize)
        return fail(SSD_ERR_UNSUPPORTED, "batch * channels exceeds the launch grid");
    *d = ssd::SelectiveDims{dims->batch, dims->seqlen, dims->channels, dims->dstate,
                            dims->ngroups};
    return check_dtype(dtype, t);
}

ssd_status_t rotate_dims(const ssd_rotate_dims_t* dims, ssd_dtype_t dtype, ssd::RotateDims* d,
                         ssd::Elt* t) {
    if (!dims) return fail(SSD_ERR_INVALID_ARG, "dims is NULL");
    ssd_status_t st = check_tokens(dims->batch, dims->seqlen);
    if (st != SSD_OK) return st;
    if (dims->ngroups < 1 || dims->dstate < 1)
        return fail(SSD_ERR_INVALID_ARG, "ngroups and dstate must be >= 1");
    if (dims->dstate > 256) return fail(SSD_ERR_UNSUPPORTED, "dstate must be <= 256");
    if (dims->ngroups > 65535) return fail(SSD_ERR_UNSUPPORTED, "ngroups must be <= 65535");
    if (dims->rotary < 0 || dims->rotary % 2 != 0 || dims->rotary > dims->dstate)
        return fail(SSD_ERR_INVALID_ARG, "rotary (%lld) must be even and in 0..dstate",
                    (long long)dims->rotary);
    *d = ssd::RotateDims{dims->batch, dims->seqlen, dims->ngroups, dims->dstate, dims->rotary};
    return check_dtype(dtype, t);
}

#define REQUIRE_STRIDE(p)                                                                \
    do {                                                                                 \
        if (!(p)) return fail(SSD_ERR_INVALID_ARG, "%s is NULL", #p);                    \
    } while (0)

// A view: any pointer aligned to its element.
ssd_status_t check_view(const void* p, const char* name, ssd::Elt t) {
    if (!p) return fail(SSD_ERR_INVALID_ARG, "%s is NULL", name);
    if (!ssd::aligned_to(p, t == ssd::Elt::F32 ? 4 : 2))
        return fail(SSD_ERR_INVALID_ARG, "%s is not aligned to its element", name);
    return SSD_OK;
}

#define REQUIRE_VIEW(p)                                                                  \
    do {                                                                                 \
        ssd_status_t st_view_ = check_view((p), #p, t);                                  \
        if (st_view_ != SSD_OK) return st_view_;                                         \
    } while (0)

#define REQUIRE_LENS(p)                                                                  \
    do {                                                                                 \
        if ((p) && !ssd::aligned_to((p), 4))                                             \
            return fail(SSD_ERR_INVALID_ARG, "%s is not aligned to its element", #p);    \
    } while (0)

ssd::Stride stride_of(const ssd_stride_t& s) { return ssd::Stride{s.batch, s.token}; }

// Tokens of a view lie less than 2^31 elements apart (kernels keep the distance
// in 32 bits), and not in descending order.
ssd_status_t check_stride(const ssd_stride_t& s, const char* name) {
    if (s.token < 0 || s.batch < 0)
        return fail(SSD_ERR_INVALID_ARG, "%s strides must be >= 0", name);
    if (s.token > kMaxSize)
        return fail(SSD_ERR_UNSUPPORTED, "%s token stride must be below 2^31", name);
    return SSD_OK;
}

// The step calls ignore the token strides.
#define CHECK_BATCH_STRIDE(s, name)                                                      \
    do {                                                                                 \
        if ((s).batch < 0)                                                               \
            return fail(SSD_ERR_INVALID_ARG, "%s strides must be >= 0", name);           \
    } while (0)

#define CHECK_STRIDE(s, name)                                                            \
    do {                                                                                 \
        ssd_status_t st_stride_ = check_stride((s), name);                               \
        if (st_stride_ != SSD_OK) return st_stride_;                                     \
    } while (0)

}  // namespace

extern "C" {

// ---------------------------------------------------------------- causal convolution
ssd_status_t ssd_causal_conv_fwd(const void* x, const ssd_stride_t* x_stride,
                                 const float* weight, const float* bias, const void* init_state,
                                 const int32_t* seq_lens, int silu, void* y, void* final_state,
                                 const ssd_conv_dims_t* dims, ssd_dtype_t dtype, void* stream) {
    ssd::clear_error_detail();
    ssd::ConvDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = conv_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(bias); OPTIONAL_PTR(init_state); OPTIONAL_PTR(final_state);
    REQUIRE_LENS(seq_lens);
    REQUIRE_STRIDE(x_stride);
    CHECK_STRIDE(*x_stride, "x");
    if (d.b == 0 || (d.L == 0 && !final_state)) return SSD_OK;
    REQUIRE_PTR(weight);
    if (d.L > 0) {
        REQUIRE_VIEW(x);
        REQUIRE_PTR(y);
    }
    REQUIRE_DEVICE(weight);
    cudaError_t e = ssd::launch_conv_fwd(x, stride_of(*x_stride), weight, bias, init_state,
                                         seq_lens, silu != 0, y, final_state, d, t,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "convolution kernel");
}

ssd_status_t ssd_causal_conv_bwd_workspace_size(const ssd_conv_dims_t* dims, ssd_dtype_t dtype,
                                                size_t* bytes) {
    ssd::clear_error_detail();
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::ConvDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = conv_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    *bytes = ssd::conv_bwd_workspace_bytes(d);
    return SSD_OK;
}

ssd_status_t ssd_causal_conv_bwd(const void* x, const ssd_stride_t* x_stride,
                                 const float* weight, const float* bias, const void* init_state,
                                 const int32_t* seq_lens, int silu, const void* dy, int dy_f32,
                                 const void* dfinal_state, void* dx, float* dweight,
                                 float* dbias, void* dinit_state, const ssd_conv_dims_t* dims,
                                 ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    ssd::clear_error_detail();
    ssd::ConvDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = conv_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(bias); OPTIONAL_PTR(init_state); OPTIONAL_PTR(dfinal_state);
    OPTIONAL_PTR(dinit_state);
    REQUIRE_LENS(seq_lens);
    REQUIRE_STRIDE(x_stride);
    CHECK_STRIDE(*x_stride, "x");
    REQUIRE_PTR(weight); REQUIRE_PTR(dweight); REQUIRE_PTR(dbias);
    if (d.b > 0 && d.L > 0) {
        REQUIRE_VIEW(x);
        REQUIRE_PTR(dy);
        REQUIRE_PTR(dx);
    }
    const size_t need = ssd::conv_bwd_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(SSD_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed",
                    workspace_bytes, need);
    if (need > 0) REQUIRE_PTR(workspace);
    REQUIRE_DEVICE(weight);
    cudaError_t e = ssd::launch_conv_bwd(x, stride_of(*x_stride), weight, bias, init_state,
                                         seq_lens, silu != 0, dy, dy_f32 != 0, dfinal_state, dx,
                                         dweight, dbias, dinit_state,
                                         static_cast<float*>(workspace), d, t,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "convolution gradient kernels");
}

ssd_status_t ssd_causal_conv_step(void* state, const void* x, const ssd_stride_t* x_stride,
                                  const float* weight, const float* bias, int silu, void* y,
                                  const ssd_conv_dims_t* dims, ssd_dtype_t dtype, void* stream) {
    ssd::clear_error_detail();
    ssd::ConvDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_conv_dims_t one{};
    if (dims) one = *dims;
    one.seqlen = 1;
    ssd_status_t st = conv_dims(dims ? &one : nullptr, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(bias);
    REQUIRE_STRIDE(x_stride);
    CHECK_BATCH_STRIDE(*x_stride, "x");
    if (d.b == 0) return SSD_OK;
    REQUIRE_PTR(state); REQUIRE_PTR(weight); REQUIRE_PTR(y);
    REQUIRE_VIEW(x);
    REQUIRE_DEVICE(state);
    cudaError_t e = ssd::launch_conv_step(state, x, x_stride->batch, weight, bias, silu != 0, y,
                                          d, t, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "convolution step kernel");
}

// ---------------------------------------------------------------- selective scan
namespace {
ssd::SelectiveArgs selective_args(const void* x, const void* dt, const float* A, const void* B,
                                  const void* C, const float* D, const void* z,
                                  const float* dt_bias, int softplus, const float* init,
                                  const int32_t* lens, const ssd_selective_strides_t& st) {
    return ssd::SelectiveArgs{x, dt, B, C, z, stride_of(st.x), stride_of(st.dt),
                              stride_of(st.B), stride_of(st.C), stride_of(st.z), A, D, dt_bias,
                              init, lens, softplus != 0};
}
}  // namespace

ssd_status_t ssd_selective_scan_fwd_workspace_size(const ssd_selective_dims_t* dims,
                                                   ssd_dtype_t dtype, size_t* bytes) {
    ssd::clear_error_detail();
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::SelectiveDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = selective_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    *bytes = ssd::selective_fwd_workspace_bytes(d, t);
    return SSD_OK;
}

ssd_status_t ssd_selective_scan_fwd(const void* x, const void* dt, const float* A, const void* B,
                                    const void* C, const float* D, const void* z,
                                    const float* dt_bias, int softplus,
                                    const float* init_states, const int32_t* seq_lens, void* y,
                                    float* final_states, const ssd_selective_strides_t* strides,
                                    const ssd_selective_dims_t* dims, ssd_dtype_t dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    ssd::clear_error_detail();
    ssd::SelectiveDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = selective_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(D); OPTIONAL_PTR(dt_bias); OPTIONAL_PTR(init_states); OPTIONAL_PTR(final_states);
    REQUIRE_LENS(seq_lens);
    REQUIRE_STRIDE(strides);
    CHECK_STRIDE(strides->x, "x"); CHECK_STRIDE(strides->dt, "dt");
    CHECK_STRIDE(strides->B, "B"); CHECK_STRIDE(strides->C, "C");
    if (z) CHECK_STRIDE(strides->z, "z");
    if (d.b == 0 || (d.L == 0 && !final_states)) return SSD_OK;
    REQUIRE_PTR(A);
    if (d.L > 0) {
        REQUIRE_VIEW(x); REQUIRE_VIEW(dt); REQUIRE_VIEW(B); REQUIRE_VIEW(C);
        if (z) REQUIRE_VIEW(z);
        REQUIRE_PTR(y);
    }
    const size_t need = ssd::selective_fwd_workspace_bytes(d, t);
    if (workspace_bytes < need)
        return fail(SSD_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed",
                    workspace_bytes, need);
    if (need > 0) REQUIRE_PTR(workspace);
    REQUIRE_DEVICE(A);
    cudaError_t e = ssd::launch_selective_fwd(
        selective_args(x, dt, A, B, C, D, z, dt_bias, softplus, init_states, seq_lens, *strides),
        y, final_states, static_cast<float*>(workspace), d, t, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "selective scan kernels");
}

ssd_status_t ssd_selective_scan_bwd_workspace_size(const ssd_selective_dims_t* dims,
                                                   ssd_dtype_t dtype, size_t* bytes) {
    ssd::clear_error_detail();
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::SelectiveDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = selective_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    *bytes = ssd::selective_bwd_workspace_bytes(d, t);
    return SSD_OK;
}

ssd_status_t ssd_selective_scan_bwd(const void* x, const void* dt, const float* A, const void* B,
                                    const void* C, const float* D, const void* z,
                                    const float* dt_bias, int softplus,
                                    const float* init_states, const int32_t* seq_lens,
                                    const void* dy, const float* dfinal_states, void* dx,
                                    void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz,
                                    float* ddt_bias, float* dinit_states,
                                    const ssd_selective_strides_t* strides,
                                    const ssd_selective_dims_t* dims, ssd_dtype_t dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    ssd::clear_error_detail();
    ssd::SelectiveDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = selective_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(D); OPTIONAL_PTR(dt_bias); OPTIONAL_PTR(init_states);
    OPTIONAL_PTR(dfinal_states); OPTIONAL_PTR(dD); OPTIONAL_PTR(ddt_bias);
    OPTIONAL_PTR(dinit_states);
    REQUIRE_LENS(seq_lens);
    REQUIRE_STRIDE(strides);
    CHECK_STRIDE(strides->x, "x"); CHECK_STRIDE(strides->dt, "dt");
    CHECK_STRIDE(strides->B, "B"); CHECK_STRIDE(strides->C, "C");
    if (z) CHECK_STRIDE(strides->z, "z");
    REQUIRE_PTR(A); REQUIRE_PTR(dA);
    if (d.b > 0 && d.L > 0) {
        REQUIRE_VIEW(x); REQUIRE_VIEW(dt); REQUIRE_VIEW(B); REQUIRE_VIEW(C);
        REQUIRE_PTR(dy); REQUIRE_PTR(dx); REQUIRE_PTR(ddt); REQUIRE_PTR(dB); REQUIRE_PTR(dC);
        if (z) { REQUIRE_VIEW(z); REQUIRE_PTR(dz); }
    }
    const size_t need = ssd::selective_bwd_workspace_bytes(d, t);
    if (workspace_bytes < need)
        return fail(SSD_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed",
                    workspace_bytes, need);
    if (need > 0) REQUIRE_PTR(workspace);
    REQUIRE_DEVICE(A);
    const ssd::SelectiveGrads g{dy, dfinal_states, dx, ddt, dB, dC, dz,
                                dA, dD, ddt_bias, dinit_states};
    cudaError_t e = ssd::launch_selective_bwd(
        selective_args(x, dt, A, B, C, D, z, dt_bias, softplus, init_states, seq_lens, *strides),
        g, static_cast<float*>(workspace), d, t, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "selective scan gradient kernels");
}

ssd_status_t ssd_selective_step(float* state, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z,
                                const float* dt_bias, int softplus, void* y,
                                const ssd_selective_strides_t* strides,
                                const ssd_selective_dims_t* dims, ssd_dtype_t dtype,
                                void* stream) {
    ssd::clear_error_detail();
    ssd::SelectiveDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_selective_dims_t one{};
    if (dims) one = *dims;
    one.seqlen = 1;
    ssd_status_t st = selective_dims(dims ? &one : nullptr, dtype, &d, &t);
    if (st != SSD_OK) return st;
    OPTIONAL_PTR(D); OPTIONAL_PTR(dt_bias);
    REQUIRE_STRIDE(strides);
    CHECK_BATCH_STRIDE(strides->x, "x"); CHECK_BATCH_STRIDE(strides->dt, "dt");
    CHECK_BATCH_STRIDE(strides->B, "B"); CHECK_BATCH_STRIDE(strides->C, "C");
    if (z) CHECK_BATCH_STRIDE(strides->z, "z");
    if (d.b == 0) return SSD_OK;
    REQUIRE_PTR(state); REQUIRE_PTR(A); REQUIRE_PTR(y);
    REQUIRE_VIEW(x); REQUIRE_VIEW(dt); REQUIRE_VIEW(B); REQUIRE_VIEW(C);
    if (z) REQUIRE_VIEW(z);
    REQUIRE_DEVICE(state);
    cudaError_t e = ssd::launch_selective_step(
        state, selective_args(x, dt, A, B, C, D, z, dt_bias, softplus, nullptr, nullptr, *strides),
        y, d, t, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "selective step kernel");
}

// ---------------------------------------------------------------- norm and rotation of B and C
ssd_status_t ssd_bc_norm_rotate_fwd(const void* B, const ssd_stride_t* B_stride, const void* C,
                                    const ssd_stride_t* C_stride, const float* B_weight,
                                    const float* C_weight, int weight_per_group,
                                    const int64_t* positions, const float* freq, float eps,
                                    int interleaved, void* B_out, void* C_out,
                                    const ssd_rotate_dims_t* dims, ssd_dtype_t dtype,
                                    void* stream) {
    ssd::clear_error_detail();
    ssd::RotateDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = rotate_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    if (!(eps >= 0.f)) return fail(SSD_ERR_INVALID_ARG, "eps must be >= 0");
    REQUIRE_STRIDE(B_stride); REQUIRE_STRIDE(C_stride);
    CHECK_STRIDE(*B_stride, "B"); CHECK_STRIDE(*C_stride, "C");
    if (d.b == 0 || d.L == 0) return SSD_OK;
    REQUIRE_VIEW(B); REQUIRE_VIEW(C);
    REQUIRE_PTR(B_weight); REQUIRE_PTR(C_weight); REQUIRE_PTR(B_out); REQUIRE_PTR(C_out);
    if (d.R > 0) { REQUIRE_PTR(positions); REQUIRE_PTR(freq); }
    REQUIRE_DEVICE(B);
    const ssd::RotateArgs r{B, C, stride_of(*B_stride), stride_of(*C_stride), B_weight, C_weight,
                            weight_per_group != 0, positions, freq, eps, interleaved != 0};
    cudaError_t e = ssd::launch_norm_rotate_fwd(r, B_out, C_out, d, t,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "norm and rotation kernel");
}

ssd_status_t ssd_bc_norm_rotate_bwd_workspace_size(const ssd_rotate_dims_t* dims,
                                                   ssd_dtype_t dtype, size_t* bytes) {
    ssd::clear_error_detail();
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::RotateDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = rotate_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    *bytes = ssd::norm_rotate_bwd_workspace_bytes(d);
    return SSD_OK;
}

ssd_status_t ssd_bc_norm_rotate_bwd(const void* B, const ssd_stride_t* B_stride, const void* C,
                                    const ssd_stride_t* C_stride, const float* B_weight,
                                    const float* C_weight, int weight_per_group,
                                    const int64_t* positions, const float* freq, float eps,
                                    int interleaved, const void* dB_out, const void* dC_out,
                                    int grad_f32, void* dB, void* dC, float* dB_weight,
                                    float* dC_weight, const ssd_rotate_dims_t* dims,
                                    ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    ssd::clear_error_detail();
    ssd::RotateDims d{}; ssd::Elt t = ssd::Elt::BF16;
    ssd_status_t st = rotate_dims(dims, dtype, &d, &t);
    if (st != SSD_OK) return st;
    if (!(eps >= 0.f)) return fail(SSD_ERR_INVALID_ARG, "eps must be >= 0");
    REQUIRE_STRIDE(B_stride); REQUIRE_STRIDE(C_stride);
    CHECK_STRIDE(*B_stride, "B"); CHECK_STRIDE(*C_stride, "C");
    REQUIRE_PTR(B_weight); REQUIRE_PTR(C_weight);
    REQUIRE_PTR(dB_weight); REQUIRE_PTR(dC_weight);
    if (d.b > 0 && d.L > 0) {
        REQUIRE_VIEW(B); REQUIRE_VIEW(C);
        REQUIRE_PTR(dB_out); REQUIRE_PTR(dC_out); REQUIRE_PTR(dB); REQUIRE_PTR(dC);
        if (d.R > 0) { REQUIRE_PTR(positions); REQUIRE_PTR(freq); }
    }
    const size_t need = ssd::norm_rotate_bwd_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(SSD_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed",
                    workspace_bytes, need);
    if (need > 0) REQUIRE_PTR(workspace);
    REQUIRE_DEVICE(B_weight);
    const ssd::RotateArgs r{B, C, stride_of(*B_stride), stride_of(*C_stride), B_weight, C_weight,
                            weight_per_group != 0, positions, freq, eps, interleaved != 0};
    cudaError_t e = ssd::launch_norm_rotate_bwd(r, dB_out, dC_out, grad_f32 != 0, dB, dC,
                                                dB_weight, dC_weight,
                                                static_cast<float*>(workspace), d, t,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "norm and rotation gradient kernels");
}

}  // extern "C"
