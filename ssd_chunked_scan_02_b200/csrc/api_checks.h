// api_checks.h -- error reporting and argument checks shared by the C-ABI
// entry points (defined in ssd_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssd.h"

namespace ssd {

// Clears, or records, this host thread's message for ssd_last_error_detail().
void clear_error_detail();
void set_error_detail(const char* fmt, ...);
ssd_status_t fail(ssd_status_t s, const char* fmt, ...);
ssd_status_t cuda_fail(cudaError_t e, const char* where);

// A tensor handed to the kernels must be device memory of the current device:
// tensor maps, the status word and scratch are looked up per current device,
// and a kernel on one GPU given another GPU's (or unregistered host) memory
// faults or reads the wrong memory.  Checked once per call, after every other
// validation, on the call's main input.
ssd_status_t check_current_device(const void* p, const char* name);

inline bool aligned_to(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace ssd

#define REQUIRE_DEVICE(p)                                                                \
    do {                                                                                 \
        ssd_status_t st_dev_ = ssd::check_current_device((p), #p);                       \
        if (st_dev_ != SSD_OK) return st_dev_;                                           \
    } while (0)

#define REQUIRE_PTR(p)                                                                   \
    do {                                                                                 \
        if (!(p)) return ssd::fail(SSD_ERR_INVALID_ARG, "%s is NULL", #p);               \
        if (!ssd::aligned16(p))                                                          \
            return ssd::fail(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p);      \
    } while (0)
#define OPTIONAL_PTR(p)                                                                  \
    do {                                                                                 \
        if ((p) && !ssd::aligned16(p))                                                   \
            return ssd::fail(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p);      \
    } while (0)
