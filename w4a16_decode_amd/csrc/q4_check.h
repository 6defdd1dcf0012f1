// Argument checks and error reporting shared by the C ABI front ends (q4_api.cpp,
// q4_attn_api.cpp). Host code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/q4.h"

namespace q4 {

constexpr int64_t kMaxDim = int64_t(1) << 30;
// A launch has fewer than 2^32 threads: workgroups of 256 it may have.
constexpr int64_t kMaxGroups256 = (int64_t(1) << 24) - 1;

// Record the calling thread's last error and return its status; ok() clears it.
q4_status fail(q4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
q4_status ok();
q4_status hip_status(hipError_t e, const char* what);

// The checks of a product (q4_gemm, or with asym q4_gemm_asym) and, for B > 0, its
// arguments with the launch shape the library picks; the channel splits of that shape
// for valid sizes, else 0 (q4_api.cpp).
struct GemmArgs;
q4_status gemm_args(const void* x, int64_t B, const void* packed, const void* scales, const void* zeros, bool asym,
                    int64_t out, int64_t in, int32_t group, void* y, GemmArgs* a);
int gemm_splits(int64_t B, int64_t out, int64_t in, int32_t group, bool asym);

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace q4
