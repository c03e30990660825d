// Argument checks shared by the C-ABI front ends (api.hip, serving.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/q4gsw.h"

namespace q4gsw {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxM = int64_t(1) << 23;

inline int esize(int32_t dt) { return dt == Q4GSW_F32 ? 4 : 2; }
inline bool act_dtype_ok(int32_t dt) { return dt == Q4GSW_F32 || dt == Q4GSW_F16 || dt == Q4GSW_BF16; }
inline bool scale_dtype_ok(int32_t dt) { return dt == Q4GSW_F32 || dt == Q4GSW_F16; }
inline bool finite_f(double v) { return v == v && v - v == 0.0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};
inline Range range_of(const void* p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline q4gsw_status hip_status(hipError_t e) { return e == hipSuccess ? Q4GSW_OK : Q4GSW_E_HIP; }

inline bool ws_ok(const void* ws, uint64_t ws_bytes, uint64_t need) {
    return need == 0 || (ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}

}  // namespace q4gsw
