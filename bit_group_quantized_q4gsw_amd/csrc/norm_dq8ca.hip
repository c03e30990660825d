// Residual addition, root-mean-square norm and per-row int8 codes in one pass over the row.
//
//   h = round(x + residual) in the residual's type,  t = h * weight (fp32),
//   codes and zero point of the row t as dq8ca_quantize defines them (every step in fp32),
//   row scale = step * fp32(1 / sqrt(mean(h^2) + eps)).
//
// The norm's factor is one positive number per row, so it does not change which code a value gets:
// it goes into the row's scale, and the row's range, the sum of squares and the codes all come
// from one read of x and the residual, the row staying in registers.  The sum of squares is held
// in 64 bits: the squares are exact there, and at one fma a value its cost is hidden behind the
// memory traffic.
//
// Codes leave in the row layout of the int8-activation GEMM (dq8ca.hip: k_pad long, octets in the
// order 0, 4, 1, 5, 2, 6, 3, 7, padding 0, minus the zero point), so linears of the same rows
// start at once; optionally the values scale * (code - zero) go out as fp32 too.
//
// Bound: HBM: 4096 rows of 8192, bf16, with h and values written, 369 MB in 82 us, 4.5 TB/s (a large
// copy: 4.72); 4 rows of 2048 take 3.1 us, two rounds of loads and one join.
#include "device.h"
#include "internal.h"

#include <float.h>

namespace q4gsw {
namespace {

constexpr int kOcts = 4;                 // octets a thread keeps
constexpr int kMaxThreads = 1024;

struct NormArgs {
    const void *x, *residual, *weight;   // residual may be null
    void* h;                             // may be null
    int8_t* q;
    float* scale;
    int32_t* nzp;
    float* values;                       // may be null
    int64_t K, ld;
    float eps;
};

// v as the type RT holds it, and back
template <int RT>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (RT == kF16) return (float)(_Float16)v;
    else if constexpr (RT == kBF16) return (float)(__bf16)v;
    else return v;
}

template <int RT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
    if constexpr (RT == kF16) static_cast<uint16_t*>(p)[i] = bitcast<uint16_t>((_Float16)v);
    else if constexpr (RT == kBF16) static_cast<uint16_t*>(p)[i] = bitcast<uint16_t>((__bf16)v);
    else static_cast<float*>(p)[i] = v;
}

template <int T>
__device__ __forceinline__ void load8(const void* x, int64_t e, float (&v)[8]) {
    if constexpr (T == kF32) {
        const f4 a = bitcast<f4>(ldg16(static_cast<const float*>(x) + e));
        const f4 b = bitcast<f4>(ldg16(static_cast<const float*>(x) + e + 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u4 a = ldg16(static_cast<const uint16_t*>(x) + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = T == kF16 ? f16_bits_to_f32((uint16_t)(a[i] & 0xFFFFu)) : bitcast<float>(a[i] << 16);
            v[2 * i + 1] = T == kF16 ? f16_bits_to_f32((uint16_t)(a[i] >> 16)) : bitcast<float>(a[i] & 0xFFFF0000u);
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t e, const float (&v)[8]) {
    if constexpr (T == kF32) {
        f4* d = reinterpret_cast<f4*>(static_cast<float*>(p) + e);
        d[0] = f4{v[0], v[1], v[2], v[3]};
        d[1] = f4{v[4], v[5], v[6], v[7]};
    } else {
        u4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == kF16) w[i] = bitcast<uint32_t>(h2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
            else w[i] = bitcast<uint32_t>(b2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
        }
        *reinterpret_cast<u4*>(static_cast<uint16_t*>(p) + e) = w;
    }
}

struct RowStats {
    float lo, hi;
    double ss;
    __device__ void add(float h, float t) {
        lo = t < lo ? t : lo;
        hi = t > hi ? t : hi;
        ss = fma((double)h, (double)h, ss);
    }
};

struct RowCodes {
    float inv, row;                      // row: the scale with the norm's factor
    int z;
    __device__ int operator()(float t) const {
        const int c = (int)rintf(t * inv) + z;
        return c < -128 ? -128 : (c > 127 ? 127 : c);
    }
};

__device__ __forceinline__ RowCodes row_codes(RowStats s, int64_t K, float eps) {
    __shared__ float s_lo[kMaxThreads / 64], s_hi[kMaxThreads / 64];
    __shared__ double s_ss[kMaxThreads / 64];
    const int tid = threadIdx.x;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float l2 = __shfl_xor(s.lo, off), h2_ = __shfl_xor(s.hi, off);
        s.lo = l2 < s.lo ? l2 : s.lo;
        s.hi = h2_ > s.hi ? h2_ : s.hi;
        s.ss += __shfl_xor(s.ss, off);
    }
    if ((tid & 63) == 0) {
        s_lo[tid >> 6] = s.lo;
        s_hi[tid >> 6] = s.hi;
        s_ss[tid >> 6] = s.ss;
    }
    __syncthreads();
    s.lo = s_lo[0];
    s.hi = s_hi[0];
    s.ss = s_ss[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) {
        s.lo = s_lo[w] < s.lo ? s_lo[w] : s.lo;
        s.hi = s_hi[w] > s.hi ? s_hi[w] : s.hi;
        s.ss += s_ss[w];
    }
    RowCodes r;
    float step = (s.hi - s.lo) / 255.0f;
    if (step < FLT_MIN) step = FLT_MIN;
    r.inv = 1.0f / step;
    const int z = -128 - (int)rintf(s.lo * r.inv);
    r.z = z < -128 ? -128 : (z > 127 ? 127 : z);
    r.row = (float)(1.0 / sqrt(s.ss / (double)K + (double)eps)) * step;
    return r;
}

// k-offset held by byte position p of a GEMM-layout octet
__device__ constexpr int kPerm[8] = {0, 4, 1, 5, 2, 6, 3, 7};

// One workgroup per row, the row in registers (K % 8 == 0, K <= 8 kOcts blockDim, every pointer
// 16-byte aligned).
template <int XT, int RT>
__global__ __launch_bounds__(kMaxThreads) void norm_dq8ca_kernel(NormArgs a) {
    const int64_t m = blockIdx.x, base = m * a.K, octs = a.K >> 3;
    const int tid = threadIdx.x, nt = blockDim.x;
    float t[kOcts][8];
    RowStats s{0.0f, 0.0f, 0.0};
#pragma unroll
    for (int i = 0; i < kOcts; ++i) {
        const int64_t o = tid + (int64_t)i * nt;
        if (o >= octs) break;
        float h[8], w[8];
        load8<XT>(a.x, base + 8 * o, h);
        if (a.residual) {
            float r[8];
            load8<RT>(a.residual, base + 8 * o, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] += r[e];
        }
        load8<RT>(a.weight, 8 * o, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = rounded<RT>(h[e]);
            t[i][e] = h[e] * w[e];
            s.add(h[e], t[i][e]);
        }
        if (a.h) store8<RT>(a.h, base + 8 * o, h);
    }
    const RowCodes rc = row_codes(s, a.K, a.eps);
#pragma unroll
    for (int i = 0; i < kOcts; ++i) {
        const int64_t o = tid + (int64_t)i * nt;
        if (o >= octs) break;
        int c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = rc(t[i][e]);
        uint32_t wd[2] = {0u, 0u};
#pragma unroll
        for (int p = 0; p < 8; ++p) wd[p >> 2] |= (uint32_t)(c[kPerm[p]] & 0xFF) << (8 * (p & 3));
        *reinterpret_cast<u2*>(a.q + m * a.ld + 8 * o) = u2{wd[0], wd[1]};
        if (a.values) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = rc.row * (float)(c[e] - rc.z);
            store8<kF32>(a.values, base + 8 * o, v);
        }
    }
    for (int64_t o = octs + tid; o < a.ld / 8; o += nt) *reinterpret_cast<u2*>(a.q + m * a.ld + 8 * o) = u2{0u, 0u};
    if (tid == 0) {
        a.scale[m] = rc.row;
        a.nzp[m] = -rc.z;
    }
}

// Any K and alignment: the row is read twice, element by element.
template <int XT, int RT>
__global__ __launch_bounds__(256) void norm_dq8ca_any_kernel(NormArgs a) {
    const int64_t m = blockIdx.x, base = m * a.K;
    const int tid = threadIdx.x;
    auto value = [&](int64_t k) {
        float h = load_elem<XT>(a.x, base + k);
        if (a.residual) h += load_elem<RT>(a.residual, base + k);
        return rounded<RT>(h);
    };
    RowStats s{0.0f, 0.0f, 0.0};
    for (int64_t k = tid; k < a.K; k += 256) {
        const float h = value(k);
        s.add(h, h * load_elem<RT>(a.weight, k));
    }
    const RowCodes rc = row_codes(s, a.K, a.eps);
    // an octet of codes a thread: its values, then its bytes in layout order
    for (int64_t o = tid; o < a.ld / 8; o += 256) {
        uint32_t wd[2] = {0u, 0u};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t k = 8 * o + kPerm[p];
            if (k >= a.K) continue;
            const float h = value(k);
            const int c = rc(h * load_elem<RT>(a.weight, k));
            wd[p >> 2] |= (uint32_t)(c & 0xFF) << (8 * (p & 3));
            if (a.h) store_elem<RT>(a.h, base + k, h);
            if (a.values) a.values[base + k] = rc.row * (float)(c - rc.z);
        }
        *reinterpret_cast<u2*>(a.q + m * a.ld + 8 * o) = u2{wd[0], wd[1]};
    }
    if (tid == 0) {
        a.scale[m] = rc.row;
        a.nzp[m] = -rc.z;
    }
}

template <int XT>
hipError_t norm_launch(const NormArgs& a, int r_dtype, int64_t M, hipStream_t s) {
    uintptr_t bits = 0;
    for (const void* p : {a.x, a.residual, a.weight, (const void*)a.h, (const void*)a.values}) bits |= reinterpret_cast<uintptr_t>(p);
    const int64_t octs = a.K >> 3;
    const unsigned nt = octs <= 256 * kOcts ? 256 : (octs <= 512 * kOcts ? 512 : 1024);
    // a grid takes fewer than 2^32 threads: millions of wide rows take 256 a row
    const bool vec = a.K % 8 == 0 && (bits & 15u) == 0 && octs <= (int64_t)kOcts * kMaxThreads && M * (int64_t)nt < (int64_t(1) << 32);
    const dim3 grid((unsigned)M), block(vec ? nt : 256u);
#define Q4GSW_NORM(RT)                                                                  \
    if (vec) hipLaunchKernelGGL((norm_dq8ca_kernel<XT, RT>), grid, block, 0, s, a);       \
    else hipLaunchKernelGGL((norm_dq8ca_any_kernel<XT, RT>), grid, block, 0, s, a);
    switch (r_dtype) {
        case kF32: Q4GSW_NORM(kF32) break;
        case kF16: Q4GSW_NORM(kF16) break;
        default: Q4GSW_NORM(kBF16) break;
    }
#undef Q4GSW_NORM
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_dq8ca(const void* x, int x_dtype, const void* residual, int r_dtype, const void* weight,
                                int64_t M, int64_t K, float eps, void* h, const Dq8caRows& rows, float* values,
                                hipStream_t s) {
    if (M > 0x7fffffff) return hipErrorInvalidConfiguration;
    const NormArgs a{x, residual, weight, h, rows.codes, rows.scale, rows.nzp, values, K, rows.ld, eps};
    switch (x_dtype) {
        case kF32: return norm_launch<kF32>(a, r_dtype, M, s);
        case kF16: return norm_launch<kF16>(a, r_dtype, M, s);
        default: return norm_launch<kBF16>(a, r_dtype, M, s);
    }
}

}  // namespace q4gsw
