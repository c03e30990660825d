// Shared by the attention kernels over the 4-bit cache (kv_rows.hip, kv_prompt.hip).
#pragma once
#include "kv4.h"

namespace q4gsw {

struct KvAttnArgs {
    KvView c;
    KvSeqs sq;
    const void* q;           // token rows of q_ld elements, [hq][dim] dense, of dtype
    int64_t q_ld;
    int dtype;
    void* out;               // [tokens][hq][dim] of dtype (one split)
    float* part;             // more: [split][tokens][hq][dim] sums, not divided by the weights' sum
    float* ml;               //       [split][tokens][hq] pairs (reference exponent, weights' sum)
    int hq, group;           // query heads; of them per head of the cache
    int max_new;             // rows of later new tokens are not computed
    int window;              // 0: none
    float cap_in, cap_out;   // 1 / cap and cap log2(e); 0: no cap
    float scale;             // dim^-1/2
    int splits, chunk;       // blocks of 32 tokens per split (the last split takes the rest)
    int row_tiles;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoKey = -3.0e38f;   // reference exponent of a row that has seen no key
// Weights are 2^(score - reference + kLift): the reference moves only when a score passes it by
// more than kSlack, so a weight is at most 2^(kLift + kSlack) = 2^14, a finite fp16, and the
// largest weight of a row is at least 2^kLift, 2^30 times fp16's smallest step.
constexpr float kLift = 6.0f, kSlack = 8.0f;

// The last place that the window of the row at `place` has left behind; -1: none (no window, or a row
// nearer to the start than the window is long; places may be negative and windows as long as an
// int: their difference may not fit one).
__device__ __forceinline__ int kv_left_behind(const KvAttnArgs& a, int place) {
    return a.window && place >= a.window ? place - a.window : -1;
}

// What the rows [r0, r0 + nr) of one (sequence, cache head) see: row r is new token r / group,
// query head r % group; its place is p0 + r / group.
struct KvSpan {
    int pmin, pmax;          // places of the first and last row
    int64_t lo, hi;          // 32-token blocks [lo, hi) of this split
};
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs& a, const KvSeq& s, int r0, int nr, int split) {
    KvSpan r;
    const int p0 = s.len - s.m;
    r.pmin = p0 + r0 / a.group;
    r.pmax = p0 + (r0 + nr - 1) / a.group;
    int64_t first = a.window ? (int64_t)r.pmin - a.window + 1 : 0;
    first = first < 0 ? 0 : first;
    int64_t end = r.pmax < 0 ? 0 : (r.pmax >> 5) + 1;
    const int64_t room = (int64_t)a.sq.table_cols << a.c.bpp_log2;
    end = end < room ? end : room;
    r.lo = (first >> 5) + (int64_t)split * a.chunk;
    r.hi = split == a.splits - 1 ? end : (r.lo + a.chunk < end ? r.lo + a.chunk : end);
    return r;
}

// Factor 2^(14 - e), e the exponent of a row's largest magnitude, that brings the row into fp16's
// range (every bf16 or fp16 value of it down to 2^-19 of the largest stays exact; fp32 values
// round to 11 bits), and its inverse.  A zero row gets any factor; NaN stay, and an infinity makes the
// whole row NaN: its scores would be infinite or NaN, and where all that a row sees are -inf the weights
// would add up to 0, as if it saw no key.
__device__ __forceinline__ void row_factor(float amax, float& mul, float& inv) {
    int eb = (int)(bitcast<uint32_t>(amax) >> 23) & 0xFF;
    eb = eb < 15 ? 15 : eb;
    mul = eb == 255 ? __builtin_nanf("") : bitcast<float>((uint32_t)(268 - eb > 254 ? 254 : 268 - eb) << 23);
    inv = bitcast<float>((uint32_t)(eb - 14) << 23);
}

// cap * tanh(x / cap) * log2(e), with in = 1 / cap and out = cap log2(e).  tanh z = 1 - 2 / (1 + e^2z)
// is off by a few 2^-24 absolute, so below 1/8 its series takes over (next term 2^-24 relative).
__device__ __forceinline__ float capped_log2(float x, float in, float out) {
    const float z = x * in;
    const float big = fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * (2.0f * kLog2e))), 1.0f);
    const float z2 = z * z;
    const float small = fmaf(z * z2, fmaf(z2, fmaf(z2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), z);
    return out * (fabsf(z) < 0.125f ? small : big);
}

// Maximum of v over lanes l, l ^ 16, l ^ 32, l ^ 48, in every lane (NaN counts as nothing).
__device__ __forceinline__ float wave_max_rows(float v) {
    const uint32_t a = bitcast<uint32_t>(v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const float s = fmaxf(bitcast<float>(r[0]), bitcast<float>(r[1]));
    const uint32_t b = bitcast<uint32_t>(s);
    const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(bitcast<float>(h[0]), bitcast<float>(h[1]));
}

// Four neighbouring channels of an output row.
__device__ __forceinline__ void store4(void* out, int dtype, int64_t e, f4 v) {
    if (dtype == kF32) {
        *reinterpret_cast<f4*>(static_cast<float*>(out) + e) = v;
    } else if (dtype == kF16) {
        const h2 a = {(_Float16)v[0], (_Float16)v[1]}, b = {(_Float16)v[2], (_Float16)v[3]};
        *reinterpret_cast<u2*>(static_cast<uint16_t*>(out) + e) = u2{bitcast<uint32_t>(a), bitcast<uint32_t>(b)};
    } else {
        const b2 a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
        *reinterpret_cast<u2*>(static_cast<uint16_t*>(out) + e) = u2{bitcast<uint32_t>(a), bitcast<uint32_t>(b)};
    }
}

// A lane's part of a query row: octets at e0 + stride * i, i < N, 16-byte aligned.  load issues all
// of its loads together; convert makes operand fragments of them: the row's largest magnitude is
// joined over the lanes that share the row by `join`, and fp16 pairs times 2^k go to frag (zeros
// where ok is false).  Returns the factor back, 2^-k.
template <int N>
struct QueryRow {
    u4 raw[2 * N];                       // 16-bit types use the first N

    __device__ __forceinline__ void load(const void* q, int dtype, int64_t e0, int stride) {
        if (dtype == kF32) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                raw[2 * i] = ldg16(static_cast<const float*>(q) + e0 + stride * i);
                raw[2 * i + 1] = ldg16(static_cast<const float*>(q) + e0 + stride * i + 4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) raw[i] = ldg16(static_cast<const uint16_t*>(q) + e0 + stride * i);
        }
    }

    template <int DT, class Join>
    __device__ __forceinline__ float convert(bool ok, Join join, u4 (&frag)[N]) const {
        auto value = [&](int i, int e) -> float {            // element e (0..7) of octet i
            if constexpr (DT == kF32) return bitcast<float>(raw[i * 2 + (e >> 2)][e & 3]);
            else if constexpr (DT == kF16) return (float)bitcast<h2>(raw[i][e >> 1])[e & 1];
            else return bitcast<float>((e & 1) ? raw[i][e >> 1] & 0xFFFF0000u : raw[i][e >> 1] << 16);
        };
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(value(i, e)));
        }
        float mul, inv;
        amax = join(amax);
        row_factor(ok ? amax : 0.0f, mul, inv);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const h2 p = {(_Float16)(value(i, 2 * e) * mul), (_Float16)(value(i, 2 * e + 1) * mul)};
                frag[i][e] = ok ? bitcast<uint32_t>(p) : 0u;
            }
        }
        return inv;
    }

    template <class Join>
    __device__ __forceinline__ float convert(int dtype, bool ok, Join join, u4 (&frag)[N]) const {
        if (dtype == kF32) return convert<kF32>(ok, join, frag);
        if (dtype == kF16) return convert<kF16>(ok, join, frag);
        return convert<kBF16>(ok, join, frag);
    }
};

// Waves a SIMD holds of the kernel of few rows: what its registers allow (89, 122, 148, 202 and 256
// for 64 .. 256 channels: sums D / 4, queries D / 8).
constexpr int kv_rows_waves(int D) { return D == 64 ? 4 : (D <= 128 ? 3 : 2); }

// The kernel of many rows: blocks of 32 tokens in a tile (two, but one where two with the remainders
// that `prec` keeps do not fit LDS twice), bytes of its two stages of keys and values, and how many of
// its workgroups of `waves` a CU of 160 KB holds: registers allow two waves a SIMD up to 128 channels and one
// above.
constexpr int prompt_blocks(int D, bool prec) { return prec && D > 128 ? 1 : 2; }
constexpr int prompt_lds(int D, bool prec) { return 2 * prompt_blocks(D, prec) * (D / 16) * 1024 * (prec ? 4 : 2); }
constexpr int prompt_fit(int D, bool prec, int waves) {
    const int by_regs = (D <= 128 ? 8 : 4) / waves, by_lds = 160 * 1024 / prompt_lds(D, prec);
    return by_regs < by_lds ? by_regs : by_lds;
}

// kv_rows.hip: `waves` (4 or 8) per workgroup, tiles of 16 rows.
hipError_t launch_kv_rows(const KvAttnArgs& a, int waves, hipStream_t s);
// kv_prompt.hip: 32 rows a wave, `waves` 4, or 8 up to 128 channels; a.chunk even.
hipError_t launch_kv_prompt(const KvAttnArgs& a, int waves, hipStream_t s);
// The join of the splits' partials into out.
hipError_t launch_kv_join(const KvAttnArgs& a, hipStream_t s);

}  // namespace q4gsw
