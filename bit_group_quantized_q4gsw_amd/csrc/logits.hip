// Penalties for repeated tokens, biases and a grammar's mask on logits, in one pass (gfx950).
//
//   x = logit;  of a token seen so far: x = x > 0 ? x / repetition : x * repetition;  of one generated n > 0
//   times: x = (x - frequency n) - presence;  x += bias;  masked: -inf;  every step in fp32 as written.
//
// A workgroup takes a run of the vocabulary and one or more rows.  It counts, in LDS, how often the tokens of
// its run stand in the row's history (bit 31: among the prompt's; below: how often generated), by
// integer atomics, whose order does not matter; rows of one sequence (a tree's nodes) share that count, and
// each adds its own path's tokens and takes them off again.  Of biases of one token the last entry counts:
// the largest index wins by an integer maximum.  Then the run is read, adjusted and written once.
//
// Bound: HBM for large vocabularies; few rows are latency (history, LDS, logits).
#include "logits.h"

namespace q4gsw {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kPrompt = 0x80000000u;

template <int DT>
__device__ __forceinline__ f4 load_logits(const void* p, int64_t at) {
    if constexpr (DT == kF32) return *reinterpret_cast<const f4*>(static_cast<const float*>(p) + at);
    const u2 w = *reinterpret_cast<const u2*>(static_cast<const uint16_t*>(p) + at);
    f4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        v[e] = DT == kF16 ? f16_bits_to_f32(h) : bf16_bits_to_f32(h);
    }
    return v;
}

template <int DT>
__device__ __forceinline__ void store_logits(void* p, int64_t at, f4 v) {
    if constexpr (DT == kF32) {
        *reinterpret_cast<f4*>(static_cast<float*>(p) + at) = v;
    } else {
        u2 w;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            w[e] = DT == kF16 ? bitcast<uint32_t>(h2{(_Float16)v[2 * e], (_Float16)v[2 * e + 1]})
                              : bitcast<uint32_t>(b2{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]});
        *reinterpret_cast<u2*>(static_cast<uint16_t*>(p) + at) = w;
    }
}

template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t at, float v) {
    if constexpr (DT == kF32) static_cast<float*>(p)[at] = v;
    else if constexpr (DT == kF16) static_cast<uint16_t*>(p)[at] = bitcast<uint16_t>((_Float16)v);
    else static_cast<uint16_t*>(p)[at] = bitcast<uint16_t>((__bf16)v);
}

// The last sequence that begins at `row` or before; -1: none.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int batch, int64_t row) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
        const bool before = b0 + lane < batch && cu[min(b0 + lane, batch - 1)] <= row;
        count += __popcll(__ballot(before));
    }
    return __builtin_amdgcn_readfirstlane(count) - 1;
}

// The logit of a token seen before and generated n times.
__device__ __forceinline__ float penalised(float y, uint32_t n, float rep, float freq, float pres) {
#pragma clang fp contract(off)               // a product that is rounded before the difference
    y = y > 0.0f ? y / rep : y * rep;
    if (n) y = (y - freq * (float)n) - pres;
    return y;
}

// 4 Q x 256 tokens of the vocabulary a workgroup, a quad a thread and step.
template <int DT, int Q>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs a) {
    constexpr int C = 4 * Q * kThreads;
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    const int tid = threadIdx.x;
    const int64_t v0 = (int64_t)(blockIdx.x % a.chunks) * C;
    const int64_t row0 = (int64_t)(blockIdx.x / a.chunks) * a.rows_per_group;
    const int64_t row1 = min(row0 + a.rows_per_group, a.rows);
    const bool counted = a.history || a.ids;
    uint32_t* const s_count = lds;                            // [C], where tokens are counted
    uint32_t* const s_bias = lds + (counted ? C : 0);         // [C], where biases are given: entry + 1
    const KvTree tree(reinterpret_cast<uint8_t*>(s_bias + (a.bias_ids ? C : 0)), a.max_new);

    int seq = -1;
    int64_t first = 0;                                        // the sequence's rows
    int nodes = 0, tree0 = 0;
    for (int64_t row = row0; row < row1; ++row) {
        const int b = a.cu ? sequence_of(a.cu, a.batch, row) : (int)row;
        if (b < 0) continue;
        if (b != seq) {
            if (a.cu) {
                first = max(a.cu[b], 0);
                const int64_t end = min((int64_t)a.cu[b + 1], a.rows);
                nodes = (int)min(end - first, (int64_t)a.max_new);
            } else {
                first = row;
                nodes = 1;
            }
        }
        if (row - first >= nodes) continue;                   // behind the last sequence, or past max_new
        if (b != seq) {
            seq = b;
            __syncthreads();                                  // the last row's reads are done
            if (counted)
                for (int j = tid; j < C / 4; j += kThreads) reinterpret_cast<u4*>(s_count)[j] = u4{0u, 0u, 0u, 0u};
            if (a.bias_ids)
                for (int j = tid; j < C / 4; j += kThreads) reinterpret_cast<u4*>(s_bias)[j] = u4{0u, 0u, 0u, 0u};
            __syncthreads();
            if (a.history) {
                const int32_t* h = a.history + (int64_t)b * a.history_ld;
                const int n = min(max(a.history_len[b], 0), a.history_cols), prompt = a.prompt_len ? a.prompt_len[b] : 0;
                for (int j = tid; j < n; j += kThreads) {
                    const int64_t at = (int64_t)h[j] - v0;
                    if (at < 0 || at >= C) continue;
                    if (j < prompt) atomicOr(&s_count[at], kPrompt);
                    else atomicAdd(&s_count[at], 1u);
                }
            }
            if (a.bias_ids) {
                const int32_t* ids = a.bias_ids + (int64_t)b * a.bias_ld;
                for (int j = tid; j < a.bias_cols; j += kThreads) {
                    const int64_t at = (int64_t)ids[j] - v0;
                    if (at >= 0 && at < C) atomicMax(&s_bias[at], (uint32_t)j + 1u);
                }
            }
            tree0 = (int)(row - first);
            if (a.parents) KvTree(tree).build(a.parents, first, nodes, tree0, (int)min(row1 - row, (int64_t)nodes - tree0), 0);
        }
        const int node = (int)(row - first);
        // a chain's row has all rows up to it behind it: only single tokens and short drafts come so
        auto path = [&](uint32_t by) {
            const int last = a.parents ? nodes : node + 1;
            for (int j = tid; j < last; j += kThreads) {
                if (a.parents && !((tree.bits[(node - tree0) * tree.stride + 1 + (j >> 5)] >> (j & 31)) & 1u)) continue;
                const int64_t at = (int64_t)a.ids[first + j] - v0;
                if (at >= 0 && at < C) atomicAdd(&s_count[at], by);
            }
        };
        if (a.ids) path(1u);
        __syncthreads();

        const float rep = a.repetition ? a.repetition[b] : 1.0f, pres = a.presence ? a.presence[b] : 0.0f;
        const float freq = a.frequency ? a.frequency[b] : 0.0f;
        const float* bias = a.bias + (a.bias_ids ? (int64_t)b * a.bias_ld : 0);
        const uint32_t* mask = a.mask ? a.mask + row * a.mask_ld : nullptr;
        f4 x[Q];
#pragma unroll
        for (int k = 0; k < Q; ++k) {
            const int64_t v = v0 + 4 * (tid + k * kThreads);
            if (a.quads) {
                if (v < a.V) x[k] = load_logits<DT>(a.logits, row * a.ld + v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e < a.V) x[k][e] = load_elem<DT>(a.logits, row * a.ld + v + e);
            }
        }
#pragma unroll
        for (int k = 0; k < Q; ++k) {
            const int at = 4 * (tid + k * kThreads);
            const int64_t v = v0 + at;
            if (v >= a.V) continue;
            const u4 c = counted ? *reinterpret_cast<const u4*>(s_count + at) : u4{0u, 0u, 0u, 0u};
            const u4 w = a.bias_ids ? *reinterpret_cast<const u4*>(s_bias + at) : u4{0u, 0u, 0u, 0u};
            const uint32_t allowed = mask ? mask[v >> 5] >> (v & 31) : 15u;      // v is a multiple of 4
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = x[k][e];
                if (c[e]) y = penalised(y, c[e] & ~kPrompt, rep, freq, pres);
                if (w[e]) y += bias[w[e] - 1];
                x[k][e] = (allowed >> e) & 1u ? y : -INFINITY;
            }
            if (a.quads) {
                store_logits<DT>(a.out, row * a.out_ld + v, x[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e < a.V) store_logit<DT>(a.out, row * a.out_ld + v + e, x[k][e]);
            }
        }
        if (a.ids) {
            __syncthreads();
            path(0u - 1u);
        }
    }
}

constexpr int kWide = 4;                 // quads a thread where there is work for all CUs

int chunks_of(int64_t V, int quads) { return (int)((V + 4 * quads * kThreads - 1) / (4 * quads * kThreads)); }

int quads_of(const LogitsArgs& a) { return a.rows * chunks_of(a.V, kWide) >= 512 ? kWide : 1; }

// Rows of one sequence share the count of its history, as long as 1024 workgroups are left.
int group_rows(const LogitsArgs& a, int chunks) {
    if (!a.cu || !(a.history || a.bias_ids)) return 1;
    int64_t n = (a.rows + a.batch - 1) / a.batch;
    if (n > a.rows * chunks / 1024) n = a.rows * chunks / 1024;
    return (int)(n < 1 ? 1 : (n > 16 ? 16 : n));
}

template <int DT, int Q>
hipError_t launch(const LogitsArgs& a, hipStream_t s) {
    constexpr int C = 4 * Q * kThreads;
    size_t lds = (a.history || a.ids ? 4 * C : 0) + (a.bias_ids ? 4 * C : 0);
    if (a.parents) lds += tree_bytes(a.max_new, a.rows_per_group);
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    hipLaunchKernelGGL((logits_kernel<DT, Q>), dim3((unsigned)(groups * a.chunks)), dim3(kThreads), lds, s, a);
    return hipGetLastError();
}

}  // namespace

bool logits_launch_ok(const LogitsArgs& a) {
    return a.rows <= ((int64_t(1) << 32) / kThreads - 1) / chunks_of(a.V, 1);
}

hipError_t launch_logits(LogitsArgs a, int dtype, hipStream_t s) {
    const int quads = quads_of(a);
    a.chunks = chunks_of(a.V, quads);
    a.rows_per_group = group_rows(a, a.chunks);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.out);
    a.quads = a.V % 4 == 0 && a.ld % 4 == 0 && a.out_ld % 4 == 0 && (at & (dtype == kF32 ? 15u : 7u)) == 0;
#define Q4GSW_LOGITS(DT) return quads == 1 ? launch<DT, 1>(a, s) : launch<DT, kWide>(a, s)
    switch (dtype) {
        case kF32: Q4GSW_LOGITS(kF32);
        case kF16: Q4GSW_LOGITS(kF16);
        default: Q4GSW_LOGITS(kBF16);
    }
#undef Q4GSW_LOGITS
}

}  // namespace q4gsw
