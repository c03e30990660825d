// Penalties for repeated tokens, biases and a grammar's mask on logits, in one pass (gfx950).
//
//   x = logit;  of a token seen so far: x = x > 0 ? x / repetition : x * repetition;  of one generated n > 0
//   times: x = (x - frequency n) - presence;  x += bias;  masked: -inf;  every step in fp32 as written.
//
// A workgroup takes a run of the vocabulary and one or more rows.  Few tokens are touched by more than
// the mask: those that stand in the sequence's history, among the tokens of its rows, or in its list of
// biases.  The history's are counted in LDS (bit 31: among the prompt's; low bits: how often generated) by
// integer atomics, whose order does not matter, and the first mark of a token lists it.  Of biases of one
// token the largest index wins by an integer maximum.  The rows' runs are then copied, masked, at the width
// of memory (not at all where the call is in place and nothing is masked), and the listed tokens of every
// row are computed from the logits once more, a thread each, over what the copy wrote; what a row's own path
// adds to a count is found by comparing its tokens, few rows' tokens being in one run.  So rows of one
// sequence share its count and wait for nothing of each other.
//
// Bound: HBM for large vocabularies: masking alone runs at a copy's rate (110 rows of 128256 fp32 logits: 24 us,
// 4.7 TB/s); counts of 4096 tokens a sequence, paths and biases make it 36 us, since all workgroups count at
// the same time and memory waits.  Few rows are latency: 8 rows of 32000 over 600 tokens 5 us a call.
// Long histories bound all: every workgroup reads its sequence's whole (8 rows of 32000 or of 128256 over 8192 tokens 11 us,
// 32768 30, 131072 88; 112 rows of 128256 in trees: 54, 124 and 379).
#include "logits.h"

namespace q4gsw {
namespace {

constexpr int kRows = 4;                 // most rows of a workgroup
constexpr int kThreads = 256, kOwnLoads = kTreeMax / kThreads, kLoads = 8, kItems = 2;
// Of a token's count: among the prompt's; listed; one of the rows' tokens.
constexpr uint32_t kPrompt = 0x80000000u, kListed = 0x40000000u, kOwn = 0x20000000u;

__host__ __device__ constexpr int in_quads(int n) { return (n + 3) & ~3; }

// Vectors in memory at the alignment of an element, which vector loads and stores take.
typedef uint32_t u4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2_at2 __attribute__((ext_vector_type(2), aligned(2)));

// Four neighbouring logits as they lie in memory.
template <int DT>
struct Quad {
    uint32_t w[DT == kF32 ? 4 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (DT == kF32) {
            const u4_at4 v = *reinterpret_cast<const u4_at4*>(static_cast<const float*>(p) + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = v[e];
        } else {
            const u2_at2 v = *reinterpret_cast<const u2_at2*>(static_cast<const uint16_t*>(p) + at);
            w[0] = v[0];
            w[1] = v[1];
        }
    }
    // bit e of `allowed` clear: logit e is -inf
    __device__ __forceinline__ void mask(uint32_t allowed) {
        if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (allowed >> e) & 1u ? w[e] : 0xFF800000u;
        } else {
            constexpr uint32_t none = DT == kF16 ? 0xFC00u : 0xFF80u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t lo = (allowed >> (2 * e)) & 1u ? w[e] & 0xFFFFu : none;
                const uint32_t hi = (allowed >> (2 * e + 1)) & 1u ? w[e] & 0xFFFF0000u : none << 16;
                w[e] = lo | hi;
            }
        }
    }
    __device__ __forceinline__ void store(void* p, int64_t at) const {
        if constexpr (DT == kF32) *reinterpret_cast<u4_at4*>(static_cast<float*>(p) + at) = u4_at4{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u2_at2*>(static_cast<uint16_t*>(p) + at) = u2_at2{w[0], w[1]};
    }
    // one by one, `n` of them (a row's last)
    __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
        for (uint32_t& v : w) v = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= n) break;
            if constexpr (DT == kF32) w[e] = static_cast<const uint32_t*>(p)[at + e];
            else w[e >> 1] |= (uint32_t)static_cast<const uint16_t*>(p)[at + e] << (16 * (e & 1));
        }
    }
    __device__ __forceinline__ void store(void* p, int64_t at, int64_t n) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= n) break;
            if constexpr (DT == kF32) static_cast<uint32_t*>(p)[at + e] = w[e];
            else static_cast<uint16_t*>(p)[at + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
};

template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t at, float v) {
    if constexpr (DT == kF32) static_cast<float*>(p)[at] = v;
    else if constexpr (DT == kF16) static_cast<uint16_t*>(p)[at] = bitcast<uint16_t>((_Float16)v);
    else static_cast<uint16_t*>(p)[at] = bitcast<uint16_t>((__bf16)v);
}

// The sequence that `row` is in and its rows [first, end); false: none.
struct Rows {
    int b;
    int64_t first, end;
    __device__ __forceinline__ bool find(const LogitsArgs& a, int64_t row) {
        if (!a.cu) {
            b = (int)row;
            first = row;
            end = row + 1;
            return true;
        }
        const int lane = threadIdx.x & 63;
        int count = 0, lo = 0, hi = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            lo = a.cu[min(b0 + lane, a.batch - 1)];
            hi = a.cu[min(b0 + lane, a.batch - 1) + 1];
            count += __popcll(__ballot(b0 + lane < a.batch && lo <= row));
        }
        b = __builtin_amdgcn_readfirstlane(count) - 1;
        if (b < 0) return false;
        if (a.batch <= 64) {
            first = __builtin_amdgcn_readlane(lo, b);
            end = __builtin_amdgcn_readlane(hi, b);
        } else {
            first = a.cu[b];
            end = a.cu[b + 1];
        }
        if (first < 0) first = 0;
        end = min(min(end, first + a.max_new), a.rows);
        return row >= first && row < end;                     // an offset may lie behind the next one
    }
};

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
    const bool listed = a.history || a.ids || a.bias_ids, copied = a.mask || a.out != a.logits;
    uint32_t* const s_count = lds;                            // [C]
    uint32_t* const s_bias = lds + C;                         // [C], where biases are given: entry + 1
    uint32_t* const s_listed = lds + (a.bias_ids ? 2 * C : C);
    uint16_t* const s_list = reinterpret_cast<uint16_t*>(s_listed + 4);                       // [C]
    int32_t* const s_ids = reinterpret_cast<int32_t*>(s_list + C);                            // [max_new in quads], where given
    const KvTree tree(reinterpret_cast<uint8_t*>(s_ids + (a.ids ? in_quads(a.max_new) : 0)), a.max_new);

    auto here = [&](int64_t id) -> bool { return id >= v0 && id < v0 + C && id < a.V; };
    // a token's first mark lists it
    auto mark = [&](int at, uint32_t old) {
        if (!(old & kListed) && !(atomicOr(&s_count[at], kListed) & kListed)) s_list[atomicAdd(s_listed, 1u)] = (uint16_t)at;
    };
    Quad<DT> x[kRows][Q];
    uint32_t allowed[kRows][Q];

    for (int64_t row = row0; row < row1;) {
        Rows in;
        if (!in.find(a, row)) {                               // of no sequence, or past max_new
            ++row;
            continue;
        }
        const int b = in.b, nodes = (int)(min(in.end, row1) - in.first), node0 = (int)(row - in.first);
        const int64_t first = in.first, end = first + nodes;

        // every load that depends on no other is on its way before the first use of one
        if (copied) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (row + r >= end) break;
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int64_t v = v0 + 4 * (tid + k * kThreads), l = row + r;         // its quad's mask is in one word
                    if (v >= a.V) continue;
                    if (v + 4 <= a.V) x[r][k].load(a.logits, l * a.ld + v);
                    else x[r][k].load(a.logits, l * a.ld + v, a.V - v);
                    if (a.mask) allowed[r][k] = a.mask[l * a.mask_ld + (v >> 5)];
                }
            }
        }
        const float rep = a.repetition ? a.repetition[b] : 1.0f, pres = a.presence ? a.presence[b] : 0.0f;
        const float freq = a.frequency ? a.frequency[b] : 0.0f;
        if (listed) {
            const int32_t* hist = a.history + (int64_t)b * a.history_ld;
            const int32_t* biased = a.bias_ids + (int64_t)b * a.bias_ld;
            const int held = a.history && a.history_cols ? a.history_len[b] : 0, prompt = a.prompt_len ? a.prompt_len[b] : 0;
            int old[kLoads], own[kOwnLoads], up[kOwnLoads], bias_id = -1;
            if (a.history && a.history_cols)
#pragma unroll
                for (int k = 0; k < kLoads; ++k) old[k] = hist[min(tid + k * kThreads, a.history_cols - 1)];
#pragma unroll
            for (int k = 0; k < kOwnLoads; ++k) {
                const int64_t j = first + min(tid + k * kThreads, nodes - 1);
                if (a.ids) own[k] = a.ids[j];
                if (a.parents) up[k] = a.parents[j];
            }
            if (a.bias_ids && tid < a.bias_cols) bias_id = biased[tid];

            __syncthreads();                                  // the last sequence's reads are done
            for (int j = tid; j < (a.bias_ids ? C / 2 : C / 4); j += kThreads) reinterpret_cast<u4*>(lds)[j] = u4{0u, 0u, 0u, 0u};
            if (tid == 0) *s_listed = 0u;
            if (a.ids)
#pragma unroll
                for (int k = 0; k < kOwnLoads; ++k) {
                    const int j = tid + k * kThreads;
                    if (j >= nodes) break;
                    s_ids[j] = own[k];
                    if (a.parents) tree.put(j, up[k]);
                }
            __syncthreads();
            const int n = min(max(held, 0), a.history_cols);
            for (int j0 = tid; j0 < n; j0 += kLoads * kThreads) {
                if (j0 != tid)
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) old[k] = hist[min(j0 + k * kThreads, n - 1)];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int j = j0 + k * kThreads;
                    if (j >= n || !here(old[k])) continue;
                    const int at = (int)(old[k] - v0);
                    mark(at, j < prompt ? atomicOr(&s_count[at], kPrompt) : atomicAdd(&s_count[at], 1u));
                }
            }
            if (a.ids)
#pragma unroll
                for (int k = 0; k < kOwnLoads; ++k)
                    if (tid + k * kThreads < nodes && here(own[k])) mark((int)(own[k] - v0), atomicOr(&s_count[own[k] - v0], kOwn));
            if (a.bias_ids) {
                for (int j = tid; j < a.bias_cols; j += kThreads) {
                    const int id = j == tid ? bias_id : biased[j];
                    if (!here(id)) continue;
                    atomicMax(&s_bias[id - v0], (uint32_t)j + 1u);
                    mark((int)(id - v0), 0u);
                }
            }
            if (a.parents && tid < (int)(end - row)) tree.climb(node0 + tid, 0, tree.bits + tid * tree.stride);
        }

        if (copied) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (row + r >= end) break;
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int64_t v = v0 + 4 * (tid + k * kThreads), l = row + r;
                    if (v >= a.V) continue;
                    if (a.mask) x[r][k].mask(allowed[r][k] >> (v & 31));
                    if (v + 4 <= a.V) x[r][k].store(a.out, l * a.out_ld + v);
                    else x[r][k].store(a.out, l * a.out_ld + v, a.V - v);
                }
            }
        }
        if (listed) {
            __syncthreads();
            const int n = (int)*s_listed, items = n * (int)(end - row);
            // the loads of kItems of them together
            for (int i0 = tid; i0 < items; i0 += kItems * kThreads) {
                int at[kItems], r[kItems];
                uint32_t word[kItems], w[kItems];
                float y[kItems], bias[kItems];
#pragma unroll
                for (int k = 0; k < kItems; ++k) {
                    const int it = min(i0 + k * kThreads, items - 1);
                    r[k] = it / n;
                    at[k] = s_list[it - r[k] * n];
                    const int64_t v = v0 + at[k], l = row + r[k];
                    word[k] = a.mask ? a.mask[l * a.mask_ld + (v >> 5)] : ~0u;
                    y[k] = load_elem<DT>(a.logits, l * a.ld + v);
                    w[k] = a.bias_ids ? s_bias[at[k]] : 0u;
                    bias[k] = w[k] ? a.bias[(int64_t)b * a.bias_ld + (w[k] - 1)] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kItems; ++k) {
                    const int64_t v = v0 + at[k], l = row + r[k];
                    if (i0 + k * kThreads >= items || !((word[k] >> (v & 31)) & 1u)) continue;
                    uint32_t c = s_count[at[k]];
                    if (c & kOwn) {
                        const int node = (int)(l - first);
                        const uint32_t* bits = tree.bits + r[k] * tree.stride + 1;
                        for (int j = 0; j <= node; j += 4) {
                            const u4 id = *reinterpret_cast<const u4*>(s_ids + j);
                            uint32_t on = a.parents ? bits[j >> 5] >> (j & 31) : ~0u;
                            if (node - j < 3) on &= (2u << (node - j)) - 1u;
#pragma unroll
                            for (int e = 0; e < 4; ++e) c += (on >> e) & (id[e] == (uint32_t)v ? 1u : 0u);
                        }
                    }
                    c &= ~(kListed | kOwn);
                    float z = y[k];
                    if (c) z = penalised(z, c & ~kPrompt, rep, freq, pres);
                    if (w[k]) z += bias[k];
                    store_logit<DT>(a.out, l * a.out_ld + v, z);
                }
            }
        }
        row = end;
    }
}

// Quads a thread where there is work for all CUs: 110 rows of 128256 logits in trees over 4096 tokens take 36 us with
// two of them and up to four rows a workgroup, 39 with three, 42 with four, 55 with two and one row.
constexpr int kWide = 2;

int chunks_of(int64_t V, int quads) { return (int)((V + 4 * quads * kThreads - 1) / (4 * quads * kThreads)); }

int quads_of(const LogitsArgs& a) { return a.rows * chunks_of(a.V, kWide) >= 512 ? kWide : 1; }

int lds_bytes(const LogitsArgs& a, int quads, int rows) {
    const int C = 4 * quads * kThreads;
    if (!a.history && !a.ids && !a.bias_ids) return 0;
    return 4 * C + (a.bias_ids ? 4 * C : 0) + 16 + 2 * C + (a.ids ? 4 * in_quads(a.max_new) : 0) + (a.parents ? tree_bytes(a.max_new, rows) : 0);
}

// Rows of one sequence share the count of its history: as many to a workgroup as let all workgroups run at once.
int group_rows(const LogitsArgs& a, int quads, int chunks) {
    if (!a.cu || !(a.history || a.bias_ids)) return 1;
    const int lds = lds_bytes(a, quads, kRows), fit = 160 * 1024 / lds < 8 ? 160 * 1024 / lds : 8;
    int64_t n = (a.rows * chunks + 256 * fit - 1) / (256 * fit);
    const int64_t most = (a.rows + a.batch - 1) / a.batch;
    if (n > most) n = most;
    return (int)(n > kRows ? kRows : n);
}

template <int DT, int Q>
hipError_t launch(const LogitsArgs& a, hipStream_t s) {
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    hipLaunchKernelGGL((logits_kernel<DT, Q>), dim3((unsigned)(groups * a.chunks)), dim3(kThreads), lds_bytes(a, Q, a.rows_per_group), s, a);
    return hipGetLastError();
}

}  // namespace

bool logits_launch_ok(const LogitsArgs& a) {
    return a.rows <= ((int64_t(1) << 32) / kThreads - 1) / chunks_of(a.V, 1);
}

hipError_t launch_logits(LogitsArgs a, int dtype, hipStream_t s) {
    const int quads = quads_of(a);
    a.chunks = chunks_of(a.V, quads);
    a.rows_per_group = group_rows(a, quads, a.chunks);
#define Q4GSW_LOGITS(DT) return quads == 1 ? launch<DT, 1>(a, s) : launch<DT, kWide>(a, s)
    switch (dtype) {
        case kF32: Q4GSW_LOGITS(kF32);
        case kF16: Q4GSW_LOGITS(kF16);
        default: Q4GSW_LOGITS(kBF16);
    }
#undef Q4GSW_LOGITS
}

}  // namespace q4gsw
