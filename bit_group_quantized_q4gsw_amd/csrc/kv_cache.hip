// Keys and values of new tokens into the paged 4-bit cache, and back out of it (layout: kv4.h).
//
// Per token, head and run of 32 channels x, every step in fp32 as written (rint: half to even):
//   scale = fp16(min(max|x| / 7, 8188)),  inv = 1 / scale,
//   value = clamp(rint(x inv), -8, 7), and 0 where the scale is 0 or x is NaN (a NaN also counts
//   as 0 in the maximum).  8188 is 65504 / 8: value * scale stays a finite fp16.
//
// One workgroup per (32-token block, head), so the nibbles that eight tokens share in a word of
// values are all written by one workgroup: a word some of whose tokens are not new is read,
// merged and written back; no atomics.  A sequence of m new tokens touches at most m / 32 + 2
// blocks, and floor(cu[b] / 32) + 2 b is then a first workgroup for sequence b that no other
// sequence's range reaches: the grid needs no scan of the lengths, and every workgroup finds its
// sequence by counting the first workgroups that are not after it, 64 sequences a load.
//
// Bound: HBM for the read-out (it writes 4 bytes an element: 13000 tokens of 8 heads of 128 in 25 us,
// 4.8 TB/s); the append reads 2 bytes and writes 0.56 a 16-bit element and takes 22.5 us for them, some
// 15 of it the codes' VALU (two IEEE divisions an octet, eight steps an element).  Single tokens take 6
// and 4 us, which is three rounds of loads.
#include "internal.h"
#include "kv_tree.h"

namespace q4gsw {
namespace {

constexpr int kThreads = 256;

struct BlockAt {
    int t0, t1;          // the block's new tokens: places [t0, t1); none if t0 >= t1
    int64_t row0;        // token row of place 0 (may lie before the sequence's first)
    int page, sub;       // its page (negative or past the cache: none holds the block) and block of the page
    __device__ __forceinline__ uint8_t* unit(const KvView& c, int head) const {
        return page >= 0 && page < c.pages ? c.data + kv_unit(c, page, head, sub) : nullptr;
    }
};

// The block that workgroup `w` serves.  Places before 0 (more new tokens than the length) count on
// downwards, so that every row of a sequence belongs to one workgroup.  A batch of up to 64 takes one
// round of loads for its sequence and one for its page, which nothing here waits for.
__device__ __forceinline__ BlockAt find_block(const KvView& c, const KvSeqs& sq, int64_t w) {
    BlockAt r{0, 0, 0, -1, 0};
    const int lane = threadIdx.x & 63;
    int count = 0, lo = 0, hi = 0, len = 0;
    for (int b0 = 0; b0 < sq.batch; b0 += 64) {
        const int b = min(b0 + lane, sq.batch - 1);
        lo = sq.cu[b];
        hi = sq.cu[b + 1];
        len = sq.lens[b];
        const bool before = b0 + lane < sq.batch && (int64_t)(max(lo, 0) >> 5) + 2 * (int64_t)b <= w;
        count += __popcll(__ballot(before));
    }
    if (count == 0) return r;
    const int b = __builtin_amdgcn_readfirstlane(min(count, sq.batch) - 1);
    KvSeq s;
    if (sq.batch <= 64)
        s = kv_seq(sq.tokens, __builtin_amdgcn_readlane(lo, b), __builtin_amdgcn_readlane(hi, b), __builtin_amdgcn_readlane(len, b));
    else
        s = kv_seq(sq, b);
    const int64_t k = w - ((s.first_row >> 5) + 2 * (int64_t)b);
    const int64_t p0 = (int64_t)s.len - s.m;            // place of the first new token
    const int64_t blk = (p0 >> 5) + k;
    if (k < 0 || 32 * blk >= s.len) return r;
    r.t0 = (int)max(p0 - 32 * blk, (int64_t)0);
    r.t1 = (int)min(s.len - 32 * blk, (int64_t)32);
    r.row0 = s.first_row + 32 * blk - p0;
    const int64_t at = blk >> c.bpp_log2;
    if (blk < 0 || at >= sq.table_cols) return r;
    r.page = sq.table[(int64_t)b * sq.table_ld + at];
    r.sub = (int)(blk & ((1 << c.bpp_log2) - 1));
    return r;
}

// 8 elements as they lie in memory, from a 16-byte aligned place, and as fp32
template <int XT>
struct Raw8 {
    u4 w[XT == kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* x, int64_t e) {
        if constexpr (XT == kF32) {
            w[0] = ldg16(static_cast<const float*>(x) + e);
            w[1] = ldg16(static_cast<const float*>(x) + e + 4);
        } else {
            w[0] = ldg16(static_cast<const uint16_t*>(x) + e);
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (XT == kF32) return bitcast<float>(w[i >> 2][i & 3]);
        const uint32_t h = w[0][i >> 1];
        if constexpr (XT == kF16) return f16_bits_to_f32((uint16_t)((i & 1) ? h >> 16 : h & 0xFFFFu));
        return bitcast<float>((i & 1) ? h & 0xFFFF0000u : h << 16);
    }
};

// v as a whole number, saturated; NaN gives 0
__device__ __forceinline__ int to_int(float v) {
    int r;
    asm("v_cvt_i32_f32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}

// 24 bytes more a token: the four tokens that a wave gathers at once lie in other banks
template <int D>
constexpr int kVcRow = D + 24;

// The whole workgroup: tokens [t0, t1) of a unit, from keys' words in plane order, values' codes
// [token][channel] and scales in layout order in LDS.
template <int D>
__device__ __forceinline__ void store_block(uint8_t* unit, int t0, int t1, const uint32_t* s_kw, const uint8_t* s_vc,
                                            const uint16_t* s_ksc, const uint16_t* s_vsc) {
    constexpr int G = D / 32;
    const int tid = threadIdx.x;
    // words of one plane in address order: lane and word of 4-byte place n
    auto place = [](int n, int& w, int& lane) {
        const int p = n >> 8;
        if ((G & 1) && p == G / 2) {
            lane = (n & 255) >> 1;
            w = 4 * p + (n & 1);
        } else {
            lane = (n & 255) >> 2;
            w = 4 * p + (n & 3);
        }
    };
    uint32_t* kw = reinterpret_cast<uint32_t*>(unit);
    uint32_t* vw = reinterpret_cast<uint32_t*>(unit + 512 * G);
    uint16_t* ksc = reinterpret_cast<uint16_t*>(unit + 1024 * G);
    uint16_t* vsc = ksc + 32 * G;
    for (int n = tid; n < 128 * G; n += kThreads) {
        int w, lane;
        place(n, w, lane);
        const int i = lane & 15, q = lane >> 4;
        const int t = kv_tok(i >> 2, 4 * (w & 1) + (i & 3));
        if (t >= t0 && t < t1) kw[n] = s_kw[n];
        uint32_t word = 0, mask = 0;
#pragma unroll
        for (int slot = 0; slot < 8; ++slot) {
            const int tt = kv_tok(q, slot);
            if (tt < t0 || tt >= t1) continue;
            word |= (uint32_t)s_vc[tt * kVcRow<D> + 16 * w + i] << (4 * nib_pos(slot));
            mask |= 0xFu << (4 * nib_pos(slot));
        }
        if (mask == 0xFFFFFFFFu) vw[n] = word;
        else if (mask) vw[n] = (vw[n] & ~mask) | word;
    }
    for (int n = tid; n < 32 * G; n += kThreads) {
        const int t = kv_tok(n / (8 * G), n & 7);
        if (t < t0 || t >= t1) continue;
        ksc[n] = s_ksc[n];
        vsc[n] = s_vsc[n];
    }
}

// Four lanes hold the 32 channels of a scale, 8 each.  The arithmetic follows the definition step
// by step, IEEE division included, so the codes are the definition's bit for bit.  Each item (a
// token's k-octet) is one coalesced 16-byte load; the codes go through LDS because a word of
// values joins eight tokens, which also lets whole words leave in layout order.
template <int XT, int D>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvView c, KvSeqs sq, const void* __restrict__ k, int64_t k_ld,
                                                             const void* __restrict__ v, int64_t v_ld) {
    constexpr int G = D / 32, kOct = D / 8, kItems = 32 * kOct;
    __shared__ uint32_t s_kw[128 * G];                     // keys' words in plane order
    __shared__ __attribute__((aligned(16))) uint8_t s_vc[32 * kVcRow<D>];    // values' codes [token][channel]
    __shared__ uint16_t s_sc[2][32 * G];                   // scales in layout order
    const int tid = threadIdx.x, head = blockIdx.y;
    const BlockAt at = find_block(c, sq, blockIdx.x);
    if (at.t0 >= at.t1) return;

    // every load of the thread before the first use of one
    constexpr int kPer = (kItems + kThreads - 1) / kThreads;
    Raw8<XT> raw[2][kPer];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int it = tid + j * kThreads, t = it / kOct, o = it - t * kOct;
            if (t >= at.t0 && t < at.t1) raw[kv][j].load(kv ? v : k, (at.row0 + t) * (kv ? v_ld : k_ld) + head * D + 8 * o);
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int it = tid + j * kThreads, t = it / kOct, o = it - t * kOct, g = o >> 2;
            if (t < at.t0 || t >= at.t1) continue;         // a group's four lanes stay together
            const Raw8<XT>& x = raw[kv][j];
            float amax = 0.0f;                             // fmaxf passes NaN over
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
            amax = fmaxf(amax, __shfl_xor(amax, 1));
            amax = fmaxf(amax, __shfl_xor(amax, 2));
            const _Float16 sh = (_Float16)fminf(amax / 7.0f, 8188.0f);
            const float s = (float)sh;
            const float inv = s > 0.0f ? 1.0f / s : 0.0f;
            uint32_t code[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = to_int(rintf(x[e] * inv));
                code[e] = (uint32_t)((r < -8 ? -8 : (r > 7 ? 7 : r)) + 8);
            }
            const int q = kv_q(t), slot = kv_slot(t);
            if (kv == 0) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) w |= code[e] << (4 * nib_pos(e));
                s_kw[kv_word_off<G>(2 * g + (slot >> 2), 16 * (o & 3) + 4 * q + (slot & 3)) >> 2] = w;
            } else {
                u2 w = {0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e >> 2] |= code[e] << (8 * (e & 3));
                *reinterpret_cast<u2*>(&s_vc[t * kVcRow<D> + 8 * o]) = w;
            }
            if ((o & 3) == 0) s_sc[kv][(q * G + g) * 8 + slot] = bitcast<uint16_t>(sh);
        }
    }
    __syncthreads();
    uint8_t* const unit = at.unit(c, head);
    if (!unit) return;

    store_block<D>(unit, at.t0, at.t1, s_kw, s_vc, s_sc[0], s_sc[1]);
}

// The new tokens' rows back as fp32: value * scale, exact (4 + 11 bits).  A token whose place has
// no page of the cache gives zeros.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvView c, KvSeqs sq, float* __restrict__ k, float* __restrict__ v) {
    constexpr int G = D / 32, kOct = D / 8;
    __shared__ __attribute__((aligned(16))) uint8_t s_unit[1152 * G];
    const int tid = threadIdx.x, head = blockIdx.y;
    const BlockAt at = find_block(c, sq, blockIdx.x);
    if (at.t0 >= at.t1) return;
    const uint8_t* const unit = at.unit(c, head);
    // a block without a page reads as a unit of zeros: scale 0
    for (int n = tid; n < 72 * G; n += kThreads)
        *reinterpret_cast<u4*>(&s_unit[16 * n]) = unit ? ldg16(unit + 16 * n) : u4{0u, 0u, 0u, 0u};
    __syncthreads();
    const uint16_t* ksc = reinterpret_cast<const uint16_t*>(s_unit + 1024 * G);
    const uint16_t* vsc = ksc + 32 * G;
    for (int it = tid; it < 32 * kOct; it += kThreads) {
        const int t = it / kOct, o = it - t * kOct, g = o >> 2;
        if (t < at.t0 || t >= at.t1) continue;
        const int q = kv_q(t), slot = kv_slot(t);
        const int64_t dst = ((at.row0 + t) * c.heads + head) * D + 8 * o;
        const uint32_t w =
            *reinterpret_cast<const uint32_t*>(&s_unit[kv_word_off<G>(2 * g + (slot >> 2), 16 * (o & 3) + 4 * q + (slot & 3))]);
        const float ks = f16_bits_to_f32(ksc[(q * G + g) * 8 + slot]);
        float x[8];
        word_codes_minus8_f32(w, x);
        f4 lo, hi;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = x[e] * ks;
            hi[e] = x[4 + e] * ks;
        }
        *reinterpret_cast<f4*>(k + dst) = lo;
        *reinterpret_cast<f4*>(k + dst + 4) = hi;
        const float vs = f16_bits_to_f32(vsc[(q * G + g) * 8 + slot]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ch = 8 * o + e;
            const uint32_t vwd =
                *reinterpret_cast<const uint32_t*>(&s_unit[512 * G + kv_word_off<G>(ch >> 4, 16 * q + (ch & 15))]);
            const float y = (float)((int)((vwd >> (4 * nib_pos(slot))) & 15u) - 8) * vs;
            if (e < 4) lo[e] = y;
            else hi[e - 4] = y;
        }
        *reinterpret_cast<f4*>(v + dst) = lo;
        *reinterpret_cast<f4*>(v + dst + 4) = hi;
    }
}

// The accepted path of each tree in a row: the nodes on the way from a root to leaf[b] (kv_tree.h) move, as
// they are, to places p0, p0 + 1, ... behind the p0 tokens before the tree.  One workgroup per (sequence,
// head) and cache.  Node numbers rise along the path, so the k-th node's place is p0 + k or later: block
// after block of destinations is gathered into LDS and then stored as the append stores one, and what a
// block still has to read lies behind all that is written so far.  Nodes in place already are skipped.
//
// Bound: latency: the climb, then per block a page number, the codes, and the merge of values' words: 4 sequences of 13
// nodes, 8 heads of 64 and 2 caches 5 us; 64 of 31 to 61 nodes, 8 heads of 128, 4 caches (2048 workgroups, all at once) 15.
struct KeepArgs {
    uint8_t* data[kKeepCaches];
    KvView c;                            // of every cache, but for the data
    KvSeqs sq;
    const int32_t* parents;
    const int32_t* leaf;
    int max_new;
    int32_t* kept;
    int32_t* path;                       // may be null
};

template <int D>
__global__ __launch_bounds__(kThreads) void kv_keep_kernel(KeepArgs a) {
    constexpr int G = D / 32, kOct = D / 8;
    __shared__ uint32_t s_kw[128 * G];
    __shared__ __attribute__((aligned(16))) uint8_t s_vc[32 * kVcRow<D>];
    __shared__ uint16_t s_sc[2][32 * G];
    __shared__ int16_t s_up[kTreeMax], s_back[kTreeMax];   // parents, path from the leaf back
    __shared__ int s_count;
    const int tid = threadIdx.x, b = blockIdx.x / a.c.heads, head = blockIdx.x % a.c.heads;
    const KvSeq s = kv_seq(a.sq, b);
    const int nodes = min(s.m, a.max_new), leaf = a.leaf[b];
    for (int j = tid; j < nodes; j += kThreads) s_up[j] = tree_parent(a.parents[s.first_row + j], j);
    __syncthreads();
    if (tid == 0) {
        int n = 0;
        if (leaf >= 0 && leaf < nodes)
            for (int j = leaf; j >= 0; j = s_up[j]) s_back[n++] = (int16_t)j;
        s_count = n;
    }
    __syncthreads();
    const int count = s_count;
    auto node = [&](int k) -> int { return s_back[count - 1 - k]; };
    const int p0 = s.len - s.m;          // may be negative: such places are none
    if (blockIdx.y == 0 && head == 0) {
        if (tid == 0) a.kept[b] = max(p0 + count, 0);
        if (a.path)
            for (int k = tid; k < a.max_new; k += kThreads) a.path[(int64_t)b * a.max_new + k] = k < count ? node(k) : -1;
    }
    int still = 0;                       // nodes in place: the first ones
    for (int k0 = 0; k0 < count; k0 += kThreads) still += __syncthreads_count(k0 + tid < count && node(k0 + tid) == k0 + tid);
    if (still >= count) return;

    KvView c = a.c;
    c.data = a.data[blockIdx.y];
    const int sub_mask = (1 << c.bpp_log2) - 1;
    auto unit_of = [&](int place) -> uint8_t* {
        const int64_t blk = place >> 5, at = blk >> c.bpp_log2;
        if (place < 0 || at >= a.sq.table_cols) return nullptr;
        const int page = a.sq.table[(int64_t)b * a.sq.table_ld + at];
        return page >= 0 && page < c.pages ? c.data + kv_unit(c, page, head, (int)(blk & sub_mask)) : nullptr;
    };
    const int first = max(p0 + still, 0), end = p0 + count;
    for (int64_t blk = first >> 5; 32 * blk < end; ++blk) {
        const int base = (int)(32 * blk), t0 = max(first - base, 0), t1 = min(end - base, 32);
        for (int it = tid; it < 32 * kOct; it += kThreads) {
            const int t = it / kOct, o = it - t * kOct, g = o >> 2;
            if (t < t0 || t >= t1) continue;
            const int from = p0 + node(base + t - p0), ft = from & 31;
            const uint8_t* src = unit_of(from);
            const int q = kv_q(t), slot = kv_slot(t), fq = kv_q(ft), fslot = kv_slot(ft);
            uint32_t key = 0x88888888u;                    // no page there: zeros
            uint16_t ks = 0, vs = 0;
            u2 w = {0x08080808u, 0x08080808u};
            if (src) {
                key = *reinterpret_cast<const uint32_t*>(src + kv_word_off<G>(2 * g + (fslot >> 2), 16 * (o & 3) + 4 * fq + (fslot & 3)));
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int ch = 8 * o + e;
                    v[e] = *reinterpret_cast<const uint32_t*>(src + 512 * G + kv_word_off<G>(ch >> 4, 16 * fq + (ch & 15)));
                }
                ks = reinterpret_cast<const uint16_t*>(src + 1024 * G)[(fq * G + g) * 8 + fslot];
                vs = reinterpret_cast<const uint16_t*>(src + 1088 * G)[(fq * G + g) * 8 + fslot];
                w = u2{0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e >> 2] |= ((v[e] >> (4 * nib_pos(fslot))) & 15u) << (8 * (e & 3));
            }
            s_kw[kv_word_off<G>(2 * g + (slot >> 2), 16 * (o & 3) + 4 * q + (slot & 3)) >> 2] = key;
            *reinterpret_cast<u2*>(&s_vc[t * kVcRow<D> + 8 * o]) = w;
            if ((o & 3) == 0) {
                s_sc[0][(q * G + g) * 8 + slot] = ks;
                s_sc[1][(q * G + g) * 8 + slot] = vs;
            }
        }
        __syncthreads();
        if (uint8_t* const unit = unit_of(base)) store_block<D>(unit, t0, t1, s_kw, s_vc, s_sc[0], s_sc[1]);
        __syncthreads();
    }
}

template <int XT>
hipError_t append_dims(const KvView& c, const KvSeqs& sq, const void* k, int64_t k_ld, const void* v, int64_t v_ld, dim3 grid,
                       hipStream_t s) {
#define Q4GSW_KV_APPEND(D) \
    case D: hipLaunchKernelGGL((kv_append_kernel<XT, D>), grid, dim3(kThreads), 0, s, c, sq, k, k_ld, v, v_ld); break;
    switch (c.dim) {
        Q4GSW_KV_APPEND(64)
        Q4GSW_KV_APPEND(96)
        Q4GSW_KV_APPEND(128)
        Q4GSW_KV_APPEND(192)
        Q4GSW_KV_APPEND(256)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_KV_APPEND
    return hipGetLastError();
}

dim3 block_grid(const KvView& c, const KvSeqs& sq) {
    return dim3((unsigned)(sq.tokens / 32 + 2 * (int64_t)sq.batch), (unsigned)c.heads);
}

}  // namespace

hipError_t launch_kv_append(const KvView& c, const KvSeqs& sq, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                            int dtype, hipStream_t s) {
    const dim3 grid = block_grid(c, sq);
    switch (dtype) {
        case kF32: return append_dims<kF32>(c, sq, k, k_ld, v, v_ld, grid, s);
        case kF16: return append_dims<kF16>(c, sq, k, k_ld, v, v_ld, grid, s);
        default: return append_dims<kBF16>(c, sq, k, k_ld, v, v_ld, grid, s);
    }
}

hipError_t launch_kv_read(const KvView& c, const KvSeqs& sq, float* k, float* v, hipStream_t s) {
    const dim3 grid = block_grid(c, sq);
#define Q4GSW_KV_READ(D) \
    case D: hipLaunchKernelGGL((kv_read_kernel<D>), grid, dim3(kThreads), 0, s, c, sq, k, v); break;
    switch (c.dim) {
        Q4GSW_KV_READ(64)
        Q4GSW_KV_READ(96)
        Q4GSW_KV_READ(128)
        Q4GSW_KV_READ(192)
        Q4GSW_KV_READ(256)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_KV_READ
    return hipGetLastError();
}

hipError_t launch_kv_keep(const KvView* caches, int count, const KvSeqs& sq, const int32_t* parents, const int32_t* leaf,
                          int max_new, int32_t* kept, int32_t* path, hipStream_t s) {
    KeepArgs a{{}, caches[0], sq, parents, leaf, max_new, kept, path};
    for (int i = 0; i < count; ++i) a.data[i] = caches[i].data;
    const dim3 grid((unsigned)(sq.batch * caches[0].heads), (unsigned)count);
#define Q4GSW_KV_KEEP(D) \
    case D: hipLaunchKernelGGL((kv_keep_kernel<D>), grid, dim3(kThreads), 0, s, a); break;
    switch (caches[0].dim) {
        Q4GSW_KV_KEEP(64)
        Q4GSW_KV_KEEP(96)
        Q4GSW_KV_KEEP(128)
        Q4GSW_KV_KEEP(192)
        Q4GSW_KV_KEEP(256)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_KV_KEEP
    return hipGetLastError();
}

}  // namespace q4gsw
