// Low-rank adapters of many requests beside one projection (gfx950).
//
//   out[m] = y[m] + alpha_s (x[m] A_s^T) B_s^T,   s = slot[m];  A_s [rank, K], B_s [N, rank].
//
// A set holds its slots' factors in 16 bits, laid out when a slot is loaded for the matrix operands that
// read them (adapter_set.h), so odd ranks, widths and alignments cost nothing later.  Two launches:
//   * t[m] = x[m] A_s^T: a workgroup takes 16 rows, one or more of the adapters among them and 16 ranks;
//     its waves share K and add up in LDS.  Factors are the first operand of the 16x16x32 product, rows the
//     second.  Rows of other adapters are not loaded: they are zeros there, and their columns of the product are
//     not stored;
//   * out = y + alpha t B_s^T: factors as the first operand of the 16x16x16 product, so that a lane ends
//     with eight neighbouring columns of one row.  With few rows the waves of a workgroup share the adapters of
//     16 rows (a row is its adapter's wave's alone), with many they share the columns.
// Beside a linear whose K is split, the launch that sums the splits adds the terms (adapters_fwd, 64 rows of 32 adapters,
// K = 2048, N = 8192: 24 us against 27 with the sum in a launch of its own).
// Few rows of small factors take one launch, in which every workgroup of the second computes t itself.
// Rows need no order: adapters are found among each 16 rows by comparison, and one that many tiles share
// is read from L2 by all but the first.
//
// Bound: bytes of the factors and latency: 61 rows of 48 adapters, rank 32, K = 8192, N = 2048, fp32 rows, fp16 factors:
// 11.4 us (29 MB through L2, 18 from HBM) + 4.7 us; 64 rows of 32 adapters, rank 16, K = 2048, N = 8192: 5.4 us and the sum.  Prompts:
// the second launch's y, read and written: 2048 rows of 8192: 7.4 + 30 us for 134 MB.
//
// Numbers: products of 16-bit factors are exact in the matrix unit's fp32, so what rows and t lose on
// their way into 16-bit operands is all that is lost.  They enter as sums of parts: with bf16 factors one
// part of a bf16 row, two of fp16 (exact: 11 bits in 8 + 8), three of fp32 (exact: 24 in 3 x 8) and of t; with
// fp16 factors, after a power of two per row (and, in x, per 256 columns) that brings the largest value to
// 2^14, one part of an fp16 row (as it is) or bf16 row, two of fp32 and of t (22 bits of the largest).
#include "adapter_set.h"
#include "internal.h"
#include "kv_attention.h"   // row_factor, wave_max_rows

namespace q4gsw {
namespace {

// rows of y and out in memory, at the alignment of an element, which vector loads and stores take
typedef float f4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

template <int FT>
__device__ __forceinline__ f4 mfma32(u4 a, u4 b, f4 c) {
    if constexpr (FT == kF16) return mfma_f16(a, b, c);
    else return mfma_bf16(a, b, c);
}
// 16x16x16: lane l holds A[l % 16][4 (l / 16) + 0..3], B[4 (l / 16) + 0..3][l % 16]; D as in 16x16x32.
template <int FT>
__device__ __forceinline__ f4 mfma16(u2 a, u2 b, f4 c) {
    if constexpr (FT == kF16) return __builtin_amdgcn_mfma_f32_16x16x16f16(bitcast<h4>(a), bitcast<h4>(b), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(bitcast<s4v>(a), bitcast<s4v>(b), c, 0, 0, 0);
}

template <int FT, int XT>
constexpr int row_parts() {
    if (FT == XT) return 1;
    if (FT == kF16) return XT == kF32 ? 2 : 1;
    return XT == kF32 ? 3 : 2;
}

// v0 and v1 as one pair of a part, which is taken off them.
template <int FT>
__device__ __forceinline__ uint32_t take_part(float& v0, float& v1) {
    if constexpr (FT == kF16) {
        const h2 p = {(_Float16)v0, (_Float16)v1};
        v0 -= (float)p[0];
        v1 -= (float)p[1];
        return bitcast<uint32_t>(p);
    } else {
        const uint32_t p = bitcast<uint32_t>(b2{(__bf16)v0, (__bf16)v1});
        v0 -= bitcast<float>(p << 16);
        v1 -= bitcast<float>(p & 0xFFFF0000u);
        return p;
    }
}

// The adapters among 16 rows: `mine` is the slot of row lane % 16 (-1: none); bit i of the result: row i
// is the first of its adapter.
__device__ __forceinline__ int row_slot(const AdapterArgs& a, int64_t tile, int i) {
    const int64_t m = 16 * tile + i;
    const int s = m < a.M ? a.slot[m] : -1;
    return s >= 0 && s < a.set.slots ? s : -1;
}
__device__ __forceinline__ uint32_t first_rows(int mine, int i) {
    bool again = mine < 0;
#pragma unroll
    for (int j = 0; j < 15; ++j) again |= j < i && __builtin_amdgcn_readlane(mine, j) == mine;
    return (uint32_t)__ballot(!again) & 0xFFFFu;
}

// Columns k .. k + 7 of a row of x, as they lie in memory; zeros past K.
template <int XT, bool VEC>
struct Octet {
    u4 w[XT == kF32 ? 2 : 1];
    __device__ __forceinline__ void clear() {
        for (u4& v : w) v = u4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ void load(const void* x, int64_t row, int64_t k, int64_t K) {
        if constexpr (VEC && XT == kF32) {
            if (k < K) w[0] = ldg16(static_cast<const float*>(x) + row + k);
            if (k + 4 < K) w[1] = ldg16(static_cast<const float*>(x) + row + k + 4);
        } else if constexpr (VEC) {
            if (k < K) w[0] = ldg16(static_cast<const uint16_t*>(x) + row + k);
        } else if constexpr (XT == kF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) w[e >> 2][e & 3] = static_cast<const uint32_t*>(x)[row + k + e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) w[0][e >> 1] |= (uint32_t)static_cast<const uint16_t*>(x)[row + k + e] << (16 * (e & 1));
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (XT == kF32) return bitcast<float>(w[e >> 2][e & 3]);
        else if constexpr (XT == kF16) return (float)bitcast<h2>(w[0][e >> 1])[e & 1];
        else return bitcast<float>((e & 1) ? w[0][e >> 1] & 0xFFFF0000u : w[0][e >> 1] << 16);
    }
};

constexpr int kWaves = 8;                // of a workgroup, which share a chunk of K
constexpr int kMostChunks = 4;

// Steps [s0, s1) of 32 columns of t for 16 rows and 16 ranks: lane (i, q) gets ranks 4 q .. + 3 of row i, where
// `match`.  A: the adapter's runs of these ranks, `stride` bytes a step, at this lane.
template <int FT, int XT, bool VEC>
__device__ __forceinline__ f4 down_part(const AdapterArgs& a, const uint8_t* A, int64_t stride, int64_t row, bool match, int q,
                                        int64_t s0, int64_t s1) {
    constexpr int P = row_parts<FT, XT>();
    constexpr bool SCALED = FT == kF16 && XT != kF16;
    constexpr int kSteps = 8;                             // loaded together
    f4 sum = {0.f, 0.f, 0.f, 0.f};
    for (; s0 < s1; s0 += kSteps) {
        u4 av[kSteps];
        Octet<XT, VEC> xv[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            av[s] = u4{0u, 0u, 0u, 0u};
            xv[s].clear();
            if (s0 + s < s1) av[s] = ldg16(A + (s0 + s) * stride);
        }
        if (match) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                if (s0 + s < s1) xv[s].load(a.x, row, 32 * (s0 + s) + 8 * q, a.K);
        }
        float mul = 1.0f, inv = 1.0f;
        if constexpr (SCALED) {
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(xv[s][e]));
            row_factor(wave_max_rows(amax), mul, inv);
        }
        f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if constexpr (FT == XT) {
                acc = mfma32<FT>(av[s], xv[s].w[0], acc);
            } else {
                u4 part[P];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v0 = xv[s][2 * e], v1 = xv[s][2 * e + 1];
                    if constexpr (SCALED) {
                        v0 *= mul;
                        v1 *= mul;
                    }
#pragma unroll
                    for (int p = 0; p < P; ++p) part[p][e] = take_part<FT>(v0, v1);
                }
#pragma unroll
                for (int p = 0; p < P; ++p) acc = mfma32<FT>(av[s], part[p], acc);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = SCALED ? fmaf(acc[e], inv, sum[e]) : sum[e] + acc[e];
    }
    return sum;
}

// t of 16 rows, 16 ranks and a chunk of K: t[chunk][m][rank].
template <int FT, int XT, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void down_kernel(AdapterArgs a) {
    __shared__ f4 s_sum[kWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int64_t id = blockIdx.x;
    const int chunk = (int)(id % a.chunks);
    id /= a.chunks;
    const int rt = (int)(id % a.rank_tiles);
    id /= a.rank_tiles;
    const int group = (int)(id % a.groups);
    const int64_t tile = id / a.groups;
    const int mine = row_slot(a, tile, i);
    uint32_t firsts = first_rows(mine, i);
    const int64_t m = 16 * tile + i, row = m * a.K;
    // the waves from a.share on have none of it, so that one launch for few rows, whose waves share K alike, sums in the same order
    const int64_t steps = a.set.k_pad >> 5, parts = a.chunks * a.share, per = (steps + parts - 1) / parts;
    const int64_t begin = wave < a.share ? per * (chunk * a.share + wave) : steps, s1 = min(begin + per, steps);
    for (int n = 0; firsts; firsts &= firsts - 1, ++n) {
        if (n % a.groups != group) continue;
        const int slot = __builtin_amdgcn_readlane(mine, __builtin_ctz(firsts));
        const bool match = mine == slot;
        const uint8_t* A = a.set.data + slot * a.set.slot_bytes + 1024 * (int64_t)rt + 16 * lane;
        s_sum[wave][lane] = down_part<FT, XT, VEC>(a, A, 1024 * (int64_t)a.rank_tiles, row, match, q, begin, s1);
        __syncthreads();
        if (tid < 256) {
            const int l = tid >> 2, e = tid & 3, ri = l & 15;
            float t = s_sum[0][l][e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) t += s_sum[w][l][e];
            if (__shfl(mine, ri) == slot) a.t[(chunk * a.M + 16 * tile + ri) * (16 * a.rank_tiles) + 16 * rt + 4 * (l >> 4) + e] = t;
        }
        __syncthreads();
    }
}

// t of row m, ranks 16 s + 4 q .. + 3: its chunks in order.
template <int S>
__device__ __forceinline__ void row_terms(const AdapterArgs& a, int64_t m, int q, f4 (&tv)[S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const float* t = a.t + m * (16 * S) + 16 * s + 4 * q;
        f4 v[kMostChunks];
#pragma unroll
        for (int c = 0; c < kMostChunks; ++c) v[c] = *reinterpret_cast<const f4*>(t + min(c, a.chunks - 1) * a.M * (16 * S));
        tv[s] = v[0];
#pragma unroll
        for (int c = 1; c < kMostChunks; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) tv[s][e] += c < a.chunks ? v[c][e] : 0.0f;
    }
}

// alpha t as the parts of an operand; the factor that the products take then (fp16 factors).
template <int FT, int S, int P>
__device__ __forceinline__ float term_parts(f4 (&tv)[S], float alpha, u2 (&part)[S][P]) {
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tv[s][e] *= alpha;
            amax = fmaxf(amax, fabsf(tv[s][e]));
        }
    float mul = 1.0f, inv = 1.0f;
    if constexpr (FT == kF16) row_factor(wave_max_rows(amax), mul, inv);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v0 = tv[s][2 * e] * mul, v1 = tv[s][2 * e + 1] * mul;
#pragma unroll
            for (int p = 0; p < P; ++p) part[s][p][e] = take_part<FT>(v0, v1);
        }
    return inv;
}

// out = y + alpha t B^T for 16 rows, S steps of 16 ranks.  kMany: 256 columns, 64 a wave.  kFew: 32 J columns,
// the adapters of the rows dealt to the waves.  kOne: as kFew, of one tile of rows, and t is computed here, by every
// workgroup once more (XT: the rows' type, which the others do not look at).
enum UpKind { kFew, kMany, kOne };
template <int FT, int S, UpKind KIND, int XT>
__global__ __launch_bounds__(KIND == kOne ? 64 * kWaves : 256) void up_kernel(AdapterArgs a) {
    constexpr bool MANY = KIND == kMany;
    constexpr int NW = KIND == kOne ? kWaves : 4;
    constexpr int J = MANY || S == 1 ? 2 : 1;             // blocks of 32 columns a wave
    constexpr int kBatch = MANY ? 1 : 4;                  // adapters whose factors are loaded together
    constexpr int P = FT == kF16 ? 2 : 3;
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t tile = blockIdx.x / a.col_groups, m = 16 * tile + i;
    const int64_t blk0 = (int64_t)(blockIdx.x % a.col_groups) * (MANY ? 4 * J : J) + (MANY ? wave * J : 0);
    const int64_t blocks = a.set.n_pad >> 5;
    if (MANY && blk0 >= blocks) return;
    const int mine = row_slot(a, tile, i);
    uint32_t firsts = first_rows(mine, i);
    bool here = m < a.M && (mine >= 0 || a.y != a.out);   // rows that this wave writes
    if constexpr (!MANY) {
        uint32_t left = firsts;
        firsts = 0;
        here = here && mine < 0 && wave == 0;
        for (int n = 0; left; left &= left - 1, ++n) {
            if (n % NW != wave) continue;
            firsts |= left & (0u - left);
            here |= mine == __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        }
        if (KIND != kOne && !__any(here)) return;
    }

    // ---- what the columns hold so far and the first factors: on their way while t is computed ----
    const float alpha = mine >= 0 ? a.set.alpha[mine] : 0.0f;
    f4 acc[J][2], base[J][2];
    auto col = [&](int j, int h) -> int64_t { return 32 * (blk0 + j) + 8 * q + 4 * h; };
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            acc[j][h] = base[j][h] = f4{0.f, 0.f, 0.f, 0.f};
            const int64_t n = col(j, h);
            if (here) {
                if (n + 4 <= a.N) {
                    base[j][h] = *reinterpret_cast<const f4_at4*>(a.y + m * a.N + n);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < a.N) base[j][h][e] = a.y[m * a.N + n + e];
                }
            }
        }
    u4 b[kBatch][J][S];
    int slot[kBatch];
    auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            slot[k] = -1;
            if (!firsts) continue;
            slot[k] = __builtin_amdgcn_readlane(mine, __builtin_ctz(firsts));
            firsts &= firsts - 1;
            const uint8_t* B = a.set.data + slot[k] * a.set.slot_bytes + a.set.b_offset + 16 * lane;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (blk0 + j < blocks) b[k][j][s] = ldg16(B + ((blk0 + j) * S + s) * 1024);
        }
    };
    fetch();

    // ---- t ----
    f4 tv[S];
#pragma unroll
    for (int s = 0; s < S; ++s) tv[s] = f4{0.f, 0.f, 0.f, 0.f};
    if constexpr (KIND == kOne) {
        // a.share waves take one adapter's K, the others the next adapters'
        __shared__ f4 s_t[kWaves][S][64];
        const int ways = kWaves / a.share, way = wave / a.share;
        const int64_t steps = a.set.k_pad >> 5, per = (steps + a.share - 1) / a.share, begin = per * (wave % a.share);
        int first = 0;
#pragma unroll
        for (int j = 15; j >= 0; --j) first = __builtin_amdgcn_readlane(mine, j) == mine ? j : first;
        uint32_t left = first_rows(mine, i);
        int order = mine >= 0 ? __popc(left & ((1u << first) - 1u)) : -1;     // of the row's adapter
        for (; left; order -= ways) {
            uint32_t one = 0u;                                // the wave's adapter of this turn
            for (int w = 0; w < ways; ++w) {
                const uint32_t low = left & (0u - left);
                one = w == way ? low : one;
                left ^= low;
            }
            if (one) {
                const int slot = __builtin_amdgcn_readlane(mine, __builtin_ctz(one));
                const uint8_t* A = a.set.data + slot * a.set.slot_bytes + 16 * lane;
#pragma unroll
                for (int s = 0; s < S; ++s)
                    s_t[wave][s][lane] = down_part<FT, XT, true>(a, A + 1024 * s, 1024 * S, m * a.K, mine == slot, q, begin, min(begin + per, steps));
            }
            __syncthreads();
            if (order >= 0 && order < ways) {
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    tv[s] = s_t[order * a.share][s][lane];
                    for (int w = 1; w < a.share; ++w)
#pragma unroll
                        for (int e = 0; e < 4; ++e) tv[s][e] += s_t[order * a.share + w][s][lane][e];
                }
            }
            __syncthreads();
        }
        if (!__any(here)) return;
    } else if (here && mine >= 0) {
        row_terms<S>(a, m, q, tv);
    }
    u2 part[S][P];
    const float inv = term_parts<FT, S, P>(tv, alpha, part);

    for (; slot[0] >= 0; fetch()) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (slot[k] < 0) break;
            // a row's products are its own column: rows of other adapters are left as they are, whatever
            // this one's factors hold
            const bool match = mine == slot[k];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (blk0 + j >= blocks) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int p = 0; p < P; ++p) d = mfma16<FT>(u2{b[k][j][s][2 * h], b[k][j][s][2 * h + 1]}, part[s][p], d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][h][e] = match ? d[e] : acc[j][h][e];
                }
            }
        }
    }
    if (!here) return;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = col(j, h);
            f4 v = base[j][h];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = FT == kF16 ? fmaf(acc[j][h][e], inv, v[e]) : v[e] + acc[j][h][e];
            if (n + 4 <= a.N) {
                *reinterpret_cast<f4_at4*>(a.out + m * a.N + n) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < a.N) a.out[m * a.N + n + e] = v[e];
            }
        }
}

// The sums of a projection's K splits and the adapters' terms in one launch: a workgroup takes a 32x32 tile of
// the partials (fragment layout, internal.h), a wave 16 rows and half the columns of it.  Roles are swapped against
// up_kernel: t is the first operand, so that a lane ends with four rows of one column, as the partials lie.
template <int FT, int S>
__global__ __launch_bounds__(256) void join_kernel(AdapterArgs a, const float* __restrict__ part, int splits, int64_t ntn,
                                                   int64_t plane) {
    constexpr int P = FT == kF16 ? 2 : 3;
    constexpr int kBatch = 8 / S > 2 ? 8 / S : 2;         // adapters whose factors are loaded together
    constexpr int kPlanes = 4;                            // partials loaded together
    __shared__ float s_tile[32][33];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), mh = wave >> 1, h = wave & 1;
    const int64_t tm = blockIdx.x / ntn, tn = blockIdx.x % ntn;
    if (32 * tn >= a.N) return;                           // columns that only the packed weight has
    const float* src = part + (int64_t)blockIdx.x * 1024 + 4 * (64 * (2 * mh + (q >> 1)) + 32 * (q & 1) + adapter_col(i, h));
    f4 p[kPlanes];
#pragma unroll
    for (int k = 0; k < kPlanes; ++k) p[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(src + (k < splits ? k : 0) * plane));

    const int64_t m = 32 * tm + 16 * mh + i;
    const int mine = row_slot(a, 2 * tm + mh, i);
    uint32_t firsts = first_rows(mine, i);
    f4 tv[S];
    float alpha = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) tv[s] = f4{0.f, 0.f, 0.f, 0.f};
    if (mine >= 0) {
        row_terms<S>(a, m, q, tv);
        alpha = a.set.alpha[mine];
    }
    u2 b[kBatch][S];
    int slot[kBatch];
    auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            slot[k] = -1;
            if (!firsts) continue;
            slot[k] = __builtin_amdgcn_readlane(mine, __builtin_ctz(firsts));
            firsts &= firsts - 1;
            const uint8_t* B = a.set.data + slot[k] * a.set.slot_bytes + a.set.b_offset + tn * S * 1024 + 16 * lane + 8 * h;
#pragma unroll
            for (int s = 0; s < S; ++s) b[k][s] = *reinterpret_cast<const u2*>(B + 1024 * s);
        }
    };
    fetch();

    f4 sum = p[0];
#pragma unroll
    for (int k = 1; k < kPlanes; ++k)
        if (k < splits) sum += p[k];
    for (int s0 = kPlanes; s0 < splits; s0 += kPlanes) {
#pragma unroll
        for (int k = 0; k < kPlanes; ++k)
            p[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(src + (s0 + k < splits ? s0 + k : 0) * plane));
#pragma unroll
        for (int k = 0; k < kPlanes; ++k)
            if (s0 + k < splits) sum += p[k];
    }

    u2 parts[S][P];
    const float inv = term_parts<FT, S, P>(tv, alpha, parts);
    int of[4];                                            // slots of the lane's rows
#pragma unroll
    for (int e = 0; e < 4; ++e) of[e] = __shfl(mine, 4 * q + e);
    f4 acc = {0.f, 0.f, 0.f, 0.f};
    for (; slot[0] >= 0; fetch()) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (slot[k] < 0) break;
            f4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int e = 0; e < P; ++e) d = mfma16<FT>(parts[s][e], b[k][s], d);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = of[e] == slot[k] ? d[e] : acc[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float f = FT == kF16 ? __shfl(inv, 4 * q + e) : 1.0f;
        s_tile[16 * mh + 4 * q + e][adapter_col(i, h)] = of[e] < 0 ? sum[e] : (FT == kF16 ? fmaf(acc[e], f, sum[e]) : sum[e] + acc[e]);
    }
    __syncthreads();
    const int row = tid >> 3, c4 = 4 * (tid & 7);
    const int64_t mo = 32 * tm + row, n = 32 * tn + c4;
    if (mo >= a.M) return;
    float* dst = a.out + mo * a.N + n;
    if (n + 4 <= a.N) {
        *reinterpret_cast<f4_at4*>(dst) = f4_at4{s_tile[row][c4], s_tile[row][c4 + 1], s_tile[row][c4 + 2], s_tile[row][c4 + 3]};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) dst[e] = s_tile[row][c4 + e];
    }
}

// One slot's factors into the set, 16 bytes a thread, and its alpha; zeros past rank, K and N.
template <int FT, int ST>
__global__ __launch_bounds__(256) void load_kernel(AdapterSet set, int slot, const void* A, const void* B, int rank, float alpha) {
    const int64_t R = set.rank_tiles, a_units = set.k_pad / 32 * R * 64, b_units = set.n_pad / 32 * R * 64;
    uint8_t* const base = set.data + slot * set.slot_bytes;
    for (int64_t u = blockIdx.x * 256 + threadIdx.x; u < a_units + b_units; u += (int64_t)gridDim.x * 256) {
        const bool b = u >= a_units;
        const int64_t v = b ? u - a_units : u;
        const int lane = (int)(v & 63), i = lane & 15, q = lane >> 4;
        const int64_t tile = (v >> 6) % R, at = (v >> 6) / R;           // at: step of 32 columns, or block of 32 outputs
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (b) {
                const int64_t n = 32 * at + adapter_col(i, e >> 2), r = 16 * tile + 4 * q + (e & 3);
                f[e] = n < set.N && r < rank ? load_elem<ST>(B, n * rank + r) : 0.0f;
            } else {
                const int64_t r = 16 * tile + i, k = 32 * at + 8 * q + e;
                f[e] = k < set.K && r < rank ? load_elem<ST>(A, r * set.K + k) : 0.0f;
            }
        }
        u4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (FT == kF16) w[e] = bitcast<uint32_t>(h2{(_Float16)f[2 * e], (_Float16)f[2 * e + 1]});
            else w[e] = bitcast<uint32_t>(b2{(__bf16)f[2 * e], (__bf16)f[2 * e + 1]});
        }
        *reinterpret_cast<u4*>(base + (b ? set.b_offset : 0) + 16 * v) = w;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) set.alpha[slot] = alpha;
}

template <int FT, int XT>
hipError_t down_launch(const AdapterArgs& a, bool vec, dim3 grid, dim3 block, hipStream_t s) {
    if (vec) hipLaunchKernelGGL((down_kernel<FT, XT, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((down_kernel<FT, XT, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int FT>
hipError_t up_launch(const AdapterArgs& a, bool many, dim3 grid, hipStream_t s) {
#define Q4GSW_UP(S)                                                                                   \
    case S:                                                                                           \
        if (many) hipLaunchKernelGGL((up_kernel<FT, S, kMany, kF32>), grid, dim3(256), 0, s, a);      \
        else hipLaunchKernelGGL((up_kernel<FT, S, kFew, kF32>), grid, dim3(256), 0, s, a);            \
        break;
    switch (a.rank_tiles) {
        Q4GSW_UP(1)
        Q4GSW_UP(2)
        Q4GSW_UP(3)
        Q4GSW_UP(4)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_UP
    return hipGetLastError();
}

template <int FT, int XT>
hipError_t one_launch(const AdapterArgs& a, dim3 grid, hipStream_t s) {
    if (a.rank_tiles == 1) hipLaunchKernelGGL((up_kernel<FT, 1, kOne, XT>), grid, dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((up_kernel<FT, 2, kOne, XT>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

// How a call's work is cut.  Adapters of a tile of single tokens are all unlike, those of long prompts
// mostly one: up to 256 rows every one has workgroups of its own, beyond that two share them: the host cannot tell
// which it has, and more workgroups than adapters cost prompts what fewer cost single tokens (us, 16 of them a tile / two,
// K = N = 2048, rank 16, bf16: 257 rows of 32 adapters in no order 11.6 / 20.9, 512 rows 14.7 / 22.8, 2048 rows 39 / 34;
// prompts of four adapters 10.4 / 9.8, 12.4 / 10.2, 36 / 17).  A chunk is 2048 columns, so that a wave has all of its loads on their way at once or twice, unless rows fill the GPU.
struct Cut {
    int64_t tiles;
    int chunks, groups;
    bool many, one;                      // the column groups are up_kernel's: kMany, else kFew and, if one launch may do, kOne
    int64_t col_groups;
};
Cut cut_of(const AdapterSet& set, int64_t M) {
    Cut c;
    c.tiles = (M + 15) / 16;
    const int64_t steps = set.k_pad / 32;
    c.many = c.tiles * ((set.N + 255) / 256) >= 1024;
    const int cols = c.many ? 256 : (set.rank_tiles == 1 ? 64 : 32);
    c.col_groups = (set.N + cols - 1) / cols;
    // One launch, in which every workgroup computes t again, where that costs less than the other launch: up to 128 KB of factors, read
    // by at most one workgroup a CU (us in one launch / two, bf16, rank 16: K = 2048 and N up to 16384, 1 row 5.8 / 7.7, 2 rows 7.7 / 8.0,
    // 4 rows, 256 KB, 11.5 / 8.5; 16 rows of K = 256 8.8 / 10.0, of 512 11.7 / 10.0; 1 row of K = 8192 8.5 / 7.8; 1 row of K = 2048 and
    // N = 20000, two workgroups on some CUs, 9.7 / 7.9, N = 131072 33 / 10).  So few groups of so few rows are never kMany's.
    c.one = c.col_groups <= 256 && M <= 16 && set.rank_tiles <= 2 && M * set.rank_tiles * 32 * set.k_pad <= (128 << 10);
    // rows of x that one launch cannot load, since they are not aligned, are summed in its order: one chunk
    c.chunks = (int)(c.one || c.tiles >= 1024 || steps <= 64 ? 1 : (steps >= 64 * kMostChunks ? kMostChunks : (steps + 63) / 64));
    c.groups = M <= 256 ? (int)(M < 16 ? M : 16) : 2;
    return c;
}

}  // namespace

bool adapters_launch_ok(const AdapterSet& set, int64_t M) {
    const Cut c = cut_of(set, M);
    // threads of a grid; one launch for all, whose workgroups are twice as large, has at most 256 of them
    const int64_t most = (int64_t(1) << 32) - 1;
    return c.tiles * c.groups * set.rank_tiles <= most / (64 * kWaves * c.chunks) && c.tiles <= most / 256 / c.col_groups;
}

uint64_t adapters_ws_bytes(const AdapterSet& set, int64_t M) {
    return (uint64_t)cut_of(set, M).chunks * M * 16 * set.rank_tiles * 4;
}

hipError_t launch_adapters_load(const AdapterSet& set, int slot, const void* A, const void* B, int src_dtype, int rank, float alpha,
                                hipStream_t s) {
    const int64_t units = (set.k_pad + set.n_pad) / 32 * set.rank_tiles * 64;
    const int64_t want = (units + 255) / 256;
    const dim3 grid((unsigned)(want < 4096 ? want : 4096));
#define Q4GSW_LOAD(FT, ST) hipLaunchKernelGGL((load_kernel<FT, ST>), grid, dim3(256), 0, s, set, slot, A, B, rank, alpha)
    if (set.dtype == kF16) {
        if (src_dtype == kF32) Q4GSW_LOAD(kF16, kF32);
        else if (src_dtype == kF16) Q4GSW_LOAD(kF16, kF16);
        else Q4GSW_LOAD(kF16, kBF16);
    } else {
        if (src_dtype == kF32) Q4GSW_LOAD(kBF16, kF32);
        else if (src_dtype == kF16) Q4GSW_LOAD(kBF16, kF16);
        else Q4GSW_LOAD(kBF16, kBF16);
    }
#undef Q4GSW_LOAD
    return hipGetLastError();
}

namespace {

AdapterArgs args_of(const AdapterSet& set, const Cut& c, const void* x, int64_t M, const int32_t* slot, const float* y, float* out,
                    void* t) {
    AdapterArgs a{set, x, M, set.K, set.N, slot, y, out, static_cast<float*>(t), c.chunks, c.groups, set.rank_tiles, c.col_groups, kWaves};
    // a wave has the loads of 8 steps on their way at once
    const int64_t steps = set.k_pad >> 5;
    a.share = steps <= 8 ? 1 : (steps <= 16 ? 2 : (steps <= 32 ? 4 : kWaves));
    return a;
}

// rows of x hold aligned octets
bool octets(const AdapterSet& set, const void* x, int x_dtype) {
    return (set.K * (x_dtype == kF32 ? 4 : 2)) % 16 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
}

hipError_t launch_down(const AdapterArgs& a, const Cut& c, int x_dtype, hipStream_t s) {
    const dim3 down((unsigned)(c.tiles * c.groups * a.rank_tiles * c.chunks)), block(64 * kWaves);
    const bool vec = octets(a.set, a.x, x_dtype);
#define Q4GSW_DOWN(FT)                                                                                        \
    (x_dtype == kF32 ? down_launch<FT, kF32>(a, vec, down, block, s)                                          \
                     : (x_dtype == kF16 ? down_launch<FT, kF16>(a, vec, down, block, s) : down_launch<FT, kBF16>(a, vec, down, block, s)))
    return a.set.dtype == kF16 ? Q4GSW_DOWN(kF16) : Q4GSW_DOWN(kBF16);
#undef Q4GSW_DOWN
}

template <int FT>
hipError_t join_launch(const AdapterArgs& a, const float* part, int splits, int64_t width, hipStream_t s) {
    const dim3 grid((unsigned)((a.M + 31) / 32 * (width / 32)));
    const int64_t plane = frag_plane_floats(a.M, width);
#define Q4GSW_JOIN(S) \
    case S: hipLaunchKernelGGL((join_kernel<FT, S>), grid, dim3(256), 0, s, a, part, splits, width / 32, plane); break;
    switch (a.rank_tiles) {
        Q4GSW_JOIN(1)
        Q4GSW_JOIN(2)
        Q4GSW_JOIN(3)
        Q4GSW_JOIN(4)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_JOIN
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters_add(const AdapterSet& set, const void* x, int x_dtype, int64_t M, const int32_t* slot, const float* y,
                               float* out, void* ws, hipStream_t s) {
    const Cut c = cut_of(set, M);
    const AdapterArgs a = args_of(set, c, x, M, slot, y, out, ws);
    const dim3 up((unsigned)(c.tiles * c.col_groups));
    if (c.one && octets(set, x, x_dtype)) {
#define Q4GSW_ONE(FT) \
    (x_dtype == kF32 ? one_launch<FT, kF32>(a, up, s) : (x_dtype == kF16 ? one_launch<FT, kF16>(a, up, s) : one_launch<FT, kBF16>(a, up, s)))
        return set.dtype == kF16 ? Q4GSW_ONE(kF16) : Q4GSW_ONE(kBF16);
#undef Q4GSW_ONE
    }
    const hipError_t e = launch_down(a, c, x_dtype, s);
    if (e != hipSuccess) return e;
    return set.dtype == kF16 ? up_launch<kF16>(a, c.many, up, s) : up_launch<kBF16>(a, c.many, up, s);
}

hipError_t launch_adapters_join(const AdapterSet& set, const void* x, int x_dtype, int64_t M, const int32_t* slot, const float* part,
                                int splits, int64_t width, float* out, void* t, hipStream_t s) {
    const Cut c = cut_of(set, M);
    const AdapterArgs a = args_of(set, c, x, M, slot, out, out, t);
    const hipError_t e = launch_down(a, c, x_dtype, s);
    if (e != hipSuccess) return e;
    return set.dtype == kF16 ? join_launch<kF16>(a, part, splits, width, s) : join_launch<kBF16>(a, part, splits, width, s);
}

}  // namespace q4gsw
