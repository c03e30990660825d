// Attention of few rows (single tokens, drafts) over the 4-bit cache.
//
//   score[r, t] = q[r] . k[t] / sqrt(dim) (optionally cap tanh(score / cap)), t <= place of r,
//   t > place - window;  out[r] = sum_t softmax(score)[r, t] v[t].
//
// Rows are the new tokens of one sequence times the query heads of one head of the cache.  Every
// wave works alone on 32-token blocks: 4 KB of codes and 0.5 KB of scales per block (dim 128)
// come straight from memory into the lanes that use them, 16 bytes a lane, one block ahead.
//   * scores: 16x16x32 MFMA, keys as the first operand, so a lane holds the scores of eight
//     tokens of one row.  With one tile of rows (R 1) the keys' codes enter as fp16 code + bias,
//     unpacked by 5 VALU a word; the product starts from -bias * sum(q) and every run of 32
//     channels is one MFMA, whose fp32 sum is multiplied by the token's scale: exact products.
//     With two tiles that multiplication would double, and the scale is multiplied into the
//     unpacked fp16 codes instead (one rounding, 2^-11).
//   * weights: running reference and sum of a softmax in fp32; the reference moves only when some
//     score passes it by kSlack, so most blocks need no exchange between lanes and no rescaling.
//   * sums: 16x16x32 MFMA, values (code - 8) * scale in fp16 (one rounding) as the first operand;
//     the weights, rounded to fp16, are the second operand as the lane holds them.
// The waves of a workgroup join through LDS at the end; splits of the cache's length join in a
// second launch (kv_join_kernel).
//
// Bound: HBM for long caches (36 * dim bytes per 32 tokens and head).
#include "kv_attention.h"

namespace q4gsw {
namespace {

template <int G, int R>
struct Block {
    uint32_t k[2 * G], v[2 * G];
    uint32_t ks[R == 1 ? 4 * G : G];
    uint32_t vs[4 * G];
};

// Words 0 .. 2 G - 1 of this lane.
template <int G>
__device__ __forceinline__ void load_plane(const uint8_t* p, int lane, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
        const u4 x = ldg16(p + 1024 * i + 16 * lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = x[e];
    }
    if constexpr (G & 1) {
        const u2 x = *reinterpret_cast<const u2*>(p + 512 * (G - 1) + 8 * lane);
        w[2 * G - 2] = x[0];
        w[2 * G - 1] = x[1];
    }
}

template <int G, int R>
__device__ __forceinline__ void load_block(const uint8_t* unit, int lane, Block<G, R>& b) {
    const int i = lane & 15, q = lane >> 4;
    load_plane<G>(unit, lane, b.k);
    const uint8_t* sc = unit + 1024 * G;
    if constexpr (R == 1) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const u4 x = ldg16(sc + 16 * G * q + 16 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) b.ks[4 * g + e] = x[e];
        }
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) b.ks[g] = *reinterpret_cast<const uint32_t*>(sc + 4 * G * i + 4 * g);
    }
    load_plane<G>(unit + 512 * G, lane, b.v);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const u4 x = ldg16(sc + 64 * G + 16 * G * q + 16 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) b.vs[4 * g + e] = x[e];
    }
}

template <int D, int R>
__global__ __launch_bounds__(512) void kv_rows_kernel(KvAttnArgs a) {
    constexpr int G = D / 32, C = D / 16;
    extern __shared__ __attribute__((aligned(16))) float smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int i = lane & 15, qd = lane >> 4;

    int id = blockIdx.x;
    const int split = id % a.splits;
    id /= a.splits;
    const int head = id % a.c.heads;
    id /= a.c.heads;
    const int b = id % a.sq.batch;
    const int rt0 = id / a.sq.batch;

    const KvSeq s = kv_seq(a.sq, b);
    const int rows = min(s.m, a.max_new) * a.group;
    const int r0 = rt0 * 16 * R;
    if (r0 >= rows) return;
    const int nr = min(16 * R, rows - r0);
    const KvSpan sp = kv_span(a, s, r0, nr, split);

    // ---- queries: operand fragments, factors, places ----
    u4 bq[R][G];
    float cb[R == 1 ? G : 1];            // R 1: -bias * sum of the run's queries
    float f[R];
    int pr[R];
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const int r = r0 + 16 * rt + i;
        const bool ok = r < rows;
        const int tok = ok ? r / a.group : 0, gh = ok ? r - tok * a.group : 0;
        pr[rt] = ok ? s.len - s.m + tok : sp.pmax;
        const int64_t base = (s.first_row + tok) * a.q_ld + (int64_t)(head * a.group + gh) * D;
        float x[8 * G];
        float amax = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            load_q8(a.q, a.dtype, base + 32 * g + 8 * qd, x + 8 * g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[8 * g + e] = ok ? x[8 * g + e] : 0.0f;
                amax = fmaxf(amax, fabsf(x[8 * g + e]));
            }
        }
        amax = wave_max_rows(amax);
        float mul, inv;
        row_factor(amax, mul, inv);
        f[rt] = a.scale * inv;
        if (a.cap_out == 0.0f) f[rt] *= kLog2e;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const h2 p = {(_Float16)(x[8 * g + 2 * e] * mul), (_Float16)(x[8 * g + 2 * e + 1] * mul)};
                bq[rt][g][e] = bitcast<uint32_t>(p);
                if constexpr (R == 1) sum += ((float)p[0] + (float)p[1]) * ((e & 1) ? kBiasOdd : kBiasEven);
            }
            if constexpr (R == 1) cb[g] = -wave_sum_rows(sum);
        }
    }

    f4 o[R][C];
    float mref[R], l[R];
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        mref[rt] = kNoKey;
        l[rt] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) o[rt][c] = f4{0.f, 0.f, 0.f, 0.f};
    }

    auto compute = [&](const Block<G, R>& bl, int64_t blk) {
        f4 sc[R][2];
        if constexpr (R == 1) {
#pragma unroll
            for (int ab = 0; ab < 2; ++ab) {
                sc[0][ab] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const f4 p = mfma_f16(codes_biased_f16(bl.k[2 * g + ab]), bq[0][g], f4{cb[g], cb[g], cb[g], cb[g]});
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const h2 ks = bitcast<h2>(bl.ks[j * G + g]);
                        sc[0][ab][j] = fmaf((float)ks[ab], p[j], sc[0][ab][j]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int ab = 0; ab < 2; ++ab) {
#pragma unroll
                for (int rt = 0; rt < R; ++rt) sc[rt][ab] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const h2 ks = bitcast<h2>(bl.ks[g]);
                    const h2 kk = {ks[ab], ks[ab]};
                    const u4 kf = codes_scaled_f16(bl.k[2 * g + ab], kk, kk, kk, kk);
#pragma unroll
                    for (int rt = 0; rt < R; ++rt) sc[rt][ab] = mfma_f16(kf, bq[rt][g], sc[rt][ab]);
                }
            }
        }
        const int t0 = (int)(32 * blk);
        const int tl = t0 + 16 * (qd >> 1) + 4 * (qd & 1);     // + 8 ab + j
        const bool edge = t0 + 31 > sp.pmin || (a.window && t0 <= sp.pmax - a.window);
        const bool tail = t0 + 32 > s.len;
        u4 pw[R];
#pragma unroll
        for (int rt = 0; rt < R; ++rt) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = sc[rt][e >> 2][e & 3];
            float fl = f[rt];
            if (a.cap_out != 0.0f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = capped_log2(x[e] * fl, a.cap_in, a.cap_out);
                fl = 1.0f;
            }
            if (edge) {
                const int last = pr[rt], gone = a.window ? pr[rt] - a.window : -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = tl + 8 * (e >> 2) + (e & 3);
                    x[e] = t <= last && t > gone ? x[e] : -INFINITY;
                }
            }
            float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * fl;
            if (__any(mx > mref[rt] + kSlack)) {
                const float mn = fmaxf(mref[rt], wave_max_rows(mx));
                const float w = __builtin_amdgcn_exp2f(mref[rt] - mn);
                mref[rt] = mn;
                l[rt] *= w;
#pragma unroll
                for (int c = 0; c < C; ++c) o[rt][c] *= w;
            }
            const float off = kLift - mref[rt];
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(x[e], fl, off));
            l[rt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
            for (int e = 0; e < 4; ++e) pw[rt][e] = bitcast<uint32_t>(h2{(_Float16)p[2 * e], (_Float16)p[2 * e + 1]});
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t vs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) vs[e] = bl.vs[4 * g + e];
            if (tail) {                  // places past the length may hold anything: their values count as 0
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tl + 8 * (e >> 1) + 2 * (e & 1);
                    vs[e] = t + 1 < s.len ? vs[e] : (t < s.len ? vs[e] & 0xFFFFu : 0u);
                }
            }
#pragma unroll
            for (int c = 2 * g; c < 2 * g + 2; ++c) {
                const u4 vf = codes_scaled_f16(bl.v[c], bitcast<h2>(vs[0]), bitcast<h2>(vs[1]), bitcast<h2>(vs[2]),
                                               bitcast<h2>(vs[3]));
#pragma unroll
                for (int rt = 0; rt < R; ++rt) o[rt][c] = mfma_f16(vf, pw[rt], o[rt][c]);
            }
        }
    };

    // ---- the wave's blocks: lo + wave, + waves, ...; page numbers 64 at a time in a register ----
    const int64_t first = sp.lo + wave;
    const int64_t left = sp.hi - first;
    const int64_t n = left > 0 ? (left + waves - 1) / waves : 0;
    const int sub_mask = (1 << a.c.bpp_log2) - 1;
    int pages = -1;
    auto fetch = [&](int64_t it, Block<G, R>& bl) -> bool {
        if (it >= n) return false;
        const int64_t blk = first + it * waves;
        if ((it & 63) == 0) {
            const int64_t mine = first + (it + lane) * waves;
            pages = mine < sp.hi ? a.sq.table[(int64_t)b * a.sq.table_ld + (mine >> a.c.bpp_log2)] : -1;
        }
        const int page = __builtin_amdgcn_readlane(pages, (int)(it & 63));
        if (page < 0 || page >= a.c.pages) return false;
        load_block<G, R>(a.c.data + kv_unit(a.c, page, head, (int)(blk & sub_mask)), lane, bl);
        return true;
    };
    Block<G, R> b0, b1;
    bool h0 = fetch(0, b0);
    for (int64_t it = 0; it < n; it += 2) {
        const bool h1 = fetch(it + 1, b1);
        if (h0) compute(b0, first + it * waves);
        h0 = fetch(it + 2, b0);
        if (h1) compute(b1, first + (it + 1) * waves);
    }

    // ---- join the waves, one tile of 16 rows after the other ----
    float* const s_ml = smem;                                // [waves][16][2]
    float* const s_o = smem + 32 * waves;                    // [waves][rows of a tile][D + 4]
    const int tile_rows = min(16, a.max_new * a.group);
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const int nt = min(16, nr - 16 * rt);
        if (nt <= 0) break;
        if (rt) __syncthreads();
        const float lsum = wave_sum_rows(l[rt]);
        if (qd == 0) {
            s_ml[2 * (16 * wave + i)] = mref[rt];
            s_ml[2 * (16 * wave + i) + 1] = lsum;
        }
        if (i < nt) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                *reinterpret_cast<f4*>(&s_o[(wave * tile_rows + i) * (D + 4) + 16 * c + 4 * qd]) = o[rt][c];
        }
        __syncthreads();
        for (int e = tid; e < nt * (D / 4); e += blockDim.x) {
            const int row = e / (D / 4), c4 = e - row * (D / 4);
            float m = kNoKey;
            for (int w = 0; w < waves; ++w) m = fmaxf(m, s_ml[2 * (16 * w + row)]);
            float ls = 0.0f;
            f4 acc = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < waves; ++w) {
                const float wt = __builtin_amdgcn_exp2f(s_ml[2 * (16 * w + row)] - m);
                ls = fmaf(wt, s_ml[2 * (16 * w + row) + 1], ls);
                acc += wt * *reinterpret_cast<const f4*>(&s_o[(w * tile_rows + row) * (D + 4) + 4 * c4]);
            }
            const int r = r0 + 16 * rt + row, tok = r / a.group;
            const int64_t orow = (s.first_row + tok) * a.hq + head * a.group + (r - tok * a.group);
            if (a.splits == 1) {
                // a row that no key is seen by has a sum of exactly 0 and gives zeros
                const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                store4(a.out, a.dtype, orow * D + 4 * c4, acc * inv);
            } else {
                const int64_t prow = (int64_t)split * a.sq.tokens * a.hq + orow;
                *reinterpret_cast<f4*>(a.part + prow * D + 4 * c4) = acc;
                if (c4 == 0) {
                    a.ml[2 * prow] = m;
                    a.ml[2 * prow + 1] = ls;
                }
            }
        }
    }
}

// out[row] = sum_s 2^(m_s - m) part_s / sum_s 2^(m_s - m) l_s, in split order per thread and then
// over the threads' fixed order.  A split that saw no key (l 0) is not read.
template <int D>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttnArgs a) {
    constexpr int kQuads = D / 4, kPar = 256 / kQuads;
    __shared__ float s_red[4];
    __shared__ __attribute__((aligned(16))) f4 s_acc[kPar * kQuads];
    __shared__ float s_l[kPar];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, rows = a.sq.tokens * a.hq;
    const f4* part = reinterpret_cast<const f4*>(a.part);
    const u2* ml = reinterpret_cast<const u2*>(a.ml);
    float m = kNoKey;
    for (int sp = tid; sp < a.splits; sp += 256) m = fmaxf(m, bitcast<float>(ml[sp * rows + row][0]));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if ((tid & 63) == 0) s_red[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const int c4 = tid % kQuads, p = tid / kQuads;
    if (p < kPar) {
        f4 acc = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.0f;
        for (int sp = p; sp < a.splits; sp += kPar) {
            const u2 x = ml[sp * rows + row];
            const float lw = bitcast<float>(x[1]);
            if (lw == 0.0f) continue;
            const float w = __builtin_amdgcn_exp2f(bitcast<float>(x[0]) - m);
            ls = fmaf(w, lw, ls);
            acc += w * part[(sp * rows + row) * kQuads + c4];
        }
        s_acc[p * kQuads + c4] = acc;
        if (c4 == 0) s_l[p] = ls;
    }
    __syncthreads();
    if (tid >= kQuads) return;
    f4 acc = s_acc[tid];
    float ls = s_l[0];
    for (int j = 1; j < kPar; ++j) {
        acc += s_acc[j * kQuads + tid];
        ls += s_l[j];
    }
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    store4(a.out, a.dtype, row * D + 4 * tid, acc * inv);
}

}  // namespace

template <int D>
static hipError_t rows_launch(const KvAttnArgs& a, int r, int waves, hipStream_t s) {
    const int64_t blocks = (int64_t)a.splits * a.c.heads * a.sq.batch * a.row_tiles;
    const int rows = a.max_new * a.group < 16 ? a.max_new * a.group : 16;
    const size_t lds = sizeof(float) * (size_t)waves * (32 + (size_t)rows * (D + 4));
    const dim3 grid((unsigned)blocks), block(64 * waves);
    if constexpr (D <= 128) {
        if (r == 2) {
            hipLaunchKernelGGL((kv_rows_kernel<D, 2>), grid, block, lds, s, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((kv_rows_kernel<D, 1>), grid, block, lds, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_rows(const KvAttnArgs& a, int r, int waves, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return rows_launch<64>(a, r, waves, s);
        case 96: return rows_launch<96>(a, r, waves, s);
        case 128: return rows_launch<128>(a, r, waves, s);
        case 192: return rows_launch<192>(a, r, waves, s);
        case 256: return rows_launch<256>(a, r, waves, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_kv_join(const KvAttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.sq.tokens * a.hq));
#define Q4GSW_KV_JOIN(D) \
    case D: hipLaunchKernelGGL((kv_join_kernel<D>), grid, dim3(256), 0, s, a); break;
    switch (a.c.dim) {
        Q4GSW_KV_JOIN(64)
        Q4GSW_KV_JOIN(96)
        Q4GSW_KV_JOIN(128)
        Q4GSW_KV_JOIN(192)
        Q4GSW_KV_JOIN(256)
        default: return hipErrorInvalidValue;
    }
#undef Q4GSW_KV_JOIN
    return hipGetLastError();
}

}  // namespace q4gsw
