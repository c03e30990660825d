// Attention of few rows (single tokens, drafts) over the 4-bit cache.
//
//   score[r, t] = q[r] . k[t] / sqrt(dim) (optionally cap tanh(score / cap)), t <= place of r,
//   t > place - window;  out[r] = sum_t softmax(score)[r, t] v[t].
//
// Rows are the new tokens of one sequence times the query heads of one head of the cache.  Every
// wave works alone on 32-token blocks, each a unit of 36 dim bytes that LDS-DMA brings into the
// wave's own two LDS stages (no registers, no barrier; the next unit loads while one is used).
//   * scores: 16x16x32 MFMA, keys as the first operand, so a lane holds the scores of eight tokens
//     of one row.  The codes enter as fp16 integers and every run of 32 channels is one MFMA, whose
//     fp32 sum is multiplied by the token's scale: exact products (a scale multiplied into fp16
//     codes would round, and scores feel that rounding most: twice the output's own).  The codes are
//     unpacked to their values: with the bias of their unpacking left in and taken out of the sum
//     (4 of 9 VALU a word less) a sum would start a thousand times above its result, and queries whose
//     channels have an offset in common lost up to 12 of its bits.
//   * weights: running reference and sum of a softmax in fp32; the reference moves only when some
//     score passes it by kSlack, so most blocks need no exchange between lanes and no rescaling.
//   * sums: 16x16x32 MFMA, values' codes as the first operand; the second, which the lane holds
//     already, is weight * scale, one fp16 rounding a run of channels.  The reference carries the
//     power of two above the largest scale so far (vlog), which keeps the products in fp16's range.
// The waves of a workgroup join through LDS at the end; splits of the cache's length join in a
// second launch (kv_join_kernel).
//
// Bound: HBM for long caches (36 * dim bytes per 32 tokens and head): 64 sequences of 4096 .. 16384
// tokens, 8 heads of 128, 719 MB in 152 us, 4.7 TB/s (a large copy: 4.72).  At 128 channels a unit
// costs some 290 VALU and 16 products a wave, two thirds of the time its bytes take.  Short caches are
// latency: 3 us to the first unit, 2 us for the waves' join, 4 to 5 us for the splits' join.
#include "kv_attention.h"

namespace q4gsw {
namespace {

// The next unit into this wave's LDS, 1 KB an instruction.
template <int D>
__device__ __forceinline__ void fetch_unit(const uint8_t* unit, lds_u8* dst, int lane) {
    constexpr int kBytes = 36 * D, kFull = kBytes / 1024, kRest = kBytes % 1024;
#pragma unroll
    for (int i = 0; i < kFull; ++i) dma16(unit + 1024 * i + 16 * lane, dst + 1024 * i);
    if constexpr (kRest != 0) {
        if (lane < kRest / 16) dma16(unit + 1024 * kFull + 16 * lane, dst + 1024 * kFull);
    }
}

// Wait until at most N of this wave's vector-memory loads are outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Words 2 g and 2 g + 1 of `lane` in a code plane.
template <int G>
__device__ __forceinline__ u2 word_pair(const uint8_t* plane, int g, int lane) {
    return *reinterpret_cast<const u2*>(plane + kv_word_off<G>(2 * g, lane));
}

template <int D>
__global__ __launch_bounds__(512, kv_rows_waves(D)) void kv_rows_kernel(KvAttnArgs a) {
    constexpr int G = D / 32, C = D / 16, kUnit = 36 * D, kLoads = (kUnit + 1023) / 1024;
    extern __shared__ __attribute__((aligned(16))) float smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int i = lane & 15, qd = lane >> 4;

    // Sequences and heads run fastest and each split starts three further on: workgroups go to the
    // XCDs in turn, so every sequence's splits (the late ones empty in short sequences) reach all of them.
    const int pairs = a.sq.batch * a.c.heads;
    const int id = blockIdx.x / pairs;
    const int split = id % a.splits;
    const int rt0 = id / a.splits;
    const int pair = (int)((blockIdx.x % pairs + 3u * (unsigned)split) % (unsigned)pairs);
    const int head = pair % a.c.heads, b = pair / a.c.heads;

    // ---- page numbers of the wave's blocks, 64 at a time in a register ----
    auto page_numbers = [&](int64_t blk) -> int {            // of blocks blk + lane * waves
        const int64_t col = (blk + (int64_t)lane * waves) >> a.c.bpp_log2;
        return col < a.sq.table_cols ? a.sq.table[(int64_t)b * a.sq.table_ld + col] : -1;
    };
    // without a window the first ones do not wait for the sequence's numbers
    int pages = -1;
    if (!a.window) pages = page_numbers((int64_t)split * a.chunk + wave);

    const KvSeq s = kv_seq(a.sq, b);
    const int rows = min(s.m, a.max_new) * a.group;
    const int r0 = rt0 * 16;
    if (r0 >= rows) return;
    const int nr = min(16, rows - r0);
    const KvSpan sp = kv_span(a, s, r0, nr, split);
    auto out_row = [&](int row) -> int64_t {
        const int r = r0 + row, tok = r / a.group;
        return (s.first_row + tok) * a.hq + head * a.group + (r - tok * a.group);
    };
    if (sp.hi <= sp.lo && a.splits > 1) {                    // a split past the sequence's end
        if (tid < nr) {
            const int64_t prow = (int64_t)split * a.sq.tokens * a.hq + out_row(tid);
            a.ml[2 * prow] = kNoKey;
            a.ml[2 * prow + 1] = 0.0f;
        }
        return;
    }

    // ---- queries and the first block's unit: all loads in flight together ----
    u4 bq[G];
    const bool ok = i < nr;
    const int tok = ok ? (r0 + i) / a.group : 0, gh = ok ? r0 + i - tok * a.group : 0;
    const int place = ok ? s.len - s.m + tok : sp.pmax;
    QueryRow<G> qr;
    qr.load(a.q, a.dtype, (s.first_row + tok) * a.q_ld + (int64_t)(head * a.group + gh) * D + 8 * qd, 32);

    const int64_t first = sp.lo + wave;
    const int64_t left = sp.hi - first;
    const int n = left > 0 ? (int)((left + waves - 1) / waves) : 0;
    const int sub_mask = (1 << a.c.bpp_log2) - 1;
    lds_u8* const ring = (lds_u8*)smem + wave * 2 * kUnit;
    uint8_t* const ring_r = reinterpret_cast<uint8_t*>(smem) + wave * 2 * kUnit;
    if (a.window) pages = page_numbers(first);
    // loads block `it` into its stage; false for a page outside the cache (page 0 is loaded instead, so
    // that every block has the same number of loads)
    auto fetch = [&](int it) -> bool {
        const int64_t blk = first + (int64_t)it * waves;
        if (it && (it & 63) == 0) {
            pages = page_numbers(blk);
            // used here, so that the wait for it stays on this path and spares the stages in flight
            asm volatile("" : "+v"(pages));
        }
        const int page = __builtin_amdgcn_readlane(pages, it & 63);
        const bool ok = page >= 0 && page < a.c.pages;
        fetch_unit<D>(a.c.data + kv_unit(a.c, ok ? page : 0, head, (int)(blk & sub_mask)), ring + (it & 1) * kUnit, lane);
        return ok;
    };
    bool have = n > 0 && fetch(0);

    float f = a.scale * qr.convert(a.dtype, ok, wave_max_rows, bq);
    if (a.cap_out == 0.0f) f *= kLog2e;

    f4 o[C];
    float mref = kNoKey, l = 0.0f;
    float vlog = -40.0f, vlim = 0x1p-40f;    // no scale so far is above vlim = 2^vlog
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = f4{0.f, 0.f, 0.f, 0.f};
    const Unpack unpack;
    auto rescale = [&](float w) {
        l *= w;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= w;
    };

    auto compute = [&](uint8_t* unit, int64_t blk) {
        f4 sc[2];
        sc[0] = sc[1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g && (g & 3) == 0 && D >= 256) __builtin_amdgcn_sched_barrier(0);
            const u2 kw = word_pair<G>(unit, g, lane);
            const u4 ks = *reinterpret_cast<const u4*>(unit + 1024 * G + (qd * G + g) * 16);
#pragma unroll
            for (int ab = 0; ab < 2; ++ab) {
                const h2 s01 = bitcast<h2>(ks[2 * ab]), s23 = bitcast<h2>(ks[2 * ab + 1]);
                const f4 p = mfma_f16(unpack.values(kw[ab]), bq[g], f4{0.f, 0.f, 0.f, 0.f});
                sc[ab][0] = fmaf((float)s01[0], p[0], sc[ab][0]);
                sc[ab][1] = fmaf((float)s01[1], p[1], sc[ab][1]);
                sc[ab][2] = fmaf((float)s23[0], p[2], sc[ab][2]);
                sc[ab][3] = fmaf((float)s23[1], p[3], sc[ab][3]);
            }
        }
        const int t0 = (int)(32 * blk);
        const int tl = t0 + 16 * (qd >> 1) + 4 * (qd & 1);     // + 8 ab + j
        const bool edge = t0 + 31 > sp.pmin || t0 <= kv_left_behind(a, sp.pmax);
        const bool tail = t0 + 32 > s.len;
        if (tail) {
            // places past the length may hold anything: their values' scales become 0 in the stage
#pragma unroll
            for (int g = 0; g < G; ++g) {
                u4* const at = reinterpret_cast<u4*>(unit + 1088 * G + (qd * G + g) * 16);
                u4 vs = *at;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tl + 8 * (e >> 1) + 2 * (e & 1);
                    vs[e] = t + 1 < s.len ? vs[e] : (t < s.len ? vs[e] & 0xFFFFu : 0u);
                }
                *at = vs;
            }
        }
        auto scales = [&](int g) { return *reinterpret_cast<const u4*>(unit + 1088 * G + (qd * G + g) * 16); };
        us2 vm = {0, 0};                 // scales are not negative: their bits order like their values
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const u4 vs = scales(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) vm = __builtin_elementwise_max(vm, bitcast<us2>(vs[e]));
        }
        float vmax = f16_bits_to_f32(vm[0] > vm[1] ? vm[0] : vm[1]);
        if (__any(vmax > vlim)) {
            vmax = wave_max_rows(vmax);
            const int ex = (int)(bitcast<uint32_t>(vmax) >> 23) - 126;     // 2^ex > vmax
            const float nl = (float)ex;
            rescale(__builtin_amdgcn_exp2f(vlog - nl));
            vlog = nl;
            vlim = __builtin_amdgcn_exp2f(nl);
        }
        float x[8], p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sc[e >> 2][e & 3];
        float fl = f;
        if (a.cap_out != 0.0f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = capped_log2(x[e] * fl, a.cap_in, a.cap_out);
            fl = 1.0f;
        }
        if (edge) {
            const int gone = kv_left_behind(a, place);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = tl + 8 * (e >> 2) + (e & 3);
                x[e] = t <= place && t > gone ? x[e] : -INFINITY;
            }
        }
        const float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * fl;
        if (__any(mx > mref + kSlack)) {
            const float mn = fmaxf(mref, wave_max_rows(mx));
            rescale(__builtin_amdgcn_exp2f(mref - mn));
            mref = mn;
        }
        const float off = kLift - vlog - mref;
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(x[e], fl, off));
        l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g && (g & 3) == 0 && D >= 256) __builtin_amdgcn_sched_barrier(0);
            const u2 vw = word_pair<G>(unit + 512 * G, g, lane);
            const u4 vs = scales(g);
            u4 pw;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const h2 v2 = bitcast<h2>(vs[e]);
                const h2 w = {(_Float16)fmaf((float)v2[0], p[2 * e], 0.0f), (_Float16)fmaf((float)v2[1], p[2 * e + 1], 0.0f)};
                pw[e] = bitcast<uint32_t>(w);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) o[2 * g + c] = mfma_f16(unpack.values(vw[c]), pw, o[2 * g + c]);
        }
    };

    for (int it = 0; it < n; ++it) {
        bool next = false;
        if (it + 1 < n) {
            // the stage's last reads are done before new bytes may land in it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            next = fetch(it + 1);
            wait_loads<kLoads>();
        } else {
            wait_loads<0>();
        }
        if (have) compute(ring_r + (it & 1) * kUnit, first + (int64_t)it * waves);
        have = next;
    }
    mref += vlog;

    // ---- join the waves ----
    float* const s_ml = smem;                                // [waves][16][2]
    float* const s_o = smem + 32 * waves;                    // [waves][rows of a tile][D + 4]
    const int tile_rows = min(16, a.max_new * a.group);
    const float lsum = wave_sum_rows(l);
    __syncthreads();
    if (qd == 0) {
        s_ml[2 * (16 * wave + i)] = mref;
        s_ml[2 * (16 * wave + i) + 1] = lsum;
    }
    if (i < nr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            *reinterpret_cast<f4*>(&s_o[(wave * tile_rows + i) * (D + 4) + 16 * c + 4 * qd]) = o[c];
    }
    __syncthreads();
    for (int e = tid; e < nr * (D / 4); e += blockDim.x) {
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
        const int64_t orow = out_row(row);
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

// out[row] = sum_s 2^(m_s - m) part_s / sum_s 2^(m_s - m) l_s: a thread takes every kPar-th split,
// kBatch of them in flight, on a running reference of its own, and the threads of a channel join in
// a fixed order.  A split that saw no key (l 0) wrote no sums: what stands there is loaded but not used.
constexpr int kJoinBatch = 4;
constexpr int join_splits(int D, int threads) { return kJoinBatch * (threads / (D / 4)); }   // in one round

template <int D, int THREADS>
__global__ __launch_bounds__(THREADS) void kv_join_kernel(KvAttnArgs a) {
    constexpr int kQuads = D / 4, kPar = THREADS / kQuads, kBatch = kJoinBatch;
    __shared__ __attribute__((aligned(16))) f4 s_acc[kPar * kQuads];
    __shared__ float s_l[kPar], s_m[kPar];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, rows = a.sq.tokens * a.hq;
    const f4* part = reinterpret_cast<const f4*>(a.part);
    const u2* ml = reinterpret_cast<const u2*>(a.ml);
    const int c4 = tid % kQuads, p = tid / kQuads;
    if (p < kPar) {
        f4 acc = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.0f, m = kNoKey;
        for (int sp = p; sp < a.splits; sp += kBatch * kPar) {
            u2 x[kBatch];
            f4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t at = min(sp + j * kPar, a.splits - 1) * rows + row;
                x[j] = ml[at];
                v[j] = part[at * kQuads + c4];
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float lw = bitcast<float>(x[j][1]);
                if (sp + j * kPar >= a.splits || lw == 0.0f) continue;
                const float mw = bitcast<float>(x[j][0]), mn = fmaxf(m, mw);
                const float keep = __builtin_amdgcn_exp2f(m - mn), w = __builtin_amdgcn_exp2f(mw - mn);
                m = mn;
                ls = fmaf(w, lw, ls * keep);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, v[j][e], acc[e] * keep);
            }
        }
        s_acc[p * kQuads + c4] = acc;
        if (c4 == 0) {
            s_l[p] = ls;
            s_m[p] = m;
        }
    }
    __syncthreads();
    if (tid >= kQuads) return;
    float m = kNoKey, ls = 0.0f;
    f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kPar; ++j) m = fmaxf(m, s_m[j]);
#pragma unroll
    for (int j = 0; j < kPar; ++j) {
        const float w = __builtin_amdgcn_exp2f(s_m[j] - m);
        ls = fmaf(w, s_l[j], ls);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, s_acc[j * kQuads + tid][e], acc[e]);
    }
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    store4(a.out, a.dtype, row * D + 4 * tid, acc * inv);
}

}  // namespace

template <int D>
static hipError_t rows_launch(const KvAttnArgs& a, int waves, hipStream_t s) {
    const int64_t blocks = (int64_t)a.splits * a.c.heads * a.sq.batch * a.row_tiles;
    const int rows = a.max_new * a.group < 16 ? a.max_new * a.group : 16;
    const size_t join = sizeof(float) * (size_t)waves * (32 + (size_t)rows * (D + 4)), ring = (size_t)waves * 2 * 36 * D;
    const size_t lds = join > ring ? join : ring;
    hipLaunchKernelGGL((kv_rows_kernel<D>), dim3((unsigned)blocks), dim3(64 * waves), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_rows(const KvAttnArgs& a, int waves, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return rows_launch<64>(a, waves, s);
        case 96: return rows_launch<96>(a, waves, s);
        case 128: return rows_launch<128>(a, waves, s);
        case 192: return rows_launch<192>(a, waves, s);
        case 256: return rows_launch<256>(a, waves, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_kv_join(const KvAttnArgs& a, hipStream_t s) {
    // one wave a row where it takes the splits in one round
    const dim3 grid((unsigned)(a.sq.tokens * a.hq));
#define Q4GSW_KV_JOIN(D)                                                                                                  \
    case D:                                                                                                               \
        if (a.splits <= join_splits(D, 64)) hipLaunchKernelGGL((kv_join_kernel<D, 64>), grid, dim3(64), 0, s, a);           \
        else hipLaunchKernelGGL((kv_join_kernel<D, 256>), grid, dim3(256), 0, s, a);                                        \
        break;
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
