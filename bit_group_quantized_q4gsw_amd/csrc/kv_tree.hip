// Attention of trees of drafted tokens over the 4-bit cache, 17 rows of a cache head and more (fewer:
// kv_rows.hip; so many that a workgroup's waves can share what one of them unpacks: kv_prompt.hip).
//
// As in kv_rows.hip every wave works alone on 32-token units that LDS-DMA brings into its own two stages,
// and the waves of a workgroup join at the end; but a tile is 32 rows and the products are 32x32x16, so a
// unit is unpacked once for 32 rows.  A unit lies in memory for the 16x16x32 product: word 2 g + ab of lane
// (i, q) is row i of half ab, channels or tokens octet q.  The 32x32x16 operand wants the two halves in the
// two lower 16-lane rows and the same halves of the next octet in the upper two, which a row swap and a
// half swap of the two words give: a0 a1 a2 a3, b0 b1 b2 b3 -> a0 b0 a1 b1, a2 b2 a3 b3, the operands of two
// products.  A lane then holds the scores of 16 tokens of one row, in the order in which the products of the
// values want their weights.
//
// bf16 queries: scales are multiplied into the codes (one fp16 rounding, below the output's own).  fp16 and fp32
// queries (PREC): every run of 32 channels is a sum of its own that takes the token's scale in fp32, and
// values' scales go into the weights, one rounding a run, as in kv_rows.hip; see there for the reference
// and the ranges.
//
// Bound: VALU: a unit of 128 channels costs a wave some 360 of them (PREC 430), 2500 cycles of its SIMD with the 16
// products, for 32 rows, where two tiles of 16 cost 580.  Three or four stages instead of two change nothing.
// 16 sequences of 1024 .. 4096 tokens, 32 / 8 heads of 128, 16 nodes each: bf16 39 us, fp16 47 (tiles of 16 rows: 53).
#include "kv_attention.h"

namespace q4gsw {
namespace {

__device__ __forceinline__ float max_halves(float v) {
    const uint32_t a = bitcast<uint32_t>(v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    return fmaxf(bitcast<float>(r[0]), bitcast<float>(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
    const uint32_t a = bitcast<uint32_t>(v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    return bitcast<float>(r[0]) + bitcast<float>(r[1]);
}

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

// Words 2 g and 2 g + 1 of a code plane as the operands of two 32x32x16 products.
template <int G>
__device__ __forceinline__ u2 operand_words(const uint8_t* plane, int g, int lane) {
    const u2 w = *reinterpret_cast<const u2*>(plane + kv_word_off<G>(2 * g, lane));
    const auto r = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);       // a0 b0 a2 b2, a1 b1 a3 b3
    const auto h = __builtin_amdgcn_permlane32_swap(r[0], r[1], false, false);       // a0 b0 a1 b1, a2 b2 a3 b3
    return u2{h[0], h[1]};
}

__device__ __forceinline__ u4 scaled(const u4& c, h2 s0, h2 s1, h2 s2, h2 s3) {
    const h2 ss[4] = {s0, s1, s2, s3};
    u4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = bitcast<uint32_t>(bitcast<h2>(c[e]) * ss[e]);
    return r;
}

constexpr int kJoinLd = 36;              // floats of a row's 32 channels in the join

template <int D, bool PREC>
__global__ __launch_bounds__(64 * kv_tree_most(D), kv_tree_waves(D, PREC)) void kv_tree_kernel(KvAttnArgs a) {
    constexpr int G = D / 32, S = D / 16, kUnit = 36 * D, kLoads = (kUnit + 1023) / 1024;
    extern __shared__ __attribute__((aligned(16))) float smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int i = lane & 15, qd = lane >> 4;             // lane of a unit
    const int rl = lane & 31, h = lane >> 5;             // products: row or column, half

    // the order of kv_rows.hip: every sequence's splits reach all XCDs
    const int pairs = a.sq.batch * a.c.heads;
    const int id = blockIdx.x / pairs;
    const int split = id % a.splits;
    const int rt0 = id / a.splits;
    const int pair = (int)((blockIdx.x % pairs + 3u * (unsigned)split) % (unsigned)pairs);
    const int head = pair % a.c.heads, b = pair / a.c.heads;

    const KvSeq s = kv_seq(a.sq, b);
    const int rows = min(s.m, a.max_new) * a.group;
    const int r0 = rt0 * 32;
    if (r0 >= rows) return;
    const int nr = min(32, rows - r0);
    const KvSpan sp = kv_span<true>(a, s, r0, nr, split);
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

    // page numbers of the wave's blocks, 64 at a time in a register
    auto page_numbers = [&](int64_t blk) -> int {            // of blocks blk + lane * waves
        const int64_t col = (blk + (int64_t)lane * waves) >> a.c.bpp_log2;
        return col < a.sq.table_cols ? a.sq.table[(int64_t)b * a.sq.table_ld + col] : -1;
    };
    const int64_t first = sp.lo + wave;
    const int64_t left = sp.hi - first;
    const int n = left > 0 ? (int)((left + waves - 1) / waves) : 0;
    const int sub_mask = (1 << a.c.bpp_log2) - 1;
    lds_u8* const ring = (lds_u8*)smem + wave * 2 * kUnit;
    uint8_t* const ring_r = reinterpret_cast<uint8_t*>(smem) + wave * 2 * kUnit;
    int pages = page_numbers(first);

    // ---- queries and the first block's unit: all loads in flight together ----
    u4 bq[S];
    const bool ok = rl < nr;
    const int tok0 = r0 / a.group, p0 = s.len - s.m;
    const int tok = ok ? (r0 + rl) / a.group : tok0, gh = ok ? r0 + rl - tok * a.group : 0;
    QueryRow<S> qr;
    qr.load(a.q, a.dtype, (s.first_row + tok) * a.q_ld + (int64_t)(head * a.group + gh) * D + 8 * h, 16);
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
    const KvTree tree(reinterpret_cast<uint8_t*>(smem) + a.tree_at, a.max_new);
    tree.build(a.parents, s.first_row, min(s.m, a.max_new), tok0, (r0 + nr - 1) / a.group + 1 - tok0, a.window);
    const int position = ok ? p0 + tree.depth(tok - tok0) : sp.pmax;

    float f = a.scale * qr.convert(a.dtype, ok, max_halves, bq);
    if (a.cap_out == 0.0f) f *= kLog2e;

    f32x16 o[G];
    const f32x16 zero = {};
#pragma unroll
    for (int g = 0; g < G; ++g) o[g] = zero;
    float mref = kNoKey, l = 0.0f;
    float vlog = PREC ? -40.0f : 0.0f, vlim = 0x1p-40f;      // PREC: no scale so far is above vlim = 2^vlog
    const Unpack unpack;
    auto rescale = [&](float w) {
        l *= w;
#pragma unroll
        for (int g = 0; g < G; ++g) o[g] *= w;
    };

    auto compute = [&](uint8_t* unit, int64_t blk) {
        const int t0 = (int)(32 * blk);
        if (t0 + 32 > s.len) {
            // places past the length may hold anything: their values' scales become 0 in the stage
            const int tl = t0 + 16 * (qd >> 1) + 4 * (qd & 1);
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
        auto scales = [&](int kv, int q, int g) { return *reinterpret_cast<const u4*>(unit + (kv ? 1088 : 1024) * G + (q * G + g) * 16); };
        // ---- scores: register e holds token 16 (e / 4 % 2) + 8 (e / 8) + 4 h + e % 4 ----
        f32x16 sc = zero;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const u2 kw = operand_words<G>(unit, g, lane);
            if constexpr (PREC) {
                f32x16 p = mfma32_f16(unpack.values(kw[0]), bq[2 * g], zero);
                p = mfma32_f16(unpack.values(kw[1]), bq[2 * g + 1], p);
                const u4 s0 = scales(0, h, g), s1 = scales(0, 2 + h, g);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const u4& ks = e & 4 ? s1 : s0;
                    const int slot = 4 * (e >> 3) + (e & 3);
                    sc[e] = fmaf((float)bitcast<h2>(ks[slot >> 1])[slot & 1], p[e], sc[e]);
                }
            } else {
                // a lane's operand is one token's: key row i of half qd & 1
                const _Float16 k = bitcast<_Float16>(*reinterpret_cast<const uint16_t*>(
                    unit + 1024 * G + 2 * (((i >> 2) * G + g) * 8 + 4 * (qd & 1) + (i & 3))));
                const h2 kk = {k, k};
                sc = mfma32_f16(scaled(unpack.values(kw[0]), kk, kk, kk, kk), bq[2 * g], sc);
                sc = mfma32_f16(scaled(unpack.values(kw[1]), kk, kk, kk, kk), bq[2 * g + 1], sc);
            }
        }
        float fl = f;
        if (a.cap_out != 0.0f) {
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[e] = capped_log2(sc[e] * fl, a.cap_in, a.cap_out);
            fl = 1.0f;
        }
        if (t0 + 32 > p0 || t0 <= kv_left_behind(a, sp.pmax)) {
            const int gone = kv_left_behind(a, position);
            const uint32_t seen = tree.block(tok - tok0, t0, p0) >> (4 * h);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = 16 * ((e >> 2) & 1) + 8 * (e >> 3) + (e & 3);
                sc[e] = ((seen >> t) & 1u) && t0 + t + 4 * h > gone ? sc[e] : -INFINITY;
            }
        }
        if constexpr (PREC) {
            us2 vm = {0, 0};             // scales are not negative: their bits order like their values
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const u4 vs = scales(1, qd, g);
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
        }
        float mx = sc[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[e]);
        mx *= fl;
        if (__any(mx > mref + kSlack)) {
            const float mn = fmaxf(mref, max_halves(mx));
            rescale(__builtin_amdgcn_exp2f(mref - mn));
            mref = mn;
        }
        const float off = kLift - vlog - mref;
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            sc[e] = __builtin_amdgcn_exp2f(fmaf(sc[e], fl, off));
            sum += sc[e];
        }
        l += sum;
        // ---- sums: octet 2 st + h of the tokens is registers 4 st + j and 8 + 4 st + j ----
        u4 pw[2];
        if constexpr (!PREC) {
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 4 * st + 8 * (e >> 1) + 2 * (e & 1);
                    pw[st][e] = bitcast<uint32_t>(h2{(_Float16)sc[at], (_Float16)sc[at + 1]});
                }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const u2 vw = operand_words<G>(unit + 512 * G, g, lane);
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const u4 vs = scales(1, 2 * st + h, g);
                if constexpr (PREC) {
                    u4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = 4 * st + 8 * (e >> 1) + 2 * (e & 1);
                        const h2 v2 = bitcast<h2>(vs[e]);
                        w[e] = bitcast<uint32_t>(h2{(_Float16)fmaf((float)v2[0], sc[at], 0.0f), (_Float16)fmaf((float)v2[1], sc[at + 1], 0.0f)});
                    }
                    o[g] = mfma32_f16(unpack.values(vw[st]), w, o[g]);
                } else {
                    o[g] = mfma32_f16(scaled(unpack.values(vw[st]), bitcast<h2>(vs[0]), bitcast<h2>(vs[1]), bitcast<h2>(vs[2]), bitcast<h2>(vs[3])),
                                      pw[st], o[g]);
                }
            }
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

    // ---- join the waves, 32 channels at a time ----
    float* const s_ml = smem;                                // [waves][32][2]
    float* const s_o = smem + 64 * waves;                    // [waves][32][kJoinLd]
    const float lsum = sum_halves(l);
    __syncthreads();
    if (h == 0) {
        s_ml[2 * (32 * wave + rl)] = mref;
        s_ml[2 * (32 * wave + rl) + 1] = lsum;
    }
    const int row = tid >> 3, c4 = tid & 7;                  // of threads 0 .. 255
    float m = kNoKey, ls = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f4*>(&s_o[(32 * wave + rl) * kJoinLd + 8 * e + 4 * h]) = f4{o[g][4 * e], o[g][4 * e + 1], o[g][4 * e + 2], o[g][4 * e + 3]};
        __syncthreads();
        if (tid < 256 && row < nr) {
            if (g == 0) {
                for (int w = 0; w < waves; ++w) m = fmaxf(m, s_ml[2 * (32 * w + row)]);
                for (int w = 0; w < waves; ++w)
                    ls = fmaf(__builtin_amdgcn_exp2f(s_ml[2 * (32 * w + row)] - m), s_ml[2 * (32 * w + row) + 1], ls);
            }
            f4 acc = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < waves; ++w) {
                const float wt = __builtin_amdgcn_exp2f(s_ml[2 * (32 * w + row)] - m);
                acc += wt * *reinterpret_cast<const f4*>(&s_o[(32 * w + row) * kJoinLd + 4 * c4]);
            }
            const int64_t orow = out_row(row);
            if (a.splits == 1) {
                // a row that no key is seen by has a sum of exactly 0 and gives zeros
                const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                store4(a.out, a.dtype, orow * D + 32 * g + 4 * c4, acc * inv);
            } else {
                const int64_t prow = (int64_t)split * a.sq.tokens * a.hq + orow;
                *reinterpret_cast<f4*>(a.part + prow * D + 32 * g + 4 * c4) = acc;
                if (g == 0 && c4 == 0) {
                    a.ml[2 * prow] = m;
                    a.ml[2 * prow + 1] = ls;
                }
            }
        }
        __syncthreads();
    }
}

template <int D>
hipError_t launch(KvAttnArgs a, int waves, hipStream_t s) {
    const int64_t blocks = (int64_t)a.splits * a.c.heads * a.sq.batch * a.row_tiles;
    const int join = 4 * waves * (64 + 32 * kJoinLd), ring = waves * 2 * 36 * D;
    a.tree_at = join > ring ? join : ring;
    const size_t lds = a.tree_at + tree_lds(a, 32);
    if (a.dtype != kBF16) hipLaunchKernelGGL((kv_tree_kernel<D, true>), dim3((unsigned)blocks), dim3(64 * waves), lds, s, a);
    else hipLaunchKernelGGL((kv_tree_kernel<D, false>), dim3((unsigned)blocks), dim3(64 * waves), lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_tree(const KvAttnArgs& a, int waves, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return launch<64>(a, waves, s);
        case 96: return launch<96>(a, waves, s);
        case 128: return launch<128>(a, waves, s);
        case 192: return launch<192>(a, waves, s);
        case 256: return launch<256>(a, waves, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace q4gsw
