// Attention of many rows (prompts, or chunks of them) over the 4-bit cache.
//
// A workgroup holds 32 rows per wave (rows: new tokens of a sequence times the query heads of one
// head of the cache) and walks the keys in tiles.  A tile's codes are unpacked once per workgroup,
// scale multiplied in, to fp16 in LDS, in the operand order of the 32x32x16 MFMA, so each wave's
// operand read is 1 KB in lane order.  Two stages: while a tile is used, the next one is unpacked
// into the other stage from codes that were loaded a tile earlier.
//   * scores: keys as the first operand: a lane holds the scores of 16 of 32 tokens of one row;
//   * weights: running reference and sum of a softmax in fp32 (see kv_attention.h), rounded to
//     fp16 in the registers where they arose, which is the second operand of the next product;
//   * sums: values as the first operand, 32 channels of a row in a lane's 16 accumulators.
// Rounding code * scale to fp16 (2^-11) is below a bf16 output's own rounding but twice an fp16
// output's, since scores feel it; with PREC (fp16 and fp32 outputs) the exact remainder of every
// key and value is kept beside it and enters by a second product: rms error 2.2e-4 .. 2.8e-4 (without the
// values' remainder 2.8e-4 .. 3.4e-4 in four fifths of the time).  fp32 queries round to 11 bits as in the
// other kernel: behind int8 rows their own error is 2^-8, and a second part of the query would double
// the scores' products once more.
//
// Bound: MFMA and the softmax's VALU, about even at 128 channels (a wave's turn of 64 keys: 32 products of
// 32 cycles, some 230 VALU of 4 and more) and hardly overlapping between the two waves of a SIMD:
// three chunks of 2048 rows behind 6144 keys, 32 / 8 heads of 128, take 781 us in bf16, 924 TFLOP/s (a
// large library product: 1206), and 1207 us in fp16; unlike chunks in bf16 (1024 .. 2048 rows of 8192 tokens and
// fewer) run at 830 to 860 TFLOP/s.
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

// Instruction kinds of __builtin_amdgcn_sched_group_barrier
constexpr int kSchedValu = 0x2, kSchedMfma = 0x8, kSchedRead = 0x100;

// The sequence with `rank` longer ones before it (batches of more than 64: in their order).
__device__ __forceinline__ int by_length(const KvSeqs& sq, int rank, int lane) {
    if (sq.batch > 64) return rank;
    const int mine = lane < sq.batch ? sq.lens[lane] : 0;
    int before = lane < sq.batch ? 0 : 64;
    for (int j = 0; j < sq.batch; ++j) {
        const int other = __builtin_amdgcn_readlane(mine, j);
        before += other > mine || (other == mine && j < lane);
    }
    return __builtin_ctzll(__ballot(before == rank));
}

template <int D, int NW, bool PREC, bool TREE>
__global__ __launch_bounds__(64 * NW, (D <= 128 ? 2 : 1)) void kv_prompt_kernel(KvAttnArgs a) {
    constexpr int G = D / 32, S = D / 16, TB = prompt_blocks(D, PREC);
    constexpr int kFrags = TB * S;                       // operand KBs of the keys (and of the values) of a tile
    constexpr int kPlane = kFrags * 1024, kStage = kPlane * (PREC ? 4 : 2);     // keys, values, their remainders
    constexpr int kPairs = TB * G, kPer = (kPairs + NW - 1) / NW;   // (block, run) pairs a wave unpacks
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, qd = lane >> 4;             // unpacking: lane of a unit
    const int rl = lane & 31, h = lane >> 5;             // products: row or column, half

    // the longest sequence first, its last rows first, so that the last workgroups to start are short
    // (three unlike chunks of 2048 rows: 645 -> 620 us); cache heads fastest, so that with eight of them
    // one head's keys and values stay in one XCD's L2
    int id = blockIdx.x;
    const int head = id % a.c.heads;
    id /= a.c.heads;
    const int split = id % a.splits;
    id /= a.splits;
    const int rt0 = a.row_tiles - 1 - id % a.row_tiles;
    const int b = by_length(a.sq, id / a.row_tiles, lane);

    const KvSeq s = kv_seq(a.sq, b);
    const int rows = min(s.m, a.max_new) * a.group;
    const int r0 = rt0 * 32 * NW;
    if (r0 >= rows) return;
    const KvSpan sp = kv_span<TREE>(a, s, r0, min(32 * NW, rows - r0), split);
    const int64_t nb = sp.hi - sp.lo;
    const int n = nb > 0 ? (int)((nb + TB - 1) / TB) : 0;

    // ---- the wave's rows ----
    const int r = r0 + 32 * wave + rl;
    const bool ok = r < rows;
    const int tok = ok ? r / a.group : 0, gh = ok ? r - tok * a.group : 0;
    const int p0 = s.len - s.m;
    int place = ok ? p0 + tok : sp.pmax;
    const int wmin = TREE ? p0 : p0 + (r0 + 32 * wave) / a.group;                       // places of the wave's rows
    const int wmax = min(p0 + (r0 + 32 * wave + 31) / a.group, sp.pmax);
    const bool active = r0 + 32 * wave < rows;
    u4 bq[S];
    float f;
    {
        const int64_t base = (s.first_row + tok) * a.q_ld + (int64_t)(head * a.group + gh) * D;
        QueryRow<S> qr;
        qr.load(a.q, a.dtype, base + 8 * h, 16);
        f = a.scale * qr.convert(a.dtype, ok, max_halves, bq);
        if (a.cap_out == 0.0f) f *= kLog2e;
    }
    const int tok0 = r0 / a.group;
    const KvTree tree(lds + 2 * kStage, a.max_new);
    if constexpr (TREE) {
        tree.build(a.parents, s.first_row, min(s.m, a.max_new), tok0,
                           (min(r0 + 32 * NW, rows) - 1) / a.group + 1 - tok0, a.window);
        if (ok) place = p0 + tree.depth(tok - tok0);     // its position
    }

    // ---- tiles: codes to registers two tiles ahead, unpacked into LDS one ahead ----
    const Unpack unpack;
    struct Codes {
        u2 k, v;
        uint32_t ks;                     // scales of the two keys' words
        u4 vs;                           // of the eight tokens of the values' words
    };
    Codes cr[kPer];
    const int sub_mask = (1 << a.c.bpp_log2) - 1;
    int pages = -1;                      // page numbers of blocks 64 k + lane of the span
    int page_of[TB];
    uint32_t hidden = 0;                 // bits TB t ..: block of the tile t tiles before the last loaded has no page
    auto load = [&](int t) {
        const int at = t * TB;
        if ((at & 63) == 0) {
            const int64_t mine = sp.lo + at + lane;
            pages = mine < sp.hi ? a.sq.table[(int64_t)b * a.sq.table_ld + (mine >> a.c.bpp_log2)] : -1;
            asm volatile("" : "+v"(pages));
        }
        hidden <<= TB;
#pragma unroll
        for (int u = 0; u < TB; ++u) {
            const int page = __builtin_amdgcn_readlane(pages, (at + u) & 63);
            const bool bad = page < 0 || page >= a.c.pages;
            hidden |= (uint32_t)bad << u;
            page_of[u] = bad ? 0 : page;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p = wave + NW * j;
            if (p >= kPairs) break;
            const int u = p / G, g = p - u * G;
            const int64_t blk = sp.lo + at + u;
            const uint8_t* unit = a.c.data + kv_unit(a.c, TB == 1 || u == 0 ? page_of[0] : page_of[TB - 1], head, (int)(blk & sub_mask));
            const int off = kv_word_off<G>(2 * g, lane);
            cr[j].k = *reinterpret_cast<const u2*>(unit + off);
            cr[j].v = *reinterpret_cast<const u2*>(unit + 512 * G + off);
            const uint16_t* ks = reinterpret_cast<const uint16_t*>(unit + 1024 * G) + ((i >> 2) * G + g) * 8 + (i & 3);
            cr[j].ks = ks[0] | (uint32_t)ks[4] << 16;
            cr[j].vs = *reinterpret_cast<const u4*>(unit + 1088 * G + (qd * G + g) * 16);
        }
    };
    auto put = [&](uint8_t* at, const u4& c, h2 s0, h2 s1, h2 s2, h2 s3) {
        const h2 ss[4] = {s0, s1, s2, s3};
        u4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const h2 x = bitcast<h2>(c[e]) * ss[e];
            hi[e] = bitcast<uint32_t>(x);
            if constexpr (PREC) lo[e] = bitcast<uint32_t>(__builtin_elementwise_fma(bitcast<h2>(c[e]), ss[e], -x));
        }
        *reinterpret_cast<u4*>(at) = hi;
        if constexpr (PREC) *reinterpret_cast<u4*>(at + 2 * kPlane) = lo;
    };
    auto store = [&](int t) {            // tile t, the last loaded
        uint8_t* stage = lds + (t & 1) * kStage;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p = wave + NW * j;
            if (p >= kPairs) break;
            const int u = p / G, g = p - u * G;
            u4 vs = cr[j].vs;
            const int t0 = (int)(32 * (sp.lo + t * TB + u));
            const bool bad = (hidden >> u) & 1;
            if (bad || t0 + 32 > s.len) {            // such places may hold anything: their values count as 0
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tk = t0 + kv_tok(qd, 2 * e);
                    vs[e] = bad || tk >= s.len ? 0u : (tk + 1 < s.len ? vs[e] : vs[e] & 0xFFFFu);
                }
            }
            const h2 k2 = bitcast<h2>(cr[j].ks);
#pragma unroll
            for (int ab = 0; ab < 2; ++ab) {
                const h2 kk = {k2[ab], k2[ab]};
                uint8_t* at = stage + (u * S + 2 * g + (qd >> 1)) * 1024 + 16 * (kv_tok(i >> 2, 4 * ab + (i & 3)) + 32 * (qd & 1));
                put(at, unpack.values(cr[j].k[ab]), kk, kk, kk, kk);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint8_t* at = stage + kPlane + (u * S + 2 * g + (qd >> 1)) * 1024 + 16 * (16 * c + i + 32 * (qd & 1));
                put(at, unpack.values(cr[j].v[c]), bitcast<h2>(vs[0]), bitcast<h2>(vs[1]), bitcast<h2>(vs[2]), bitcast<h2>(vs[3]));
            }
        }
    };

    f32x16 o[G];
    const f32x16 zero = {};
#pragma unroll
    for (int g = 0; g < G; ++g) o[g] = zero;
    float mref = kNoKey, l = 0.0f;

    auto compute = [&](int t, uint32_t gone_blocks) {
        const int t0 = (int)(32 * (sp.lo + t * TB));
        if (!active || t0 > wmax || t0 + 32 * TB - 1 <= kv_left_behind(a, wmin)) return;
        const uint8_t* stage = lds + (t & 1) * kStage;
        f32x16 sc[TB];
#pragma unroll
        for (int u = 0; u < TB; ++u) sc[u] = zero;
        // operands are read kAhead products ahead of their use
        constexpr int kProducts = TB * S * (PREC ? 2 : 1), kAhead = kProducts < 6 ? kProducts : 6;
#pragma unroll
        for (int k = 0; k < S; ++k) {
#pragma unroll
            for (int u = 0; u < TB; ++u) {
                const uint8_t* at = stage + (u * S + k) * 1024 + 16 * lane;
                sc[u] = mfma32_f16(*reinterpret_cast<const u4*>(at), bq[k], sc[u]);
                if constexpr (PREC) sc[u] = mfma32_f16(*reinterpret_cast<const u4*>(at + 2 * kPlane), bq[k], sc[u]);
            }
        }
        __builtin_amdgcn_sched_group_barrier(kSchedRead, kAhead, 0);
#pragma unroll
        for (int j = 0; j < kProducts; ++j) {
            __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
            if (j + kAhead < kProducts) __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
        }
        float fl = f;
        if (a.cap_out != 0.0f) {
#pragma unroll
            for (int u = 0; u < TB; ++u) {
#pragma unroll
                for (int e = 0; e < 16; ++e) sc[u][e] = capped_log2(sc[u][e] * fl, a.cap_in, a.cap_out);
            }
            fl = 1.0f;
        }
        if (t0 + 32 * TB - (TREE ? 0 : 1) > wmin || t0 <= kv_left_behind(a, wmax) || gone_blocks) {
            const int gone = kv_left_behind(a, place);
#pragma unroll
            for (int u = 0; u < TB; ++u) {
                const bool bad = (gone_blocks >> u) & 1;
                uint32_t seen = 0u;                  // bit j: the row sees place t0 + 32 u + 4 h + j
                // a block past the wave's last row is not in the tree's words
                if constexpr (TREE) seen = t0 + 32 * u <= wmax ? tree.block(ok ? tok - tok0 : 0, t0 + 32 * u, p0) >> (4 * h) : 0u;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int tk = t0 + 32 * u + 8 * (e >> 2) + 4 * h + (e & 3);
                    const bool near = TREE ? (seen >> (8 * (e >> 2) + (e & 3))) & 1u : tk <= place;
                    sc[u][e] = near && tk > gone && !bad ? sc[u][e] : -INFINITY;
                }
            }
        }
        float mx = sc[0][0];
#pragma unroll
        for (int u = 0; u < TB; ++u) {
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sc[u][e]);
        }
        mx *= fl;
        if (__any(mx > mref + kSlack)) {
            const float mn = fmaxf(mref, max_halves(mx));
            const float w = __builtin_amdgcn_exp2f(mref - mn);
            mref = mn;
            l *= w;
#pragma unroll
            for (int g = 0; g < G; ++g) o[g] *= w;
        }
        const float off = kLift - mref;
        // 16 tokens a step; a step's operands are read a step ahead, and the weights of the next step
        // are computed under the products of this one
        constexpr int kSteps = 2 * TB, kStep = G * (PREC ? 2 : 1);
        auto operands = [&](int st, u4 (&v)[kStep]) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint8_t* at = stage + kPlane + ((st >> 1) * S + 2 * g + (st & 1)) * 1024 + 16 * lane;
                v[g] = *reinterpret_cast<const u4*>(at);
                if constexpr (PREC) v[G + g] = *reinterpret_cast<const u4*>(at + 2 * kPlane);
            }
        };
        auto weights = [&](int st) -> u4 {
            u4 p;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __builtin_amdgcn_exp2f(fmaf(sc[st >> 1][8 * (st & 1) + 2 * e], fl, off));
                const float y = __builtin_amdgcn_exp2f(fmaf(sc[st >> 1][8 * (st & 1) + 2 * e + 1], fl, off));
                sum += x + y;
                p[e] = bitcast<uint32_t>(h2{(_Float16)x, (_Float16)y});
            }
            l += sum;
            return p;
        };
        u4 v[2][kStep];
        operands(0, v[0]);
        u4 p = weights(0);
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            u4 next = p;
            if (st + 1 < kSteps) {
                operands(st + 1, v[(st + 1) & 1]);
                next = weights(st + 1);
            }
#pragma unroll
            for (int j = 0; j < kStep; ++j) o[j % G] = mfma32_f16(v[st & 1][j], p, o[j % G]);
            p = next;
        }
        __builtin_amdgcn_sched_group_barrier(kSchedRead, kStep, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedValu, 30, 1);
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            if (st + 1 < kSteps) __builtin_amdgcn_sched_group_barrier(kSchedRead, kStep, 1);
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 1);
                if (st + 1 < kSteps) __builtin_amdgcn_sched_group_barrier(kSchedValu, (28 + kStep - 1) / kStep, 1);
            }
        }
    };

    if (n > 0) {
        load(0);
        store(0);
        if (n > 1) load(1);
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            // bits of tile t: the last loaded is tile t + 1, where there is one
            const uint32_t gone = (t + 1 < n ? hidden >> TB : hidden) & ((1u << TB) - 1);
            if (t + 1 < n) store(t + 1);
            if (t + 2 < n) load(t + 2);
            compute(t, gone);
            __syncthreads();
        }
    }

    l = sum_halves(l);
    if (!ok) return;
    const int64_t orow = (s.first_row + tok) * a.hq + head * a.group + gh;
    if (a.splits == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store4(a.out, a.dtype, orow * D + 32 * g + 8 * e + 4 * h,
                       f4{o[g][4 * e] * inv, o[g][4 * e + 1] * inv, o[g][4 * e + 2] * inv, o[g][4 * e + 3] * inv});
        }
        return;
    }
    const int64_t prow = (int64_t)split * a.sq.tokens * a.hq + orow;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f4*>(a.part + prow * D + 32 * g + 8 * e + 4 * h) =
                f4{o[g][4 * e], o[g][4 * e + 1], o[g][4 * e + 2], o[g][4 * e + 3]};
    }
    if (h == 0) {
        a.ml[2 * prow] = mref;
        a.ml[2 * prow + 1] = l;
    }
}

template <int D, int NW, bool PREC>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
    constexpr int lds = prompt_lds(D, PREC);
    const int64_t blocks = (int64_t)a.splits * a.c.heads * a.sq.batch * a.row_tiles;
    if (a.parents)
        hipLaunchKernelGGL((kv_prompt_kernel<D, NW, PREC, true>), dim3((unsigned)blocks), dim3(64 * NW),
                           lds + tree_lds(a, 32 * NW), s, a);
    else
        hipLaunchKernelGGL((kv_prompt_kernel<D, NW, PREC, false>), dim3((unsigned)blocks), dim3(64 * NW), lds, s, a);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const KvAttnArgs& a, int waves, hipStream_t s) {
    const bool prec = a.dtype != kBF16;
    if constexpr (D <= 128) {
        if (waves == 8) return prec ? launch<D, 8, true>(a, s) : launch<D, 8, false>(a, s);
    }
    return prec ? launch<D, 4, true>(a, s) : launch<D, 4, false>(a, s);
}

}  // namespace

hipError_t launch_kv_prompt(const KvAttnArgs& a, int waves, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return launch_d<64>(a, waves, s);
        case 96: return launch_d<96>(a, waves, s);
        case 128: return launch_d<128>(a, waves, s);
        case 192: return launch_d<192>(a, waves, s);
        case 256: return launch_d<256>(a, waves, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace q4gsw
