// The paged cache of 4-bit keys and values: layout and unpacking (gfx950).
//
// A page holds page_size tokens (a power of two, 32 or more) of every head.  Tokens are kept in
// blocks of 32: the unit of one (page, head, block) is 36 * dim contiguous bytes, G = dim / 32
// scale groups,
//     [keys' codes 512 G][values' codes 512 G][keys' scales 64 G][values' scales 64 G],
// and the units of a page run head by head, block by block.  A unit is laid out for the MFMA
// operands that read it, so no lane ever exchanges a code with another:
//   * a code plane is 2 G 32-bit words for each of 64 lanes, lane = i + 16 q; words 4p .. 4p + 3
//     of all lanes are one 1 KB run of 16 bytes a lane (with G odd the last two words are a run
//     of 8 bytes a lane);
//   * token t of the block, t = 16 u + 8 ab + 4 h + j (bits u, ab, h, two bits j), has key row
//     i = 4 q + j with q = 2 u + h.  Keys' word 2 g + ab of lane (i, q') holds that row's
//     channels 32 g + 8 q' .. + 7: a 16x16x32 operand row;
//   * values' word c of lane (i, q) holds channel 16 c + i of the eight tokens of q, slots
//     4 ab + j.  These are the tokens whose scores lane (any row, q) of the 16x16 products of
//     the keys' rows holds, and half h of a 32x32 product holds in registers 8 u + 4 ab + j, so
//     the probabilities enter the second product from the registers they were computed in;
//   * entry k of a word (channel or token slot) is its nibble nib_pos(k); code = value + 8;
//   * scales are fp16, keys' and values' alike [q][g][slot]: the scales of the tokens of q.
#pragma once
#include "device.h"

namespace q4gsw {

typedef uint16_t us2 __attribute__((ext_vector_type(2)));

constexpr int kKvTok = 32;               // tokens of a block
constexpr int kKvGroup = 32;             // channels of a scale
constexpr int kKvMinPage = 32, kKvMaxPage = 4096;

__host__ __device__ inline int64_t kv_unit_bytes(int dim) { return 36 * (int64_t)dim; }

// Head widths with kernel instances.
inline bool kv_dim_ok(int dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256; }

struct KvView {
    uint8_t* data;
    int64_t pages;
    int page_size, heads, dim;
    int bpp_log2;                        // log2 of the blocks per page
};

// One sequence per entry: its newest cu[b + 1] - cu[b] tokens (rows cu[b] .. of the token arrays)
// are the last of the lens[b] that its pages table[b][0 ..] hold.
struct KvSeqs {
    const int32_t* table;
    int64_t table_ld;
    int table_cols;
    const int32_t* cu;
    const int32_t* lens;
    int batch;
    int64_t tokens;
};

struct KvSeq {
    int64_t first_row;                   // token row of its first new token
    int m;                               // new tokens
    int len;                             // tokens in the cache with them
};

// The sequence's numbers with every row inside [0, tokens] and every length at least 0.
__device__ __forceinline__ KvSeq kv_seq(int64_t tokens, int64_t lo, int64_t hi, int len) {
    KvSeq r;
    lo = lo < 0 ? 0 : (lo > tokens ? tokens : lo);
    hi = hi < lo ? lo : (hi > tokens ? tokens : hi);
    r.first_row = lo;
    r.m = (int)(hi - lo);
    r.len = len < 0 ? 0 : len;
    return r;
}
__device__ __forceinline__ KvSeq kv_seq(const KvSeqs& s, int b) { return kv_seq(s.tokens, s.cu[b], s.cu[b + 1], s.lens[b]); }

// Byte offset of word w of `lane` in a code plane.
template <int G>
__host__ __device__ __forceinline__ constexpr int kv_word_off(int w, int lane) {
    const int p = w >> 2;
    const int per = ((2 * G) & 3) == 2 && p == G / 2 ? 8 : 16;
    return p * 1024 + lane * per + (w & 3) * 4;
}

// Where token t of a block stands: q and the slot 4 ab + j of the values' words; key row
// i = 4 q + j of operand ab.
__host__ __device__ __forceinline__ constexpr int kv_q(int t) { return 2 * (t >> 4) + ((t >> 2) & 1); }
__host__ __device__ __forceinline__ constexpr int kv_slot(int t) { return 4 * ((t >> 3) & 1) + (t & 3); }
__host__ __device__ __forceinline__ constexpr int kv_tok(int q, int slot) {
    return 16 * (q >> 1) + 8 * (slot >> 2) + 4 * (q & 1) + (slot & 3);
}

// A word as four fp16 pairs of code - 8, exactly.  A nibble at bits 0..3 of a half under the exponent
// of 2^10 reads 1024 + code, one at bits 4..7 under that of 2^6 reads 64 + code: pairs 0 and 2 are
// off by 1024 + 8, pairs 1 and 3 by 64 + 8, and one shift serves a word.
constexpr float kBiasEven = 1032.0f, kBiasOdd = 72.0f;
// The constants are held in registers, which makes a biased pair one v_and_or_b32: 9 VALU a word.
struct Unpack {
    uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u, even = 0x64006400u, odd = 0x54005400u;
    __device__ __forceinline__ Unpack() {
        asm volatile("" : "+s"(lo), "+s"(hi));
        asm volatile("" : "+v"(even), "+v"(odd));
    }
    __device__ __forceinline__ u4 values(uint32_t w) const {
        const uint32_t w8 = w >> 8;
        const u4 b = {(w & lo) | even, (w & hi) | odd, (w8 & lo) | even, (w8 & hi) | odd};
        const h2 e = {(_Float16)kBiasEven, (_Float16)kBiasEven}, o = {(_Float16)kBiasOdd, (_Float16)kBiasOdd};
        return u4{bitcast<uint32_t>(bitcast<h2>(b[0]) - e), bitcast<uint32_t>(bitcast<h2>(b[1]) - o),
                  bitcast<uint32_t>(bitcast<h2>(b[2]) - e), bitcast<uint32_t>(bitcast<h2>(b[3]) - o)};
    }
};

// Bytes of the unit of (page, head, block in the page).
__device__ __forceinline__ int64_t kv_unit(const KvView& c, int64_t page, int head, int sub) {
    return (((page * c.heads + head) << c.bpp_log2) + sub) * kv_unit_bytes(c.dim);
}

}  // namespace q4gsw
