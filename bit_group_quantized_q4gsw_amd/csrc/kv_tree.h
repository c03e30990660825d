// Trees of drafted tokens over the 4-bit cache: what the attention kernels and the move of accepted
// paths share.
//
// The m new tokens of a sequence are nodes 0 .. m - 1; up[j] is node j's parent, a smaller number, or -1
// (a root).  A node sees the places before the tree, its ancestors and itself.  Attention keeps, per
// token of a workgroup's rows, that set as bits in LDS: word 0 stands for the 32 places before the tree
// (all ones), then a bit a node, then a word of zeros, and the node's depth last, so the 32 bits of any
// block of the cache that a row may see are two words and a funnel shift.
//
// Each thread climbs from one node: its ancestors come in falling order, so a word of bits is complete
// when the next smaller one begins, and every word is written once.  A step is one dependent LDS read,
// some 0.09 us; the climb runs while the first keys are on their way, but one of a deep tree is longer (1024 tokens, 8
// heads of 64, bf16, nodes in a chain against a star: 16 nodes 10.5 and 9.4 us, 64 15 and 9.5, 512 57 and 10.4).
#pragma once
#include "kv4.h"

namespace q4gsw {

constexpr int kTreeMax = 512;            // nodes of a sequence

__host__ __device__ inline int tree_words(int nodes) { return (nodes + 31) >> 5; }
__host__ __device__ inline int tree_stride(int nodes) { return tree_words(nodes) + 3; }
// Tokens that `rows` rows in a row may belong to, `group` rows a token.
__host__ __device__ inline int tree_tokens(int rows, int group, int nodes) {
    const int n = (rows + group - 2) / group + 1;
    return n < nodes ? n : nodes;
}
// Bytes of the parents (16 bits each) and the bits of `tokens` tokens.
__host__ __device__ inline int tree_bytes(int nodes, int tokens) {
    return 4 * ((nodes + 1) / 2) + 4 * tokens * tree_stride(nodes);
}

__device__ __forceinline__ int16_t tree_parent(int raw, int node) { return (int16_t)(raw >= 0 && raw < node ? raw : -1); }

struct KvTree {
    int16_t* up;
    uint32_t* bits;                      // [token - first][stride]
    int stride, words;

    __device__ __forceinline__ KvTree(uint8_t* at, int nodes)
        : up(reinterpret_cast<int16_t*>(at)), bits(reinterpret_cast<uint32_t*>(at + 4 * ((nodes + 1) / 2))),
          stride(tree_stride(nodes)), words(tree_words(nodes)) {}

    // The set of `node` (below `nodes`), of its ancestors only those fewer than `window` steps up (0: all).
    __device__ __forceinline__ void climb(int node, int window, uint32_t* row) const {
        row[0] = ~0u;
        row[words + 1] = 0u;
        uint32_t word = 0u;
        int w = words - 1, depth = 0;
        for (int j = node;;) {
            for (; w > (j >> 5); --w) {
                row[1 + w] = word;
                word = 0u;
            }
            if (!window || depth < window) word |= 1u << (j & 31);
            const int p = up[j];
            if (p < 0) break;
            j = p;
            ++depth;
        }
        for (; w >= 0; --w) {
            row[1 + w] = word;
            word = 0u;
        }
        row[words + 2] = (uint32_t)depth;
    }
    // The parent of `node` as the caller gave it.
    __device__ __forceinline__ void put(int node, int raw) const { up[node] = tree_parent(raw, node); }
    // All threads of the workgroup: the parents of the first `nodes` nodes of the sequence at token row
    // `first_row`, then the sets of tokens [tok0, tok0 + tokens).
    __device__ __forceinline__ void build(const int32_t* parents, int64_t first_row, int nodes, int tok0, int tokens, int window) const {
        for (int j = threadIdx.x; j < nodes; j += blockDim.x)
            put(j, parents[first_row + j]);
        __syncthreads();
        for (int t = threadIdx.x; t < tokens; t += blockDim.x) climb(tok0 + t, window, bits + t * stride);
        __syncthreads();
    }
    __device__ __forceinline__ int depth(int token) const { return (int)bits[token * stride + words + 2]; }
    // Bits of the 32 places from t0 on, which is not past the last node; p0: the place of node 0.
    __device__ __forceinline__ uint32_t block(int token, int t0, int p0) const {
        const int at = t0 < p0 - 32 ? 0 : t0 - p0 + 32;
        const uint32_t* row = bits + token * stride + (at >> 5);
        return __builtin_amdgcn_alignbit(row[1], row[0], at & 31);
    }
};

}  // namespace q4gsw
