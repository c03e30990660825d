// Sets of low-rank adapters: layout in memory and launches (adapter_set.hip).
//
// A slot is the factors of one adapter in 16 bits, both in runs of 1 KB, 16 bytes a lane (lane = i + 16 q),
// zeros past its rank, K and N:
//   * A, runs [step of 32 columns][tile of 16 ranks]: lane (i, q) holds rank 16 tile + i, columns 32 step
//     + 8 q .. + 7: a 16x16x32 operand;
//   * B, runs [block of 32 outputs][step of 16 ranks]: lane (i, q) holds ranks 16 step + 4 q .. + 3 of
//     output 32 block + adapter_col(i, 0), then of adapter_col(i, 1): two 16x16x16 operands whose products
//     leave eight neighbouring outputs in a lane.
// Behind the slots stand their alphas, fp32.
#pragma once
#include "device.h"

namespace q4gsw {

constexpr int kAdapterRank = 64, kAdapterSlots = 1 << 20;

// The output of a block whose ranks lane i holds in half h: the product's rows 4 q' + r are outputs 8 q' + 4 h + r.
__host__ __device__ __forceinline__ constexpr int adapter_col(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

struct AdapterSet {
    uint8_t* data;
    float* alpha;
    int64_t N, K, n_pad, k_pad;
    int64_t slot_bytes, b_offset;
    int slots, rank_tiles, dtype;
};

struct AdapterArgs {
    AdapterSet set;
    const void* x;
    int64_t M, K, N;
    const int32_t* slot;
    const float* y;
    float* out;
    float* t;                // [chunk][M][16 rank_tiles]
    int chunks;              // of K
    int groups;              // workgroups that share a tile's adapters in the first launch
    int rank_tiles;
    int64_t col_groups;
    int share;               // waves that share a chunk of K
};

bool adapters_launch_ok(const AdapterSet& set, int64_t M);
uint64_t adapters_ws_bytes(const AdapterSet& set, int64_t M);
// One slot's A [rank][K] and B [N][rank] in src_dtype.
hipError_t launch_adapters_load(const AdapterSet& set, int slot, const void* A, const void* B, int src_dtype, int rank, float alpha,
                                hipStream_t s);
hipError_t launch_adapters_add(const AdapterSet& set, const void* x, int x_dtype, int64_t M, const int32_t* slot, const float* y,
                               float* out, void* ws, hipStream_t s);
// out = the sums of `splits` planes of partials [M rounded up to 32, width] in the fragment layout (internal.h)
// + the adapters' terms; t: adapters_ws_bytes bytes beside the partials.
hipError_t launch_adapters_join(const AdapterSet& set, const void* x, int x_dtype, int64_t M, const int32_t* slot, const float* part,
                                int splits, int64_t width, float* out, void* t, hipStream_t s);

}  // namespace q4gsw
