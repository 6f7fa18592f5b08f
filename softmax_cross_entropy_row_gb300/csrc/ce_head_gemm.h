// Host-side interface of the projection's matrix products (ce_head_gemm.cu).
// Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "ce_device.cuh"

namespace ce {

// One matrix product is computed in tiles of kTileM x kTileN, each by a pair
// of CTAs (kTileM / 2 rows of the tile per CTA), kTileK of the contraction per
// stage.
constexpr int kTileM = 256;
constexpr int kTileN = 256;
constexpr int kTileK = 64;

// What becomes of a tile.
enum HeadEpilogue {
    kEpiLogits = 0,  // row maxima and sums of exponentials, the exponentials in 16 bits
    kEpiOut = 1,     // scaled, rounded to 16 bits
    kEpiF32 = 2,     // fp32, stored (partial sums)
    kEpiAdd = 3,     // fp32, added to what is there
};

// Which way the operands lie: the logits (both rows along K), the gradient of
// the hidden states (weights along N) and of the weights (both along M, N).
enum HeadProduct { kProdLogits = 0, kProdHidden = 1, kProdWeight = 2 };

struct HeadGemm {
    CUtensorMap a, b, out;
    int tiles_m, tiles_n, splits;  // output tiles, parts of the contraction
    int k_blocks;                  // stages of the whole contraction
    int group_m;                   // tile rows that are walked together
    long long split_rows;          // output rows from one part to the next
    const float *scale;            // kEpiOut: device factor
    float alpha;                   //          times this
    int rows, cols;                // of the product
    // kEpiLogits
    float exp_scale;               // log2(e) / temperature
    float shift;                   // the exponentials are kept times 2^shift
    const int32_t *targets;        // nullptr: none
    float2 *stats;                 // [tiles_n][rows]: (M, S), sum of e^z = S 2^M over the tile
    float *zt;                     // [rows] target logits
    int write_exp;                 // 0: the statistics alone
    int *failed;                   // set when a wait gave up
    int clear_failed;              // the call's first launch clears it
    int *err;                      // error counters
};

cudaError_t launch_head_gemm(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, bool bf16,
                             int sms, cudaStream_t s);

}  // namespace ce
