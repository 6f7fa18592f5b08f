// Host-side interface of the projection's matrix products (ce_head_gemm.cu),
// and what their kernels and the row kernels (ce_head_rows.cu) agree on.
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
// Columns of a tile that one warp drains; the logits' statistics are per half
// tile.
constexpr int kStatN = kTileN / 2;

// What the launches of one call share on the device.
struct HeadInfo {
    int count;    // rows that count (not ignored, not without a list)
    float out;    // factor of the gradients (what is not in the rows' own)
    float norm;   // what the rows' own factors are divided by
    int failed;   // a bounded wait gave up
    int rescue;   // a row's reference exponent was too low
};

// What becomes of a tile.
enum HeadEpilogue {
    kEpiStats = 0,  // row maxima and sums of exponentials alone
    kEpiKeep = 1,   // these, and the exponentials relative to the tile's maxima
    kEpiRef = 2,    // these, and the exponentials relative to a given exponent per row
    kEpiOut = 3,    // scaled, rounded to 16 bits
    kEpiF32 = 4,    // fp32, stored
    kEpiAdd = 5,    // fp32, added to what is there
};

// Which way the operands lie: the logits (both rows along K), the gradient of
// the hidden states (weights along N) and of the weights (both along M, N).
// For few rows the logits are formed the other way round, Z^T = W H^T (score):
// the classes then fill the tensor cores' 256 rows and the memory's whole rate
// goes into the weights' copies.
enum HeadProduct { kProdLogits = 0, kProdHidden = 1, kProdWeight = 2, kProdScore = 3 };
constexpr int kScoreRows = 64;  // rows of the batch, at most
constexpr int kScoreStats = 8;  // statistics per tile: 32 classes each

struct HeadGemm {
    CUtensorMap a, b, out;
    CUtensorMap packed;            // the hidden states without the rows that do not count
    const HeadInfo *info;
    int B;                         // rows of the call
    int dynamic;                   // only the rows that count: [first, first + rows) of them
    int first, rows;               // rows of this piece, at most
    int C, D;
    int tile_n;                    // kEpiStats: width of a tile (else kTileN)
    int tile_m;                    // score: classes of a tile, in two halves (else kTileM)
    int group_m;                   // tile rows that are walked together
    int may_split;                 // the last tiles' contraction may be split
    float *parts;                  // fp32 tiles of the split parts (kMaxParts a pair)
    float alpha;                   // kEpiOut: times info->out
    // logits
    float exp_scale;               // log2(e) / temperature
    float shift;                   // kEpiKeep: the exponentials are kept times 2^shift
    const int32_t *targets;        // [B], nullptr: none
    const int *perm;               // the counting rows' places, nullptr: all in order
    float2 *stats;                 // [half column tiles][rows]
    float *zt;                     // [rows] target logits (kEpiStats, kEpiKeep)
    const float *ref;              // [rows] reference exponents
    const int *only_if;            // nullptr, or: nothing to do unless set
    int clear_failed, clear_rescue;
    // dhidden
    const float *row_mul;          // row i's factor row_mul[i * row_mul_stride], or nullptr
    int row_mul_stride;
    unsigned char *dhidden;        // [B][D]
    int *failed, *rescue;
    long long wait_limit;          // cycles after which a wait gives up
    int skip_row;                  // test hook: the tile row from this row on lacks a copy; -1
    int *err;                      // error counters
};

// Parts of tiles whose contraction is split, at most, per pair of CTAs.
constexpr int kMaxParts = 4;

// The tiles of a product over `pairs` pairs of CTAs: whole rounds of tiles are
// computed whole; the contraction of the `rest` tiles of the last round is
// split into `splits` parts each, so that all pairs share them.
struct HeadWork {
    int rows;       // rows of this piece
    int tiles_m, tiles_n, k_blocks;
    int full, rest, splits, units;
};

#ifdef __CUDACC__
// The parts (of at most 64, and kMaxParts per pair) that cost `rest` tiles of
// k_blocks stages the least: a stage takes about 0.35 us, a part more, for its
// 256 KB written and read and the launch that adds them up.  Every lane of the
// warp tries two numbers and all get the answer.
__device__ __forceinline__ int head_splits(int rest, int k_blocks, int pairs) {
    const int lane = threadIdx.x & 31;
    unsigned best = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 1 + 32 * i;
        if (s > 1 && (rest * s > kMaxParts * pairs || k_blocks < 8 * s)) continue;
        const unsigned rounds = (unsigned)(rest * s + pairs - 1) / (unsigned)pairs;
        const unsigned ns = rounds * ((unsigned)(k_blocks + s - 1) / (unsigned)s) * 350u +
                            (s > 1 ? 4000u + 80u * (unsigned)(rest * s) : 0u);
        // in units of 64 ns, the number of parts below
        best = min(best, (min(ns, 0xfffffffu) / 64u) << 6 | (unsigned)(s - 1));
    }
    return (int)(__reduce_min_sync(0xffffffffu, best) & 63u) + 1;
}
// Called by whole warps.
__device__ __forceinline__ HeadWork head_work(const HeadGemm &p, HeadProduct prod, int count,
                                              int pairs) {
    HeadWork w;
    w.rows = p.rows;
    if (p.dynamic) w.rows = min(max(count - p.first, 0), p.rows);
    const int m = prod == kProdWeight || prod == kProdScore ? p.C : w.rows;
    const int n = prod == kProdLogits ? p.C : prod == kProdScore ? w.rows : p.D;
    const int k = prod == kProdLogits || prod == kProdScore ? p.D
                  : prod == kProdHidden ? p.C : w.rows;
    w.tiles_m = (m + p.tile_m - 1) / p.tile_m;
    w.tiles_n = (n + p.tile_n - 1) / p.tile_n;
    w.k_blocks = (k + kTileK - 1) / kTileK;
    const int tiles = w.tiles_m * w.tiles_n;
    w.full = tiles;
    w.rest = 0;
    w.splits = 1;
    if (p.may_split && tiles > 0) {
        const int rest = tiles % pairs;
        w.splits = rest > 0 ? head_splits(rest, w.k_blocks, pairs) : 1;
        if (w.splits > 1) {
            w.rest = rest;
            w.full = tiles - rest;
        }
    }
    w.units = w.full + w.rest * w.splits;
    return w;
}
#endif

// Tile t of the walk: groups of group_m tile rows, down the columns of each,
// so that pairs working at the same time share operands in L2.
__host__ __device__ inline void head_tile(const HeadGemm &p, const HeadWork &w, int t, int *mt,
                                          int *nt) {
    const int per_group = p.group_m * w.tiles_n;
    const int g = t / per_group;
    t -= g * per_group;
    const int first = g * p.group_m;
    const int gm = p.group_m < w.tiles_m - first ? p.group_m : w.tiles_m - first;
    *nt = t / gm;
    *mt = first + (t - *nt * gm);
}

cudaError_t launch_head_gemm(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, bool bf16,
                             int pairs, cudaStream_t s);
// The split parts of a product added up, in their order (nothing to do where
// nothing was split).  out: dhidden's rows or the weights' gradient.
cudaError_t launch_head_join(const HeadGemm &p, HeadProduct prod, void *out, bool bf16, int pairs,
                             cudaStream_t s);
// out[i] = alpha info->out parts[i], n elements (a multiple of 8), to 16 bits.
cudaError_t launch_head_convert(const float *parts, long long n, const HeadInfo *info, float alpha,
                                void *out, bool bf16, int sms, cudaStream_t s);

}  // namespace ce
