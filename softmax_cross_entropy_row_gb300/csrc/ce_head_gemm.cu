// The three matrix products of a vocabulary projection and its loss, on the
// tensor cores (tcgen05) of CTA pairs:
//   logits  Z = H W^T        H [rows][D], W [C][D]: both operands lie along K
//   score   Z^T = W H^T      the same for few rows
//   hidden  dH = E W         E [rows][C] along K, W along N
//   weight  dW = E^T H       E along M, H along N
// A persistent kernel: each pair of CTAs takes tiles of 256 x 256 in turn.
// One thread per CTA streams 64-wide slices of the operands into a ring of
// six stages by TMA (each CTA of the pair loads its 128 rows of A and its
// half of B, so a stage is 32 KB per SM and an operand byte is loaded once per
// pair), one thread of the first CTA issues the matrix instructions, and eight
// warps per CTA (32 rows and half of the columns each) drain the finished
// accumulator while the next tile's is being formed (two accumulators of 256
// columns: all of tensor memory).
//
// The logits never leave the SM as logits: their epilogue turns a tile into
// its rows' maximum and sum of exponentials (without the target's class), and,
// when gradients follow, into 16-bit exponentials.
#include <math.h>

#include "ce_head_gemm.h"
#include "ce_launch.h"
#include "ce_tcgen05.cuh"

namespace ce {
namespace {

constexpr int kCtaRows = kTileM / 2;                  // rows of A and of B per CTA
constexpr int kOperandBytes = kCtaRows * kTileK * 2;  // 16 KB
// The ring: six stages of 16 + 16 KB; with few rows as B eleven of 16 + 4 KB.
constexpr int kMaxStages = 11;
__host__ __device__ constexpr int stages_of(int prod) { return prod == kProdScore ? 11 : 6; }
__host__ __device__ constexpr int stage_bytes(int prod) {
    return kOperandBytes + (prod == kProdScore ? kScoreRows / 2 * kTileK * 2 : kOperandBytes);
}
constexpr int kEpiWarp0 = 4;                       // warps 4..11: the epilogue
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kEpiBufBytes = 32 * 128;             // 32 rows of 128 bytes
constexpr uint32_t kTmemCols = 512;

struct Barriers {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem;
};

__host__ __device__ constexpr int box_bytes(int prod) {
    return prod == kProdScore ? 0 : kEpiWarps * kEpiBufBytes;
}
constexpr int smem_bytes(int prod) {
    return stages_of(prod) * stage_bytes(prod) + box_bytes(prod) + 1024 /* alignment */ +
           (int)sizeof(Barriers);
}

// Work unit u: a tile, and the part [k0, k1) of its contraction.
struct Unit {
    int mt, nt, k0, k1;
    int part;  // -1: all of it, else the part's place among the parts
};
__device__ __forceinline__ Unit unit_of(const HeadGemm &p, const HeadWork &w, int u) {
    Unit r;
    int tile = u, split = 0, splits = 1;
    r.part = -1;
    if (u >= w.full) {
        r.part = u - w.full;
        splits = w.splits;
        tile = w.full + r.part / splits;
        split = r.part % splits;
    }
    head_tile(p, w, tile, &r.mt, &r.nt);
    r.k0 = (int)((long long)w.k_blocks * split / splits);
    r.k1 = (int)((long long)w.k_blocks * (split + 1) / splits);
    return r;
}

// 16 bytes of row `row` of a 128-byte wide staging box, in TMA's 128-byte
// swizzle (16-byte piece c of row r lies at piece c ^ (r mod 8)).
__device__ __forceinline__ void stage16(unsigned char *box, int row, int piece, uint4 v) {
    *reinterpret_cast<uint4 *>(box + row * 128 + ((piece ^ (row & 7)) << 4)) = v;
}

// Element j of v set to x (selects, no indexing).
__device__ __forceinline__ void put(float (&v)[32], int j, float x) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i == j ? x : v[i];
}
__device__ __forceinline__ float pick(const float (&v)[32], int j) {
    float x = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) x = i == j ? v[i] : x;
    return x;
}

// The epilogue's staging box of one warp.  open() waits until the box's last
// store has read it (it has had the time of a TMEM load and the arithmetic).
struct Stager {
    unsigned char *box;
    __device__ __forceinline__ void open() {
        if ((threadIdx.x & 31) == 0) bulk_wait_read<0>();
        __syncwarp();
    }
    template <typename F>
    __device__ __forceinline__ void close(F issue) {
        fence_proxy_async();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            issue(box);
            bulk_commit();
        }
    }
};

// The staged box (32 rows of 128 bytes) to 32 rows of a row-major matrix, 16
// bytes per lane: rows `at` (each lane's own row's address, nullptr: none),
// as many of their bytes as are inside.
__device__ __forceinline__ void unstage(const unsigned char *box, unsigned char *at, int bytes) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3), piece = lane & 7;
        unsigned char *dst = reinterpret_cast<unsigned char *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), r));
        if (dst != nullptr && piece * 16 < bytes)
            *reinterpret_cast<uint4 *>(dst + piece * 16) =
                *reinterpret_cast<const uint4 *>(box + r * 128 + ((piece ^ (r & 7)) << 4));
    }
    __syncwarp();
}

// Row m0 + lane of this piece, and its target's column in this tile (-1:
// elsewhere, or none).
struct LogitRow {
    int row, target;
    bool counts;
};
__device__ __forceinline__ LogitRow logit_row(const HeadGemm &p, const HeadWork &w, int m0, int n0,
                                              int cols) {
    LogitRow r;
    r.row = m0 + (threadIdx.x & 31);
    r.counts = r.row < w.rows;
    r.target = -1;
    if (p.targets != nullptr && r.counts) {
        const int at = p.first + r.row;
        r.target = __ldg(p.targets + (p.perm ? p.perm[at] : at)) - n0;
        if (r.target >= cols) r.target = -1;
    }
    return r;
}

// Columns c .. c + 31 of a tile of `cols`, the target and what lies outside
// read as -inf.
__device__ __forceinline__ void load_logits(float (&v)[32], uint32_t acc, int c, int cols,
                                            const LogitRow &r) {
    tmem_ld32(acc + c, v);
    tmem_wait_ld(v);
    if ((unsigned)(r.target - c) < 32u) put(v, r.target - c, -INFINITY);
    if (c + 32 > cols) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (c + i >= cols) v[i] = -INFINITY;
    }
}
__device__ __forceinline__ float max32(const float (&v)[32]) {
    float a = v[0], b = v[1];
#pragma unroll
    for (int i = 2; i < 32; i += 2) {
        a = fmaxf(a, v[i]);
        b = fmaxf(b, v[i + 1]);
    }
    return fmaxf(a, b);
}
// 2^(v exp_scale - M) of 32 logits: added to `sum`, and (KEEP) staged as
// pieces piece0 .. of this lane's row.
template <typename E, bool KEEP>
__device__ __forceinline__ void exponentials(const float (&v)[32], float exp_scale, float M,
                                             unsigned long long &sum, unsigned char *box,
                                             int piece0, bool zero) {
    const unsigned long long sc2 = f2_pack(exp_scale, exp_scale), nM2 = f2_pack(-M, -M);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        unsigned long long e2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]), sc2, nM2), a, b);
            e2[i] = f2_pack(ex2(a), ex2(b));
            sum = f2_add(sum, e2[i]);
        }
        if (KEEP)
            stage16(box, threadIdx.x & 31, piece0 + q,
                    zero ? make_uint4(0u, 0u, 0u, 0u) : E::pack2(e2));
    }
}

// The tile's maxima first, then its exponentials relative to them: (M, S) with
// the tile's sum of exponentials S 2^M.
template <typename E, bool KEEP>
__device__ __forceinline__ void epi_tile_max(const HeadGemm &p, const HeadWork &w, const Unit &u,
                                             uint32_t acc, int m0, int half, Stager &st) {
    const int n0 = u.nt * p.tile_n + half * (p.tile_n / 2);
    const int cols = min(p.tile_n / 2, p.C - n0);
    const LogitRow r = logit_row(p, w, m0, n0, cols);
    float v[32];
    float m = -INFINITY;
    for (int c = 0; c < cols; c += 32) {
        tmem_ld32(acc + c, v);
        tmem_wait_ld(v);
        if ((unsigned)(r.target - c) < 32u) {
            p.zt[r.row] = pick(v, r.target - c);
            put(v, r.target - c, -INFINITY);
        }
        if (c + 32 > cols) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i >= cols) v[i] = -INFINITY;
        }
        m = fmaxf(m, max32(v));
    }
    const float M = m == -INFINITY ? 0.f : m * p.exp_scale - p.shift;
    unsigned long long sum = 0ull;
    for (int c0 = 0; c0 < cols; c0 += 64) {
        load_logits(v, acc, c0, cols, r);
        if (KEEP) st.open();
        exponentials<E, KEEP>(v, p.exp_scale, M, sum, st.box, 0, !r.counts);
        if (KEEP || c0 + 32 < cols) {
            load_logits(v, acc, c0 + 32, cols, r);
            exponentials<E, KEEP>(v, p.exp_scale, M, sum, st.box, 4, !r.counts);
        }
        if (KEEP) st.close([&](const void *src) { tma_store(&p.out, src, n0 + c0, m0); });
    }
    if (r.counts) {
        float a, b;
        f2_unpack(sum, a, b);
        p.stats[(size_t)(2 * u.nt + half) * p.rows + r.row] =
            make_float2(m == -INFINITY ? -INFINITY : M, a + b);
    }
}

// Few rows: stages k, k + 4, .. of a contraction add to an accumulator of their
// own (64 columns each; tensor memory has the room), and the four sums are
// added in fp32.  The tensor core's additions cut off low bits: on 64 rows x
// 128256 classes x 4096 the loss was off by 2.8e-6 with one accumulator.
constexpr int kScoreChains = 4;

// This lane's class against 32 rows of the batch.  A row's maximum
// and sum over the warp's classes: one reduction instruction per row for the
// maximum, a transposing tree of shuffles (lane i ends with row i) for the sum.
__device__ __forceinline__ void epi_score(const HeadGemm &p, const Unit &u, uint32_t acc,
                                          int class0, int classes, int stat, int row0,
                                          int chains) {
    const int lane = threadIdx.x & 31;
    float v[32], e[32];
    tmem_ld32(acc + row0, v);
    tmem_wait_ld(v);
    for (int i = 1; i < chains; ++i) {
        tmem_ld32(acc + i * kScoreRows + row0, e);
        tmem_wait_ld(e);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += e[j];
    }
    const int row = row0 + lane;
    int target = -1;
    if (p.targets != nullptr && row < p.rows) target = __ldg(p.targets + p.first + row);
    float mine = -INFINITY;  // row `row`'s maximum
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (lane >= classes) v[i] = -INFINITY;
        const int t = __shfl_sync(0xffffffffu, target, i);
        if (t >= 0 && t == class0 + lane && lane < classes && row0 + i < p.rows) {
            p.zt[row0 + i] = v[i];
            v[i] = -INFINITY;
        }
        const float m = warp_max(v[i]);
        if (i == lane) mine = m;
        const float M = m == -INFINITY ? 0.f : m * p.exp_scale;
        e[i] = ex2(fmaf(v[i], p.exp_scale, -M));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float give = up ? e[i] : e[i + o], keep = up ? e[i + o] : e[i];
            e[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    if (row < p.rows)
        p.stats[(size_t)(u.mt * kScoreStats + stat) * p.rows + row] =
            make_float2(mine == -INFINITY ? -INFINITY : mine * p.exp_scale, e[0]);
}

// Exponentials relative to the row's given exponent, in one pass: (m, S) with
// the tile's largest exponent m and its sum of exponentials S 2^ref.
template <typename E>
__device__ __forceinline__ void epi_ref(const HeadGemm &p, const HeadWork &w, const Unit &u,
                                        uint32_t acc, int m0, int half, Stager &st) {
    const int n0 = u.nt * kTileN + half * kStatN;
    const int cols = min(kStatN, p.C - n0);
    const LogitRow r = logit_row(p, w, m0, n0, cols);
    const float M = r.counts ? p.ref[r.row] : 0.f;
    float v[32];
    float m = -INFINITY;
    unsigned long long sum = 0ull;
    for (int c0 = 0; c0 < cols; c0 += 64) {
        load_logits(v, acc, c0, cols, r);
        m = fmaxf(m, max32(v));
        st.open();
        exponentials<E, true>(v, p.exp_scale, M, sum, st.box, 0, !r.counts);
        load_logits(v, acc, c0 + 32, cols, r);
        m = fmaxf(m, max32(v));
        exponentials<E, true>(v, p.exp_scale, M, sum, st.box, 4, !r.counts);
        st.close([&](const void *src) { tma_store(&p.out, src, n0 + c0, m0); });
    }
    if (r.counts) {
        float a, b;
        f2_unpack(sum, a, b);
        p.stats[(size_t)(2 * u.nt + half) * p.rows + r.row] = make_float2(m * p.exp_scale, a + b);
    }
}

// A part of a tile in fp32 to its place among the parts.
__device__ __forceinline__ void epi_part(const HeadGemm &p, const Unit &u, uint32_t acc, int row0,
                                         int half, Stager &st) {
    const int lane = threadIdx.x & 31;
    float *at = p.parts + (size_t)u.part * (kTileM * kTileN) + (size_t)(row0 + lane) * kTileN +
                half * kStatN;
    float v[32];
    st.open();  // a store of the tile before may still read the box
    unsigned char *box = st.box;
#pragma unroll 1
    for (int c = 0; c < kStatN; c += 32) {
        tmem_ld32(acc + c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float x[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            stage16(box, lane, q, Elem<float>::pack(x));
        }
        unstage(box, reinterpret_cast<unsigned char *>(at + c), 128);
    }
}

// The hidden states' gradient: row i's sum times its own factor, to its
// place in the call's batch.
template <typename E>
__device__ __forceinline__ void epi_hidden(const HeadGemm &p, const HeadWork &w, const Unit &u,
                                           uint32_t acc, int m0, int half, float f, Stager &st) {
    const int lane = threadIdx.x & 31;
    const int row = m0 + lane;
    const bool counts = row < w.rows;
    unsigned char *at = nullptr;
    if (counts) {
        if (p.row_mul) f *= p.row_mul[(size_t)row * p.row_mul_stride];
        const int b = p.perm ? p.perm[p.first + row] : p.first + row;
        at = p.dhidden + (size_t)b * p.D * 2;
    }
    float v[32];
    const int n0 = u.nt * kTileN + half * kStatN;
    const int cols = min(kStatN, p.D - n0);
    unsigned char *box = st.box;
#pragma unroll 1
    for (int c0 = 0; c0 < cols; c0 += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tmem_ld32(acc + c0 + 32 * h, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = f * v[8 * q + i];
                stage16(box, lane, 4 * h + q, E::pack(x));
            }
        }
        unstage(box, at ? at + (size_t)(n0 + c0) * 2 : nullptr, (cols - c0) * 2);
    }
}

// The weights' gradient in 16 bits (`zero`: no row counts).  All 128 columns are
// read first and the accumulator is handed back (`release`) before they are
// stored.
template <typename E, typename R>
__device__ __forceinline__ void epi_weight(const HeadGemm &p, const Unit &u, uint32_t acc, int m0,
                                           int half, float f, bool zero, Stager &st, R release) {
    const int lane = threadIdx.x & 31;
    float v[4][32];
    const int n0 = u.nt * kTileN + half * kStatN;
    const int cols = min(kStatN, p.D - n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_ld32(acc + 32 * i, v[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_wait_ld(v[i]);
    release();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (c * 64 >= cols) break;
        uint4 w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = zero ? 0.f : f * v[2 * c + q / 4][q % 4 * 8 + i];
            w[q] = E::pack(x);
        }
        st.open();
#pragma unroll
        for (int q = 0; q < 8; ++q) stage16(st.box, lane, q, w[q]);
        st.close([&](const void *src) { tma_store(&p.out, src, n0 + 64 * c, m0); });
    }
}

// The weights' gradient in fp32, over several pieces of the rows.
template <bool ADD>
__device__ __forceinline__ void epi_f32(const HeadGemm &p, const Unit &u, uint32_t acc, int m0,
                                        int half, bool zero, Stager &st) {
    const int lane = threadIdx.x & 31;
    float v[32];
    const int n0 = u.nt * kTileN + half * kStatN;
    const int cols = min(kStatN, p.D - n0);
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
        tmem_ld32(acc + c, v);
        tmem_wait_ld(v);
        st.open();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float x[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            stage16(st.box, lane, q, zero ? make_uint4(0u, 0u, 0u, 0u) : Elem<float>::pack(x));
        }
        st.close([&](const void *src) {
            if (ADD)
                tma_add(&p.out, src, n0 + c, m0);
            else
                tma_store(&p.out, src, n0 + c, m0);
        });
    }
}

// Waits that give up end the role's loop; every other role then gives up at
// its own next wait, so all threads reach the end of the kernel.
__device__ __forceinline__ bool wait_or_fail(const HeadGemm &p, uint64_t *bar, uint32_t parity,
                                             long long more = 0) {
    if (mbar_wait_limit(bar, parity, p.wait_limit + more)) return true;
    *reinterpret_cast<volatile int *>(p.failed) = 1;
    atomicAdd(&p.err[kErrTimeout], 1);
    return false;
}

template <int PROD, int EPI, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    head_gemm_kernel(const __grid_constant__ HeadGemm p) {
    using E = Elem<T>;
    constexpr bool kAMn = PROD == kProdWeight;
    constexpr bool kBMn = PROD == kProdHidden || PROD == kProdWeight;
    constexpr int kStages = stages_of(PROD);
    constexpr int kStageBytes = stage_bytes(PROD);
    constexpr bool kBf16 = E::kNegInfWord == Elem<__nv_bfloat16>::kNegInfWord;
    extern __shared__ unsigned char smem_raw[];
    // 1024-byte aligned (a swizzle atom), at the same offset in both CTAs
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *boxes = smem + kStages * kStageBytes;
    Barriers &bar = *reinterpret_cast<Barriers *>(boxes + box_bytes(PROD));

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.acc_full[i], 1);
            mbar_init(&bar.acc_empty[i], 2 * kEpiWarps);  // of both CTAs
        }
        fence_mbar_init();
        prefetch_map(&p.a);
        prefetch_map(&p.b);
        prefetch_map(&p.out);
        prefetch_map(&p.packed);
    }
    if (warp == 2) tmem_alloc_pair(&bar.tmem, kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&bar.tmem);
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (p.clear_failed) *reinterpret_cast<volatile int *>(p.failed) = 0;
        if (p.clear_rescue) *reinterpret_cast<volatile int *>(p.rescue) = 0;
    }
    const bool skip =
        p.only_if != nullptr && *reinterpret_cast<const volatile int *>(p.only_if) == 0;
    const int count = p.dynamic ? p.info->count : p.B;
    const bool packed = count < p.B;
    const HeadWork work = head_work(p, (HeadProduct)PROD, count, pairs);
    const int units = skip || (EPI == kEpiAdd && work.rows == 0) ? 0 : work.units;
    // the operand that is the hidden states (logits: A; weights: B)
    const CUtensorMap *map_a = PROD == kProdLogits && packed ? &p.packed : &p.a;
    const CUtensorMap *map_b = PROD == kProdWeight && packed ? &p.packed : &p.b;
    const int half_n = p.tile_n / 2;  // rows of B per CTA
    const int half_m = p.tile_m / 2;  // rows of A per CTA (the rest of its 128 do not matter)

    if (warp == 0 && lane == 0) {
        // ---- the producer: this CTA's halves of A and B
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int w = pair; ok && w < units; w += pairs) {
            const Unit u = unit_of(p, work, w);
            const int m0 = u.mt * p.tile_m + rank * half_m;
            const int n0 = u.nt * p.tile_n + rank * half_n;
            for (int k = u.k0; k < u.k1; ++k) {
                if (!(ok = wait_or_fail(p, &bar.empty[s], ph ^ 1u))) break;
                // test hook: this stage's copies are left out
                const bool skip_copy = p.skip_row >= 0 && k == u.k0 &&
                                       u.mt * p.tile_m == p.skip_row / kTileM * kTileM;
                if (rank == 0 && !skip_copy)
                    mbar_arrive_expect_tx(&bar.full[s], 2 * (half_m + half_n) * kTileK * 2);
                const uint32_t fb = mapa(&bar.full[s], 0);
                if (!skip_copy) {
                    unsigned char *da = smem + s * kStageBytes;
                    unsigned char *db = da + kOperandBytes;
                    if constexpr (kAMn) {
                        tma_load_pair(da, map_a, m0, k * kTileK, fb);
                        tma_load_pair(da + kOperandBytes / 2, map_a, m0 + 64, k * kTileK, fb);
                    } else {
                        tma_load_pair(da, map_a, k * kTileK, m0, fb);
                    }
                    if constexpr (kBMn) {
                        tma_load_pair(db, map_b, n0, k * kTileK, fb);
                        tma_load_pair(db + kOperandBytes / 2, map_b, n0 + 64, k * kTileK, fb);
                    } else {
                        tma_load_pair(db, map_b, k * kTileK, n0, fb);
                    }
                }
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && rank == 0) {
            // copies still in flight land before shared memory is given up
            // (the pair's copies all complete on this CTA's barriers)
            const int n = min(issued, kStages);
            for (int i = 0; i < n; ++i) {
                s = s == 0 ? kStages - 1 : s - 1;
                if (s == kStages - 1) ph ^= 1u;
                mbar_wait_limit(&bar.full[s], ph, kWaitLimitCycles);
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- the matrix instructions of the pair
        const uint32_t idesc = instr_desc(kBf16, kAMn, kBMn, kTileM, p.tile_n);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        int it = 0;
        for (int w = pair; ok && w < units; w += pairs, ++it) {
            const Unit u = unit_of(p, work, w);
            const int ab = it & 1;
            if (!(ok = wait_or_fail(p, &bar.acc_empty[ab], ((it >> 1) & 1) ^ 1))) break;
            tc_fence_after();
            constexpr int kChains = PROD == kProdScore ? kScoreChains : 1;
            for (int k = u.k0; k < u.k1; ++k) {
                const uint32_t d = tmem + ab * kTileN +
                                   (kChains > 1 ? (k % kChains) * kScoreRows : 0);
                if (!(ok = wait_or_fail(p, &bar.full[s], ph))) break;
                tc_fence_after();
                const uint32_t a = smem_addr(smem + s * kStageBytes);
                const uint32_t b = a + kOperandBytes;
#pragma unroll
                for (int kk = 0; kk < kTileK / 16; ++kk) {
                    const uint64_t ad = kAMn ? smem_desc(a + kk * 2048, kOperandBytes / 2, 1024)
                                             : smem_desc(a + kk * 32, 16, 1024);
                    const uint64_t bd = kBMn ? smem_desc(b + kk * 2048, kOperandBytes / 2, 1024)
                                             : smem_desc(b + kk * 32, 16, 1024);
                    mma_pair(d, ad, bd, idesc, k >= u.k0 + kChains || kk > 0);
                }
                commit_pair(&bar.empty[s]);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) commit_pair(&bar.acc_full[ab]);
        }
    } else if (warp >= kEpiWarp0) {
        // ---- the epilogue: warp w drains lanes 32 (w mod 4) .., half of the
        // columns
        const int quad = warp & 3;
        const int half = (warp - kEpiWarp0) >> 2;
        Stager st;
        st.box = boxes + (warp - kEpiWarp0) * kEpiBufBytes;
        float f = 1.f;
        if constexpr (EPI == kEpiOut) f = p.alpha * p.info->out;
        // a whole contraction may lie between two finished accumulators
        const long long acc_more = 4096LL * work.k_blocks;
        // rows of the product; of the logits also those up to the next 64,
        // whose kept exponentials are zeros (the last stage of E^T H reads them)
        const int rows = PROD == kProdWeight ? p.C
                         : PROD == kProdLogits ? (work.rows + 63) / 64 * 64 : work.rows;
        const bool zero = work.k_blocks == 0;
        int it = 0;
        for (int w = pair; w < units; w += pairs, ++it) {
            const Unit u = unit_of(p, work, w);
            const int ab = it & 1;
            if (!wait_or_fail(p, &bar.acc_full[ab], (it >> 1) & 1, acc_more)) break;
            tc_fence_after();
            const uint32_t acc =
                tmem + ((uint32_t)(quad * 32) << 16) + ab * kTileN + half * (p.tile_n / 2);
            const int row0 = rank * kCtaRows + quad * 32;
            const int m0 = u.mt * kTileM + row0;
            bool released = false;
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa(&bar.acc_empty[ab], 0));
                released = true;
            };
            if constexpr (PROD == kProdScore) {
                // this warp's classes, and every second 32 rows of the batch
                const int class0 = u.mt * p.tile_m + rank * half_m + quad * 32;
                const int classes = min(half_m - quad * 32, p.C - class0);
                for (int r0 = half * 32; r0 < work.rows; r0 += 64)
                    epi_score(p, u, tmem + ((uint32_t)(quad * 32) << 16) + ab * kTileN, class0,
                              classes, rank * 4 + quad, r0, min(kScoreChains, work.k_blocks));
            } else if (m0 < rows) {
                if constexpr (EPI == kEpiStats || EPI == kEpiKeep)
                    epi_tile_max<E, EPI == kEpiKeep>(p, work, u, acc, m0, half, st);
                if constexpr (EPI == kEpiRef) epi_ref<E>(p, work, u, acc, m0, half, st);
                if constexpr (EPI == kEpiOut) {
                    if (u.part >= 0)
                        epi_part(p, u, acc, row0, half, st);
                    else if constexpr (PROD == kProdHidden)
                        epi_hidden<E>(p, work, u, acc, m0, half, f, st);
                    else
                        epi_weight<E>(p, u, acc, m0, half, f, zero, st, release);
                }
                if constexpr (EPI == kEpiF32) epi_f32<false>(p, u, acc, m0, half, zero, st);
                if constexpr (EPI == kEpiAdd) epi_f32<true>(p, u, acc, m0, half, zero, st);
            }
            if (!released) release();
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------- the parts
// A warp adds 128 columns of a row of a
// split tile, its parts in order.
template <int PROD, typename T>
__global__ void __launch_bounds__(256)
    head_join_kernel(const __grid_constant__ HeadGemm p, unsigned char *out, int pairs) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const HeadWork work =
        head_work(p, (HeadProduct)PROD, p.dynamic ? p.info->count : p.B, pairs);
    const int m_rows = PROD == kProdWeight ? p.C : work.rows;
    const float f0 = p.alpha * p.info->out;
    for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < work.rest * kTileM * 2;
         i += gridDim.x * 8) {
        const int r = i / (kTileM * 2), y = i / 2 % kTileM, x = i % 2 * 128 + lane * 4;
        int mt, nt;
        head_tile(p, work, work.full + r, &mt, &nt);
        const int row = mt * kTileM + y, col = nt * kTileN + x;
        if (row >= m_rows || col >= p.D) continue;
        const float *src = p.parts + (size_t)r * work.splits * (kTileM * kTileN) +
                           (size_t)y * kTileN + x;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int q = 0; q < work.splits; ++q) {
            const float4 a = __ldcg(
                reinterpret_cast<const float4 *>(src + (size_t)q * (kTileM * kTileN)));
            v.x += a.x;
            v.y += a.y;
            v.z += a.z;
            v.w += a.w;
        }
        float f = f0;
        size_t at = row;
        if (PROD == kProdHidden) {
            if (p.row_mul) f *= p.row_mul[(size_t)row * p.row_mul_stride];
            at = p.perm ? p.perm[p.first + row] : p.first + row;
        }
        *reinterpret_cast<uint2 *>(out + (at * p.D + col) * 2) =
            make_uint2(E::pack2(f * v.x, f * v.y), E::pack2(f * v.z, f * v.w));
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
    head_convert_kernel(const float *parts, long long n, const HeadInfo *info, float alpha,
                        unsigned char *out) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const float f = alpha * info->out;
    const long long step = (long long)gridDim.x * 256 * 8;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += step) {
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(parts + i));
        const float4 b = __ldcg(reinterpret_cast<const float4 *>(parts + i + 4));
        const float v[8] = {f * a.x, f * a.y, f * a.z, f * a.w, f * b.x, f * b.y, f * b.z, f * b.w};
        *reinterpret_cast<uint4 *>(out + i * 2) = E::pack(v);
    }
}

cudaLaunchConfig_t config(unsigned ctas, unsigned threads, size_t smem, cudaStream_t s,
                          cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int PROD, int EPI, typename T>
cudaError_t launch_t(const HeadGemm &p, int pairs, cudaStream_t s) {
    const void *f = reinterpret_cast<const void *>(head_gemm_kernel<PROD, EPI, T>);
    cudaError_t e = ensure_smem_attr(f, smem_bytes(PROD));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)(2 * pairs), kThreads, smem_bytes(PROD), s, attr);
    return cudaLaunchKernelEx(&cfg, head_gemm_kernel<PROD, EPI, T>, p);
}

template <typename T>
cudaError_t launch_of(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, int pairs,
                      cudaStream_t s) {
    if (prod == kProdScore && epi == kEpiStats)
        return launch_t<kProdScore, kEpiStats, T>(p, pairs, s);
    if (prod == kProdLogits && epi == kEpiStats)
        return launch_t<kProdLogits, kEpiStats, T>(p, pairs, s);
    if (prod == kProdLogits && epi == kEpiKeep)
        return launch_t<kProdLogits, kEpiKeep, T>(p, pairs, s);
    if (prod == kProdLogits && epi == kEpiRef)
        return launch_t<kProdLogits, kEpiRef, T>(p, pairs, s);
    if (prod == kProdHidden && epi == kEpiOut)
        return launch_t<kProdHidden, kEpiOut, T>(p, pairs, s);
    if (prod == kProdWeight && epi == kEpiOut)
        return launch_t<kProdWeight, kEpiOut, T>(p, pairs, s);
    if (prod == kProdWeight && epi == kEpiF32)
        return launch_t<kProdWeight, kEpiF32, T>(p, pairs, s);
    if (prod == kProdWeight && epi == kEpiAdd)
        return launch_t<kProdWeight, kEpiAdd, T>(p, pairs, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_head_gemm(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, bool bf16,
                             int pairs, cudaStream_t s) {
    return bf16 ? launch_of<__nv_bfloat16>(p, prod, epi, pairs, s)
                : launch_of<__half>(p, prod, epi, pairs, s);
}

cudaError_t launch_head_join(const HeadGemm &p, HeadProduct prod, void *out, bool bf16, int pairs,
                             cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)(8 * pairs), 256, 0, s, attr);
    unsigned char *o = static_cast<unsigned char *>(out);
    if (prod == kProdHidden)
        return bf16 ? cudaLaunchKernelEx(&cfg, head_join_kernel<kProdHidden, __nv_bfloat16>, p, o,
                                         pairs)
                    : cudaLaunchKernelEx(&cfg, head_join_kernel<kProdHidden, __half>, p, o, pairs);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_join_kernel<kProdWeight, __nv_bfloat16>, p, o,
                                     pairs)
                : cudaLaunchKernelEx(&cfg, head_join_kernel<kProdWeight, __half>, p, o, pairs);
}

cudaError_t launch_head_convert(const float *parts, long long n, const HeadInfo *info, float alpha,
                                void *out, bool bf16, int sms, cudaStream_t s) {
    long long ctas = (n / 8 + 255) / 256;
    if (ctas > 16LL * sms) ctas = 16LL * sms;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)ctas, 256, 0, s, attr);
    unsigned char *o = static_cast<unsigned char *>(out);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_convert_kernel<__nv_bfloat16>, parts, n, info,
                                     alpha, o)
                : cudaLaunchKernelEx(&cfg, head_convert_kernel<__half>, parts, n, info, alpha, o);
}

}  // namespace ce
