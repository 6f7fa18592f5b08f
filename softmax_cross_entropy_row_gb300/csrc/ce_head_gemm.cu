// The three matrix products of a vocabulary projection and its loss, on the
// tensor cores (tcgen05) of CTA pairs:
//   logits  Z = H W^T        H [rows][D], W [C][D]: both operands lie along K
//   hidden  dH = E W         E [rows][C] along K, W along N
//   weight  dW = E^T H       E along M, H along N
// A persistent kernel: each pair of CTAs takes tiles of 256 x 256 in turn.
// One thread per CTA streams 64-wide slices of the operands into a ring of
// six stages by TMA (each CTA of the pair loads its 128 rows of A and its
// half of B, so a stage is 32 KB per SM and an operand byte is loaded once per
// pair), one thread of the first CTA issues the matrix instructions, and four
// warps per CTA drain the finished accumulator while the next tile's is being
// formed (two accumulators of 256 columns: all of tensor memory).
//
// The logits never leave the SM as logits: their epilogue turns a tile into
// its rows' maximum and sum of exponentials (without the target's class, whose
// logit is kept in fp32), and, when gradients follow, into 16-bit exponentials
// relative to the tile's maximum.
#include <math.h>

#include "ce_head_gemm.h"
#include "ce_launch.h"
#include "ce_tcgen05.cuh"

namespace ce {
namespace {

constexpr int kStages = 6;
constexpr int kCtaRows = kTileM / 2;               // rows of A and of B per CTA
constexpr int kOperandBytes = kCtaRows * kTileK * 2;  // 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kThreads = 256;
constexpr int kEpiWarp0 = 4;                       // warps 4..7: the epilogue
constexpr int kEpiBufs = 2;
constexpr int kEpiBufBytes = 32 * 128;             // 32 rows of 128 bytes
constexpr uint32_t kTmemCols = 512;

struct Barriers {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem;
};

constexpr int kSmemBytes =
    kStages * kStageBytes + 4 * kEpiBufs * kEpiBufBytes + 1024 /* alignment */ + sizeof(Barriers);

// The tile and part of work unit u: groups of group_m tile rows, walked down
// the columns of the group, so that neighbouring pairs share operands in L2.
struct Unit {
    int mt, nt, split;
};
__device__ __forceinline__ Unit unit_of(const HeadGemm &p, int u) {
    Unit r;
    const int tiles = p.tiles_m * p.tiles_n;
    r.split = u / tiles;
    u -= r.split * tiles;
    const int per_group = p.group_m * p.tiles_n;
    const int g = u / per_group;
    u -= g * per_group;
    const int first = g * p.group_m;
    const int gm = min(p.group_m, p.tiles_m - first);
    r.nt = u / gm;
    r.mt = first + (u - r.nt * gm);
    return r;
}
__device__ __forceinline__ void k_range(const HeadGemm &p, int split, int &k0, int &k1) {
    k0 = (int)((long long)p.k_blocks * split / p.splits);
    k1 = (int)((long long)p.k_blocks * (split + 1) / p.splits);
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

// The epilogue's staging boxes of one warp: two, so that one is filled while
// the other is on its way out.
struct Stager {
    unsigned char *base;
    int n;
    __device__ __forceinline__ unsigned char *open() {
        // the group that used this box two commits ago has been read
        if ((threadIdx.x & 31) == 0) bulk_wait_read<kEpiBufs - 1>();
        __syncwarp();
        return base + n * kEpiBufBytes;
    }
    template <typename F>
    __device__ __forceinline__ void close(F issue) {
        fence_proxy_async();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            issue(base + n * kEpiBufBytes);
            bulk_commit();
        }
        n ^= 1;
    }
};

template <typename E>
__device__ __forceinline__ void epi_logits(const HeadGemm &p, const Unit &u, uint32_t acc, int m0,
                                           Stager &st) {
    const int lane = threadIdx.x & 31;
    const int row = m0 + lane;
    const int n0 = u.nt * kTileN;
    const int cols = min(kTileN, p.cols - n0);
    int t = -1;
    if (p.targets != nullptr && row < p.rows) t = __ldg(p.targets + row) - n0;
    if (t >= cols) t = -1;
    float v[32];
    // the tile's maximum, the target left out
    float m = -INFINITY;
    for (int c = 0; c < cols; c += 32) {
        tmem_ld32(acc + c, v);
        tmem_wait_ld(v);
        if ((unsigned)(t - c) < 32u) {
            p.zt[row] = pick(v, t - c);
            put(v, t - c, -INFINITY);
        }
        if (c + 32 > cols) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i >= cols) v[i] = -INFINITY;
        }
        float a = v[0], b = v[1];
#pragma unroll
        for (int i = 2; i < 32; i += 2) {
            a = fmaxf(a, v[i]);
            b = fmaxf(b, v[i + 1]);
        }
        m = fmaxf(m, fmaxf(a, b));
    }
    // e^(z / T) = 2^(z exp_scale - M), M the fp32 value all of the tile uses
    const float M = m == -INFINITY ? 0.f : m * p.exp_scale - p.shift;
    const unsigned long long sc2 = f2_pack(p.exp_scale, p.exp_scale);
    const unsigned long long nM2 = f2_pack(-M, -M);
    unsigned long long sum2 = 0ull;
    for (int c0 = 0; c0 < cols; c0 += 64) {
        unsigned char *box = nullptr;
        if (p.write_exp) box = st.open();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 32 * h;
            tmem_ld32(acc + c, v);
            tmem_wait_ld(v);
            if ((unsigned)(t - c) < 32u) put(v, t - c, -INFINITY);
            if (c + 32 > cols) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i >= cols) v[i] = -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                unsigned long long e2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]), sc2, nM2), a,
                              b);
                    e2[i] = f2_pack(ex2(a), ex2(b));
                    sum2 = f2_add(sum2, e2[i]);
                }
                if (p.write_exp) stage16(box, lane, 4 * h + q, E::pack2(e2));
            }
        }
        if (p.write_exp) {
            st.close([&](const void *src) { tma_store(&p.out, src, n0 + c0, m0); });
        }
    }
    if (row < p.rows) {
        float a, b;
        f2_unpack(sum2, a, b);
        p.stats[(size_t)u.nt * p.rows + row] =
            make_float2(m == -INFINITY ? -INFINITY : M, a + b);
    }
}

template <typename E>
__device__ __forceinline__ void epi_out(const HeadGemm &p, const Unit &u, uint32_t acc, int m0,
                                        float f, Stager &st) {
    const int lane = threadIdx.x & 31;
    float v[32];
#pragma unroll 1
    for (int c0 = 0; c0 < min(kTileN, p.cols - u.nt * kTileN); c0 += 64) {
        unsigned char *box = st.open();
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
        st.close([&](const void *src) { tma_store(&p.out, src, u.nt * kTileN + c0, m0); });
    }
}

template <bool ADD>
__device__ __forceinline__ void epi_f32(const HeadGemm &p, const Unit &u, uint32_t acc, int m0,
                                        Stager &st) {
    const int lane = threadIdx.x & 31;
    const int y = (int)(u.split * p.split_rows) + m0;
    float v[32];
#pragma unroll 1
    for (int c = 0; c < min(kTileN, p.cols - u.nt * kTileN); c += 32) {
        unsigned char *box = st.open();
        tmem_ld32(acc + c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float x[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            stage16(box, lane, q, Elem<float>::pack(x));
        }
        st.close([&](const void *src) {
            if (ADD)
                tma_add(&p.out, src, u.nt * kTileN + c, y);
            else
                tma_store(&p.out, src, u.nt * kTileN + c, y);
        });
    }
}

// Waits that give up end the role's loop; every other role then gives up at
// its own next wait, so all threads reach the end of the kernel.
__device__ __forceinline__ bool wait_or_fail(const HeadGemm &p, uint64_t *bar, uint32_t parity,
                                             long long limit = kWaitLimitCycles) {
    if (mbar_wait_limit(bar, parity, limit)) return true;
    *reinterpret_cast<volatile int *>(p.failed) = 1;
    atomicAdd(&p.err[kErrTimeout], 1);
    return false;
}

template <int PROD, int EPI, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    head_gemm_kernel(const __grid_constant__ HeadGemm p) {
    using E = Elem<T>;
    constexpr bool kAMn = PROD == kProdWeight;
    constexpr bool kBMn = PROD != kProdLogits;
    constexpr bool kBf16 = E::kNegInfWord == Elem<__nv_bfloat16>::kNegInfWord;
    constexpr uint32_t kIdesc = instr_desc(kBf16, kAMn, kBMn, kTileM, kTileN);
    extern __shared__ unsigned char smem_raw[];
    // 1024-byte aligned (a swizzle atom), at the same offset in both CTAs
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *boxes = smem + kStages * kStageBytes;
    Barriers &bar = *reinterpret_cast<Barriers *>(boxes + 4 * kEpiBufs * kEpiBufBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int pairs = gridDim.x >> 1;
    const int units = p.tiles_m * p.tiles_n * p.splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.acc_full[i], 1);
            mbar_init(&bar.acc_empty[i], 8);  // four warps of each CTA
        }
        fence_mbar_init();
        prefetch_map(&p.a);
        prefetch_map(&p.b);
        prefetch_map(&p.out);
    }
    if (warp == 2) tmem_alloc_pair(&bar.tmem, kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&bar.tmem);
    pdl_trigger();
    pdl_wait();
    if (p.clear_failed && blockIdx.x == 0 && threadIdx.x == 0)
        *reinterpret_cast<volatile int *>(p.failed) = 0;

    if (warp == 0 && lane == 0) {
        // ---- the producer: this CTA's halves of A and B
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int w = pair; ok && w < units; w += pairs) {
            const Unit u = unit_of(p, w);
            const int m0 = u.mt * kTileM + rank * kCtaRows;
            const int n0 = u.nt * kTileN + rank * kCtaRows;
            int k0, k1;
            k_range(p, u.split, k0, k1);
            for (int k = k0; k < k1; ++k) {
                if (!(ok = wait_or_fail(p, &bar.empty[s], ph ^ 1u))) break;
                if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], 2 * kStageBytes);
                const uint32_t fb = mapa(&bar.full[s], 0);
                unsigned char *da = smem + s * kStageBytes;
                unsigned char *db = da + kOperandBytes;
                if constexpr (kAMn) {
                    tma_load_pair(da, &p.a, m0, k * kTileK, fb);
                    tma_load_pair(da + kOperandBytes / 2, &p.a, m0 + 64, k * kTileK, fb);
                } else {
                    tma_load_pair(da, &p.a, k * kTileK, m0, fb);
                }
                if constexpr (kBMn) {
                    tma_load_pair(db, &p.b, n0, k * kTileK, fb);
                    tma_load_pair(db + kOperandBytes / 2, &p.b, n0 + 64, k * kTileK, fb);
                } else {
                    tma_load_pair(db, &p.b, k * kTileK, n0, fb);
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
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        int it = 0;
        for (int w = pair; ok && w < units; w += pairs, ++it) {
            const Unit u = unit_of(p, w);
            int k0, k1;
            k_range(p, u.split, k0, k1);
            const int ab = it & 1;
            if (!(ok = wait_or_fail(p, &bar.acc_empty[ab], ((it >> 1) & 1) ^ 1))) break;
            tc_fence_after();
            const uint32_t d = tmem + ab * kTileN;
            for (int k = k0; k < k1; ++k) {
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
                    mma_pair(d, ad, bd, kIdesc, k > k0 || kk > 0);
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
        // ---- the epilogue: warp w drains lanes 32 (w mod 4) ..
        const int quad = warp & 3;
        Stager st;
        st.base = boxes + (warp - kEpiWarp0) * kEpiBufs * kEpiBufBytes;
        st.n = 0;
        float f = 1.f;
        if constexpr (EPI == kEpiOut) f = p.alpha * (p.scale ? __ldg(p.scale) : 1.f);
        // a whole contraction may lie between two finished accumulators
        const long long acc_limit = kWaitLimitCycles + 4096LL * p.k_blocks;
        int it = 0;
        for (int w = pair; w < units; w += pairs, ++it) {
            const Unit u = unit_of(p, w);
            const int ab = it & 1;
            if (!wait_or_fail(p, &bar.acc_full[ab], (it >> 1) & 1, acc_limit)) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + ab * kTileN;
            const int m0 = u.mt * kTileM + rank * kCtaRows + quad * 32;
            if (m0 < p.rows) {
                if constexpr (EPI == kEpiLogits) epi_logits<E>(p, u, acc, m0, st);
                if constexpr (EPI == kEpiOut) epi_out<E>(p, u, acc, m0, f, st);
                if constexpr (EPI == kEpiF32) epi_f32<false>(p, u, acc, m0, st);
                if constexpr (EPI == kEpiAdd) epi_f32<true>(p, u, acc, m0, st);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa(&bar.acc_empty[ab], 0));
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

template <int PROD, int EPI, typename T>
cudaError_t launch_t(const HeadGemm &p, int sms, cudaStream_t s) {
    const void *f = reinterpret_cast<const void *>(head_gemm_kernel<PROD, EPI, T>);
    cudaError_t e = ensure_smem_attr(f, kSmemBytes);
    if (e != cudaSuccess) return e;
    const long long units = (long long)p.tiles_m * p.tiles_n * p.splits;
    const long long pairs = units < sms / 2 ? units : sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, head_gemm_kernel<PROD, EPI, T>, p);
}

template <typename T>
cudaError_t launch_of(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, int sms,
                      cudaStream_t s) {
    if (prod == kProdLogits && epi == kEpiLogits)
        return launch_t<kProdLogits, kEpiLogits, T>(p, sms, s);
    if (prod == kProdHidden && epi == kEpiOut) return launch_t<kProdHidden, kEpiOut, T>(p, sms, s);
    if (prod == kProdHidden && epi == kEpiF32) return launch_t<kProdHidden, kEpiF32, T>(p, sms, s);
    if (prod == kProdWeight && epi == kEpiOut) return launch_t<kProdWeight, kEpiOut, T>(p, sms, s);
    if (prod == kProdWeight && epi == kEpiF32) return launch_t<kProdWeight, kEpiF32, T>(p, sms, s);
    if (prod == kProdWeight && epi == kEpiAdd) return launch_t<kProdWeight, kEpiAdd, T>(p, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_head_gemm(const HeadGemm &p, HeadProduct prod, HeadEpilogue epi, bool bf16,
                             int sms, cudaStream_t s) {
    return bf16 ? launch_of<__nv_bfloat16>(p, prod, epi, sms, s)
                : launch_of<__half>(p, prod, epi, sms, s);
}

}  // namespace ce
