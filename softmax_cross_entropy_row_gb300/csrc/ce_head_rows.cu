// Row kernels around the matrix products of a vocabulary projection's loss:
// everything that is not a matrix product.  A row's statistics come per column
// tile j, as a reference exponent M_j (log2) and the sum of exponentials S_j
// 2^M_j.  Its exponentials E_c are kept in 16 bits relative to
//   one exponent M per row (bf16, whose range is fp32's): a class known to be
//     likely, the target or the teacher's best, gives it before the product;
//     then G_c = mul E_c with one factor per row, which goes into the rows of
//     the products' other side, and E is written and read once; or to
//   one exponent per tile (f16): G_c = mul 2^(M_j - M) E_c, a pass over E.
// What is kept for the target, or the listed classes, is replaced by what makes
// their gradient exact: with S_rest the sum without the target, G_t = -mul
// S_rest (no difference of near values is formed).
#include <math.h>

#include "ce_head_rows.h"
#include "ce_launch.h"

namespace ce {
namespace {

cudaLaunchConfig_t config(unsigned gx, unsigned gy, unsigned threads, cudaStream_t s,
                          cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(gx, gy, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// The piece's rows that count.
__device__ __forceinline__ int piece_rows(const HeadRows &p) {
    if (!p.dynamic) return p.rows;
    return min(max(p.info->count - p.first, 0), p.rows);
}
// The batch's row of the piece's row i.
__device__ __forceinline__ int batch_row(const HeadRows &p, int i) {
    return p.perm ? p.perm[p.first + i] : p.first + i;
}

// ------------------------------------------------------------------- prep
// One CTA: the rows that count, in order, and the factors that keep the rows'
// own gradients within [-1, 1], so that they fit 16 bits whatever the upstream
// gradient is.
constexpr int kPrepThreads = 1024;
__global__ void __launch_bounds__(kPrepThreads) head_prep_kernel(HeadPrep p) {
    __shared__ float norms[32];
    __shared__ int counts[32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // each warp has a run of rows, 32 at a time: first their count, then, with
    // the counts of the warps before it, their places
    const long long run = (p.B + 1023) / 1024 * 32;
    const long long b0 = min(p.B, run * warp), b1 = min(p.B, b0 + run);
    int n = 0, bad = 0;
    float norm = 0.f;
#pragma unroll 4
    for (long long b = b0 + lane; b < b1; b += 32) {
        bool c;
        float w = p.scale_per_row ? fabsf(__ldg(p.scale + b)) : 1.f;
        if (p.targets) {
            const int t = __ldg(p.targets + b);
            c = t != p.ignore_index;
            bad += c && (t < 0 || t >= p.C);
        } else {
            const float mass = p.mass[b];
            c = mass != 0.f;
            w *= fmaxf(fabsf(mass), 1.f);
        }
        n += c;
        if (c) norm = fmaxf(norm, w);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    norm = warp_max(norm);
    if (lane == 0) {
        counts[warp] = n;
        norms[warp] = norm;
    }
    if (p.perm && bad) atomicAdd(&p.err[kErrBadTarget], bad);
    __syncthreads();
    const int before = lane < warp ? counts[lane] : 0;
    int at = __reduce_add_sync(0xffffffffu, before);
    const int total = __reduce_add_sync(0xffffffffu, counts[lane]);
    norm = warp_max(norms[lane]);
    if (p.perm) {
#pragma unroll 4
        for (long long i = b0; i < b1; i += 32) {
            const long long b = i + lane;
            bool c = false;
            float mass = 0.f;
            if (b < b1) {
                if (!p.targets) mass = p.mass[b];
                c = p.targets ? __ldg(p.targets + b) != p.ignore_index : mass != 0.f;
            }
            const unsigned those = __ballot_sync(0xffffffffu, c);
            const int place = at + __popc(those & ((1u << lane) - 1u));
            at += __popc(those);
            if (c) {
                p.pos[b] = place;
                p.perm[place] = (int)b;
            } else if (b < b1) {
                p.pos[b] = -1;
                p.loss[b] = !p.targets && signbit(mass) ? NAN : 0.f;
            }
        }
    }
    if (threadIdx.x == 0) {
        if (!(norm > 0.f) || isinf(norm)) norm = 1.f;
        const float up = p.scale != nullptr && !p.scale_per_row ? __ldg(p.scale) : 1.f;
        const float by = p.mean_of_all ? (float)p.B : (float)max(total, 1);
        p.info->count = total;
        p.info->norm = norm;
        p.info->out = p.alpha * norm * up * (p.mean ? 1.f / by : 1.f);
    }
}

// ------------------------------------------------------------------- pack
// A warp per row of the batch (and per row of padding): the hidden states of
// the rows that count together, if not all do; zeros as the gradient of the
// others; the logit of one likely class, whose exponent is the row's reference
// (rounded to an integer: powers of two scale the exponentials exactly).
template <typename T>
__global__ void __launch_bounds__(256) head_pack_kernel(HeadPack p) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long b = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int count = p.info->count, nv = p.D / 8;
    if (b >= p.B) {  // rows count .. of the last 64 are zeros
        const long long at = count + (b - p.B);
        if (count < p.B && at < ((long long)count + 63) / 64 * 64)
            for (int v = lane; v < nv; v += 32)
                reinterpret_cast<uint4 *>(p.packed + (size_t)at * p.D * 2)[v] =
                    make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int pos = p.pos[b];
    if (pos < 0) {
        if (p.dhidden)
            for (int v = lane; v < nv; v += 32)
                reinterpret_cast<uint4 *>(p.dhidden + (size_t)b * p.D * 2)[v] =
                    make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const uint4 *h = reinterpret_cast<const uint4 *>(p.hidden + (size_t)b * p.D * 2);
    uint4 *to = reinterpret_cast<uint4 *>(p.packed + (size_t)pos * p.D * 2);
    const bool dot = p.targets != nullptr && p.ref != nullptr;
    int c = dot ? __ldg(p.targets + b) : 0;
    const bool has = c >= 0 && c < p.C;
    if (!has) c = 0;  // any class: its logit is not above the largest
    const uint4 *w = reinterpret_cast<const uint4 *>(p.weight + (size_t)c * p.D * 2);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (dot || count < p.B) {
#pragma unroll 4
        for (int v = lane; v < nv; v += 32) {
            const uint4 x = __ldg(h + v);
            if (count < p.B) to[v] = x;
            if (dot) {
                float a[8], y[8];
                E::unpack(x, a);
                E::unpack(__ldg(w + v), y);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j & 3] = fmaf(a[j], y[j], acc[j & 3]);
            }
        }
    }
    if (p.ref == nullptr) return;
    float z = warp_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
    if (!dot) {
        z = -INFINITY;
        for (int k = lane; k < p.K; k += 32) {
            const int i = __ldg(p.idx + b * p.K + k);
            if (i >= 0 && i < p.C) z = fmaxf(z, p.zk[b * p.K + k]);
        }
        z = warp_max(z);
    }
    if (lane == 0) {
        const float r = rintf(z * p.exp_scale);
        p.ref[pos] = fabsf(r) <= 1e30f ? r : 0.f;
        if (dot) p.zt[pos] = z;
    }
}

// ---------------------------------------------------------------- teacher
// A warp per row: the teacher's log-probabilities over its list.
template <typename V>
__device__ __forceinline__ float teacher_value(const void *val, long long i) {
    return Elem<V>::load_global(static_cast<const unsigned char *>(val) + i * Elem<V>::kBytes);
}
__device__ __forceinline__ float teacher_at(const HeadTeacher &p, long long i) {
    return p.val_dtype == 0   ? teacher_value<float>(p.val, i)
           : p.val_dtype == 1 ? teacher_value<__nv_bfloat16>(p.val, i)
                              : teacher_value<__half>(p.val, i);
}

__global__ void __launch_bounds__(256) head_teacher_kernel(HeadTeacher p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long b = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (b >= p.B) return;
    const long long i0 = b * p.K;
    float m = -INFINITY;
    bool bad = false;
    for (int k = lane; k < p.K; k += 32) {
        const int c = __ldg(p.idx + i0 + k);
        if (c < -1 || c >= p.C) bad = true;
        if (c >= 0 && c < p.C) m = fmaxf(m, teacher_at(p, i0 + k));
    }
    m = warp_max(m);
    float ref;  // log of what the exponentials are divided by, relative to m
    if (p.lse != nullptr) {
        ref = __ldg(p.lse + b) - m * p.inv_t;
    } else {
        float s = 0.f;
        for (int k = lane; k < p.K; k += 32) {
            const int c = __ldg(p.idx + i0 + k);
            if (c >= 0 && c < p.C) s += expf((teacher_at(p, i0 + k) - m) * p.inv_t);
        }
        ref = logf(warp_sum(s));
    }
    float mass = 0.f;
    for (int k = lane; k < p.K; k += 32) {
        const int c = __ldg(p.idx + i0 + k);
        float lq = -INFINITY;
        if (c >= 0 && c < p.C && m != -INFINITY) {  // m = -inf: no place has a probability
            lq = (teacher_at(p, i0 + k) - m) * p.inv_t - ref;
            mass += expf(lq);
        }
        p.logq[i0 + k] = lq;
    }
    mass = warp_sum(mass);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        p.mass[b] = bad ? -mass : mass;
        if (bad) atomicAdd(&p.err[kErrBadTarget], 1);
    }
}

// A warp per place of a list: z = hidden_b . weight_c in fp32.
template <typename T>
__global__ void __launch_bounds__(256) head_dots_kernel(HeadTeacher p) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * 8;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < p.B * p.K; i += warps) {
        const int c = __ldg(p.idx + i);
        if (c < 0 || c >= p.C) continue;
        const uint4 *h = reinterpret_cast<const uint4 *>(p.hidden + (size_t)(i / p.K) * p.D * 2);
        const uint4 *w = reinterpret_cast<const uint4 *>(p.weight + (size_t)c * p.D * 2);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int v = lane; v < p.D / 8; v += 32) {
            float a[8], x[8];
            E::unpack(__ldg(h + v), a);
            E::unpack(__ldg(w + v), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j & 3] = fmaf(a[j], x[j], acc[j & 3]);
        }
        const float z = warp_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
        if (lane == 0) p.zk[i] = z;
    }
}

// ------------------------------------------------------------- statistics
// R rows per CTA, 256 / R threads a row, each over every (256 / R)-th tile;
// joined in a tree whose shape depends on R alone.
struct MS {
    float M, S;
};
__device__ __forceinline__ MS join(MS a, MS b) {
    const float M = fmaxf(a.M, b.M);
    if (M == -INFINITY) return {M, a.S + b.S};
    return {M, a.S * ex2(a.M - M) + b.S * ex2(b.M - M)};
}

// Above this sum (relative to the reference exponent) the exponentials come
// near the top of bf16's range, and their factors near its bottom.
constexpr float kRescueSum = 1.152921504606847e18f;  // 2^60

template <int R, typename T>
__global__ void __launch_bounds__(256) head_rows_kernel(HeadRows p) {
    using E = Elem<T>;
    constexpr int P = 256 / R;
    __shared__ MS sh[256];
    pdl_trigger();
    pdl_wait();
    if (p.only_if != nullptr && *reinterpret_cast<const volatile int *>(p.only_if) == 0) return;
    const int rows = piece_rows(p);
    const int r = threadIdx.x % R;
    const int part = threadIdx.x / R;
    const int row = blockIdx.x * R + r;
    if (blockIdx.x * R >= rows) return;
    const bool per_row = p.ref != nullptr;
    MS acc = {-INFINITY, 0.f};
    if (row < rows) {
        const float2 *st = p.stats + row;
        if (per_row) {
#pragma unroll 8
            for (int j = part; j < p.tiles; j += P) {
                const float2 v = __ldcg(st + (size_t)j * p.rows);
                acc.M = fmaxf(acc.M, v.x);
                acc.S += v.y;
            }
        } else {
#pragma unroll 8
            for (int j = part; j < p.tiles; j += P) {
                const float2 v = __ldcg(st + (size_t)j * p.rows);
                acc = join(acc, {v.x, v.y});
            }
        }
    }
    sh[threadIdx.x] = acc;
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (part < o) {
            const MS x = sh[threadIdx.x], y = sh[threadIdx.x + o * R];
            sh[threadIdx.x] = per_row ? MS{fmaxf(x.M, y.M), x.S + y.S} : join(x, y);
        }
    }
    if (part != 0 || row >= rows) return;
    MS a = sh[threadIdx.x];
    const int b = batch_row(p, row);
    // the row's own factor, relative to the largest
    float w = 1.f;
    if (p.want_grad) w = (p.row_scale ? __ldg(p.row_scale + b) : 1.f) / p.info->norm;
    HeadRow out;
    const int t = p.targets ? __ldg(p.targets + b) : -1;
    const bool has = t >= 0 && t < p.C;
    const float zt = has ? p.zt[row] * p.exp_scale : -INFINITY;
    if (per_row) {
        if (p.flag_rescue && !(a.S <= kRescueSum)) {
            // the products are formed again with the row's largest exponent
            const float top = ceilf(fmaxf(a.M, zt));
            p.ref[row] = fabsf(top) <= 1e30f ? top : 0.f;
            *reinterpret_cast<volatile int *>(&p.info->rescue) = 1;
            return;
        }
        a.M = p.ref[row];
    }
    if (p.targets != nullptr) {
        float l;
        if (!p.want_grad && t == p.ignore_index) {
            l = 0.f;
            out = {0.f, 0.f, 0.f, 0.f};
        } else {
            out.M = per_row ? a.M : fmaxf(a.M, zt);
            const float rest = a.M == -INFINITY ? a.S : a.S * ex2(a.M - out.M);
            const float e = has ? ex2(zt - out.M) : 0.f;
            const float S = rest + e;
            l = rest < e ? log1pf(rest / e) : kLn2 * (log2f(S) - (zt - out.M));
            if (!has) {
                l = NAN;
                if (!p.want_grad) atomicAdd(&p.err[kErrBadTarget], 1);
            }
            out.mul = w / S * (per_row ? 1.f : p.shift_mul);
            out.target = has ? -(rest / S) * w * p.shift_mul : 0.f;
            out.log2S = log2f(S);
            if (per_row && has)
                E::store(p.exps + ((size_t)row * p.ld + t) * 2, -rest);
        }
        if (p.nan_on_failure && p.info->failed) l = NAN;
        p.loss[b] = l;
    } else {
        const float mass = fabsf(p.mass[b]);
        out.M = a.M;
        out.mul = mass * w / a.S * (per_row ? 1.f : p.shift_mul);
        // what a listed class's p - q / mass (mass p - q) is multiplied by to be kept
        out.target = per_row ? a.S : w * p.shift_mul;
        out.log2S = log2f(a.S);
    }
    p.row[row] = out;
}

// ------------------------------------------------------ kept exponentials
// A warp per 256 columns of a row (two half tiles, a factor for each half of the
// warp), eight of them in flight.
constexpr int kScaleTiles = 8;
template <typename T>
__global__ void __launch_bounds__(256) head_scale_kernel(HeadRows p) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int tiles = p.tiles / 2;
    const long long groups = (tiles + kScaleTiles - 1) / kScaleTiles;
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= groups * piece_rows(p)) return;
    const int row = (int)(i / groups);
    const int j0 = (int)(i - row * groups) * kScaleTiles;
    const HeadRow h = p.row[row];
    const int t = p.targets ? __ldg(p.targets + batch_row(p, row)) : -1;
    unsigned char *base = p.exps + ((size_t)row * p.ld) * 2;
    uint4 x[kScaleTiles];
    float f[kScaleTiles];
#pragma unroll
    for (int k = 0; k < kScaleTiles; ++k) {
        const long long c = (long long)(j0 + k) * 256 + lane * 8;
        if (c < p.ld) x[k] = *reinterpret_cast<const uint4 *>(base + c * 2);
        const int j = 2 * (j0 + k) + (lane >> 4);
        f[k] = j < p.tiles ? ex2(__ldcg(&p.stats[(size_t)j * p.rows + row].x) - h.M) * h.mul : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kScaleTiles; ++k) {
        const long long c = (long long)(j0 + k) * 256 + lane * 8;
        if (c >= p.ld) continue;
        float v[8];
        E::unpack(x[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f[k];
        if (t >= c && t < c + 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (t - c == e) v[e] = h.target;
        }
        *reinterpret_cast<uint4 *>(base + c * 2) = E::pack(v);
    }
}

// A warp per row (and per row of padding up to 64): h mul in bf16, for E^T h.
__global__ void __launch_bounds__(256) head_scale_hidden_kernel(HeadRows p) {
    using E = Elem<__nv_bfloat16>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int rows = piece_rows(p);
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (rows + 63) / 64 * 64) return;
    uint4 *to = reinterpret_cast<uint4 *>(p.scaled + (size_t)row * p.D * 2);
    const unsigned char *src = p.info->count < p.B ? p.packed : p.hidden;
    const uint4 *h = reinterpret_cast<const uint4 *>(src + (size_t)row * p.D * 2);
    const float mul = row < rows ? p.row[row].mul : 0.f;
#pragma unroll 4
    for (int v = lane; v < p.D / 8; v += 32) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) {
            float a[8];
            E::unpack(__ldcg(h + v), a);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] *= mul;
            x = E::pack(a);
        }
        to[v] = x;
    }
}

// ----------------------------------------------------------------- listed
// A warp per row: the divergence from the teacher, and the gradients of the
// listed classes, mass p_c - sum of the teacher's probabilities at c, from the
// fp32 logits (the kept exponentials' rounding must not meet the difference).
template <typename T>
__global__ void __launch_bounds__(256) head_listed_kernel(HeadRows p) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= piece_rows(p)) return;
    const HeadRow h = p.row[row];
    const int b = batch_row(p, row);
    const float signed_mass = p.mass[b];
    const float mass = fabsf(signed_mass);
    const long long i0 = (long long)b * p.K;
    float l = 0.f;
    for (int k = lane; k < p.K; k += 32) {
        const int c = __ldg(p.idx + i0 + k);
        if (c < 0 || c >= p.C) continue;
        const float lq = p.logq[i0 + k];
        const float lp2 = p.zk[i0 + k] * p.exp_scale - h.M - h.log2S;
        const float q = expf(lq);
        if (q != 0.f) l += q * (lq - kLn2 * lp2);
        if (!p.want_grad) continue;
        // one place per class writes: the first, with all of them added
        float all = 0.f;
        bool first = true;
        for (int j = 0; j < p.K; ++j) {
            if (__ldg(p.idx + i0 + j) != c) continue;
            if (j < k) first = false;
            all += expf(p.logq[i0 + j]);
        }
        if (first)
            E::store(p.exps + ((size_t)row * p.ld + c) * 2,
                     (p.ref ? ex2(lp2) - all / mass : mass * ex2(lp2) - all) * h.target);
    }
    l = warp_sum(l);
    if (lane == 0) {
        l = signbit(signed_mass) ? NAN : mass == 0.f ? 0.f : l * p.temperature * p.temperature;
        if (p.nan_on_failure && p.info->failed) l = NAN;
        p.loss[b] = l;
    }
}

// ------------------------------------------------------------------- loss
__global__ void __launch_bounds__(kTailThreads)
    head_loss_kernel(float *rows, long long B, int reduction, int mean_of_all, const HeadInfo *info,
                     float *out) {
    __shared__ float2 scratch[kTailWarps];
    pdl_trigger();
    pdl_wait();
    const bool failed = info->failed != 0;
    if (reduction == kReduceNone) {
        if (failed)
            for (long long b = threadIdx.x; b < B; b += kTailThreads) rows[b] = NAN;
        return;
    }
    Params p = {};
    p.loss_rows = rows;
    p.B = B;
    const float2 v = tail_virtual_warp(p, threadIdx.x >> 5, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        float h = 0.f, l = 0.f;
        for (int w = 0; w < kTailWarps; ++w) {
            float s, e;
            two_sum(h, scratch[w].x, s, e);
            h = s;
            l += scratch[w].y + e;
        }
        double r = (double)h + (double)l;
        if (reduction == kReduceMean) r /= mean_of_all ? (double)B : (double)max(info->count, 1);
        *out = failed ? NAN : (float)r;
    }
}

}  // namespace

cudaError_t launch_head_prep(const HeadPrep &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(1, 1, kPrepThreads, s, attr);
    return cudaLaunchKernelEx(&cfg, head_prep_kernel, p);
}

cudaError_t launch_head_teacher(const HeadTeacher &p, bool bf16, int sms, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((p.B + 7) / 8), 1, 256, s, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, head_teacher_kernel, p);
    if (e != cudaSuccess) return e;
    const long long ctas = (p.B * p.K + 7) / 8;
    cfg = config((unsigned)(ctas < 64LL * sms ? ctas : 64LL * sms), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_dots_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_dots_kernel<__half>, p);
}

cudaError_t launch_head_pack(const HeadPack &p, bool bf16, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((p.B + 64 + 7) / 8), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_pack_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_pack_kernel<__half>, p);
}

namespace {
template <typename T>
cudaError_t rows_of(const HeadRows &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    // eight rows per CTA (32 threads each), or one where that leaves SMs idle
    if (p.rows <= 256) {
        cudaLaunchConfig_t cfg = config((unsigned)p.rows, 1, 256, s, attr);
        return cudaLaunchKernelEx(&cfg, head_rows_kernel<1, T>, p);
    }
    cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 7) / 8), 1, 256, s, attr);
    return cudaLaunchKernelEx(&cfg, head_rows_kernel<8, T>, p);
}
}  // namespace

cudaError_t launch_head_rows(const HeadRows &p, bool bf16, cudaStream_t s) {
    return bf16 ? rows_of<__nv_bfloat16>(p, s) : rows_of<__half>(p, s);
}

cudaError_t launch_head_scale(const HeadRows &p, bool bf16, cudaStream_t s) {
    const long long groups = (p.tiles / 2 + kScaleTiles - 1) / kScaleTiles;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((groups * p.rows + 7) / 8), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_scale_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_scale_kernel<__half>, p);
}

cudaError_t launch_head_scale_hidden(const HeadRows &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 63) / 64 * 8), 1, 256, s, attr);
    return cudaLaunchKernelEx(&cfg, head_scale_hidden_kernel, p);
}

cudaError_t launch_head_listed(const HeadRows &p, bool bf16, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 7) / 8), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_listed_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_listed_kernel<__half>, p);
}

cudaError_t launch_head_loss(float *rows, long long B, int reduction, int mean_of_all,
                             const HeadInfo *info, float *loss_out, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(1, 1, kTailThreads, s, attr);
    return cudaLaunchKernelEx(&cfg, head_loss_kernel, rows, B, reduction, mean_of_all, info,
                              loss_out);
}

}  // namespace ce
