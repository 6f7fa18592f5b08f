// Row kernels around the matrix products of a vocabulary projection's loss:
// everything that is not a matrix product.  With (M_j, S_j) the reference
// exponent and the sum of exponentials of row b over column tile j,
//   M = max_j M_j,  S = sum_j S_j 2^(M_j - M),
//   p_c = E_c 2^(M_j - M) / S            (E_c the kept 16-bit exponential),
// and the row's gradient with respect to its logits is written over E.
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

__device__ __forceinline__ float block_max_256(float v, float *scratch) {
    v = warp_max(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) v = fmaxf(v, scratch[i]);
    return v;
}

// ------------------------------------------------------------------- prep
// One CTA: the rows that count (mean), and the factors that keep the rows'
// own gradients within [-1, 1] times the teacher's mass, so that they fit 16
// bits whatever the upstream gradient is.
constexpr int kPrepThreads = 1024;
__global__ void __launch_bounds__(kPrepThreads) head_prep_kernel(HeadPrep p) {
    __shared__ float scratch[kPrepThreads / 32];
    __shared__ int total;
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    int n = 0;
    float norm = 0.f;
    for (long long b = threadIdx.x; b < p.B; b += kPrepThreads) {
        const bool counts = p.targets == nullptr || __ldg(p.targets + b) != p.ignore_index;
        n += counts;
        float w = p.scale_per_row ? fabsf(__ldg(p.scale + b)) : 1.f;
        if (p.mass != nullptr) w *= fmaxf(p.mass[b], 1.f);
        norm = fmaxf(norm, w);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) atomicAdd(&total, n);
    norm = block_max_256(norm, scratch);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!(norm > 0.f) || isinf(norm)) norm = 1.f;
        const float up = p.scale != nullptr && !p.scale_per_row ? __ldg(p.scale) : 1.f;
        p.info->count = total;
        p.info->norm = norm;
        p.info->out = p.alpha * norm * up * (p.mean ? 1.f / (float)max(total, 1) : 1.f);
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
        if (c >= 0 && c < p.C) {
            lq = (teacher_at(p, i0 + k) - m) * p.inv_t - ref;
            mass += expf(lq);
        }
        p.logq[i0 + k] = lq;
    }
    mass = warp_sum(mass);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        p.mass[b] = mass;
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

template <int R>
__global__ void __launch_bounds__(256) head_rows_kernel(HeadRows p) {
    constexpr int P = 256 / R;
    __shared__ MS sh[256];
    pdl_trigger();
    pdl_wait();
    const int r = threadIdx.x % R;
    const int part = threadIdx.x / R;
    const int row = blockIdx.x * R + r;
    MS acc = {-INFINITY, 0.f};
    if (row < p.rows) {
        const float2 *st = p.stats + row;
#pragma unroll 8
        for (int j = part; j < p.tiles; j += P) {
            const float2 v = __ldcg(st + (size_t)j * p.rows);
            acc = join(acc, {v.x, v.y});
        }
    }
    sh[threadIdx.x] = acc;
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (part < o) sh[threadIdx.x] = join(sh[threadIdx.x], sh[threadIdx.x + o * R]);
    }
    if (part != 0 || row >= p.rows) return;
    const MS a = sh[threadIdx.x];
    // the row's own factor, relative to the largest
    float w = 1.f;
    if (p.want_grad) w = (p.row_scale ? __ldg(p.row_scale + row) : 1.f) / p.info->norm;
    HeadRow out;
    if (p.targets != nullptr) {
        const int t = __ldg(p.targets + row);
        const bool has = t >= 0 && t < p.cols;
        float l;
        if (t == p.ignore_index) {
            l = 0.f;
            out = {0.f, 0.f, 0.f, 0.f};
        } else {
            const float zt = has ? p.zt[row] * p.exp_scale : -INFINITY;
            out.M = fmaxf(a.M, zt);
            const float rest = a.M == -INFINITY ? a.S : a.S * ex2(a.M - out.M);
            const float e = has ? ex2(zt - out.M) : 0.f;
            const float S = rest + e;
            l = rest < e ? log1pf(rest / e) : kLn2 * (log2f(S) - (zt - out.M));
            if (!has) {
                l = NAN;
                atomicAdd(&p.err[kErrBadTarget], 1);
            }
            out.mul = w / S * p.shift_mul;
            out.target = has ? -(rest / S) * w * p.shift_mul : 0.f;
            out.log2S = log2f(S);
        }
        if (p.nan_on_failure && p.info->failed) l = NAN;
        p.loss[row] = l;
    } else {
        const float mass = p.mass[row];
        out.M = a.M;
        out.mul = mass == 0.f ? 0.f : mass * w / a.S * p.shift_mul;
        out.target = w * p.shift_mul;
        out.log2S = log2f(a.S);
    }
    p.row[row] = out;
}

// ------------------------------------------------------ kept exponentials
// A warp per 256 columns of a row (one tile, one factor), eight of them in
// flight; rows without a factor (ignored tokens) become zeros whatever they
// held.
constexpr int kScaleTiles = 8;
template <typename T>
__global__ void __launch_bounds__(256) head_scale_kernel(HeadRows p) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long groups = (p.tiles + kScaleTiles - 1) / kScaleTiles;
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= groups * p.rows) return;
    const int row = (int)(i / groups);
    const int j0 = (int)(i - row * groups) * kScaleTiles;
    const HeadRow h = p.row[row];
    const int t = p.targets ? __ldg(p.targets + row) : -1;
    unsigned char *base = p.exps + ((size_t)row * p.ld) * 2;
    uint4 x[kScaleTiles];
    float f[kScaleTiles];
#pragma unroll
    for (int k = 0; k < kScaleTiles; ++k) {
        const long long c = (long long)(j0 + k) * 256 + lane * 8;
        if (c < p.ld) x[k] = *reinterpret_cast<const uint4 *>(base + c * 2);
        f[k] = j0 + k < p.tiles
                   ? ex2(__ldcg(&p.stats[(size_t)(j0 + k) * p.rows + row].x) - h.M) * h.mul
                   : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kScaleTiles; ++k) {
        const long long c = (long long)(j0 + k) * 256 + lane * 8;
        if (c >= p.ld) continue;
        float v[8];
        E::unpack(x[k], v);
        const bool zero = h.mul == 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = zero ? 0.f : v[e] * f[k];
        if (t >= c && t < c + 8 && !zero) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (t - c == e) v[e] = h.target;
        }
        *reinterpret_cast<uint4 *>(base + c * 2) = E::pack(v);
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
    if (row >= p.rows) return;
    const HeadRow h = p.row[row];
    const float mass = p.mass[row];
    const long long i0 = (long long)row * p.K;
    float l = 0.f;
    bool bad = false;
    for (int k = lane; k < p.K; k += 32) {
        const int c = __ldg(p.idx + i0 + k);
        if (c < -1 || c >= p.cols) bad = true;
        const float lq = p.logq[i0 + k];
        if (c < 0 || c >= p.cols) continue;
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
                     (mass * ex2(lp2) - all) * h.target);
    }
    l = warp_sum(l);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        l = bad ? NAN : l * p.temperature * p.temperature;
        if (p.nan_on_failure && p.info->failed) l = NAN;
        p.loss[row] = l;
    }
}

// ------------------------------------------------------------------- join
template <typename T>
__global__ void __launch_bounds__(256)
    head_join_kernel(const float *parts, long long n, long long stride, int nparts,
                     const float *scale, float alpha, unsigned char *out) {
    using E = Elem<T>;
    pdl_trigger();
    pdl_wait();
    const float f = alpha * (scale ? *scale : 1.f);
    const long long step = (long long)gridDim.x * 256 * 8;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += step) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int q = 0; q < nparts; ++q) {
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(parts + q * stride + i));
            const float4 b = __ldcg(reinterpret_cast<const float4 *>(parts + q * stride + i + 4));
            v[0] += a.x;
            v[1] += a.y;
            v[2] += a.z;
            v[3] += a.w;
            v[4] += b.x;
            v[5] += b.y;
            v[6] += b.z;
            v[7] += b.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f;
        *reinterpret_cast<uint4 *>(out + i * 2) = E::pack(v);
    }
}

// ------------------------------------------------------------------- loss
__global__ void __launch_bounds__(kTailThreads)
    head_loss_kernel(float *rows, long long B, int reduction, const HeadInfo *info, float *out) {
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
        if (reduction == kReduceMean) r /= (double)max(info->count, 1);
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

cudaError_t launch_head_rows(const HeadRows &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    // enough CTAs for the rows there are: 32 rows each in a large batch, one
    // each where there are few
    if (p.rows <= 256) {
        cudaLaunchConfig_t cfg = config((unsigned)p.rows, 1, 256, s, attr);
        return cudaLaunchKernelEx(&cfg, head_rows_kernel<1>, p);
    }
    if (p.rows <= 2048) {
        cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 7) / 8), 1, 256, s, attr);
        return cudaLaunchKernelEx(&cfg, head_rows_kernel<8>, p);
    }
    cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 31) / 32), 1, 256, s, attr);
    return cudaLaunchKernelEx(&cfg, head_rows_kernel<32>, p);
}

cudaError_t launch_head_scale(const HeadRows &p, bool bf16, cudaStream_t s) {
    const long long groups = (p.tiles + kScaleTiles - 1) / kScaleTiles;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((groups * p.rows + 7) / 8), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_scale_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_scale_kernel<__half>, p);
}

cudaError_t launch_head_listed(const HeadRows &p, bool bf16, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((p.rows + 7) / 8), 1, 256, s, attr);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_listed_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, head_listed_kernel<__half>, p);
}

cudaError_t launch_head_join(const float *parts, long long n, long long part_stride, int nparts,
                             const float *scale, float alpha, void *out, bool bf16, int sms,
                             cudaStream_t s) {
    long long ctas = (n / 8 + 255) / 256;
    if (ctas > 16LL * sms) ctas = 16LL * sms;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)ctas, 1, 256, s, attr);
    unsigned char *o = static_cast<unsigned char *>(out);
    return bf16 ? cudaLaunchKernelEx(&cfg, head_join_kernel<__nv_bfloat16>, parts, n, part_stride,
                                     nparts, scale, alpha, o)
                : cudaLaunchKernelEx(&cfg, head_join_kernel<__half>, parts, n, part_stride, nparts,
                                     scale, alpha, o);
}

cudaError_t launch_head_loss(float *rows, long long B, int reduction, const HeadInfo *info,
                             float *loss_out, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(1, 1, kTailThreads, s, attr);
    return cudaLaunchKernelEx(&cfg, head_loss_kernel, rows, B, reduction, info, loss_out);
}

}  // namespace ce
