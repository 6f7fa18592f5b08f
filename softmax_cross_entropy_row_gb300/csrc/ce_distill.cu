// The divergence of a row's softmax from a teacher's top logits, with its
// gradient (ce_distill_fwd_bwd).  For a row z, temperature T, p = softmax(z /
// T) and the teacher's probabilities q_k at classes i_k (Q = sum_k q_k),
//   l    = T^2 sum_k q_k (log q_k - log p_{i_k}),
//   dz_c = T (Q p_c - sum_{k: i_k = c} q_k).
// Away from the listed classes the gradient is a multiple of the softmax, so
// the row is handled like a softmax row and the listed classes are written
// over it afterwards from their fp32 values.  HBM bound: the row is read once
// and its gradient written once.
//
// A row belongs to a group of G threads: a warp (short rows), a CTA, or a
// cluster of CTAs (few long rows).  Each thread forms its own maximum and sum
// of exponentials; the group joins them in a fixed order.  Rows that fit the
// group's registers stay there; longer ones are read a second time, from L2.
#include <math.h>

#include <map>
#include <mutex>
#include <tuple>

#include "ce_distill.h"
#include "ce_launch.h"

namespace ce {
namespace {

__device__ __forceinline__ uint4 ld_row(const uint4 *ptr) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(ptr));
    return v;
}

// A warp's prefetch of bytes [p, p + n) to L2.
__device__ __forceinline__ void prefetch_l2(const void *p, long long n) {
    const char *c = static_cast<const char *>(p);
    for (long long i = (threadIdx.x & 31) * 128LL; i < n; i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(c + i));
}

template <typename V>
__device__ __forceinline__ float value_at(const void *val, long long i) {
    return Elem<V>::load_global(static_cast<const unsigned char *>(val) + i * Elem<V>::kBytes);
}
__device__ __forceinline__ float teacher_at(const DistillParams &p, long long i) {
    return p.val_dtype == 0   ? value_at<float>(p.val, i)
           : p.val_dtype == 1 ? value_at<__nv_bfloat16>(p.val, i)
                              : value_at<__half>(p.val, i);
}

// A maximum and the sum of 2^((z - m) scale).
struct MS {
    float m, s;
};
__device__ __forceinline__ MS join(MS a, MS b, float scale) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};
    return {m, a.s * ex2((a.m - m) * scale) + b.s * ex2((b.m - m) * scale)};
}

// What a row's list comes to.
struct ListSums {
    float mass;    // sum q
    float negent;  // sum q log q
    bool bad;      // a class was out of range
};

// The teacher's list of row b, by one warp: classes and probabilities to shared
// memory (unused and bad places: class -1, probability 0), and, if `z` is
// given, the row's logits there (loaded while the probabilities are formed).
// One exponential per place: with x_k = (t_k - m) / T,
//   q_k = e^x_k / s, sum q log q = (sum e^x x) / s - log s     (s = sum e^x), or
//   q_k = e^(x_k - ref)                                        (lse given).
template <typename E>
__device__ __forceinline__ ListSums read_list(const DistillParams &p, long long b, int *cls,
                                              float *prob, float *z, const unsigned char *row) {
    const int lane = threadIdx.x & 31;
    const long long i0 = b * p.K;
    const float inv_t = 1.f / p.temperature;
    float m = -INFINITY;
    bool wrong = false;
#pragma unroll 4
    for (int k = lane; k < p.list_words; k += 32) {
        // both loads at once: an unused place's value is read and dropped
        int c = k < p.K ? __ldg(p.idx + i0 + k) : -1;
        float t = k < p.K ? teacher_at(p, i0 + k) : -INFINITY;
        if (c < -1 || c >= p.C) {
            wrong = true;
            c = -1;
        }
        if (c < 0) t = -INFINITY;
        cls[k] = c;
        prob[k] = t;
        m = fmaxf(m, t);
        // a NaN is not the maximum, but the place has to count
        if (t != t) m = fmaxf(m, -3.402823466e38f);
    }
    if (z != nullptr) {
#pragma unroll 4
        for (int k = lane; k < p.list_words; k += 32)
            z[k] = cls[k] >= 0 ? E::load_global(row + (size_t)cls[k] * E::kBytes) : 0.f;
    }
    m = warp_max(m);
    ListSums r = {0.f, 0.f, (bool)__any_sync(0xffffffffu, wrong)};
    if (m == -INFINITY) {  // no place has a probability
        for (int k = lane; k < p.list_words; k += 32) prob[k] = 0.f;
    } else if (p.lse != nullptr) {
        const float ref = __ldg(p.lse + b) - m * inv_t;
        for (int k = lane; k < p.list_words; k += 32) {
            const float x = (prob[k] - m) * inv_t - ref;
            const float q = expf(x);
            if (q != 0.f) r.negent += q * x;
            r.mass += q;
            prob[k] = q;
        }
        r.mass = warp_sum(r.mass);
        r.negent = warp_sum(r.negent);
    } else {
        float s = 0.f, sx = 0.f;
        for (int k = lane; k < p.list_words; k += 32) {
            const float x = (prob[k] - m) * inv_t;
            const float e = expf(x);
            if (e != 0.f) sx += e * x;
            s += e;
            prob[k] = e;
        }
        s = warp_sum(s);
        sx = warp_sum(sx);
        const float inv = 1.f / s;
        for (int k = lane; k < p.list_words; k += 32) prob[k] *= inv;
        r.mass = s == s ? 1.f : s;
        r.negent = sx * inv - logf(s);
    }
    __syncwarp();
    return r;
}

// What one warp keeps of a row's list, in shared memory.
struct List {
    int *cls;        // classes; -1: unused, or an earlier place has the class
    float *prob;     // probabilities, with those of the class's later places
    float *z;        // the student's logits there
    unsigned long long *acc;  // (scratch; z lies in it)
    int *key, *first;         // hash table of 2^bits >= 2 words places
};
__host__ __device__ constexpr int list_bytes(int words, int bits) {
    return words * 16 + (8 << bits);
}
__device__ __forceinline__ List list_at(unsigned char *base, int words, int bits) {
    List l;
    l.acc = reinterpret_cast<unsigned long long *>(base);
    l.z = reinterpret_cast<float *>(base);
    l.cls = reinterpret_cast<int *>(base + 8 * words);
    l.prob = reinterpret_cast<float *>(l.cls + words);
    l.key = reinterpret_cast<int *>(l.prob + words);
    l.first = l.key + (1 << bits);
    return l;
}
__device__ __forceinline__ int find(const int *key, int bits, int c) {
    unsigned at = ((unsigned)c * 2654435761u) >> (32 - bits);
    for (int n = 0; n < (1 << bits) && key[at] != c; ++n) at = (at + 1) & ((1 << bits) - 1);
    return (int)at;
}

__device__ __forceinline__ void clear_table(const List &l, int bits) {
    for (int i = threadIdx.x & 31; i < (1 << bits); i += 32) l.key[i] = -1;
    __syncwarp();
}

// cls and prob with the places of a class added up, by one warp (the table has
// been cleared).  A hash table finds out whether any class is listed twice.
// Only then the later places' probabilities are added to the first's, as
// multiples of 2^-61 of the list's mass (a power of two above it), whose sums do
// not depend on the order of the additions (z is formed anew then).  Returns
// whether that was so.
__device__ __forceinline__ bool merge_list(const List &l, int words, int bits, float mass) {
    const int lane = threadIdx.x & 31;
    const int size = 1 << bits;
    bool twice = false;
    for (int k = lane; k < words; k += 32) {
        const int c = l.cls[k];
        if (c < 0) continue;
        unsigned at = ((unsigned)c * 2654435761u) >> (32 - bits);
        for (int n = 0; n < size; ++n) {  // at most half full: ends earlier
            const int was = atomicCAS(&l.key[at], -1, c);
            twice |= was == c;
            if (was == -1 || was == c) break;
            at = (at + 1) & (size - 1);
        }
    }
    twice = __any_sync(0xffffffffu, twice);
    if (twice) {
        // 2^(61 - e), mass < 2^e (any scale will do for a mass that is none)
        const int e = (int)(__float_as_uint(mass) >> 23 & 255u) - 126;
        const float unit = e > -60 && e < 120 ? exp2f((float)(61 - e)) : 1.f;
        for (int i = lane; i < size; i += 32) l.first[i] = words;
        for (int k = lane; k < words; k += 32) l.acc[k] = 0ull;
        __syncwarp();
        for (int k = lane; k < words; k += 32)
            if (l.cls[k] >= 0) atomicMin(&l.first[find(l.key, bits, l.cls[k])], k);
        __syncwarp();
        for (int k = lane; k < words; k += 32) {
            if (l.cls[k] < 0) continue;
            const int f = l.first[find(l.key, bits, l.cls[k])];
            if (f == k) continue;
            const float q = l.prob[k];
            atomicAdd(&l.acc[f], (unsigned long long)fminf(q * unit, 4.611686e18f));  // 2^62
            l.cls[k] = -1;
        }
        __syncwarp();
        for (int k = lane; k < words; k += 32)
            l.prob[k] += (float)((double)l.acc[k] / (double)unit);
        __syncwarp();
    }
    return twice;
}

// A row's list complete: read, merged, with the row's logits in z.
template <typename E>
__device__ __forceinline__ ListSums take_list(const DistillParams &p, long long b, const List &l,
                                              int bits, const unsigned char *row) {
    const int words = p.list_words;
    clear_table(l, bits);
    const ListSums r = read_list<E>(p, b, l.cls, l.prob, l.z, row);
    if (merge_list(l, words, bits, r.mass))  // z lies in the sums' place
        for (int k = threadIdx.x & 31; k < words; k += 32)
            l.z[k] = l.cls[k] >= 0 ? E::load_global(row + (size_t)l.cls[k] * E::kBytes) : 0.f;
    __syncwarp();
    return r;
}

// The list of a later row on its way to L2.
__device__ __forceinline__ void prefetch_list(const DistillParams &p, long long b) {
    const int vs = p.val_dtype == 0 ? 4 : 2;
    prefetch_l2(p.idx + b * p.K, 4LL * p.K);
    prefetch_l2(static_cast<const unsigned char *>(p.val) + b * p.K * vs, (long long)vs * p.K);
}

// The reducing warps' shares of a row, joined by every lane of a warp.
template <int NW>
__device__ __forceinline__ MS join_parts(const MS *part, float scale) {
    const int lane = threadIdx.x & 31;
    const MS w = lane < NW ? part[lane] : MS{-INFINITY, 0.f};
    MS a;
    a.m = warp_max(w.m);
    a.s = warp_sum(w.m == -INFINITY ? w.s : w.s * ex2((w.m - a.m) * scale));
    return a;
}

// A row's place in memory: nh elements up to a 16-byte boundary, nvec whole
// vectors, the rest; this CTA's share is vectors [v0, v1) and, at the ends,
// the loose elements: elements [e0, e1).
struct Span {
    long long nh, v0, v1, tail0, e0, e1;
};
template <typename E>
__device__ __forceinline__ Span span_of(const unsigned char *row, long long C, int rank, int n) {
    Span s;
    const uint32_t ph = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
    s.nh = ph ? min((long long)((16u - ph) / E::kBytes), C) : 0LL;
    const long long nvec = (C - s.nh) / E::kVec;
    s.v0 = nvec * rank / n;
    s.v1 = nvec * (rank + 1) / n;
    s.tail0 = s.nh + nvec * E::kVec;
    s.e0 = rank == 0 ? 0 : s.nh + s.v0 * E::kVec;
    s.e1 = rank == n - 1 ? C : s.nh + s.v1 * E::kVec;
    return s;
}

// The loose element of thread t (head, then tail), or -1.
__device__ __forceinline__ long long loose(const Span &s, long long C, int t) {
    long long c = -1;
    if (t < s.nh) c = t;
    else if (s.tail0 + t - s.nh < C) c = s.tail0 + t - s.nh;
    return c >= s.e0 && c < s.e1 ? c : -1;
}

// The exponent (z - m) scale of a pair.  m scale is rounded to the multiple of
// 2^-24 |m scale| that is its fp32 value, so up to 2^6 (an error of 2^-18, of
// 3e-6 in the exponential) one fused operation does; beyond that (or where
// the product overflows: rows of the type's lowest values) the difference is
// formed first, which is exact where it matters.
struct Exponent {
    unsigned long long nm, sc, nM;
    bool small;
    __device__ __forceinline__ Exponent(float m, float scale) {
        const float M = m * scale;
        nm = f2_pack(-m, -m);
        sc = f2_pack(scale, scale);
        nM = f2_pack(-M, -M);
        small = fabsf(M) <= 64.f;
    }
    __device__ __forceinline__ unsigned long long fused(unsigned long long z) const {
        return f2_fma(z, sc, nM);
    }
    __device__ __forceinline__ unsigned long long exact(unsigned long long z) const {
        return f2_mul(f2_add(z, nm), sc);
    }
};

// V vectors added to a running maximum and sum, which is rescaled when the
// maximum grows (after a row's first vectors it hardly ever does).
template <typename E, int V>
__device__ __forceinline__ void add_vectors(MS &a, const uint4 (&x)[V], float scale) {
    typename E::MaxAcc acc = E::max_init();
#pragma unroll
    for (int k = 0; k < V; ++k) E::max_step(acc, x[k]);
    const float m = E::max_value(acc);
    if (m > a.m) {
        a.s *= ex2((a.m - m) * scale);
        a.m = m;
    }
    const float base = a.m == -INFINITY ? 0.f : a.m;
    const Exponent ex(base, scale);
    unsigned long long sum[2] = {0ull, 0ull};
    auto all = [&](auto exponent) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            unsigned long long z[E::kVec / 2];
            E::unpack2(x[k], z);
#pragma unroll
            for (int j = 0; j < E::kVec / 2; ++j) {
                float u, v;
                f2_unpack(exponent(z[j]), u, v);
                sum[j & 1] = f2_add(sum[j & 1], f2_pack(ex2(u), ex2(v)));
            }
        }
    };
    if (ex.small)
        all([&](unsigned long long z) { return ex.fused(z); });
    else
        all([&](unsigned long long z) { return ex.exact(z); });
    float u, v;
    f2_unpack(f2_add(sum[0], sum[1]), u, v);
    a.s += u + v;
}

// Vectors turned into their gradients, 2^((z - m) scale) f.
template <typename E, int V>
__device__ __forceinline__ void to_gradients(uint4 (&x)[V], const Exponent &ex, float f) {
    const unsigned long long f2 = f2_pack(f, f);
    auto all = [&](auto exponent) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            unsigned long long z[E::kVec / 2];
            E::unpack2(x[k], z);
#pragma unroll
            for (int j = 0; j < E::kVec / 2; ++j) {
                float u, v;
                f2_unpack(exponent(z[j]), u, v);
                z[j] = f2_mul(f2_pack(ex2(u), ex2(v)), f2);
            }
            x[k] = E::pack2(z);
        }
    };
    if (ex.small)
        all([&](unsigned long long z) { return ex.fused(z); });
    else
        all([&](unsigned long long z) { return ex.exact(z); });
}

template <typename E>
__device__ __forceinline__ void put_vector(unsigned char *g, const uint4 &v, bool aligned) {
    if (aligned) {
        __stcs(reinterpret_cast<uint4 *>(g), v);
    } else {
#pragma unroll
        for (int j = 0; j < E::kVec; ++j) E::store(g + j * E::kBytes, element_of<E>(v, j));
    }
}

// CTAs per SM the registers are set for: a thread keeps V vectors of its row.
constexpr int min_ctas(int g, int v, bool loop) {
    return loop ? 2 : g == 128 ? 4 : g == 32 && v < 16 ? (v == 8 ? 3 : 4) : 2;
}

template <typename T, int G, int V, bool LOOP>
__global__ void __launch_bounds__(G == 32 ? 256 : G, min_ctas(G, V, LOOP))
    distill_kernel(DistillParams p, int cluster, int bits) {
    using E = Elem<T>;
    constexpr int ES = E::kBytes;
    constexpr int NT = G == 32 ? 256 : G;
    constexpr int GROUPS = NT / G;
    constexpr int WARPS = G / 32;
    extern __shared__ unsigned char lists[];
    __shared__ MS part[2][WARPS * GROUPS];
    __shared__ float lpart[2][WARPS * GROUPS];
    __shared__ float4 mine[2];  // this CTA's share, read by the cluster
    __shared__ float masses[2], negents[2];
    __shared__ int bads[2];
    __shared__ int tail_flag;
    __shared__ float2 tail_scratch[kTailWarps];

    const int group = threadIdx.x / G;
    const int t = threadIdx.x % G;
    const int warp = t >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const long long first = (long long)(blockIdx.x / cluster) * GROUPS + group;
    const long long step = (long long)(gridDim.x / cluster) * GROUPS;
    const float scale = p.exp_scale;
    auto group_sync = [] {
        if constexpr (G == 32) __syncwarp();
        else __syncthreads();
    };

    pdl_trigger();
    pdl_wait();

    const float scalar = scalar_grad_scale(p);
    int buf = 0;
    for (long long b = first; b < p.B; b += step, buf ^= 1) {
        const unsigned char *row = p.logits + (size_t)(b * p.C) * ES;
        const Span sp = span_of<E>(row, p.C, rank, cluster);
        const uint4 *vp = reinterpret_cast<const uint4 *>(row + sp.nh * ES);
        const uint4 kNeg = make_uint4(E::kNegInfWord, E::kNegInfWord, E::kNegInfWord,
                                      E::kNegInfWord);
        uint4 x[V];
        auto load = [&](long long v) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                x[k] = v + k * G + t < sp.v1 ? ld_row(vp + v + k * G + t) : kNeg;
        };
        if constexpr (!LOOP) load(sp.v0);
        const long long lc = loose(sp, p.C, t);
        const float lz = lc >= 0 ? E::load_global(row + lc * ES) : -INFINITY;

        int *idx = reinterpret_cast<int *>(lists) + buf * 2 * p.list_words;
        float *lq = reinterpret_cast<float *>(idx + p.list_words);
        List l = {};
        ListSums sums = {0.f, 0.f, false};
        if constexpr (G == 32) {
            l = list_at(lists + group * list_bytes(p.list_words, bits), p.list_words, bits);
            if (b + step < p.B) {
                prefetch_l2(row + (size_t)(step * p.C) * ES, p.C * ES);
                prefetch_list(p, b + step);
            }
            sums = take_list<E>(p, b, l, bits, row);
        } else if (warp == 0) {
            const ListSums r = read_list<E>(p, b, idx, lq, nullptr, row);
            if (lane == 0) {
                masses[buf] = r.mass;
                negents[buf] = r.negent;
                bads[buf] = r.bad;
            }
        }

        // this thread's maximum and sum
        MS a = {lz, lz == -INFINITY ? 0.f : lz == lz ? 1.f : lz};
        if constexpr (LOOP) {
            for (long long v = sp.v0; v < sp.v1; v += (long long)V * G) {
                load(v);
                add_vectors<E, V>(a, x, scale);
            }
        } else {
            add_vectors<E, V>(a, x, scale);
        }
        // the warp's, the group's, the cluster's
        const float wm = warp_max(a.m);
        a.s = warp_sum(wm == -INFINITY ? a.s : a.s * ex2((a.m - wm) * scale));
        a.m = wm;
        if constexpr (G > 32) {
            if (lane == 0) part[buf][warp] = a;
            __syncthreads();
            a = join_parts<WARPS>(part[buf], scale);
            if (cluster > 1) {
                if (threadIdx.x == 0) mine[buf] = make_float4(a.m, a.s, 0.f, 0.f);
                cluster_sync();
                a = {-INFINITY, 0.f};
                for (int i = 0; i < cluster; ++i) {
                    const float4 v = ld_dsmem_f4(&mine[buf], i);
                    a = join(a, {v.x, v.y}, scale);
                }
            }
        } else {
            __syncwarp();
        }
        const float m = a.m, S = a.s;
        const float mass = G == 32 ? sums.mass : masses[buf];
        const float f = row_grad_factor(p, scalar, b) * p.temperature;
        const float inv = 1.f / S;

        if (writes_grad(p)) {
            unsigned char *grow = p.grad + (size_t)(b * p.C) * ES;
            unsigned char *gv = grow + sp.nh * ES;
            const bool zero = mass == 0.f;  // no list: nothing to learn, whatever the row holds
            const float fs = zero ? 0.f : mass * inv * f;
            if (lc >= 0) E::store(grow + lc * ES, zero ? 0.f : ex2((lz - m) * scale) * fs);
            const Exponent ex(m, scale);
            auto write = [&](long long v) {
                if (zero) {
#pragma unroll
                    for (int k = 0; k < V; ++k) x[k] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    to_gradients<E, V>(x, ex, fs);
                }
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const long long i = v + k * G + t;
                    if (i < sp.v1) put_vector<E>(gv + i * 16, x[k], p.grad_vec_ok);
                }
            };
            if constexpr (LOOP) {
                for (long long v = sp.v0; v < sp.v1; v += (long long)V * G) {
                    load(v);
                    write(v);
                }
            } else {
                write(sp.v0);
            }
            group_sync();
        }

        // the listed classes, and the loss
        const float log2S = log2f(S);
        if constexpr (G == 32) {
            float cross = 0.f;
            for (int k = lane; k < p.list_words; k += 32) {
                const int c = l.cls[k];
                if (c < 0) continue;
                const float lp2 = (l.z[k] - m) * scale - log2S;
                const float q = l.prob[k];
                if (q != 0.f) cross += q * lp2;
                if (writes_grad(p))
                    E::store(p.grad + (size_t)(b * p.C + c) * ES,
                             mass == 0.f ? 0.f : (mass * ex2(lp2) - q) * f);
            }
            cross = warp_sum(cross);
            if (lane == 0) {
                float loss = (sums.negent - kLn2 * cross) * p.temperature * p.temperature;
                if (mass == 0.f) loss = 0.f;
                if (sums.bad) {
                    loss = NAN;
                    atomicAdd(&p.err[kErrBadTarget], 1);
                }
                p.loss_rows[b] = loss;
            }
            __syncwarp();
            continue;
        }
        float cross = 0.f;
        for (int k = t; k < p.K; k += G) {
            const int c = idx[k];
            if (c < 0) continue;
            const bool here = c >= sp.e0 && c < sp.e1;
            if (!here && rank != 0) continue;
            const float lp2 = (E::load_global(row + (size_t)c * ES) - m) * scale - log2S;
            const float q = lq[k];
            if (q != 0.f) cross += q * lp2;
            if (!writes_grad(p) || !here) continue;
            float all = 0.f;
            bool mine_first = true;
            for (int j = 0; j < p.list_words; j += 4) {
                const int4 o = *reinterpret_cast<const int4 *>(idx + j);
                const int oc[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (oc[i] != c) continue;
                    if (j + i < k) mine_first = false;
                    all += lq[j + i];
                }
            }
            if (mine_first)
                E::store(p.grad + (size_t)(b * p.C + c) * ES,
                         mass == 0.f ? 0.f : (mass * ex2(lp2) - all) * f);
        }
        if (rank == 0) {
            cross = warp_sum(cross);
            if (lane == 0) lpart[buf][warp] = cross;
            __syncthreads();
            cross = lpart[buf][0];
            for (int i = 1; i < WARPS; ++i) cross += lpart[buf][i];
            if (t == 0) {
                float loss = (negents[buf] - kLn2 * cross) * p.temperature * p.temperature;
                if (mass == 0.f) loss = 0.f;
                if (bads[buf]) {
                    loss = NAN;
                    atomicAdd(&p.err[kErrBadTarget], 1);
                }
                p.loss_rows[b] = loss;
            }
        }
    }
    if (cluster > 1) cluster_sync();  // no CTA leaves while a peer may read its share
    finish_cta(p, &tail_flag, tail_scratch);
}

// ------------------------------------------------------------------- ring
//
// Many long rows: a CTA takes one row at a time, streamed through a ring of
// shared-memory chunks by a warp of its own (TMA bulk copies).  RESIDENT: the
// ring holds a row, whose chunks stay for the gradient; otherwise the row is
// streamed a second time, from L2.  The next row's copies are under way while
// a row is reduced, and one barrier per row holds the reducing warps.  The
// teacher's lists belong to warps of their own, which take the rows in turn:
// one reads its row's list ahead, waits until the others have passed the row's
// stores, and writes the listed classes and the loss, without their waiting
// for it (done by one of the reducing warps, it held the others up at the next
// row's barrier: 268 us on 8192 x 32000 bf16).
constexpr int kRingVecs = 4;  // per thread and chunk: chunks of 8, 16 and 32 KB
__host__ __device__ constexpr int chunk_bytes(int nt) { return nt * 16 * kRingVecs; }
constexpr int kMaxSlots = 16;

struct RingShape {
    int slots;
    int table_bits;
};

// List warps of a CTA, each with a list of its own: a row's list is read, and
// its listed classes are written, while LW - 1 other rows go through the ring,
// so the latencies of both are hidden.
__host__ __device__ constexpr int list_warps(int nt) { return nt == 128 ? 3 : 4; }

template <typename T, int NT, bool RESIDENT>
__global__ void __launch_bounds__(NT + 32 + 32 * list_warps(NT), 512 / NT)
    distill_ring_kernel(DistillParams p, RingShape rs) {
    using E = Elem<T>;
    constexpr int ES = E::kBytes;
    constexpr int V = kRingVecs;
    constexpr int CH = chunk_bytes(NT);
    constexpr int VC = CH / 16;
    constexpr int NW = NT / 32;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
    constexpr int LW = list_warps(NT);
    __shared__ uint64_t list_full[LW], row_done[LW];
    __shared__ MS joined[LW];
    __shared__ float masses[LW];
    __shared__ MS part[LW][NW];
    __shared__ int fine[LW][NW];  // the warp's waits have all been met
    __shared__ int dead;  // a wait gave up
    __shared__ int tail_flag;
    __shared__ float2 tail_scratch[kTailWarps];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int S = rs.slots;
    const int words = p.list_words;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NW);
        }
        for (int i = 0; i < LW; ++i) {
            mbar_init(&list_full[i], 1);
            mbar_init(&row_done[i], NW);
        }
        dead = 0;
        fence_mbar_init();
    }
    pdl_trigger();
    __syncthreads();
    pdl_wait();

    auto fail = [&] {
        *reinterpret_cast<volatile int *>(&dead) = 1;
        atomicAdd(&p.err[kErrTimeout], 1);
    };
    auto is_dead = [&] { return *reinterpret_cast<volatile int *>(&dead) != 0; };
    const long long limit = p.copy_wait_limit;
    const float scale = p.exp_scale;
    const bool grads = writes_grad(p);
    const int passes = grads && !RESIDENT ? 2 : 1;

    if (warp == NW) {
        // ---- the copies
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            const uint64_t keep = l2_policy_evict_last(), drop = l2_policy_evict_first();
            for (long long b = blockIdx.x; b < p.B; b += gridDim.x) {
                const unsigned char *row = p.logits + (size_t)(b * p.C) * ES;
                const Span sp = span_of<E>(row, p.C, 0, 1);
                const unsigned char *v0 = row + sp.nh * ES;
                for (int pass = 0; pass < passes; ++pass) {
                    const uint64_t policy = pass + 1 < passes ? keep : drop;
                    for (long long v = 0; v < sp.v1; v += VC) {
                        if (!mbar_wait(&empty[s], ph ^ 1u, limit)) {
                            fail();
                            goto copied;
                        }
                        // The slot was read through the generic proxy and is
                        // written through the async one: without this fence the
                        // next row's bytes could arrive before the last reads of
                        // this row's (seen with gradients stored element by
                        // element, whose stores hold the reads up).
                        fence_proxy_async();
                        const uint32_t bytes = (uint32_t)min((long long)VC, sp.v1 - v) * 16u;
                        if (!(skips_copy(p, b, b + 1) && v == 0 && pass == 0)) {
                            mbar_arrive_expect_tx(&full[s], bytes);
                            bulk_g2s_hint(ring + (size_t)s * CH, v0 + v * 16, bytes, &full[s],
                                          policy);
                        }
                        ++issued;
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
        copied:
            if (is_dead()) {  // what is in flight lands before shared memory is given up
                for (int n = min(issued, S); n > 0; --n) {
                    if (s == 0) {
                        s = S;
                        ph ^= 1u;
                    }
                    --s;
                    mbar_wait(&full[s], ph);
                }
            }
        }
    } else if (warp > NW) {
        // ---- the lists: this warp's are every LW-th of the CTA's rows
        const int j = warp - NW - 1;
        const List l = list_at(ring + (size_t)S * CH + j * list_bytes(words, rs.table_bits), words,
                               rs.table_bits);
        const float scalar = scalar_grad_scale(p);
        uint32_t ph = 0;
        for (long long b = blockIdx.x + (long long)j * gridDim.x; b < p.B;
             b += (long long)LW * gridDim.x, ph ^= 1u) {
            const unsigned char *row = p.logits + (size_t)(b * p.C) * ES;
            const long long next = b + (long long)LW * gridDim.x;
            if (next < p.B) prefetch_list(p, next);
            clear_table(l, rs.table_bits);
            const ListSums sums = read_list<E>(p, b, l.cls, l.prob, l.z, row);
            const float mass = sums.mass;
            if (lane == 0) {
                masses[j] = mass;
                mbar_arrive(&list_full[j]);  // the reducing warps need the mass alone
            }
            if (merge_list(l, words, rs.table_bits, mass))
                for (int k = lane; k < words; k += 32)
                    l.z[k] = l.cls[k] >= 0 ? E::load_global(row + (size_t)l.cls[k] * ES) : 0.f;
            if (!__all_sync(0xffffffffu, mbar_wait(&row_done[j], ph, limit))) {
                if (lane == 0) fail();
                break;
            }
            const MS a = grads ? joined[j] : join_parts<NW>(part[j], scale);
            const float f = row_grad_factor(p, scalar, b) * p.temperature;
            const float log2S = log2f(a.s);
            float cross = 0.f;
            for (int k = lane; k < words; k += 32) {
                const int c = l.cls[k];
                if (c < 0) continue;
                const float lp2 = (l.z[k] - a.m) * scale - log2S;
                const float q = l.prob[k];
                if (q != 0.f) cross += q * lp2;
                if (grads)
                    E::store(p.grad + (size_t)(b * p.C + c) * ES,
                             mass == 0.f ? 0.f : (mass * ex2(lp2) - q) * f);
            }
            cross = warp_sum(cross);
            if (lane == 0) {
                float loss = (sums.negent - kLn2 * cross) * p.temperature * p.temperature;
                if (mass == 0.f) loss = 0.f;
                if (sums.bad) {
                    loss = NAN;
                    atomicAdd(&p.err[kErrBadTarget], 1);
                }
                p.loss_rows[b] = loss;
            }
            __syncwarp();
        }
    } else {
        // ---- the rows
        const int t = threadIdx.x;
        const float scalar = scalar_grad_scale(p);
        int s = 0, lb = 0;
        uint32_t ph = 0, lph = 0;
        // A wait that gave up ends the warp's part in this row; the CTA stops
        // at its next barrier, where all warps see the same flags.
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
            return ok;
        };
        for (long long b = blockIdx.x; b < p.B; b += gridDim.x) {
            const unsigned char *row = p.logits + (size_t)(b * p.C) * ES;
            const Span sp = span_of<E>(row, p.C, 0, 1);
            const long long lc = loose(sp, p.C, t);
            const float lz = lc >= 0 ? E::load_global(row + lc * ES) : -INFINITY;
            MS a = {lz, lz == -INFINITY ? 0.f : lz == lz ? 1.f : lz};
            const int nvec = (int)sp.v1;
            // this thread's vectors of the chunk at vector v
            auto fetch = [&](int slot, int v, uint4 (&x)[V]) {
                const unsigned char *src = ring + slot * CH + t * 16;
                if (v + VC <= nvec) {
#pragma unroll
                    for (int k = 0; k < V; ++k) x[k] = lds128(src + k * NT * 16);
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        x[k] = v + k * NT + t < nvec
                                   ? lds128(src + k * NT * 16)
                                   : make_uint4(E::kNegInfWord, E::kNegInfWord, E::kNegInfWord,
                                                E::kNegInfWord);
                }
            };
            // whether a chunk is more than half there: all its rounds at once
            auto mostly = [&](int v) { return v + VC / 2 < nvec; };
            // vector k of a row's last chunk, one round at a time (a 98 KB row is
            // three chunks and a little)
            auto fetch_one = [&](int slot, int v, int k, uint4 (&x)[1]) {
                x[0] = v + k * NT + t < nvec
                           ? lds128(ring + slot * CH + (k * NT + t) * 16)
                           : make_uint4(E::kNegInfWord, E::kNegInfWord, E::kNegInfWord,
                                        E::kNegInfWord);
            };
            auto release = [&](int slot) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
            };
            auto release_row = [&](int i) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&row_done[i]);
            };
            const int s0 = s;
            for (int v = 0; v < nvec; v += VC) {
                if (wait(&full[s], ph)) {
                    if (mostly(v)) {
                        uint4 x[V];
                        fetch(s, v, x);
                        if (!RESIDENT || !grads) release(s);
                        add_vectors<E, V>(a, x, scale);
                    } else {
                        for (int k = 0; v + k * NT < nvec; ++k) {
                            uint4 x[1];
                            fetch_one(s, v, k, x);
                            add_vectors<E, 1>(a, x, scale);
                        }
                        if (!RESIDENT || !grads) release(s);
                    }
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!wait(&list_full[lb], lph) && lane == 0) fail();
            const float wm = warp_max(a.m);
            a.s = warp_sum(wm == -INFINITY ? a.s : a.s * ex2((a.m - wm) * scale));
            if (lane == 0) {
                part[lb][warp] = {wm, a.s};
                fine[lb][warp] = ok;
            }
            auto next_list = [&] {
                if (++lb == LW) {
                    lb = 0;
                    lph ^= 1u;
                }
            };
            if (!grads) {  // the list's warp joins the parts: no barrier
                if (!ok) break;
                release_row(lb);
                next_list();
                continue;
            }
            named_sync(1, NT);
            if (!__all_sync(0xffffffffu, lane >= NW || fine[lb][lane])) break;
            a = join_parts<NW>(part[lb], scale);
            const float m = a.m;
            const float inv = 1.f / a.s;
            const float mass = masses[lb];
            const float f = row_grad_factor(p, scalar, b) * p.temperature;
            if (grads) {
                unsigned char *grow = p.grad + (size_t)(b * p.C) * ES;
                unsigned char *gv = grow + sp.nh * ES;
                const bool zero = mass == 0.f;  // no list: nothing to learn, whatever the row holds
                const float fs = zero ? 0.f : mass * inv * f;
                if (lc >= 0) E::store(grow + lc * ES, zero ? 0.f : ex2((lz - m) * scale) * fs);
                int r = RESIDENT ? s0 : s;
                unsigned char *gt = gv + t * 16;
                const Exponent ex(m, scale);
                for (int v = 0; v < nvec; v += VC, gt += CH) {
                    if (!RESIDENT) wait(&full[r], ph);
                    if (ok && mostly(v)) {
                        uint4 x[V];
                        fetch(r, v, x);
                        release(r);
                        if (zero) {
#pragma unroll
                            for (int k = 0; k < V; ++k) x[k] = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            to_gradients<E, V>(x, ex, fs);
                        }
                        if (v + VC <= nvec && p.grad_vec_ok) {
#pragma unroll
                            for (int k = 0; k < V; ++k)
                                __stcs(reinterpret_cast<uint4 *>(gt + k * NT * 16), x[k]);
                        } else {
#pragma unroll
                            for (int k = 0; k < V; ++k)
                                if (v + k * NT + t < nvec)
                                    put_vector<E>(gt + k * NT * 16, x[k], p.grad_vec_ok);
                        }
                    } else if (ok) {
                        for (int k = 0; k < V && v + k * NT < nvec; ++k) {
                            uint4 x[1];
                            fetch_one(r, v, k, x);
                            if (zero)
                                x[0] = make_uint4(0u, 0u, 0u, 0u);
                            else
                                to_gradients<E, 1>(x, ex, fs);
                            if (v + k * NT + t < nvec)
                                put_vector<E>(gt + k * NT * 16, x[0], p.grad_vec_ok);
                        }
                        release(r);
                    }
                    if (++r == S) {
                        r = 0;
                        if (!RESIDENT) ph ^= 1u;
                    }
                }
                if (!RESIDENT) s = r;
                if (!ok && lane == 0) fail();
            }
            if (threadIdx.x == 0) joined[lb] = a;
            release_row(lb);
            next_list();
        }
    }
    __syncthreads();
    if (is_dead()) {  // every row whose result is in doubt reads NaN
        if (threadIdx.x == 0)
            for (long long b = blockIdx.x; b < p.B; b += gridDim.x) p.loss_rows[b] = NAN;
        __syncthreads();
    }
    finish_cta(p, &tail_flag, tail_scratch);
}

// The builds: a warp per row of up to 8 KB; the ring, its row resident or
// streamed twice; for few rows a CTA or a cluster per row, in registers or in
// two passes.
template <typename T>
const void *kernel_of(const DistillPlan &pl) {
    if (pl.ring_threads == 128)
        return reinterpret_cast<const void *>(distill_ring_kernel<T, 128, true>);
    if (pl.ring_threads == 256)
        return reinterpret_cast<const void *>(distill_ring_kernel<T, 256, true>);
    if (pl.ring_threads == 512)
        return reinterpret_cast<const void *>(distill_ring_kernel<T, 512, false>);
    if (pl.loop) return reinterpret_cast<const void *>(distill_kernel<T, 512, 8, true>);
    if (pl.group == 32 && pl.vecs == 4)
        return reinterpret_cast<const void *>(distill_kernel<T, 32, 4, false>);
    if (pl.group == 32 && pl.vecs == 8)
        return reinterpret_cast<const void *>(distill_kernel<T, 32, 8, false>);
    if (pl.group == 32) return reinterpret_cast<const void *>(distill_kernel<T, 32, 16, false>);
    if (pl.group == 128) return reinterpret_cast<const void *>(distill_kernel<T, 128, 16, false>);
    return reinterpret_cast<const void *>(distill_kernel<T, 256, 16, false>);
}
const void *kernel_of(int dtype, const DistillPlan &pl) {
    return dtype == 0   ? kernel_of<float>(pl)
           : dtype == 1 ? kernel_of<__nv_bfloat16>(pl)
                        : kernel_of<__half>(pl);
}

int threads_of(const DistillPlan &pl) {
    if (pl.ring_threads) return pl.ring_threads + 32 + 32 * list_warps(pl.ring_threads);
    return pl.group == 32 ? 256 : pl.group;
}

// Resident CTAs per SM, remembered (a captured call then asks nothing).
cudaError_t resident(const void *f, int threads, int smem, int *n) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void *, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    int &v = known[{dev, f, smem}];
    if (v == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, f, threads, smem);
        if (e != cudaSuccess) return e;
    }
    *n = v;
    return cudaSuccess;
}

}  // namespace

// Shared memory of an SM, and what a CTA of the ring needs beside the ring
// and its lists (the system's 1 KB and the kernel's static part, under 2 KB).
constexpr int kSmemPerSm = 228 * 1024;
constexpr int kSmemReserve = 3 * 1024;

cudaError_t plan_distill(long long B, long long C, int K, int dtype, bool grad, int sms,
                         DistillPlan *pl) {
    const long long row = C * (dtype == 0 ? 4 : 2);
    DistillPlan r = {};
    r.cluster = 1;
    r.vecs = 16;
    const int words = (K + 3) / 4 * 4;
    r.table_bits = 1;
    while ((1 << r.table_bits) < 2 * words) ++r.table_bits;
    // eight lists per CTA of the warp-per-row kernel: up to 256 places each
    if (row <= 8192 && 8 * list_bytes(words, r.table_bits) <= 65536) {
        r.group = 32;
        if (row <= 4096) r.vecs = 8;
        if (row <= 2048) r.vecs = 4;
    } else {
        // few rows: up to 8 CTAs each, as long as every SM then has one
        while (r.cluster < 8 && B * r.cluster * 2 <= sms && row / r.cluster > 16384) r.cluster *= 2;
        const long long share = row / r.cluster;
        r.group = share <= 128LL * 16 * 16 ? 128 : 256;
        if (share > 256LL * 16 * 16) {
            r.loop = true;
            r.group = 512;
            r.vecs = 8;
        }
    }
    if (r.group != 32 && B > sms) {
        // The ring of the smallest CTA (128 threads, four per SM, or 256, two)
        // that holds the row; longer rows are streamed twice through one of 512
        // threads.  Measured (K = 64, bf16 and fp32, fraction of the copy
        // bandwidth): 31 KB rows 0.77 in 128 threads (0.66-0.73 in 256), 62 KB
        // rows 0.86-0.88 in 256 (0.70-0.77 in 512), 94 KB rows 0.86-0.88 in 256; a
        // resident ring of 512 threads was no faster than streaming twice on
        // 98-125 KB rows (bf16 0.70-0.83 against 0.78-0.89).
        int lists = 0;
        r.cluster = 1;
        for (int nt : {128, 256, 512}) {
            r.ring_threads = nt;
            lists = list_warps(nt) * list_bytes(words, r.table_bits);
            const int room = (kSmemPerSm * nt / 512 - kSmemReserve - lists) / chunk_bytes(nt);
            r.slots = room < kMaxSlots ? room : kMaxSlots;
            if (row <= (long long)r.slots * chunk_bytes(nt)) break;
        }
        r.smem = r.slots * chunk_bytes(r.ring_threads) + lists;
    }
    const int groups = r.group == 32 ? 8 : 1;
    if (!r.ring_threads)
        r.smem = groups == 8 ? 8 * list_bytes(words, r.table_bits) : 2 * 2 * words * 4;
    const void *f = kernel_of(dtype, r);
    cudaError_t e = ensure_smem_attr(f, r.smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    if ((e = resident(f, threads_of(r), r.smem, &per_sm)) != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const long long want = (B + groups - 1) / groups * r.cluster;
    const long long most = (long long)per_sm * sms / r.cluster * r.cluster;
    r.ctas = (int)(want < most ? want : most);
    *pl = r;
    return cudaSuccess;
}

cudaError_t launch_distill(const DistillParams &p, int dtype, const DistillPlan &pl,
                           cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.ctas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads_of(pl), 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)pl.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pl.cluster > 1 ? 2 : 1;
    DistillParams q = p;
    int cluster = pl.cluster, bits = pl.table_bits;
    RingShape ring = {pl.slots, pl.table_bits};
    void *direct[] = {&q, &cluster, &bits}, *ringed[] = {&q, &ring};
    void **args = pl.ring_threads ? ringed : direct;
    return cudaLaunchKernelExC(&cfg, kernel_of(dtype, pl), args);
}

}  // namespace ce
