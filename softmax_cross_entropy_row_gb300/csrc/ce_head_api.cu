// C-ABI of the vocabulary projection's and the teacher's operators
// (ce_linear_fwd_bwd, ce_distill_fwd_bwd, ce_linear_distill_fwd_bwd in
// include/ce.h): argument checks, workspaces, the
// tensor maps of the operands and the sequence of launches.  Nothing here
// computes on the host.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "../../include/ce.h"
#include "../../include/ce_testing.h"
#include "ce_distill.h"
#include "ce_head_gemm.h"
#include "ce_head_rows.h"
#include "ce_host.h"

namespace {

// ------------------------------------------------------------- workspaces
//
// One per (device, stream), grown when a call needs more; nothing but the
// calls of that stream uses it, so an outgrown one is freed once the stream
// has drained.  A call that is being captured into a graph gets a workspace
// that belongs to that capture alone, so graphs may be replayed at the same
// time as each other and as eager calls; it is kept until
// ce_release_workspaces.
struct Buffer {
    unsigned char *base = nullptr;
    size_t bytes = 0;
};
std::mutex g_mu;  // held over a whole call: its launches use the workspace
long long g_skip_copy = -1, g_wait_limit = 0;  // ce_heads_test, under g_mu
std::map<std::tuple<int, uintptr_t, unsigned long long>, Buffer> g_buffers;
std::vector<std::pair<int, unsigned char *>> g_outgrown;  // of captures

// While it lives, this thread may allocate, free and wait although some stream
// of its is being captured (none of it becomes part of a capture).
struct Relaxed {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~Relaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

int workspace(int dev, cudaStream_t s, size_t need, unsigned char **out) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    cudaError_t e = cudaStreamGetCaptureInfo(s, &cs, &id);
    if (e != cudaSuccess) return ce::host_cuda_fail(e);
    if (cs != cudaStreamCaptureStatusActive) id = 0;
    // the per-thread default stream has one handle for all threads
    static thread_local char thread_key;
    const uintptr_t key = s == cudaStreamPerThread ? reinterpret_cast<uintptr_t>(&thread_key)
                                                   : reinterpret_cast<uintptr_t>(s);
    Buffer &b = g_buffers[{dev, key, id}];
    if (b.bytes < need) {
        const Relaxed relaxed;
        if (b.base) {
            if (id) {
                g_outgrown.push_back({dev, b.base});
            } else {
                e = cudaStreamSynchronize(s);
                if (e == cudaSuccess) e = cudaFree(b.base);
                if (e != cudaSuccess) return ce::host_cuda_fail(e);
            }
            b = Buffer();
        }
        const size_t bytes = (need + (1 << 20) - 1) >> 20 << 20;
        void *p = nullptr;
        e = ce::host_malloc_zeroed(&p, bytes, 256);
        if (e != cudaSuccess) return ce::host_cuda_fail(e);
        b.base = static_cast<unsigned char *>(p);
        b.bytes = bytes;
    }
    *out = b.base;
    return CE_OK;
}

// ------------------------------------------------------------ tensor maps

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_function(EncodeTiled *out) {
    static std::mutex mu;
    static EncodeTiled fn = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                               cudaEnableDefault, &found);
        if (e != cudaSuccess) return ce::host_cuda_fail(e);
        if (found != cudaDriverEntryPointSuccess || !f)
            return ce::host_cuda_fail(cudaErrorNotSupported);
        fn = reinterpret_cast<EncodeTiled>(f);
    }
    *out = fn;
    return CE_OK;
}

// [rows][cols] with `ld` elements from row to row; boxes of box_rows x (128
// bytes), 128-byte swizzled in shared memory.
int tensor_map(CUtensorMap *map, int dtype, const void *base, long long rows, long long cols,
               long long ld, int box_rows) {
    EncodeTiled encode;
    const int rc = encode_function(&encode);
    if (rc != CE_OK) return rc;
    const int es = dtype == CE_F32 ? 4 : 2;
    const CUtensorMapDataType type = dtype == CE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == CE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * es};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = encode(map, type, 2, const_cast<void *>(base), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? CE_OK : ce::host_cuda_fail(cudaErrorInvalidValue);
}

// ------------------------------------------------------------------ plans

// The reciprocal has to be a number too.
bool temperature_ok(float t) { return t > 0.f && isfinite(t) && isfinite(ce::kLog2e / t); }

constexpr size_t kTicketOffset = 128;          // within the workspace's first 256 bytes
constexpr long long kMaxK = 1024;             // places of a teacher's list
constexpr long long kPieceBytes = 1LL << 30;  // kept exponentials, see rows_per_piece

long long round_up(long long v, long long a) { return (v + a - 1) / a * a; }
long long ceil_div(long long v, long long a) { return (v + a - 1) / a; }

// Rows whose exponentials are kept at a time.  Several pieces need the
// weights' gradient accumulated in fp32 (4 C D bytes), so a piece is allowed
// as much as that buffer would take: a batch that fits needs no buffer.
long long rows_per_piece(long long B, long long D, long long C, bool dweight) {
    long long bytes = kPieceBytes;
    if (dweight) bytes = std::max(bytes, 4 * C * D);
    const long long r = bytes / (2 * round_up(C, 64)) / ce::kTileM * ce::kTileM;
    return std::min(round_up(B, ce::kTileM), std::max<long long>(r, ce::kTileM));
}

// Classes of a tile where the weights are read at the memory's rate: as many
// as spread evenly over the pairs (a tile's two halves are copied and computed
// in groups of 8 classes).
int score_tile(long long C, int pairs) {
    const long long rounds = ceil_div(C, (long long)ce::kTileM * pairs);
    return (int)std::min<long long>(ce::kTileM, round_up(ceil_div(C, rounds * pairs), 16));
}

// The same for the loss alone of a batch of one tile's rows: the width of its
// column tiles.
int stats_tile(long long C, long long rows, int pairs) {
    int best = ce::kTileN;
    if (rows > ce::kTileM) return best;
    long long least = 1LL << 60;
    for (int tn = ce::kTileN; tn >= 64; tn -= 32) {
        const long long rounds = ceil_div(ceil_div(C, tn), pairs);
        const long long cost = rounds * (tn + 8);
        if (cost < least) {
            least = cost;
            best = tn;
        }
    }
    return best;
}

// Whether a contraction of at most k may be split (head_splits: parts of at
// least 8 stages).
int can_split(long long k) { return ceil_div(k, ce::kTileK) >= 16; }

struct Call {
    const void *hidden, *weight;
    const int32_t *targets;  // cross-entropy
    int ignore_index;
    const int32_t *idx;  // teacher
    const void *val;
    const float *lse;
    int64_t K;
    int teacher_dtype;
    float temperature;
    int64_t B, D, C;
    int dtype, reduction;
    const float *scale;
    float *loss;
    void *dhidden, *dweight;
    void *stream;
};

int check(const Call &c) {
    const bool teacher = c.targets == nullptr;
    if (c.dtype != CE_BF16 && c.dtype != CE_F16) return CE_ERR_DTYPE;
    if (teacher && c.teacher_dtype != CE_F32 && c.teacher_dtype != CE_BF16 &&
        c.teacher_dtype != CE_F16)
        return CE_ERR_DTYPE;
    if (c.reduction != CE_REDUCE_MEAN && c.reduction != CE_REDUCE_SUM &&
        c.reduction != CE_REDUCE_NONE)
        return CE_ERR_REDUCTION;
    if (!c.hidden || !c.weight || !c.loss) return CE_ERR_NULL;
    if (teacher && (!c.idx || !c.val)) return CE_ERR_NULL;
    if (c.B < 1 || c.C < 1 || c.D < 8 || c.D % 8 || c.B > 0x7fffff00LL || c.C > 0x7fffff00LL ||
        c.D > (1 << 24))
        return CE_ERR_SHAPE;
    if (teacher && (c.K < 1 || c.K > kMaxK)) return CE_ERR_SHAPE;
    if (ceil_div(c.C, ce::kTileN) * ceil_div(std::max(c.B, c.D), ce::kTileM) * 32 > 0x7fffffffLL ||
        ceil_div(c.B, ce::kTileM) * ceil_div(c.D, ce::kTileM) * 32 > 0x7fffffffLL)
        return CE_ERR_SHAPE;
    if (teacher && !temperature_ok(c.temperature)) return CE_ERR_TEMPERATURE;
    const auto off = [](const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a; };
    const uintptr_t te = c.teacher_dtype == CE_F32 ? 4 : 2;
    if (off(c.hidden, 16) || off(c.weight, 16) || off(c.dhidden, 16) || off(c.dweight, 16) ||
        off(c.targets, 4) || off(c.idx, 4) || off(c.val, te) || off(c.lse, 4) || off(c.scale, 4) ||
        off(c.loss, 4))
        return CE_ERR_ALIGN;
    const size_t rows = c.reduction == CE_REDUCE_NONE ? (size_t)c.B * 4 : 4;
    const size_t hb = (size_t)c.B * c.D * 2, wb = (size_t)c.C * c.D * 2;
    struct Range {
        const void *p;
        size_t n;
    };
    const Range in[] = {{c.hidden, hb},
                        {c.weight, wb},
                        {c.targets, (size_t)c.B * 4},
                        {c.idx, (size_t)c.B * c.K * 4},
                        {c.val, (size_t)c.B * c.K * te},
                        {c.lse, (size_t)c.B * 4},
                        {c.scale, rows}};
    const Range out[] = {{c.loss, rows}, {c.dhidden, hb}, {c.dweight, wb}};
    for (int i = 0; i < 3; ++i) {
        for (const Range &r : in)
            if (ce::host_overlap(out[i].p, out[i].n, r.p, r.n)) return CE_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (ce::host_overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return CE_ERR_OVERLAP;
    }
    return CE_OK;
}

// Hands out the workspace's parts, 1 KB aligned (first pass: sizes alone).
struct Carver {
    unsigned char *base = nullptr;
    size_t used = 1024;  // HeadInfo
    template <typename T>
    T *take(size_t n) {
        T *p = reinterpret_cast<T *>(base + used);
        used += (n * sizeof(T) + 1023) / 1024 * 1024;
        return p;
    }
};

struct Parts {
    ce::HeadInfo *info;
    float *loss, *zt, *ref, *logq, *zk, *mass, *parts, *weight;
    float2 *stats;
    ce::HeadRow *row;
    int *perm, *pos;
    unsigned char *exps, *packed, *scaled;
};

struct Sizes {
    long long piece, pieces, ld;  // rows per piece, pieces, exponentials' row
    int tile_m, tile_n, tiles;
    bool grad, per_row, weight_f32, score;
};

Parts carve(Carver &w, const Call &c, const Sizes &z, int pairs) {
    const bool teacher = c.targets == nullptr;
    const size_t padded = round_up(c.B, 64), list = teacher ? (size_t)c.B * c.K : 0;
    Parts p = {};
    p.info = reinterpret_cast<ce::HeadInfo *>(w.base);
    p.loss = w.take<float>(c.reduction == CE_REDUCE_NONE ? 0 : round_up(c.B, 1024));
    p.stats = w.take<float2>((size_t)z.tiles * z.piece);
    p.row = w.take<ce::HeadRow>(z.piece);
    p.zt = w.take<float>(teacher ? 0 : c.B);
    p.logq = w.take<float>(list);
    p.zk = w.take<float>(list);
    p.mass = w.take<float>(teacher ? c.B : 0);
    if (!z.grad) return p;
    p.ref = w.take<float>(c.B);
    p.perm = w.take<int>(c.B);
    p.pos = w.take<int>(c.B);
    p.packed = w.take<unsigned char>(padded * c.D * 2);
    p.scaled = w.take<unsigned char>(z.per_row && c.dweight ? round_up(z.piece, 64) * c.D * 2 : 0);
    p.exps = w.take<unsigned char>((size_t)round_up(z.piece, 64) * z.ld * 2);
    p.parts = w.take<float>((size_t)ce::kMaxParts * pairs * ce::kTileM * ce::kTileN);
    p.weight = w.take<float>(c.dweight && z.weight_f32 ? (size_t)c.C * c.D : 0);
    return p;
}

#define CE_TRY(x)                                    \
    do {                                             \
        const int rc_ = (x);                         \
        if (rc_ != CE_OK) return rc_;                \
    } while (0)
#define CE_CUDA(x)                                             \
    do {                                                       \
        const cudaError_t e_ = (x);                            \
        if (e_ != cudaSuccess) return ce::host_cuda_fail(e_);  \
    } while (0)

int run(const Call &c) {
    CE_TRY(check(c));
    int dev = 0, sms = 0;
    CE_TRY(ce::host_device(&dev, &sms));
    for (const void *p : {c.hidden, c.weight, (const void *)c.targets, (const void *)c.idx, c.val,
                          (const void *)c.lse, (const void *)c.scale, (const void *)c.loss,
                          (const void *)c.dhidden, (const void *)c.dweight})
        if (p) CE_TRY(ce::host_check_device_pointer(p, dev));
    cudaStream_t s = static_cast<cudaStream_t>(c.stream);
    int *err = nullptr;
    CE_TRY(ce::host_error_counters(dev, s, &err));

    const bool teacher = c.targets == nullptr;
    const bool bf16 = c.dtype == CE_BF16, none = c.reduction == CE_REDUCE_NONE;
    const int pairs = sms / 2;
    Sizes z = {};
    z.grad = c.dhidden || c.dweight;
    z.per_row = z.grad && bf16;
    z.ld = round_up(c.C, 64);
    z.score = !z.grad && c.B <= ce::kScoreRows;
    z.tile_m = z.score ? score_tile(c.C, pairs) : ce::kTileM;
    z.tile_n = z.score ? (int)round_up(c.B, 32) : z.grad ? ce::kTileN
                                                         : stats_tile(c.C, c.B, pairs);
    z.tiles = z.score ? ce::kScoreStats * (int)ceil_div(c.C, z.tile_m)
                      : 2 * (int)ceil_div(c.C, z.tile_n);
    z.piece = z.grad ? rows_per_piece(c.B, c.D, c.C, c.dweight != nullptr)
                     : std::min(round_up(c.B, ce::kTileM),
                                std::max<long long>(ce::kTileM, kPieceBytes / (8LL * z.tiles) /
                                                                    ce::kTileM * ce::kTileM));
    z.pieces = ceil_div(c.B, z.piece);
    z.piece = std::min<long long>(z.piece, c.B);
    z.weight_f32 = z.pieces > 1;

    std::lock_guard<std::mutex> lk(g_mu);
    Carver sizer;
    carve(sizer, c, z, pairs);
    Carver w;
    CE_TRY(workspace(dev, s, sizer.used, &w.base));
    const Parts ws = carve(w, c, z, pairs);

    // f16 holds values down to 2^-24: what is kept (at most 1) is raised by
    // 2^15 so that small probabilities keep their 11 bits
    const float shift = bf16 ? 0.f : 15.f;
    const float shift_mul = bf16 ? 1.f : 32768.f;
    const float *row_scale = none ? c.scale : nullptr;
    const float exp_scale = ce::kLog2e / (teacher ? c.temperature : 1.f);
    float *loss_rows = none ? c.loss : ws.loss;

    if (teacher) {
        ce::HeadTeacher t = {};
        t.B = c.B;
        t.D = (int)c.D;
        t.C = (int)c.C;
        t.K = (int)c.K;
        t.hidden = static_cast<const unsigned char *>(c.hidden);
        t.weight = static_cast<const unsigned char *>(c.weight);
        t.idx = c.idx;
        t.val = c.val;
        t.val_dtype = c.teacher_dtype;
        t.lse = c.lse;
        t.inv_t = 1.f / c.temperature;
        t.logq = ws.logq;
        t.zk = ws.zk;
        t.mass = ws.mass;
        t.err = err;
        CE_CUDA(ce::launch_head_teacher(t, bf16, sms, s));
    }
    if (z.grad || c.reduction == CE_REDUCE_MEAN) {
        ce::HeadPrep p = {};
        p.B = c.B;
        p.C = (int)c.C;
        p.targets = c.targets;
        p.ignore_index = c.ignore_index;
        p.mass = ws.mass;
        p.scale = c.scale;
        p.scale_per_row = row_scale != nullptr;
        p.mean = c.reduction == CE_REDUCE_MEAN;
        p.mean_of_all = teacher;
        p.alpha = (teacher ? c.temperature : 1.f) / (z.per_row ? 1.f : shift_mul);
        p.perm = ws.perm;
        p.pos = ws.pos;
        p.loss = loss_rows;
        p.info = ws.info;
        p.err = err;
        CE_CUDA(ce::launch_head_prep(p, s));
    }
    if (z.grad) {
        ce::HeadPack p = {};
        p.B = c.B;
        p.C = (int)c.C;
        p.D = (int)c.D;
        p.K = (int)c.K;
        p.pos = ws.pos;
        p.hidden = static_cast<const unsigned char *>(c.hidden);
        p.weight = static_cast<const unsigned char *>(c.weight);
        p.targets = c.targets;
        p.idx = c.idx;
        p.zk = ws.zk;
        p.packed = ws.packed;
        p.dhidden = static_cast<unsigned char *>(c.dhidden);
        p.zt = ws.zt;
        p.ref = z.per_row ? ws.ref : nullptr;
        p.exp_scale = exp_scale;
        p.info = ws.info;
        CE_CUDA(ce::launch_head_pack(p, bf16, s));
    }

    for (long long i = 0; i < z.pieces; ++i) {
        const long long b0 = i * z.piece;
        const long long rows = std::min<long long>(z.piece, c.B - b0);
        const long long padded = round_up(rows, 64);
        const unsigned char *h =
            static_cast<const unsigned char *>(c.hidden) + (size_t)b0 * c.D * 2;
        const unsigned char *hp = ws.packed + (size_t)b0 * c.D * 2;
        ce::HeadGemm g = {};
        g.info = ws.info;
        g.B = (int)c.B;
        g.dynamic = z.grad;
        g.first = (int)b0;
        g.rows = (int)rows;
        g.C = (int)c.C;
        g.D = (int)c.D;
        g.tile_m = z.tile_m;
        g.tile_n = z.tile_n;
        g.alpha = 1.f;
        g.exp_scale = exp_scale;
        g.shift = shift;
        g.targets = c.targets;
        g.perm = ws.perm;
        g.stats = ws.stats;
        g.zt = teacher ? nullptr : ws.zt + b0;
        g.ref = z.per_row ? ws.ref + b0 : nullptr;
        g.failed = &ws.info->failed;
        g.rescue = &ws.info->rescue;
        g.err = err;
        g.parts = ws.parts;
        g.dhidden = static_cast<unsigned char *>(c.dhidden);
        g.skip_row = (int)std::max(-1LL, g_skip_copy >= 0 ? g_skip_copy - b0 : -1LL);
        g.wait_limit = g_wait_limit > 0 ? g_wait_limit : ce::kWaitLimitCycles;
        g.clear_failed = i == 0;
        g.clear_rescue = z.per_row;
        if (z.score) {
            CE_TRY(tensor_map(&g.a, c.dtype, c.weight, c.C, c.D, c.D, z.tile_m / 2));
            CE_TRY(tensor_map(&g.b, c.dtype, h, rows, c.D, c.D, z.tile_n / 2));
        } else {
            CE_TRY(tensor_map(&g.a, c.dtype, h, rows, c.D, c.D, ce::kTileM / 2));
            CE_TRY(tensor_map(&g.b, c.dtype, c.weight, c.C, c.D, c.D, z.tile_n / 2));
        }
        if (z.grad) {
            CE_TRY(tensor_map(&g.packed, c.dtype, hp, padded, c.D, c.D, ce::kTileM / 2));
            CE_TRY(tensor_map(&g.out, c.dtype, ws.exps, padded, z.ld, z.ld, 32));
        } else {
            g.packed = g.out = g.a;  // not used
        }
        g.group_m = 16;
        const ce::HeadEpilogue epi =
            !z.grad ? ce::kEpiStats : z.per_row ? ce::kEpiRef : ce::kEpiKeep;
        CE_CUDA(ce::launch_head_gemm(g, z.score ? ce::kProdScore : ce::kProdLogits, epi, bf16,
                                     pairs, s));

        ce::HeadRows r = {};
        r.B = (int)c.B;
        r.C = (int)c.C;
        r.D = (int)c.D;
        r.dynamic = g.dynamic;
        r.first = g.first;
        r.rows = g.rows;
        r.tiles = z.tiles;
        r.stats = ws.stats;
        r.zt = g.zt;
        r.ref = z.per_row ? ws.ref + b0 : nullptr;
        r.row = ws.row;
        r.exps = ws.exps;
        r.ld = z.ld;
        r.exp_scale = exp_scale;
        r.temperature = c.temperature;
        r.shift_mul = shift_mul;
        r.perm = ws.perm;
        r.targets = c.targets;
        r.ignore_index = c.ignore_index;
        r.logq = ws.logq;
        r.idx = c.idx;
        r.zk = ws.zk;
        r.mass = ws.mass;
        r.K = (int)c.K;
        r.row_scale = row_scale;
        r.info = ws.info;
        r.flag_rescue = 1;
        r.err = err;
        r.loss = loss_rows;
        r.want_grad = z.grad;
        r.nan_on_failure = none && !z.grad;
        r.hidden = h;
        r.packed = hp;
        r.scaled = ws.scaled;
        CE_CUDA(ce::launch_head_rows(r, bf16, s));
        if (z.per_row) {
            // again for rows whose reference exponent was too low (both find
            // nothing to do otherwise)
            g.clear_failed = g.clear_rescue = 0;
            g.only_if = r.only_if = &ws.info->rescue;
            r.flag_rescue = 0;
            CE_CUDA(ce::launch_head_gemm(g, ce::kProdLogits, epi, bf16, pairs, s));
            CE_CUDA(ce::launch_head_rows(r, bf16, s));
            g.only_if = r.only_if = nullptr;
        } else if (z.grad) {
            CE_CUDA(ce::launch_head_scale(r, bf16, s));
        }
        if (teacher) CE_CUDA(ce::launch_head_listed(r, bf16, s));

        g.clear_failed = g.clear_rescue = 0;
        g.skip_row = -1;
        if (c.dhidden) {
            CE_TRY(tensor_map(&g.a, c.dtype, ws.exps, padded, z.ld, z.ld, ce::kTileM / 2));
            CE_TRY(tensor_map(&g.b, c.dtype, c.weight, c.C, c.D, c.D, ce::kTileK));
            g.group_m = 8;
            g.may_split = can_split(c.C);
            g.row_mul = z.per_row ? &ws.row->mul : nullptr;
            g.row_mul_stride = sizeof(ce::HeadRow) / sizeof(float);
            CE_CUDA(ce::launch_head_gemm(g, ce::kProdHidden, ce::kEpiOut, bf16, pairs, s));
            if (g.may_split)
                CE_CUDA(ce::launch_head_join(g, ce::kProdHidden, c.dhidden, bf16, pairs, s));
        }
        if (c.dweight) {
            if (z.per_row) CE_CUDA(ce::launch_head_scale_hidden(r, s));
            CE_TRY(tensor_map(&g.a, c.dtype, ws.exps, padded, z.ld, z.ld, ce::kTileK));
            if (z.per_row) {
                CE_TRY(tensor_map(&g.b, c.dtype, ws.scaled, padded, c.D, c.D, ce::kTileK));
                g.packed = g.b;
            } else {
                CE_TRY(tensor_map(&g.b, c.dtype, h, rows, c.D, c.D, ce::kTileK));
                CE_TRY(tensor_map(&g.packed, c.dtype, hp, padded, c.D, c.D, ce::kTileK));
            }
            if (z.weight_f32)
                CE_TRY(tensor_map(&g.out, CE_F32, ws.weight, c.C, c.D, c.D, 32));
            else
                CE_TRY(tensor_map(&g.out, c.dtype, c.dweight, c.C, c.D, c.D, 32));
            g.group_m = 8;
            g.may_split = !z.weight_f32 && can_split(rows);
            CE_CUDA(ce::launch_head_gemm(g, ce::kProdWeight,
                                         !z.weight_f32 ? ce::kEpiOut
                                         : i == 0      ? ce::kEpiF32
                                                       : ce::kEpiAdd,
                                         bf16, pairs, s));
            if (g.may_split)
                CE_CUDA(ce::launch_head_join(g, ce::kProdWeight, c.dweight, bf16, pairs, s));
        }
    }
    if (c.dweight && z.weight_f32)
        CE_CUDA(ce::launch_head_convert(ws.weight, c.C * c.D, ws.info, 1.f, c.dweight, bf16, sms,
                                        s));
    if (!none || z.grad)
        CE_CUDA(ce::launch_head_loss(loss_rows, c.B, c.reduction, teacher, ws.info, c.loss, s));
    return CE_OK;
}

// The teacher's divergence on given logits: one launch.
struct DistillCall {
    const void *logits;
    const int32_t *idx;
    const void *val;
    const float *lse;
    int64_t B, C, K;
    int dtype, teacher_dtype;
    float temperature;
    int reduction;
    const float *scale;
    float *loss;
    void *grad, *stream;
};

int check(const DistillCall &c) {
    for (int t : {c.dtype, c.teacher_dtype})
        if (t != CE_F32 && t != CE_BF16 && t != CE_F16) return CE_ERR_DTYPE;
    if (c.reduction != CE_REDUCE_MEAN && c.reduction != CE_REDUCE_SUM &&
        c.reduction != CE_REDUCE_NONE)
        return CE_ERR_REDUCTION;
    if (!c.logits || !c.idx || !c.val || !c.loss) return CE_ERR_NULL;
    const uintptr_t es = c.dtype == CE_F32 ? 4 : 2, te = c.teacher_dtype == CE_F32 ? 4 : 2;
    if (c.B < 1 || c.C < 1 || c.K < 1 || c.K > kMaxK || c.B > 0x7fffffffLL || c.C > 0x7fffffffLL ||
        (unsigned long long)c.B * (unsigned long long)c.C > (1ull << 61) / es)
        return CE_ERR_SHAPE;
    if (!temperature_ok(c.temperature)) return CE_ERR_TEMPERATURE;
    const auto off = [](const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a; };
    if (off(c.logits, es) || off(c.grad, es) || off(c.idx, 4) || off(c.val, te) || off(c.lse, 4) ||
        off(c.scale, 4) || off(c.loss, 4))
        return CE_ERR_ALIGN;
    const size_t rows = c.reduction == CE_REDUCE_NONE ? (size_t)c.B * 4 : 4;
    const size_t zb = (size_t)c.B * c.C * es;
    const std::pair<const void *, size_t> in[] = {{c.logits, zb},
                                                  {c.idx, (size_t)c.B * c.K * 4},
                                                  {c.val, (size_t)c.B * c.K * te},
                                                  {c.lse, (size_t)c.B * 4},
                                                  {c.scale, rows}};
    for (const auto &r : in)
        if (ce::host_overlap(c.loss, rows, r.first, r.second) ||
            ce::host_overlap(c.grad, zb, r.first, r.second))
            return CE_ERR_OVERLAP;
    return ce::host_overlap(c.loss, rows, c.grad, zb) ? CE_ERR_OVERLAP : CE_OK;
}

int run(const DistillCall &c) {
    CE_TRY(check(c));
    int dev = 0, sms = 0;
    CE_TRY(ce::host_device(&dev, &sms));
    for (const void *p : {c.logits, (const void *)c.idx, c.val, (const void *)c.lse,
                          (const void *)c.scale, (const void *)c.loss, (const void *)c.grad})
        if (p) CE_TRY(ce::host_check_device_pointer(p, dev));
    cudaStream_t s = static_cast<cudaStream_t>(c.stream);
    ce::DistillParams p;
    CE_TRY(ce::host_error_counters(dev, s, &p.err));
    ce::DistillPlan plan;
    CE_CUDA(ce::plan_distill(c.B, c.C, (int)c.K, c.dtype, c.grad != nullptr, sms, &plan));

    const bool none = c.reduction == CE_REDUCE_NONE;
    std::lock_guard<std::mutex> lk(g_mu);
    unsigned char *ws = nullptr;
    CE_TRY(workspace(dev, s, 256 + (none ? 0 : (size_t)round_up(c.B, 1024) * 4), &ws));
    p.logits = static_cast<const unsigned char *>(c.logits);
    p.targets = nullptr;
    p.grad = static_cast<unsigned char *>(c.grad);
    p.loss_out = c.loss;
    p.loss_rows = none ? c.loss : reinterpret_cast<float *>(ws + 256);
    p.ticket = reinterpret_cast<unsigned int *>(ws + kTicketOffset);
    p.parts = nullptr;
    p.zt = nullptr;
    p.B = c.B;
    p.C = c.C;
    p.inv_b = (float)(1.0 / (double)c.B);
    p.lo_clip = p.hi_clip = 0;
    p.grad_vec_ok = c.grad != nullptr && (reinterpret_cast<uintptr_t>(c.grad) -
                                          reinterpret_cast<uintptr_t>(c.logits)) % 16 == 0;
    p.reduction = c.reduction;
    p.grad_base = c.reduction == CE_REDUCE_MEAN ? p.inv_b : 1.f;
    p.grad_scale = c.scale;
    p.scale_per_row = c.scale != nullptr && none;
    p.softmax = 0;
    p.idx = c.idx;
    p.val = c.val;
    p.val_dtype = c.teacher_dtype;
    p.lse = c.lse;
    p.K = (int)c.K;
    p.list_words = (int)round_up(c.K, 4);
    p.temperature = c.temperature;
    p.exp_scale = ce::kLog2e / c.temperature;
    p.skip_copy_row = g_skip_copy;
    if (g_wait_limit > 0) p.copy_wait_limit = g_wait_limit;
    CE_CUDA(ce::launch_distill(p, c.dtype, plan, s));
    return CE_OK;
}

}  // namespace

namespace ce {

int release_head_workspaces() {
    std::lock_guard<std::mutex> lk(g_mu);
    int rc = CE_OK;
    for (auto &kv : g_buffers) {
        if (!kv.second.base) continue;
        cudaSetDevice(std::get<0>(kv.first));
        const cudaError_t e = cudaFree(kv.second.base);
        if (e != cudaSuccess) rc = host_cuda_fail(e);
    }
    for (auto &b : g_outgrown) {
        cudaSetDevice(b.first);
        const cudaError_t e = cudaFree(b.second);
        if (e != cudaSuccess) rc = host_cuda_fail(e);
    }
    g_buffers.clear();
    g_outgrown.clear();
    return rc;
}

}  // namespace ce

extern "C" {

int ce_linear_fwd_bwd(const void *hidden, const void *weight, const int32_t *targets, int64_t B,
                      int64_t D, int64_t C, int dtype, int32_t ignore_index, int reduction,
                      const float *grad_scale, float *loss_out, void *dhidden_out,
                      void *dweight_out, void *stream) {
    if (!targets) return CE_ERR_NULL;
    Call c = {};
    c.hidden = hidden;
    c.weight = weight;
    c.targets = targets;
    c.ignore_index = ignore_index;
    c.temperature = 1.f;
    c.B = B;
    c.D = D;
    c.C = C;
    c.dtype = dtype;
    c.reduction = reduction;
    c.scale = grad_scale;
    c.loss = loss_out;
    c.dhidden = dhidden_out;
    c.dweight = dweight_out;
    c.stream = stream;
    return run(c);
}

int ce_distill_fwd_bwd(const void *logits, const int32_t *teacher_idx, const void *teacher_val,
                       const float *teacher_lse, int64_t B, int64_t C, int64_t K, int dtype,
                       int teacher_dtype, float temperature, int reduction,
                       const float *grad_scale, float *loss_out, void *grad_out, void *stream) {
    DistillCall c = {};
    c.logits = logits;
    c.idx = teacher_idx;
    c.val = teacher_val;
    c.lse = teacher_lse;
    c.B = B;
    c.C = C;
    c.K = K;
    c.dtype = dtype;
    c.teacher_dtype = teacher_dtype;
    c.temperature = temperature;
    c.reduction = reduction;
    c.scale = grad_scale;
    c.loss = loss_out;
    c.grad = grad_out;
    c.stream = stream;
    return run(c);
}

int ce_heads_test(int64_t skip_copy, int64_t wait_limit_cycles) {
    std::lock_guard<std::mutex> lk(g_mu);
    g_skip_copy = skip_copy >= 0 ? skip_copy : -1;
    g_wait_limit = wait_limit_cycles > 0 ? wait_limit_cycles : 0;
    return CE_OK;
}

int ce_linear_distill_fwd_bwd(const void *hidden, const void *weight, const int32_t *teacher_idx,
                              const void *teacher_val, const float *teacher_lse, int64_t B,
                              int64_t D, int64_t C, int64_t K, int dtype, int teacher_dtype,
                              float temperature, int reduction, const float *grad_scale,
                              float *loss_out, void *dhidden_out, void *dweight_out,
                              void *stream) {
    Call c = {};
    c.hidden = hidden;
    c.weight = weight;
    c.idx = teacher_idx;
    c.val = teacher_val;
    c.lse = teacher_lse;
    c.K = K;
    c.teacher_dtype = teacher_dtype;
    c.temperature = temperature;
    c.B = B;
    c.D = D;
    c.C = C;
    c.dtype = dtype;
    c.reduction = reduction;
    c.scale = grad_scale;
    c.loss = loss_out;
    c.dhidden = dhidden_out;
    c.dweight = dweight_out;
    c.stream = stream;
    return run(c);
}

}  // extern "C"
