// Host-side interface of the row kernels around the projection's matrix
// products (ce_head_rows.cu).  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include "ce_device.cuh"

namespace ce {

// What the launches of one call share on the device.
struct HeadInfo {
    int count;    // rows that count for the mean
    float out;    // factor of the gradients (what is not in the rows' own)
    float norm;   // what the rows' own factors are divided by
    int failed;   // a bounded wait gave up
};

// A row after its statistics are joined, in units of log2: p = E 2^(M_tile -
// M) mul, E the kept exponential; `target` replaces the target's element.
struct HeadRow {
    float M, mul, target, log2S;
};

struct HeadRows {
    int rows, cols;            // of this piece
    int tiles;                 // column tiles of the statistics
    const float2 *stats;       // [tiles][rows]
    const float *zt;           // [rows]
    HeadRow *row;              // [rows]
    unsigned char *exps;       // [rows][ld] 16-bit exponentials, then gradients
    long long ld;
    float exp_scale;           // log2(e) / T
    float temperature;
    float shift_mul;           // 2^shift of the kept values
    // cross-entropy
    const int32_t *targets;    // [rows] (nullptr: teacher)
    int ignore_index;
    // teacher
    const float *logq;         // [rows][K] log of the teacher's probabilities, -inf: unused
    const int32_t *idx;        // [rows][K]
    const float *zk;           // [rows][K] the student's logits there
    const float *mass;         // [rows] sum of the probabilities; NaN: a bad index
    int K;
    const float *row_scale;    // [rows] upstream gradient of each row, or nullptr
    const HeadInfo *info;
    int *err;
    float *loss;               // [rows]
    int want_grad;
    int nan_on_failure;        // the rows' losses are the call's last launch
};

struct HeadPrep {
    long long B;
    const int32_t *targets;    // nullptr: every row counts
    int ignore_index;
    const float *mass;         // teacher: [B]
    const float *scale;        // one fp32 or [B]
    int scale_per_row;
    int mean;
    float alpha;               // a constant factor of the gradients
    HeadInfo *info;
};

struct HeadTeacher {
    long long B;
    int D, C, K;
    const unsigned char *hidden, *weight;
    const int32_t *idx;        // [B][K]
    const void *val;           // [B][K]
    int val_dtype;
    const float *lse;          // [B] or nullptr
    float inv_t;
    float *logq, *zk, *mass;
    int *err;
};

cudaError_t launch_head_prep(const HeadPrep &p, cudaStream_t s);
cudaError_t launch_head_teacher(const HeadTeacher &p, bool bf16, int sms, cudaStream_t s);
// Joins the tiles' statistics; for a target also the row's loss.
cudaError_t launch_head_rows(const HeadRows &p, cudaStream_t s);
// Kept exponentials -> the rows' gradients with respect to the logits, in place.
cudaError_t launch_head_scale(const HeadRows &p, bool bf16, cudaStream_t s);
// Teacher: the row's loss, and the listed classes' gradients.
cudaError_t launch_head_listed(const HeadRows &p, bool bf16, cudaStream_t s);
// out[i] = alpha scale (part_0[i] + part_1[i] + ...), n elements a part
// (a multiple of 8), to 16 bits.
cudaError_t launch_head_join(const float *parts, long long n, long long part_stride, int nparts,
                             const float *scale, float alpha, void *out, bool bf16, int sms,
                             cudaStream_t s);
// The batch loss of B row losses in the fixed order; reduction none: only
// NaN for all rows after a failure.
cudaError_t launch_head_loss(float *rows, long long B, int reduction, const HeadInfo *info,
                             float *loss_out, cudaStream_t s);

}  // namespace ce
