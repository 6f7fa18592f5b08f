// Host-side interface of the row kernels around the projection's matrix
// products (ce_head_rows.cu).  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include "ce_head_gemm.h"

namespace ce {

// A row after its statistics are joined, exponents in units of log2: the row's
// gradient with respect to class c is `mul` times what is kept for it (a
// reference exponent per row: the exponential) or `mul` 2^(M_tile - M) times
// it (an exponent per tile).
struct HeadRow {
    float M, mul, target, log2S;
};

struct HeadPrep {
    long long B;
    int C;
    const int32_t *targets;    // nullptr: teacher
    int ignore_index;
    const float *mass;         // teacher: [B]
    const float *scale;        // one fp32 or [B]
    int scale_per_row;
    int mean;
    int mean_of_all;           // the mean divides by B
    float alpha;               // a constant factor of the gradients
    int *perm, *pos;           // [B] or nullptr: the counting rows, their places (-1)
    float *loss;               // [B]: set for the rows that do not count
    HeadInfo *info;
    int *err;
};

// Rows that count moved together, the others' hidden gradients set to zero,
// and each row's reference exponent.
struct HeadPack {
    long long B;
    int C, D, K;
    const int *pos;
    const unsigned char *hidden, *weight;
    const int32_t *targets;    // nullptr: teacher
    const int32_t *idx;
    const float *zk;           // teacher: [B][K]
    unsigned char *packed;     // [B rounded up to 64][D]
    unsigned char *dhidden;    // or nullptr
    float *zt, *ref;           // [B] or nullptr
    float exp_scale;
    const HeadInfo *info;
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
    float *logq, *zk;          // [B][K]
    float *mass;               // [B]; the sign bit: a class out of range
    int *err;
};

struct HeadRows {
    int B, C, D;
    int dynamic, first, rows;  // as in HeadGemm
    int tiles;                 // half column tiles (statistics per row)
    const float2 *stats;       // [tiles][rows]
    const float *zt;           // [rows]
    float *ref;                // [rows], or nullptr: an exponent per tile
    HeadRow *row;              // [rows]
    unsigned char *exps;       // [rows][ld] 16-bit exponentials, then gradients
    long long ld;
    float exp_scale;           // log2(e) / T
    float temperature;
    float shift_mul;           // 2^shift of what is kept with an exponent per tile
    const int *perm;           // [B]
    const int32_t *targets;    // [B] (nullptr: teacher)
    int ignore_index;
    const float *logq;         // [B][K] log of the teacher's probabilities, -inf: unused
    const int32_t *idx;        // [B][K]
    const float *zk;           // [B][K] the student's logits there
    const float *mass;         // [B]
    int K;
    const float *row_scale;    // [B] upstream gradient of each row, or nullptr
    HeadInfo *info;
    const int *only_if;        // nullptr, or: nothing to do unless set
    int flag_rescue;
    int *err;
    float *loss;               // [B]
    int want_grad;
    int nan_on_failure;        // the rows' losses are the call's last launch
    const unsigned char *hidden, *packed;  // this piece's rows
    unsigned char *scaled;     // [rows rounded up to 64][D]
};

cudaError_t launch_head_prep(const HeadPrep &p, cudaStream_t s);
cudaError_t launch_head_teacher(const HeadTeacher &p, bool bf16, int sms, cudaStream_t s);
cudaError_t launch_head_pack(const HeadPack &p, bool bf16, cudaStream_t s);
// Joins the tiles' statistics; for a target also the row's loss and gradient
// there.
cudaError_t launch_head_rows(const HeadRows &p, bool bf16, cudaStream_t s);
// Exponents per tile: kept exponentials -> the rows' gradients, in place.
cudaError_t launch_head_scale(const HeadRows &p, bool bf16, cudaStream_t s);
// A reference exponent per row: the hidden states times their rows' factors.
cudaError_t launch_head_scale_hidden(const HeadRows &p, cudaStream_t s);
// Teacher: the row's loss, and what is kept for the listed classes.
cudaError_t launch_head_listed(const HeadRows &p, bool bf16, cudaStream_t s);
// The batch loss of B row losses in the fixed order; reduction none: only
// NaN for all rows after a failure.
cudaError_t launch_head_loss(float *rows, long long B, int reduction, int mean_of_all,
                             const HeadInfo *info, float *loss_out, cudaStream_t s);

}  // namespace ce
