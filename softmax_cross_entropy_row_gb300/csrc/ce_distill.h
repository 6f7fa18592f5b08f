// Host-side interface of the teacher's divergence on given logits
// (ce_distill.cu).  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include "ce_device.cuh"

namespace ce {

struct DistillParams : ParamsEx {
    const int32_t *idx;    // [B][K], -1: unused
    const void *val;       // [B][K] the teacher's logits
    int val_dtype;
    const float *lse;      // [B] or nullptr (the list's own normaliser)
    int K;
    int list_words;        // shared-memory words of a row's list
    float temperature;
    float exp_scale;       // log2(e) / T
};

// How a row is spread: `group` threads (32: a warp per row, eight rows per
// CTA; else one CTA per row) of `vecs` 16-byte vectors each; `cluster` CTAs
// per row; `loop`: rows longer than the registers hold, read twice.
// `ring_threads` (else 0): rows go through a ring of `slots` chunks instead (of
// 512 threads: streamed twice).
struct DistillPlan {
    int group, vecs, cluster;
    bool loop;
    int ring_threads, slots, table_bits;
    int ctas;
    int smem;
};

cudaError_t plan_distill(long long B, long long C, int K, int dtype, bool grad, int sms,
                         DistillPlan *plan);
cudaError_t launch_distill(const DistillParams &p, int dtype, const DistillPlan &plan,
                           cudaStream_t s);

}  // namespace ce
