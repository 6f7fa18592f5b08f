/*
 * ce_testing.h -- test hooks of the softmax cross-entropy library.
 *
 * Not for production use: these entry points exist so that a test suite can
 * reach code paths that a correct run never takes, and see values that the
 * product entry points do not return.  The pages that define the operation
 * have no counterpart; everything else about the call is as in ce.h.
 */
#ifndef CE_TESTING_H
#define CE_TESTING_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    /* -1: none.  Otherwise the TMA copy that stages row `skip_copy_row` (its
     * tile, slice or first chunk) is never issued, so the kernel's bounded
     * wait for it must give up: the kernel counts a timeout (read it with
     * ce_get_device_errors), makes the batch loss (or that row's loss) NaN,
     * waits for its other copies and returns.  No copy is ever in flight to
     * the skipped slot. */
    int64_t skip_copy_row;
    /* 0: the library's limit (about a second).  Otherwise the number of SM
     * clock cycles after which a wait for a row copy gives up.  The waits for
     * a cluster peer's partial sums and for copies still in flight after a
     * failure keep the library's limit. */
    int64_t wait_limit_cycles;
    /* NULL, or device [B][C] fp32 (4-byte aligned, not overlapping the other
     * arguments): the kernel also writes every gradient element here as the
     * fp32 value it computed before rounding it to the logits' dtype. */
    float *grad_f32_out;
} ce_test_hooks;

/*
 * ce_fwd_bwd_test -- ce_fwd_bwd_path (same arguments, same results) with the
 * test hooks above; hooks may be NULL.  The streaming path (CE_PATH_STREAM)
 * stages nothing and records no fp32 gradient: with any hook set it returns
 * CE_ERR_PATH.  With a hook set the kernels run in their general build (the
 * one ce_fwd_bwd_ex uses), not in the plain call's.
 */
int ce_fwd_bwd_test(const void *logits, const int32_t *targets, int64_t B, int64_t C, int dtype,
                    float *loss_out, void *grad_out, void *stream, int path, int split,
                    const ce_test_hooks *hooks);

/*
 * ce_heads_test -- from now on, in calls of ce_linear_fwd_bwd,
 * ce_linear_distill_fwd_bwd and ce_distill_fwd_bwd of this process:
 *   skip_copy          >= 0: a copy is never issued, so the waits for it must
 *                      give up (the call counts timeouts and its loss, or every
 *                      row's, is NaN): the first stage of the logits' product
 *                      of the rows from this one on in steps of 256; or, of a
 *                      batch that ce_distill_fwd_bwd streams through shared
 *                      memory, the first chunk of this row.  -1: none.
 *   wait_limit_cycles  0: the library's limit (about a second); otherwise the
 *                      number of SM clock cycles after which a wait gives up
 *                      (waits for copies in flight after that keep the
 *                      library's).
 * (-1, 0) restores the ordinary state.  Not for concurrent use.
 */
int ce_heads_test(int64_t skip_copy, int64_t wait_limit_cycles);

#ifdef __cplusplus
}
#endif

#endif /* CE_TESTING_H */
