"""The bounded waits of the projection's and the distillation's kernels: a copy
that is never issued (nothing is in flight for it) makes them give up, count
timeouts and answer NaN; the next call is as if nothing had happened."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import heads  # noqa: E402
import softmax_cross_entropy_row_gb300 as ce  # noqa: E402

LIMIT = 50_000_000  # cycles, some 25 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    ce.build()
    ce.load_library()
    yield
    ce.ce_heads_test()
    torch.cuda.synchronize()


def check(call, outs, bad):
    """`call` writes `outs` (the loss first); `bad`: rows' losses that have to
    be NaN with the hook set."""
    ce.ce_heads_test()
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    assert not any(torch.isnan(x).any() for x in want)
    assert ce.ce_get_device_errors() == (0, 0)
    ce.ce_heads_test(bad, LIMIT)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        ce.ce_heads_test()
    loss = outs[0]
    assert math.isnan(loss.view(-1)[min(bad, loss.numel() - 1)].item())
    assert ce.ce_get_device_errors()[1] > 0
    call()
    torch.cuda.synchronize()
    assert ce.ce_get_device_errors() == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("reduction", [ce.CE_REDUCE_MEAN, ce.CE_REDUCE_NONE])
@pytest.mark.parametrize("B,grads,dtype", [(9, False, "bf16"), (300, False, "bf16"),
                                           (300, True, "bf16"), (300, True, "f16")])
def test_a_stage_of_the_logits_is_missing(B, grads, dtype, reduction):
    t = torch.arange(B, device="cuda", dtype=torch.int32)
    h, w = heads.projection(B, 200, 3000, dtype, 1, raised=t)
    loss = torch.empty(B if reduction == ce.CE_REDUCE_NONE else 1, device="cuda")
    outs = [loss] + ([torch.empty_like(h), torch.empty_like(w)] if grads else [])
    check(lambda: ce.ce_linear_fwd_bwd(h, w, t, *outs, reduction=reduction), outs, 0)


def test_a_stage_of_a_later_tile_row_is_missing():
    B = 700
    idx, val = heads.teacher_lists(B, 3000, 5, 2)
    h, w = heads.projection(B, 136, 3000, "bf16", 2)
    outs = [torch.empty(B, device="cuda"), torch.empty_like(h), torch.empty_like(w)]
    check(lambda: ce.ce_linear_distill_fwd_bwd(h, w, idx, val, *outs,
                                               reduction=ce.CE_REDUCE_NONE), outs, 600)


@pytest.mark.parametrize("reduction", [ce.CE_REDUCE_MEAN, ce.CE_REDUCE_NONE])
@pytest.mark.parametrize("B,C", [(700, 9000), (400, 20000), (320, 110001)])
def test_a_chunk_of_a_row_is_missing(B, C, reduction):
    idx, val = heads.teacher_lists(B, C, 20, 3)
    z = (torch.randn(B, C, device="cuda") * 2).bfloat16()
    loss = torch.empty(B if reduction == ce.CE_REDUCE_NONE else 1, device="cuda")
    outs = [loss, torch.empty_like(z)]
    check(lambda: ce.ce_distill_fwd_bwd(z, idx, val, *outs, reduction=reduction), outs, 170)
