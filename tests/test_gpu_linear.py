"""GPU tests of ce_linear_fwd_bwd and ce_linear_distill_fwd_bwd against the
definition in float64, within the bounds derived in heads.py."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import heads  # noqa: E402
import softmax_cross_entropy_row_gb300 as ce  # noqa: E402

MEAN, SUM, NONE = ce.CE_REDUCE_MEAN, ce.CE_REDUCE_SUM, ce.CE_REDUCE_NONE


@pytest.fixture(scope="module", autouse=True)
def _built():
    ce.build()
    ce.load_library()
    yield
    torch.cuda.synchronize()


def outputs(hidden, weight, reduction, grads="both"):
    B = hidden.shape[0]
    loss = torch.full((B if reduction == NONE else 1,), 7.0, device="cuda")
    dh = torch.full_like(hidden, 7.0) if grads in ("both", "hidden") else None
    dw = torch.full_like(weight, 7.0) if grads in ("both", "weight") else None
    return loss, dh, dw


def check_linear(hidden, weight, targets, dtype, reduction=MEAN, scale=None, ignore=-100,
                 grads="both"):
    loss, dh, dw = outputs(hidden, weight, reduction, grads)
    ce.ce_linear_fwd_bwd(hidden, weight, targets, loss, dh, dw, reduction=reduction,
                         grad_scale=scale, ignore_index=ignore)
    z, dz = heads.logits_of(hidden, weight)
    ref = heads.cross_entropy(z, dz, targets, dtype, reduction, scale, ignore)
    heads.within(loss, *ref.loss(reduction), "loss")
    (want_h, bound_h), (want_w, bound_w) = heads.product_bounds(ref, hidden, weight, dtype)
    if dh is not None:
        heads.within(dh, want_h, bound_h, "dhidden")
    if dw is not None:
        heads.within(dw, want_w, bound_w, "dweight")
    return loss, dh, dw


def some_targets(B, C, seed, ignored=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, C, (B,), generator=g, device="cuda", dtype=torch.int32)
    t[torch.rand(B, generator=g, device="cuda") < ignored] = -100
    return t


# one class, one row, one chunk of D; ragged in every direction around the
# tiles of 256 x 256 x 64; few rows with a long vocabulary (the hidden states'
# gradient split over it); few classes with many rows (the weights' split)
SHAPES = [(1, 8, 1), (1, 64, 7), (2, 16, 64), (3, 72, 257), (130, 128, 300), (257, 200, 1000),
          (256, 256, 256), (300, 1000, 513), (64, 512, 32000), (700, 256, 5003), (5000, 136, 97)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,D,C", SHAPES)
def test_linear_shapes(B, D, C, dtype):
    t = some_targets(B, C, B + C)
    h, w = heads.projection(B, D, C, dtype, B * 7 + D, raised=t)
    check_linear(h, w, t, dtype)
