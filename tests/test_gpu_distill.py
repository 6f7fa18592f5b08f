"""GPU tests of ce_distill_fwd_bwd against the definition in float64, within
the bounds derived in heads.py."""

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


def student(B, C, dtype, seed, idx=None, val=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B, C, generator=g, device="cuda") * 2
    if idx is not None:
        z.scatter_add_(1, idx.clamp(0, C - 1).long(),
                       torch.where((idx >= 0) & (idx < C), 0.7 * val, torch.zeros_like(val)))
    return z.to(heads.TORCH_DT[dtype])


def check_distill(z, idx, val, dtype, lse=None, T=1.0, reduction=MEAN, scale=None, grads=True,
                  grad=None):
    B, C = z.shape
    loss = torch.full((B if reduction == NONE else 1,), 7.0, device="cuda")
    if grads and grad is None:
        grad = torch.full_like(z, 7.0)
    ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, teacher_lse=lse, temperature=T,
                          reduction=reduction, grad_scale=scale)
    ref = heads.divergence(z.double(), torch.zeros(B, device="cuda").double(), idx, val.float(),
                           lse, T, dtype, reduction, scale, kept=1)
    heads.within(loss, *ref.loss(reduction), "loss")
    if grads:
        u = heads.unit(dtype) * ref.G.abs() if dtype == "f32" else 0
        heads.within(grad, ref.G, ref.dG + u + heads.SMALLEST[dtype] + 2.0 ** -126, "grad")
    return loss, grad


# (B, C, K): a warp per row (one class, ragged, 4 and 8 KB rows), a CTA per
# row (both sizes), two passes, and few long rows on a cluster of CTAs (each
# of the cluster's sizes, and too long for its registers); then many rows
# through the ring (resident, its fullest row, streamed twice, a long list)
SHAPES = [(1, 1, 1), (5, 7, 3), (300, 1000, 8), (17, 2047, 33), (9, 4096, 1), (3, 9001, 64),
          (100, 16000, 100), (400, 16000, 100), (330, 32000, 64), (320, 50257, 20), (40, 50257, 7), (2, 128256, 100),
          (1, 300001, 1024), (30, 131072, 256),
          (700, 9001, 31), (320, 53248, 5), (310, 53264, 64), (200, 130001, 1024)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,C,K", SHAPES)
def test_distill_shapes(B, C, K, dtype):
    idx, val = heads.teacher_lists(B, C, K, B + C)
    check_distill(student(B, C, dtype, C, idx, val), idx, val, dtype)
