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


@pytest.mark.parametrize("B,C", [(40, 700), (60, 9000), (400, 9000), (200, 60001)])
@pytest.mark.parametrize("reduction,T,own,grads,dtype,tdtype", [
    (SUM, 2.0, False, True, "f32", "bf16"), (NONE, 0.5, True, True, "bf16", "f16"),
    (NONE, 1.0, False, True, "f16", "f32"), (MEAN, 4.0, True, False, "f32", "f32"),
    (NONE, 1.0, True, False, "bf16", "f32"), (MEAN, 0.75, False, True, "f16", "bf16")])
def test_distill_options(B, C, reduction, T, own, grads, dtype, tdtype):
    K = 37
    idx, val = heads.teacher_lists(B, C, K, 7, empty=0.2, ragged=True)
    val = val.to(heads.TORCH_DT[tdtype])
    lse = torch.logsumexp(val.float() / T, 1) + 0.3 if own else None
    n = B if reduction == NONE else 1
    scale = torch.rand(n, device="cuda") * 2 - 0.5
    z = student(B, C, dtype, 7, idx, val.float())
    check_distill(z, idx, val, dtype, lse, T, reduction, scale, grads)


# a warp per row, a cluster per row, a CTA in two passes, the ring (resident
# and streamed twice)
KERNELS = [(30, 1000), (20, 20000), (100, 70000), (400, 20000), (200, 110001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C", KERNELS)
def test_rows_without_a_list(B, C, dtype):
    """Loss 0 and gradient 0 whatever the row and its unused places hold."""
    K = 9
    idx, val = heads.teacher_lists(B, C, K, 5, empty=0.4, ragged=True)
    idx[0], idx[1] = -1, torch.arange(K, device="cuda")
    z = student(B, C, dtype, 5)
    used = idx >= 0
    clean = torch.where(used, val, torch.zeros_like(val))
    a = check_distill(z, idx, clean, dtype, reduction=NONE)
    val[~used] = math.nan
    z[~used.any(1)] = math.nan
    z[0, ::2] = math.inf
    loss, grad = torch.full((B,), 7.0, device="cuda"), torch.full_like(z, 7.0)
    ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, reduction=NONE)
    assert torch.equal(loss, a[0]) and torch.equal(grad, a[1])
    assert (loss[~used.any(1)] == 0).all() and (grad[~used.any(1)] == 0).all()


@pytest.mark.parametrize("B,C", KERNELS)
@pytest.mark.parametrize("K", [3, 40, 500])
def test_repeated_and_bad_classes(B, C, K):
    g = torch.Generator("cuda").manual_seed(2)
    idx = torch.randint(0, max(2, K // 2), (B, K), generator=g, device="cuda", dtype=torch.int32)
    val = torch.randn(B, K, generator=g, device="cuda")
    z = student(B, C, "f32", 2)
    first = check_distill(z, idx, val, "f32", reduction=NONE)
    again = check_distill(z, idx, val, "f32", reduction=NONE)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    idx[4, 2], idx[9, 0], idx[9, 1] = C, -2, 2 ** 31 - 1
    idx[11] = -5
    ce.ce_get_device_errors()
    check_distill(z, idx, val, "f32", reduction=NONE)
    assert ce.ce_get_device_errors() == (3, 0)


@pytest.mark.parametrize("B,C,K", [(400, 3, 500), (10, 3, 1000), (400, 1000, 900), (1, 5, 4)])
def test_lists_longer_than_the_row(B, C, K):
    g = torch.Generator("cuda").manual_seed(6)
    idx = torch.randint(-1, C, (B, K), generator=g, device="cuda", dtype=torch.int32)
    val = torch.randn(B, K, generator=g, device="cuda") * 3
    for dtype in ("f32", "f16"):
        check_distill(student(B, C, dtype, 6), idx, val, dtype, reduction=NONE)


@pytest.mark.parametrize("B,C,dtype", [(460, 45362, "f16"), (741, 41035, "f16"),
                                       (620, 24577, "f32"), (500, 60001, "bf16")])
def test_slots_are_not_refilled_while_they_are_read(B, C, dtype):
    """Rows that fill the ring, a gradient aligned unlike the logits (stored
    element by element, slowly): every run has the first one's bits."""
    idx, val = heads.teacher_lists(B, C, 2, 1)
    buf = torch.randn(B * C + 8, device="cuda").mul_(3).to(heads.TORCH_DT[dtype])
    z = buf[1:1 + B * C].view(B, C)
    loss, grad = check_distill(z, idx, val, dtype, reduction=NONE)
    again = torch.empty_like(grad)
    for _ in range(150):
        again.fill_(7)
        ce.ce_distill_fwd_bwd(z, idx, val, loss, again, reduction=NONE)
        assert torch.equal(again, grad)


def test_every_list_length_fits():
    """The ring's shared memory for any K (its lists take what the row's chunks
    leave), on rows of each of its kernels."""
    for C in (9000, 20000, 110001):
        z = student(160, C, "bf16", C)
        loss = torch.empty(160, device="cuda")
        for K in range(1, 1025, 7):
            idx, val = heads.teacher_lists(160, C, K, K)
            loss.fill_(math.nan)
            ce.ce_distill_fwd_bwd(z, idx, val, loss, reduction=NONE)
            assert torch.isfinite(loss).all(), (C, K)


@pytest.mark.parametrize("B,C", KERNELS)
def test_small_probabilities_of_repeated_classes(B, C):
    """Sums of places of one class keep their bits however small they are."""
    g = torch.Generator("cuda").manual_seed(7)
    K = 120
    idx = torch.randint(0, 60, (B, K), generator=g, device="cuda", dtype=torch.int32)
    val = torch.randn(B, K, generator=g, device="cuda") * 4
    lse = torch.logsumexp(val * 2, 1)
    z = student(B, C, "f32", 7)
    for shift in (None, 0.0, 12.0, -3.0):
        check_distill(z, idx, val, "f32", None if shift is None else lse + shift, T=0.5,
                      reduction=NONE)


@pytest.mark.parametrize("B,C", KERNELS)
def test_cold_and_hot(B, C):
    """Temperatures at which the softmax is one class, and uniform."""
    idx, val = heads.teacher_lists(B, C, 5, 8)
    z = student(B, C, "f32", 8, idx, val)
    for T in (1e-3, 1e4):
        check_distill(z, idx, val, "f32", T=T, reduction=NONE)
    loss, grad = torch.empty(B, device="cuda"), torch.empty_like(z)
    ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, temperature=1e-30, reduction=NONE)
    assert not torch.isnan(grad).any() and not torch.isnan(loss).any()


@pytest.mark.parametrize("B,C", KERNELS)
def test_values_at_the_types_ends(B, C):
    """Student: -inf for classes ruled out, whole rows of the type's lowest
    value, one class far above it.  Teacher: -inf, the lowest value."""
    K = 4
    for dtype in ("f32", "bf16", "f16"):
        lowest = torch.finfo(heads.TORCH_DT[dtype]).min
        idx, val = heads.teacher_lists(B, C, K, 3)
        val[:, 1] = -math.inf
        val[:, 2] = torch.finfo(torch.float32).min
        z = student(B, C, dtype, 3)
        ruled_out = torch.rand(B, C, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) < 0.5
        ruled_out.scatter_(1, idx.long(), False)
        z[ruled_out] = -math.inf
        check_distill(z, idx, val, dtype, reduction=NONE)
        z[0] = lowest                    # uniform
        z[1] = lowest
        z[1, 7] = 3.0                    # certain
        idx[1] = torch.tensor([7, 8, -1, -1], device="cuda")
        val[1, 1] = val[1, 0]
        idx[2] = torch.tensor([C - 1, -1, -1, -1], device="cuda")
        z[2, C - 1] = -math.inf          # listed and ruled out
        loss, grad = torch.empty(B, device="cuda"), torch.empty_like(z)
        ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, reduction=NONE)
        u = heads.unit(dtype)
        free = torch.ones(C, dtype=torch.bool, device="cuda")
        free[idx[0].long()] = False
        assert ((grad[0][free].double() - 1 / C).abs() <= (u + 2.0 ** -18) / C + 2.0 ** -25).all()
        # sum q (log q - log 1/C) = log C - H(q), q on the two finite values
        q = torch.softmax(val[0, [0, 3]].double(), 0)
        want = math.log(C) + (q * q.log()).sum().item()
        assert abs(loss[0].item() - want) <= 2.0 ** -18 * math.log(C)
        # q = expf(log q): 2 ulp of 1/2, the logarithm's 2^-24, one rounding
        near = u + 3 * 2.0 ** -24
        assert abs(grad[1, 7].item() - 0.5) <= near and abs(grad[1, 8].item() + 0.5) <= near
        assert loss[1].item() > 1e3 and loss[2].item() == math.inf
        assert grad[2, C - 1].item() == -1.0 and not torch.isnan(grad[2]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C", KERNELS)
def test_unaligned_and_guarded(B, C, dtype):
    """Logits and gradient at any element offset, the same or another one mod
    16 bytes; inputs lie in NaN, outputs between guards."""
    K = 6
    idx, val = heads.teacher_lists(B, C, K, 13)
    z = student(B, C, dtype, 13, idx, val)
    want = check_distill(z, idx, val, dtype)
    for off_z, off_g in ((1, 1), (3, 0), (0, 1), (2, 3)):
        zb = torch.full((z.numel() + 64,), math.nan, dtype=z.dtype, device="cuda")
        gb = torch.full_like(zb, 3.0)
        zv = zb[16 + off_z:16 + off_z + z.numel()].view(B, C)
        gv = gb[16 + off_g:16 + off_g + z.numel()].view(B, C)
        zv.copy_(z)
        check_distill(zv, idx, val, dtype, grad=gv)
        assert (gb[:16 + off_g] == 3).all() and (gb[16 + off_g + z.numel():] == 3).all()
    loss = torch.empty(1, device="cuda")
    ce.ce_distill_fwd_bwd(z, idx, val, loss)
    assert torch.equal(loss, want[0])


@pytest.mark.parametrize("B,C", KERNELS)
def test_same_bits_on_streams_and_in_graphs(B, C):
    K = 20
    idx, val = heads.teacher_lists(B, C, K, 17, empty=0.1)
    z = student(B, C, "bf16", 17, idx, val)
    first = check_distill(z, idx, val, "bf16")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty(1, device="cuda"), torch.empty_like(z)) for _ in range(4)]
    graphs = []
    for out in outs[2:]:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            ce.ce_distill_fwd_bwd(z, idx, val, *out)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, out, g in zip(streams, outs, graphs):
            ce.ce_distill_fwd_bwd(z, idx, val, *out, stream=s)
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_distill_gradient_against_differences():
    """Central differences along a direction: off by at most r^3 d^2 / 3 a row
    (T = 1) and by the losses' own error over d."""
    B, C, K, step = 5, 200, 6, 2.0 ** -4
    idx, val = heads.teacher_lists(B, C, K, 4)
    z = (student(B, C, "f32", 4, idx, val) * 64).round() / 64
    loss, grad = check_distill(z, idx, val, "f32", reduction=SUM)
    ref = heads.divergence(z.double(), torch.zeros(B, device="cuda").double(), idx, val, None, 1.0,
                           "f32", SUM)
    err = ref.drows.sum().item() + 2.0 ** -20
    for i in range(4):
        g = torch.Generator("cuda").manual_seed(i)
        v = torch.randint(0, 2, z.shape, generator=g, device="cuda") * 2.0 - 1
        ends = []
        for sign in (1, -1):
            ce.ce_distill_fwd_bwd(z + sign * step * v, idx, val, loss, reduction=SUM)
            ends.append(loss.item())
        slope = (grad.double() * v).sum().item()
        bound = B * 8 * step ** 2 / 3 + err / step + 1e-5
        assert abs((ends[0] - ends[1]) / (2 * step) - slope) <= bound


def test_offsets_past_32_bits():
    """More than 2^31 logits; the last rows against float64."""
    B, C, K = 17000, 131073, 5
    z = torch.empty(B, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    for i in range(0, B, 1000):
        z[i:i + 1000] = torch.randn(min(1000, B - i), C, generator=g, device="cuda") * 2
    idx, val = heads.teacher_lists(B, C, K, 3)
    loss, grad = torch.empty(B, device="cuda"), torch.full_like(z, 7.0)
    ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, reduction=NONE)
    for s in (slice(0, 50), slice(B - 50, B)):
        ref = heads.divergence(z[s].double(), torch.zeros(50, device="cuda").double(), idx[s],
                               val[s], None, 1.0, "bf16", NONE, kept=1)
        heads.within(loss[s], *ref.loss(NONE), "loss")
        heads.within(grad[s], ref.G, ref.dG + 2.0 ** -126, "grad")
    assert not (grad[B // 2] == 7).any()
