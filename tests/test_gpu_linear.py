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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("grads", ["both", "hidden", "weight", "none"])
@pytest.mark.parametrize("reduction", [MEAN, SUM, NONE])
def test_linear_reductions(reduction, grads, dtype):
    B, D, C = 333, 104, 700
    t = some_targets(B, C, 5, ignored=0.3)
    h, w = heads.projection(B, D, C, dtype, 5, raised=t)
    n = B if reduction == NONE else 1
    scale = torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) * 4 - 1
    check_linear(h, w, t, dtype, reduction, scale, grads=grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 65, 128, 257])
@pytest.mark.parametrize("D,C", [(8, 1), (64, 250), (200, 5003), (264, 40000)])
def test_loss_alone(B, D, C, dtype):
    """Few rows (classes as the tiles' rows, up to 64 rows of the batch), one
    tile's and more."""
    t = some_targets(B, C, B, ignored=0.1)
    t[B // 2] = C - 1
    h, w = heads.projection(B, D, C, dtype, B + C, raised=t)
    check_linear(h, w, t, dtype, NONE, grads="none")
    check_linear(h, w, t, dtype, MEAN, grads="none")
    idx, val = heads.teacher_lists(B, C, 4, B)
    check_linear_distill(h, w, idx, val, dtype, reduction=NONE, grads="none")


def test_linear_upstream_gradients_of_any_size():
    """f16 keeps the rows' gradients relative to the largest upstream one."""
    B, D, C = 90, 64, 333
    t = some_targets(B, C, 9)
    h, w = heads.projection(B, D, C, "f16", 9, raised=t)
    scale = torch.full((B,), 3000.0, device="cuda")
    scale[::3] = -0.125
    scale[1] = 0.0
    check_linear(h * 0.01, w, t, "f16", NONE, scale, grads="hidden")
    check_linear(h, w, t, "bf16" if h.dtype == torch.bfloat16 else "f16", NONE, scale * 1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ignored_rows_take_no_part(dtype):
    """Whatever hidden states ignored rows hold: loss 0, gradient 0, nothing in
    the weights' gradient; ignore_index may be a class."""
    B, D, C = 290, 72, 310
    t = some_targets(B, C, 1)
    t[torch.arange(B, device="cuda") % 3 == 1] = 17
    h, w = heads.projection(B, D, C, dtype, 1, raised=t)
    bad = h.clone()
    bad[t == 17] = math.nan
    bad[1] = math.inf
    for reduction in (MEAN, NONE):
        loss, dh, dw = outputs(h, w, reduction)
        ce.ce_linear_fwd_bwd(bad, w, t, loss, dh, dw, reduction=reduction, ignore_index=17)
        z, dz = heads.logits_of(h, w)
        ref = heads.cross_entropy(z, dz, t, dtype, reduction, None, 17)
        (want_h, bound_h), (want_w, bound_w) = heads.product_bounds(ref, h, w, dtype)
        heads.within(loss, *ref.loss(reduction), "loss")
        heads.within(dh, want_h, bound_h, "dhidden")
        heads.within(dw, want_w, bound_w, "dweight")
        assert torch.equal(dh[t == 17], torch.zeros_like(dh[t == 17]))
    ce.ce_linear_fwd_bwd(h, w, t, loss, reduction=NONE, ignore_index=17)  # the loss alone
    assert (loss[t == 17] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("reduction", [MEAN, SUM, NONE])
def test_no_row_counts(dtype, reduction):
    h, w = heads.projection(70, 64, 300, dtype, 3)
    t = torch.full((70,), -100, dtype=torch.int32, device="cuda")
    for value in (0.5, math.nan):
        h.fill_(value)
        loss, dh, dw = outputs(h, w, reduction)
        ce.ce_linear_fwd_bwd(h, w, t, loss, dh, dw, reduction=reduction)
        for x in (loss, dh, dw):
            assert torch.equal(x, torch.zeros_like(x))
    loss.fill_(7.0)
    ce.ce_linear_fwd_bwd(h.fill_(1.0), w, t, loss, reduction=reduction)
    assert torch.equal(loss, torch.zeros_like(loss))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_targets_out_of_range(dtype):
    B, D, C = 40, 64, 200
    t = some_targets(B, C, 4)
    t[3], t[8], t[9] = C, -1, 2 ** 31 - 1
    h, w = heads.projection(B, D, C, dtype, 4, raised=t)
    ce.ce_get_device_errors()
    check_linear(h, w, t, dtype, NONE)
    assert ce.ce_get_device_errors() == (3, 0)
    check_linear(h, w, t, dtype, NONE, grads="none")
    assert ce.ce_get_device_errors() == (3, 0)
    loss, _, _ = check_linear(h, w, t, dtype, MEAN)
    assert math.isnan(loss.item())
    ce.ce_get_device_errors()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sigma", [30.0, 120.0])
def test_logits_far_apart(dtype, sigma):
    """Targets far below the largest logit: bf16's reference exponent, taken
    from the target, is too low for some rows or for all."""
    B, D, C = 300, 64, 600
    t = some_targets(B, C, 6)
    h, w = heads.projection(B, D, C, dtype, 6, sigma=sigma)
    if sigma > 100:
        t[5] = (h[5].float() @ w.float().T).argmin().int()
        z = h[5].float() @ w.float().T
        assert z.max() - z[t[5].item()] > 300
    check_linear(h, w, t, dtype, NONE)
    t[::2] = (h[::2].float() @ w.float().T).argmax(1).int()  # near-certain targets among them
    check_linear(h, w, t, dtype, NONE)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_row_that_is_not_finite(dtype):
    """NaN stays in its row's loss and hidden gradient; the weights' gradient,
    a sum over rows, has it too."""
    B, D, C = 20, 64, 300
    t = some_targets(B, C, 8)
    h, w = heads.projection(B, D, C, dtype, 8, raised=t)
    h[7, 3] = math.nan
    loss, dh, dw = outputs(h, w, NONE)
    ce.ce_linear_fwd_bwd(h, w, t, loss, dh, dw, reduction=NONE)
    rows = torch.arange(B, device="cuda") != 7
    assert torch.isnan(loss[7]) and torch.isnan(dh[7]).all() and torch.isnan(dw).any()
    keep, _, _ = outputs(h, w, NONE)
    good = h.clone()
    good[7] = 0
    dh2 = torch.empty_like(dh)
    ce.ce_linear_fwd_bwd(good, w, t, keep, dh2, None, reduction=NONE)
    assert torch.equal(loss[rows], keep[rows]) and torch.equal(dh[rows], dh2[rows])


@pytest.mark.parametrize("teacher", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_several_pieces(dtype, teacher):
    """More rows than one piece of kept exponentials holds (1 GiB), a third of
    them not counted: the weights' gradient is formed over three pieces."""
    B, D, C = 22000, 64, 50257
    if teacher:
        idx, val = heads.teacher_lists(B, C, 5, 3, empty=0.1)
        h, w = heads.projection(B, D, C, dtype, 11)
        check_linear_distill(h, w, idx, val, dtype)
    else:
        t = some_targets(B, C, 11, ignored=0.1)
        h, w = heads.projection(B, D, C, dtype, 11, raised=t)
        check_linear(h, w, t, dtype)


def test_inputs_and_outputs_inside_larger_buffers():
    """Nothing outside the tensors is read into the results or written: inputs
    lie in NaN, outputs between guards."""
    B, D, C = 70, 200, 333

    def inside(x, fill):
        n = x.numel()
        buf = torch.full((n + 4096,), fill, dtype=x.dtype, device="cuda")
        view = buf[2048:2048 + n].view(x.shape)
        view.copy_(x)
        return buf, view

    for dtype in ("bf16", "f16"):
        t = some_targets(B, C, 2, ignored=0.2)
        h, w = heads.projection(B, D, C, dtype, 2, raised=t)
        _, hv = inside(h, math.nan)
        _, wv = inside(w, math.nan)
        bh, dh = inside(torch.zeros_like(h), 3.0)
        bw, dw = inside(torch.zeros_like(w), 3.0)
        bl, loss = inside(torch.zeros(1, device="cuda"), 3.0)
        ce.ce_linear_fwd_bwd(hv, wv, t, loss, dh, dw)
        l2, dh2, dw2 = check_linear(h, w, t, dtype)
        assert torch.equal(loss, l2) and torch.equal(dh, dh2) and torch.equal(dw, dw2)
        for buf in (bh, bw, bl):
            assert (buf[:2048] == 3).all() and (buf[-2048:] == 3).all()


def test_same_bits_each_time_and_on_another_stream():
    for dtype in ("bf16", "f16"):
        t = some_targets(700, 3000, 3, ignored=0.1)
        h, w = heads.projection(700, 128, 3000, dtype, 3, raised=t)
        first = check_linear(h, w, t, dtype)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        runs = []
        for i in range(4):  # two streams at once, twice
            out = outputs(h, w, MEAN)
            torch.cuda.synchronize()
            ce.ce_linear_fwd_bwd(h, w, t, *out, stream=streams[i % 2])
            runs.append(out)
        torch.cuda.synchronize()
        for out in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_calls_from_two_threads():
    """Two host threads with a stream each, and two on one stream."""
    import threading

    cases = []
    for seed in (1, 2):
        t = some_targets(400 * seed, 1500, seed, ignored=0.2)
        h, w = heads.projection(400 * seed, 128, 1500, "bf16", seed, raised=t)
        cases.append((h, w, t, check_linear(h, w, t, "bf16")))
    own = [torch.cuda.Stream() for _ in cases]
    shared = torch.cuda.Stream()
    for streams in (own, [shared, shared]):
        wrong = []

        def work(i):
            h, w, t, want = cases[i]
            for _ in range(20):
                with torch.cuda.stream(streams[i]):
                    out = [torch.empty_like(x) for x in want]
                    ce.ce_linear_fwd_bwd(h, w, t, *out, stream=streams[i])
                    if not all(torch.equal(a, b) for a, b in zip(out, want)):
                        wrong.append(i)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        torch.cuda.synchronize()
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        torch.cuda.synchronize()
        assert not wrong


def test_graphs_replayed_at_the_same_time():
    """Two captured calls (the stream's first) replayed on two streams while an
    eager call runs: each has a workspace of its own.  A replay sees changed
    inputs."""
    cases = []
    for seed in (1, 2):
        t = some_targets(500, 2000, seed, ignored=0.2)
        h, w = heads.projection(500, 192, 2000, "bf16", seed, raised=t)
        out = outputs(h, w, MEAN)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            ce.ce_linear_fwd_bwd(h, w, t, *out)
        cases.append((h, w, t, out, g))
    streams = [torch.cuda.Stream() for _ in cases]
    for round_ in range(3):
        for h, w, t, out, g in cases:
            h.copy_(torch.roll(h, 1, 0))
            t.copy_(torch.roll(t, 1, 0))
        torch.cuda.synchronize()
        for (h, w, t, out, g), s in zip(cases, streams):
            with torch.cuda.stream(s):
                g.replay()
        check_linear(*cases[0][:3], "bf16")
        torch.cuda.synchronize()
        for h, w, t, out, g in cases:
            want = check_linear(h, w, t, "bf16")
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    ce.ce_release_workspaces()
    check_linear(*cases[0][:3], "bf16")


def test_a_growing_workspace_beside_a_capture():
    """While one stream is being captured, a call on another one may need a
    larger workspace: the capture goes on."""
    t = some_targets(300, 900, 5)
    h, w = heads.projection(300, 64, 900, "bf16", 5, raised=t)
    t2 = some_targets(900, 20000, 6)
    h2, w2 = heads.projection(900, 128, 20000, "bf16", 6, raised=t2)
    side = torch.cuda.Stream()
    small, large = outputs(h, w, MEAN), outputs(h2, w2, MEAN)
    torch.cuda.synchronize()
    ce.ce_linear_fwd_bwd(h, w, t, *small, stream=side)
    g = torch.cuda.CUDAGraph()
    out = outputs(h, w, MEAN)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ce.ce_linear_fwd_bwd(h, w, t, *out)
        ce.ce_linear_fwd_bwd(h2, w2, t2, *large, stream=side)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, small))
    assert all(torch.equal(a, b) for a, b in zip(large, check_linear(h2, w2, t2, "bf16")))


def test_gradients_against_differences():
    """Central differences of the loss along a direction.  The quotient is off
    by at most r^3 d^2 / 3 (the third derivative of a row's log-sum-exp along a
    direction is at most 2 r^3, r the spread of the logits' change), and by the
    losses' own error over d."""
    B, D, C = 6, 32, 90
    t = some_targets(B, C, 12)
    h, w = heads.projection(B, D, C, "bf16", 12, sigma=1.0, raised=t)
    h = (h * 8).round() / 8  # a step of 1/16 is exact
    step = 2.0 ** -4
    loss, dh, dw = outputs(h, w, SUM)
    ce.ce_linear_fwd_bwd(h, w, t, loss, dh, dw, reduction=SUM)
    z, dz = heads.logits_of(h, w)
    err = heads.cross_entropy(z, dz, t, "bf16", SUM).drows.sum().item() + 2.0 ** -20
    g = torch.Generator("cuda").manual_seed(3)
    for _ in range(4):
        v = (torch.randint(0, 2, h.shape, generator=g, device="cuda") * 2 - 1).to(h.dtype)
        ends = []
        for sign in (1, -1):
            at = h + sign * step * v
            assert torch.equal(at.double(), h.double() + sign * step * v.double())
            ce.ce_linear_fwd_bwd(at, w, t, loss, reduction=SUM)
            ends.append(loss.item())
        change = v.double() @ w.double().T
        r = (change.amax(1) - change.amin(1))
        slope = (dh.double() * v.double()).sum().item()
        bound = (r ** 3).sum().item() * step ** 2 / 3 + err / step
        bound += heads.unit("bf16") * 4 * dh.double().abs().sum().item()
        assert abs((ends[0] - ends[1]) / (2 * step) - slope) <= bound


def test_offsets_past_32_bits():
    """A projection of more than 2^31 elements."""
    B, D, C = 3, 2048, 1_060_000
    t = torch.tensor([C - 1, 5, C // 2], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    h = torch.randn(B, D, generator=g, device="cuda").bfloat16()
    w = torch.empty(C, D, dtype=torch.bfloat16, device="cuda")
    for i in range(0, C, 100_000):
        w[i:i + 100_000] = torch.randn(min(100_000, C - i), D, generator=g, device="cuda") * 0.04
    loss, dh, dw = outputs(h, w, NONE)
    ce.ce_linear_fwd_bwd(h, w, t, loss, dh, dw, reduction=NONE)
    z, dz = heads.logits_of(h, w)
    ref = heads.cross_entropy(z, dz, t, "bf16", NONE)
    heads.within(loss, *ref.loss(NONE), "loss")
    for i in range(0, C, 100_000):
        s = slice(i, min(C, i + 100_000))
        want = ref.G[:, s].T @ h.double()
        bound = ref.dG[:, s].T @ h.double().abs() * 1.01 + 2.0 ** -7 * want.abs() + 1e-30
        heads.within(dw[s], want, bound, "dweight")


# ------------------------------------------------------------- the teacher's


def check_linear_distill(h, w, idx, val, dtype, lse=None, T=1.0, reduction=MEAN, scale=None,
                         grads="both", hidden=None):
    loss, dh, dw = outputs(h, w, reduction, grads)
    ce.ce_linear_distill_fwd_bwd(h if hidden is None else hidden, w, idx, val, loss, dh, dw,
                                 teacher_lse=lse, temperature=T, reduction=reduction,
                                 grad_scale=scale)
    z, dz = heads.logits_of(h, w)
    ref = heads.divergence(z, dz, idx, val.float(), lse, T, dtype, reduction, scale)
    heads.within(loss, *ref.loss(reduction), "loss")
    (want_h, bound_h), (want_w, bound_w) = heads.product_bounds(ref, h, w, dtype)
    if dh is not None:
        heads.within(dh, want_h, bound_h, "dhidden")
    if dw is not None:
        heads.within(dw, want_w, bound_w, "dweight")
    return loss, dh, dw


TEACHER_SHAPES = [(1, 8, 1, 1), (2, 64, 300, 7), (77, 256, 1000, 16), (300, 72, 5003, 64),
                  (20, 512, 32000, 300), (1000, 64, 257, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,D,C,K", TEACHER_SHAPES)
def test_linear_distill_shapes(B, D, C, K, dtype):
    idx, val = heads.teacher_lists(B, C, K, B + C, ragged=K > 2)
    h, w = heads.projection(B, D, C, dtype, B + D, raised=idx[:, 0])
    check_linear_distill(h, w, idx, val, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("reduction,T,own,grads,tdtype", [
    (SUM, 2.0, False, "both", "f32"), (NONE, 0.5, True, "both", "bf16"),
    (MEAN, 4.0, True, "weight", "f16"), (NONE, 1.0, False, "hidden", "f32"),
    (NONE, 1.0, True, "none", "f32"), (MEAN, 3.0, False, "none", "bf16")])
def test_linear_distill_options(reduction, T, own, grads, tdtype, dtype):
    B, D, C, K = 190, 136, 900, 33
    idx, val = heads.teacher_lists(B, C, K, 7, empty=0.2, ragged=True)
    val = val.to(heads.TORCH_DT[tdtype])
    lse = torch.logsumexp(val.float() / T, 1) + 0.3 if own else None
    h, w = heads.projection(B, D, C, dtype, 7, raised=idx[:, 0])
    n = B if reduction == NONE else 1
    scale = torch.rand(n, device="cuda") + 0.25
    check_linear_distill(h, w, idx, val, dtype, lse, T, reduction, scale, grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_distill_rows_without_a_list(dtype):
    """Their hidden states and the values of unused places do not matter."""
    B, D, C, K = 200, 64, 400, 9
    idx, val = heads.teacher_lists(B, C, K, 5, empty=0.4, ragged=True)
    h, w = heads.projection(B, D, C, dtype, 5)
    used = idx >= 0
    val[~used] = math.nan
    bad = h.clone()
    bad[~used.any(1)] = math.nan
    clean = torch.where(used, val, torch.zeros_like(val))
    a = check_linear_distill(h, w, idx, clean, dtype, reduction=NONE)
    b = outputs(h, w, NONE)
    ce.ce_linear_distill_fwd_bwd(bad, w, idx, val, *b, reduction=NONE)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert (b[0][~used.any(1)] == 0).all() and (b[1][~used.any(1)] == 0).all()
    idx.fill_(-1)
    ce.ce_linear_distill_fwd_bwd(bad, w, idx, val, *b, reduction=NONE)
    assert all(torch.equal(x, torch.zeros_like(x)) for x in b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_distill_repeated_and_bad_classes(dtype):
    B, D, C, K = 50, 64, 300, 40
    g = torch.Generator("cuda").manual_seed(2)
    idx = torch.randint(0, 25, (B, K), generator=g, device="cuda", dtype=torch.int32)
    val = torch.randn(B, K, generator=g, device="cuda")
    h, w = heads.projection(B, D, C, dtype, 2)
    check_linear_distill(h, w, idx, val, dtype, reduction=NONE)
    idx[4, 2], idx[9, 0], idx[9, 5] = C, -2, 2 ** 31 - 1
    idx[11] = -5
    ce.ce_get_device_errors()
    check_linear_distill(h, w, idx, val, dtype, reduction=NONE)
    assert ce.ce_get_device_errors() == (3, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("away", [-2.0, 60.0, 95.0])
def test_lists_of_another_mass(dtype, away):
    """A normaliser that is not the list's: masses of e^2, e^-60 and e^-95 (a
    number without all its bits)."""
    B, D, C, K = 60, 64, 300, 5
    idx, val = heads.teacher_lists(B, C, K, 4)
    h, w = heads.projection(B, D, C, dtype, 4)
    lse = torch.logsumexp(val, 1) + away
    if away < 90:
        check_linear_distill(h, w, idx, val, dtype, lse, reduction=SUM)
        return
    loss, dh, dw = outputs(h, w, NONE)
    ce.ce_linear_distill_fwd_bwd(h, w, idx, val, loss, dh, dw, teacher_lse=lse, reduction=NONE)
    for x in (loss, dh, dw):
        assert x.float().abs().max() < 1e-36


def test_linear_distill_far_from_its_teacher():
    """bf16: the listed logits are far below the row's largest."""
    B, D, C, K = 120, 64, 500, 3
    h, w = heads.projection(B, D, C, "bf16", 3, sigma=60.0)
    z = h.float() @ w.float().T
    idx = z.topk(K, 1, largest=False).indices.int()
    val = torch.randn(B, K, device="cuda")
    assert (z.amax(1) - torch.gather(z, 1, idx.long()).amax(1)).max() > 150
    check_linear_distill(h, w, idx, val, "bf16", reduction=NONE)
    check_linear_distill(h, w, idx, val, "bf16", T=0.25, reduction=SUM)


def test_a_training_step_with_both_losses():
    """Cross-entropy on one part of a batch and distillation on the other
    through one projection, a step of gradient descent, and the same losses
    again; distillation on kept fp32 logits gives what the fused call gives."""
    B, D, C, K = 256, 128, 3000, 16
    idx, val = heads.teacher_lists(B, C, K, 21)
    t = idx[:, 0].clone()
    t[: B // 2] = -100                 # the first half has a teacher
    idx[B // 2:] = -1                  # the second half has targets
    h, w = heads.projection(B, D, C, "bf16", 21, raised=None)
    losses = []
    for step in range(2):
        lc, dhc, dwc = check_linear(h, w, t, "bf16")
        ld, dhd, dwd = check_linear_distill(h, w, idx, val, "bf16", T=2.0)
        assert (dhc[: B // 2] == 0).all() and (dhd[B // 2:] == 0).all()
        z = h.float() @ w.float().T
        loss = torch.empty(1, device="cuda")
        grad = torch.empty_like(z)
        ce.ce_distill_fwd_bwd(z, idx, val, loss, grad, temperature=2.0)
        zd, dz = heads.logits_of(h, w)
        ref = heads.divergence(zd, dz + 1e-5, idx, val, None, 2.0, "f32", MEAN)
        heads.within(loss, *ref.loss(MEAN), "loss of kept logits")
        heads.within(ld, *ref.loss(MEAN), "loss without them")
        # the gradients of the two losses, one formula: autograd in float64
        h64 = h.double().requires_grad_()
        w64 = w.double().requires_grad_()
        logits = h64 @ w64.T
        ce_loss = torch.nn.functional.cross_entropy(logits, t.long(), ignore_index=-100)
        q = torch.softmax(val.double() / 2, 1)[: B // 2]
        lp = torch.log_softmax(logits[: B // 2] / 2, 1)
        kd = 4 * (q * (q.log() - torch.gather(lp, 1, idx[: B // 2].long()))).sum() / B
        (ce_loss + kd).backward()
        for got, want in ((dhc.double() + dhd.double(), h64.grad),
                          (dwc.double() + dwd.double(), w64.grad)):
            assert (got - want).norm() <= 4 * heads.unit("bf16") * want.norm()
        losses.append(ce_loss.item() + kd.item())
        h = (h.float() - 4.0 * (dhc.float() + dhd.float())).bfloat16()
        w = (w.float() - 4.0 * (dwc.float() + dwd.float())).bfloat16()
    assert all(math.isfinite(x) for x in losses)
