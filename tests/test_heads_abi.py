"""Host-side checks of the projection's and the teacher's entry points: they
answer before any CUDA call, so they are tested without a GPU."""

import ctypes
import math

import pytest

import softmax_cross_entropy_row_gb300 as ce

NULL, SHAPE, DTYPE, ALIGN, OVERLAP, REDUCTION, TEMPERATURE = 1, 2, 3, 4, 6, 11, 12
M = 1 << 20  # addresses far apart


@pytest.fixture(scope="module")
def lib():
    ce.build()
    return ce.load_library()


def linear(lib, hidden=M, weight=2 * M, targets=3 * M, B=4, D=16, C=5, dtype=ce.CE_BF16,
           ignore=-100, reduction=0, scale=None, loss=4 * M, dh=5 * M, dw=6 * M):
    return lib.ce_linear_fwd_bwd(hidden, weight, targets, B, D, C, dtype, ignore, reduction, scale,
                                 loss, dh, dw, None)


def linear_distill(lib, hidden=M, weight=2 * M, idx=3 * M, val=7 * M, lse=None, B=4, D=16, C=5,
                   K=2, dtype=ce.CE_BF16, tdtype=ce.CE_F32, T=1.0, reduction=0, scale=None,
                   loss=4 * M, dh=5 * M, dw=6 * M):
    return lib.ce_linear_distill_fwd_bwd(hidden, weight, idx, val, lse, B, D, C, K, dtype, tdtype,
                                         ctypes.c_float(T), reduction, scale, loss, dh, dw, None)


def distill(lib, logits=M, idx=3 * M, val=7 * M, lse=None, B=4, C=5, K=2, dtype=ce.CE_F32,
            tdtype=ce.CE_F32, T=1.0, reduction=0, scale=None, loss=4 * M, grad=5 * M):
    return lib.ce_distill_fwd_bwd(logits, idx, val, lse, B, C, K, dtype, tdtype, ctypes.c_float(T),
                                  reduction, scale, loss, grad, None)


@pytest.mark.parametrize("call", [linear, linear_distill])
def test_projection_refusals(lib, call):
    for kw, status in [
            (dict(hidden=None), NULL), (dict(weight=None), NULL), (dict(loss=None), NULL),
            (dict(B=0), SHAPE), (dict(C=0), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE),
            (dict(D=-8), SHAPE), (dict(B=1 << 31), SHAPE), (dict(C=1 << 31), SHAPE),
            (dict(D=1 << 25), SHAPE), (dict(C=1 << 30, D=1 << 20), SHAPE),
            (dict(dtype=ce.CE_F32), DTYPE), (dict(dtype=9), DTYPE), (dict(reduction=3), REDUCTION),
            (dict(reduction=-1), REDUCTION),
            (dict(hidden=M + 8), ALIGN), (dict(weight=2 * M + 2), ALIGN),
            (dict(dh=5 * M + 8), ALIGN), (dict(dw=6 * M + 4), ALIGN), (dict(loss=4 * M + 2), ALIGN),
            (dict(scale=8 * M + 2), ALIGN),
            (dict(dh=M), OVERLAP), (dict(dh=2 * M + 16), OVERLAP), (dict(dw=M + 112), OVERLAP),
            (dict(dw=5 * M + 16), OVERLAP), (dict(loss=M + 4), OVERLAP),
            (dict(loss=5 * M + 4), OVERLAP), (dict(scale=4 * M), OVERLAP),
            (dict(loss=4 * M, scale=4 * M + 12, reduction=2), OVERLAP)]:
        assert call(lib, **kw) == status, kw


def test_targets_are_needed(lib):
    assert linear(lib, targets=None) == NULL
    assert linear(lib, targets=3 * M + 2) == ALIGN
    assert linear(lib, loss=3 * M + 4) == OVERLAP


@pytest.mark.parametrize("call", [distill, linear_distill])
def test_teacher_refusals(lib, call):
    for kw, status in [
            (dict(idx=None), NULL), (dict(val=None), NULL), (dict(K=0), SHAPE),
            (dict(K=1025), SHAPE), (dict(K=-1), SHAPE), (dict(tdtype=3), DTYPE),
            (dict(T=0.0), TEMPERATURE), (dict(T=-1.0), TEMPERATURE),
            (dict(T=math.inf), TEMPERATURE), (dict(T=math.nan), TEMPERATURE),
            (dict(T=2.0 ** -149), TEMPERATURE),
            (dict(idx=3 * M + 2), ALIGN), (dict(val=7 * M + 2), ALIGN),
            (dict(lse=8 * M + 2), ALIGN), (dict(val=7 * M + 1, tdtype=ce.CE_F16), ALIGN),
            (dict(loss=3 * M + 4), OVERLAP), (dict(loss=7 * M + 4), OVERLAP),
            (dict(lse=4 * M), OVERLAP)]:
        assert call(lib, **kw) == status, kw


def test_distill_refusals(lib):
    for kw, status in [
            (dict(logits=None), NULL), (dict(loss=None), NULL), (dict(B=0), SHAPE),
            (dict(C=0), SHAPE), (dict(B=1 << 31), SHAPE), (dict(C=1 << 31), SHAPE),
            (dict(dtype=4), DTYPE), (dict(reduction=5), REDUCTION), (dict(logits=M + 2), ALIGN),
            (dict(logits=M + 1, dtype=ce.CE_BF16), ALIGN), (dict(grad=5 * M + 2), ALIGN),
            (dict(grad=M), OVERLAP), (dict(grad=M + 32), OVERLAP), (dict(grad=3 * M), OVERLAP),
            (dict(grad=4 * M), OVERLAP)]:
        assert distill(lib, **kw) == status, kw


def test_binding_checks_what_the_c_layer_cannot(lib):
    torch = pytest.importorskip("torch")
    h = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(5, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    loss = torch.zeros(1)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    val = torch.zeros(4, 2)
    z = torch.zeros(4, 5)
    with pytest.raises(ValueError, match="CUDA"):
        ce.ce_linear_fwd_bwd(h, w, t, loss)
    with pytest.raises(ValueError, match="CUDA"):
        ce.ce_distill_fwd_bwd(z, idx, val, loss)
    with pytest.raises(ValueError, match="CUDA"):
        ce.ce_linear_distill_fwd_bwd(h, w, idx, val, loss)
    with pytest.raises(ValueError, match="weight"):
        ce.ce_linear_fwd_bwd(h, w.half(), t, loss)
    with pytest.raises(ValueError, match="weight"):
        ce.ce_linear_fwd_bwd(h, w[:, :8], t, loss)
    with pytest.raises(ValueError, match="hidden"):
        ce.ce_linear_fwd_bwd(h.t(), w, t, loss)
    with pytest.raises(ValueError, match="targets"):
        ce.ce_linear_fwd_bwd(h, w, t.long(), loss)
    with pytest.raises(ValueError, match="targets"):
        ce.ce_linear_fwd_bwd(h, w, t[:3], loss)
    with pytest.raises(ValueError, match="dhidden_out"):
        ce.ce_linear_fwd_bwd(h, w, t, loss, h[:2])
    with pytest.raises(ValueError, match="dweight_out"):
        ce.ce_linear_fwd_bwd(h, w, t, loss, None, w.float())
    with pytest.raises(ValueError, match="teacher_idx"):
        ce.ce_distill_fwd_bwd(z, idx.long(), val, loss)
    with pytest.raises(ValueError, match="teacher_idx"):
        ce.ce_distill_fwd_bwd(z, idx[:3], val[:3], loss)
    with pytest.raises(ValueError, match="teacher_val"):
        ce.ce_distill_fwd_bwd(z, idx, val[:, :1], loss)
    with pytest.raises(TypeError, match="teacher_val"):
        ce.ce_distill_fwd_bwd(z, idx, val.double(), loss)
    with pytest.raises(ValueError, match="teacher_lse"):
        ce.ce_distill_fwd_bwd(z, idx, val, loss, teacher_lse=torch.zeros(3))
    with pytest.raises(ValueError, match="grad_out"):
        ce.ce_distill_fwd_bwd(z, idx, val, loss, torch.zeros(4, 4))
