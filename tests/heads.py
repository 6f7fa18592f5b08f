"""Cases, fp64 references and error bounds of the vocabulary projection's and
the teacher's operators, shared by their GPU tests.

The references follow the definitions in float64 from the inputs as they were
rounded to the operands' type.  With u = finfo(type).eps / 2 the bounds count
  logits      fp32 accumulation of D products in chunks of 16, each addition
              off by at most 2^-23 of the partial sums' magnitude:
              dz = (D / 16 + 16) 2^-23 max_c sum_d |h_d w_cd|  (0 where the
              logits are given);
  statistics  a row's sum of exponentials, relative: at most 128 additions in
              a chain within a tile, a join per tile, the exponentials' own
              few ulp (2^-22) and the argument's rounding (|z| 2^-23):
              ds = (200 + C / 256) 2^-24 + 2^-21 + 2^-22 max|z|;
  kept p      two roundings to the operands' type, 2 u + u^2;
  products    (terms / 16 + 16) 2^-23 of sum |a b|, then one rounding u;
  flushing    an exponential below 2^-126 counts as 0; the row's sum is at
              least 2^-1/2 (its reference exponent is one of its classes',
              rounded), so a p off by less than 2^-125.
"""

import math

import torch

TORCH_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def unit(dtype):
    return torch.finfo(TORCH_DT[dtype]).eps / 2


def projection(B, D, C, dtype, seed, sigma=2.0, raised=None):
    """Hidden states and weights whose logits have standard deviation about
    `sigma`, raised by about 6 at `raised` (classes per row)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(C, D, generator=g, device="cuda") * (sigma / math.sqrt(D))
    h = torch.randn(B, D, generator=g, device="cuda")
    if raised is not None:
        h += (6.0 / sigma ** 2) * w[raised.clamp(0, C - 1).long()]
    return h.to(TORCH_DT[dtype]), w.to(TORCH_DT[dtype])


def logits_of(hidden, weight):
    """fp64 logits and the bound of their fp32 accumulation, per row."""
    h, w = hidden.double(), weight.double()
    D = h.shape[1]
    z = h @ w.T
    dz = (D / 16 + 16) * 2.0 ** -23 * (h.abs() @ w.abs().T).amax(1)
    return z, dz


def stat_bound(z, scale=1.0):
    """ds of each row for logits times `scale`."""
    C = z.shape[1]
    big = torch.where(torch.isfinite(z), z, torch.zeros_like(z)).abs().amax(1) * scale
    return (200 + C / 256) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * big


class Reference:
    """loss rows, their bound, G = d loss / d z times the rows' factors, |G|'s
    bound and what the pieces need."""

    def __init__(self, rows, drows, G, dG, counted):
        self.rows, self.drows, self.G, self.dG, self.counted = rows, drows, G, dG, counted

    def loss(self, reduction):
        if reduction == 2:
            return self.rows, self.drows + 2.0 ** -23 * self.rows.abs()
        s, d = self.rows.sum(), self.drows.sum()
        n = max(1, self.counted) if reduction == 0 else 1
        return (s / n).reshape(1), ((d + 2.0 ** -22 * self.rows.abs().sum()) / n).reshape(1)


def _factors(B, reduction, scale, counted):
    f = torch.ones(B, dtype=torch.float64, device="cuda")
    if scale is not None:
        f = f * scale.double()
    return f / max(1, counted) if reduction == 0 else f


def cross_entropy(z, dz, targets, dtype, reduction, scale=None, ignore_index=-100, kept=2):
    """Softmax cross-entropy; `kept` roundings of an unlisted gradient."""
    B, C = z.shape
    keep = targets != ignore_index
    valid = keep & (targets >= 0) & (targets < C)
    t = torch.where(valid, targets, torch.zeros_like(targets)).long()
    lse = torch.logsumexp(z, 1)
    r = torch.arange(B, device="cuda")
    err = 2 * dz + stat_bound(z) + 2.0 ** -22 * (lse.abs() + 1)
    rows = torch.where(keep, lse - z[r, t], torch.zeros_like(lse))
    rows = torch.where(keep & ~valid, torch.full_like(rows, math.nan), rows)
    counted = int(keep.sum())
    f = _factors(B, reduction, scale, counted)[:, None]
    p = torch.softmax(z, 1)
    y = torch.zeros_like(p)
    y[r[valid], t[valid]] = 1.0
    u = unit(dtype)
    G = torch.where(keep[:, None], p - y, torch.zeros_like(p))
    dG = kept * u * 1.01 * G.abs() + (2 * err[:, None]) * p + 2.0 ** -125
    if dtype == "f16":
        dG = dG + 2.0 ** -38 * f.abs().amax() / f.abs().clamp(min=1e-300)
    dG = torch.where(keep[:, None], dG, torch.zeros_like(dG))
    return Reference(rows, torch.where(keep, err, torch.zeros_like(err)), G * f, dG * f.abs(),
                     counted)


def teacher_lists(B, C, K, seed, empty=0.0, ragged=False):
    """Lists of K distinct classes with falling logits; `empty` rows without
    any, `ragged` lists with unused places anywhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    K_ = min(K, C)
    first = torch.randint(0, C, (B, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, C // K_), (B, 1), generator=g, device="cuda")
    idx = (first + step * torch.arange(K_, device="cuda")) % C
    if K > K_:
        idx = torch.cat([idx, torch.full((B, K - K_), -1, device="cuda")], 1)
    val = 8.0 - 1.5 * torch.log1p(torch.arange(K, device="cuda").float())
    val = val + torch.randn(B, K, generator=g, device="cuda")
    if ragged:
        idx[torch.rand(B, K, generator=g, device="cuda") < 0.3] = -1
    if empty:
        idx[torch.rand(B, generator=g, device="cuda") < empty] = -1
    return idx.int(), val


def divergence(z, dz, idx, val, lse, T, dtype, reduction, scale=None, kept=2):
    """The teacher's divergence; `kept` roundings of a gradient.  (A listed one
    is rounded once where it is kept; in bf16 its row's factor lies in the
    hidden states, rounded with them, for the weights' gradient.)"""
    B, C = z.shape
    used = (idx >= 0) & (idx < C)
    bad = ((idx < -1) | (idx >= C)).any(1)
    t = torch.where(used, val.double() / T, torch.full_like(val.double(), -math.inf))
    some = used.any(1)
    ref = lse.double() if lse is not None else torch.where(some, torch.logsumexp(t, 1),
                                                           torch.zeros(B, device="cuda").double())
    lq = t - ref[:, None]
    q = torch.where(used, torch.exp(lq), torch.zeros_like(lq))
    y = torch.zeros_like(z).scatter_add_(1, idx.clamp(0, C - 1).long(), q)
    zt = z / T
    lp = zt - torch.logsumexp(zt, 1, keepdim=True)
    at = torch.gather(lp, 1, idx.clamp(0, C - 1).long())
    terms = torch.where(q > 0, q * (lq - at), torch.zeros_like(q))
    rows = T * T * terms.sum(1)
    rows = torch.where(bad, torch.full_like(rows, math.nan), rows)
    err = 2 * dz / T + stat_bound(z, 1 / T) + 2.0 ** -22 * (torch.logsumexp(zt, 1).abs() + 1)
    # the teacher's own exponentials: K additions, logs of |t| and its normaliser
    tabs = torch.where(used, t.abs(), torch.zeros_like(t)).amax(1) + ref.abs()
    eq = (idx.shape[1] / 32 + 16) * 2.0 ** -23 + 2.0 ** -22 * (tabs + 1)
    big = torch.where(q > 0, lq.abs() + at.abs(), torch.zeros_like(q)).amax(1)
    mass = q.sum(1)
    drows = T * T * (mass * (err + eq * (1 + big) + (idx.shape[1] / 32 + 8) * 2.0 ** -23 * big))
    p = torch.exp(lp)
    f = _factors(B, reduction, scale, B)[:, None] * T
    G = mass[:, None] * p - y
    listed = torch.zeros_like(z, dtype=torch.bool)
    r = torch.arange(B, device="cuda")[:, None].expand_as(idx)
    listed[r[used], idx[used].long()] = True
    u = unit(dtype)
    kept_p = kept * u * 1.01 * torch.where(listed, G.abs(), mass[:, None] * p)
    dG = kept_p + mass[:, None] * (p * (2 * err + eq)[:, None] + 2.0 ** -125)
    dG = dG + 2 * eq[:, None] * y
    if dtype == "f16":
        w = f.abs() * mass[:, None].clamp(min=1.0)
        dG = dG + 2.0 ** -38 * w.amax() / f.abs().clamp(min=1e-300)
    return Reference(rows, torch.where(bad, torch.zeros_like(drows), drows), G * f, dG * f.abs(), B)


def product_bounds(ref, hidden, weight, dtype):
    """dhidden, dweight and their bounds from G."""
    h, w = hidden.double(), weight.double()
    u, tiny = unit(dtype), SMALLEST[dtype]
    B, C = ref.G.shape
    dh, dw = ref.G @ w, ref.G.T @ h
    eh = ref.dG @ w.abs() + (C / 16 + 64) * 2.0 ** -23 * (ref.G.abs() @ w.abs())
    ew = ref.dG.T @ h.abs() + (B / 16 + 64) * 2.0 ** -23 * (ref.G.abs().T @ h.abs())
    return (dh, eh * 1.01 + u * dh.abs() + tiny), (dw, ew * 1.01 + u * dw.abs() + tiny)


def within(got, want, bound, what):
    got = got.double().reshape(want.shape)
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got)), f"{what}: NaN in other places"
    excess = torch.where(nan, torch.zeros_like(want), (got - want).abs() - bound)
    if (excess > 0).any():
        i = int(excess.reshape(-1).argmax())
        raise AssertionError(
            f"{what}: {int((excess > 0).sum())} of {excess.numel()} beyond the bound, worst at {i}:"
            f" {got.reshape(-1)[i].item()!r} for {want.reshape(-1)[i].item()!r}, "
            f"bound {bound.expand_as(want).reshape(-1)[i].item():.3g}")
