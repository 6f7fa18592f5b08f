"""The language-model head operators as a user calls them, and what they compute.

Three operators stand behind these cases:

  linear          softmax cross-entropy of a vocabulary projection,
                  z = hidden weight^T, without keeping the logits, with the
                  gradients of the hidden states and of the projection
  distill         KL divergence from a teacher's top logits to the softmax of a
                  logits matrix, with the gradient of the logits
  linear_distill  the same divergence for logits that are themselves a
                  projection, without keeping them, with both gradients

``own`` selects the library's calls; otherwise ``run`` computes the plain form
in 32 bits with elementary torch operations.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MOST_FLOPS = 6 * 4096 * 4096 * 128256
MOST_LOGITS = 4096 * 128256
IGNORE = -100


def _linear(name, B, D, C, dtype, grads, reduction="mean", ignored=0.0, scaled=False):
    return {"name": name, "op": "linear", "B": B, "D": D, "C": C, "dtype": dtype, "grads": grads,
            "reduction": reduction, "ignored": ignored, "scaled": scaled}


def _distill(name, B, C, K, dtype, teacher, grads, temperature=1.0, lse=False, reduction="mean",
             empty=0.0, scaled=False):
    return {"name": name, "op": "distill", "B": B, "C": C, "K": K, "dtype": dtype,
            "teacher": teacher, "grads": grads, "temperature": temperature, "lse": lse,
            "reduction": reduction, "empty": empty, "scaled": scaled}


def _linear_distill(name, B, D, C, K, dtype, teacher, grads, temperature=1.0, lse=False,
                    reduction="mean", empty=0.0, scaled=False):
    c = _distill(name, B, C, K, dtype, teacher, grads, temperature, lse, reduction, empty, scaled)
    return dict(c, op="linear_distill", D=D)


def listed():
    return [
        # the log-probability of one generated token (a server's smallest call)
        _linear("linear_score_1", 1, 2048, 32000, "bf16", "none", "none"),
        # a decoding batch scored against a large vocabulary
        _linear("linear_score_64", 64, 4096, 128256, "bf16", "none", "none"),
        # a ragged fine-tuning batch, a third of its tokens prompt or padding
        _linear("linear_ragged_333", 333, 1000, 50257, "f16", "both", "mean", 0.3),
        # an ordinary training step
        _linear("linear_train_8192", 8192, 2048, 32000, "bf16", "both", "mean", 0.1),
        # a large training step
        _linear("linear_train_large", 4096, 4096, 128256, "bf16", "both"),
        # a frozen projection: the gradient of the hidden states alone, with an
        # upstream gradient for every token
        _linear("linear_frozen_1500", 1500, 2048, 50257, "bf16", "hidden", "none", 0.0, True),
        # a handful of rows of a classifier
        _distill("distill_16x1000", 16, 1000, 8, "f32", "f32", True),
        # stored teacher logits for a 32k vocabulary, softened
        _distill("distill_8192x32000", 8192, 32000, 64, "bf16", "bf16", True, 2.0),
        # a large vocabulary, the teacher's own normaliser, tokens without a list
        _distill("distill_4096x128256", 4096, 128256, 100, "bf16", "f16", True, 1.0, True, "mean",
                 0.1),
        # odd rows, an upstream gradient for every token
        _distill("distill_4099x50257", 4099, 50257, 20, "f32", "f32", True, 1.0, False, "none",
                 0.0, True),
        # distillation through a projection: a small and a large training step
        _linear_distill("linear_distill_77", 77, 1024, 32000, 16, "f16", "f32", "both"),
        _linear_distill("linear_distill_2048", 2048, 2048, 128256, 64, "bf16", "bf16", "both", 2.0,
                        False, "sum", 0.1, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "distill", "linear_distill"])
    reduction = rng.choice(["mean", "sum", "none"])
    scaled = rng.random() < 0.4
    C = _log_int(rng, 500, 131072)
    if op == "distill":
        dtype = rng.choice(["f32", "bf16", "f16"])
        most = MOST_LOGITS // (2 if dtype == "f32" else 1)
        B = min(_log_int(rng, 1, 16384), most // C)
        return dict(_distill("", B, C, _log_int(rng, 1, 256), dtype,
                             rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.8,
                             rng.choice([0.5, 1.0, 1.0, 2.0, 4.0]), rng.random() < 0.4, reduction,
                             rng.choice([0.0, 0.1]), scaled), name="")
    D = 8 * _log_int(rng, 8, 512)
    B = max(1, min(_log_int(rng, 1, 16384), MOST_FLOPS // (6 * D * C), MOST_LOGITS // C))
    dtype, grads = rng.choice(["bf16", "f16"]), rng.choice(["both", "both", "hidden", "none"])
    if op == "linear":
        return _linear("", B, D, C, dtype, grads, reduction, rng.choice([0.0, 0.3]), scaled)
    return _linear_distill("", B, D, C, _log_int(rng, 1, 128), dtype,
                           rng.choice(["f32", "bf16", "f16"]), grads,
                           rng.choice([0.5, 1.0, 1.0, 2.0, 4.0]), rng.random() < 0.4, reduction,
                           rng.choice([0.0, 0.1]), scaled)


def work(case):
    B, C, es = case["B"], case["C"], BYTES[case["dtype"]]
    rows = B if case["reduction"] == "none" else 1
    small = 4 * rows + (4 * rows if case["scaled"] else 0)
    if case["op"] != "linear":
        small += B * case["K"] * (4 + BYTES[case["teacher"]]) + (4 * B if case["lse"] else 0)
    else:
        small += 4 * B
    if case["op"] == "distill":
        n = B * C
        return {"bytes": n * es * (2 if case["grads"] else 1) + small,
                "flops": n * (8 if case["grads"] else 5)}
    D = case["D"]
    outs = {"none": 0, "hidden": B * D, "both": B * D + C * D}[case["grads"]]
    products = {"none": 1, "hidden": 2, "both": 3}[case["grads"]]
    return {"bytes": (B * D + C * D + outs) * es + small, "flops": 2 * products * B * D * C}


def _teacher(case, g):
    """A teacher's list for every row: K distinct classes, logits that fall
    off along the list, and (where a case has tokens without a list) -1 in
    every place of a row."""
    B, C, K, dev = case["B"], case["C"], case["K"], "cuda"
    K = min(K, C)
    first = torch.randint(0, C, (B, 1), generator=g, device=dev)
    step = torch.randint(1, max(2, C // K), (B, 1), generator=g, device=dev)
    idx = (first + step * torch.arange(K, device=dev)) % C
    place = torch.arange(K, device=dev, dtype=torch.float32)
    val = 9.0 - 1.5 * torch.log1p(place) + torch.randn(B, K, generator=g, device=dev)
    return idx, val


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, C, dt, dev = case["B"], case["C"], DTYPES[case["dtype"]], "cuda"
    s = {"case": case}
    rows = B if case["reduction"] == "none" else 1
    s["scale"] = (torch.rand(rows, generator=g, device=dev) + 0.5) if case["scaled"] else None
    s["loss"] = torch.empty(rows, dtype=torch.float32, device=dev)
    if case["op"] != "linear":
        idx, val = _teacher(case, g)
        boost = 0.7 * val
        s["val"] = val.to(DTYPES[case["teacher"]])
        s["lse"] = None
        if case["lse"]:
            t = s["val"].float() / case["temperature"]
            s["lse"] = torch.logsumexp(t, 1) + 0.2 * torch.rand(B, generator=g, device=dev)
        keep = torch.rand(B, 1, generator=g, device=dev) >= case["empty"]
        s["idx"] = torch.where(keep, idx, torch.full_like(idx, -1)).to(torch.int32)
    if case["op"] == "distill":
        z = torch.randn(B, C, generator=g, device=dev).mul_(2.0)
        s["logits"] = z.scatter_add_(1, idx, boost).to(dt)
        s["grad"] = torch.empty_like(s["logits"]) if case["grads"] else None
        return s
    D = case["D"]
    # logits of standard deviation 2, raised by 8 at the target (or by the
    # teacher's logits at its classes), as a trained model's are
    w = torch.randn(C, D, generator=g, device=dev).mul_(2.0 / math.sqrt(D))
    h = torch.randn(B, D, generator=g, device=dev)
    if case["op"] == "linear":
        t = torch.randint(0, C, (B,), generator=g, device=dev)
        h += 2.0 * w[t]
        lost = torch.rand(B, generator=g, device=dev) < case["ignored"]
        s["targets"] = torch.where(lost, torch.full_like(t, IGNORE), t).to(torch.int32)
    else:
        for k in range(idx.shape[1]):
            h += 0.25 * boost[:, k:k + 1] * w[idx[:, k]]
        h *= (math.sqrt(D) / h.norm(dim=1, keepdim=True)).clamp(max=1.0)
    s["hidden"], s["weight"] = h.to(dt), w.to(dt)
    s["dhidden"] = torch.empty_like(s["hidden"]) if case["grads"] != "none" else None
    s["dweight"] = torch.empty_like(s["weight"]) if case["grads"] == "both" else None
    return s


def _own(s):
    import softmax_cross_entropy_row_gb300 as ce

    case = s["case"]
    how = {"mean": ce.CE_REDUCE_MEAN, "sum": ce.CE_REDUCE_SUM,
           "none": ce.CE_REDUCE_NONE}[case["reduction"]]
    if case["op"] == "linear":
        ce.ce_linear_fwd_bwd(s["hidden"], s["weight"], s["targets"], s["loss"], s["dhidden"],
                             s["dweight"], reduction=how, grad_scale=s["scale"],
                             ignore_index=IGNORE)
        return {"loss": s["loss"], "dhidden": s["dhidden"], "dweight": s["dweight"]}
    if case["op"] == "distill":
        ce.ce_distill_fwd_bwd(s["logits"], s["idx"], s["val"], s["loss"], s["grad"],
                              teacher_lse=s["lse"], temperature=case["temperature"],
                              reduction=how, grad_scale=s["scale"])
        return {"loss": s["loss"], "grad": s["grad"]}
    ce.ce_linear_distill_fwd_bwd(s["hidden"], s["weight"], s["idx"], s["val"], s["loss"],
                                 s["dhidden"], s["dweight"], teacher_lse=s["lse"],
                                 temperature=case["temperature"], reduction=how,
                                 grad_scale=s["scale"])
    return {"loss": s["loss"], "dhidden": s["dhidden"], "dweight": s["dweight"]}


def _reduced(rows, how, count):
    return rows if how == "none" else rows.sum().reshape(1) / (count if how == "mean" else 1)


def _row_factor(s, count):
    """What row b's gradient is multiplied by: 1/count (mean) or 1, times the
    upstream gradient."""
    f = 1.0 / count if s["case"]["reduction"] == "mean" else 1.0
    return f if s["scale"] is None else f * s["scale"][:, None]


def _softmax(z):
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    return e.div_(total), (m + torch.log(total))[:, 0]


def _targets_plain(s, z, want):
    """Rows' loss and (want) the gradient of z for cross-entropy."""
    t = s["targets"].long()
    keep = t != IGNORE
    t = torch.where(keep, t, torch.zeros_like(t))[:, None]
    zt = torch.gather(z, 1, t)[:, 0]
    p, lse = _softmax(z)
    count = keep.sum().clamp(min=1)
    rows = torch.where(keep, lse - zt, torch.zeros_like(lse))
    if not want:
        return rows, count, None
    p.scatter_add_(1, t, torch.full_like(p[:, :1], -1.0))
    return rows, count, p.mul_(_row_factor(s, count) * keep[:, None])


def _teacher_plain(s, z, want):
    """Rows' loss and (want) the gradient of z for the divergence."""
    T = s["case"]["temperature"]
    here = s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    t = s["val"].float() / T
    t = torch.where(here, t, torch.full_like(t, -math.inf))
    some = here.any(1)
    if s["lse"] is None:
        m = torch.where(some, t.amax(1), torch.zeros_like(t[:, 0]))
        lse_t = m + torch.log(torch.exp(t - m[:, None]).sum(1))
    else:
        lse_t = s["lse"]
    logq = torch.where(here, t - lse_t[:, None], torch.zeros_like(t))
    q = torch.where(here, torch.exp(logq), torch.zeros_like(t))
    z = z / T
    zk = torch.gather(z, 1, at)
    p, lse = _softmax(z)
    rows = T * T * (q * (logq - (zk - lse[:, None]))).sum(1)
    if not want:
        return rows, z.shape[0], None
    p.mul_(q.sum(1, keepdim=True)).scatter_add_(1, at, -q)
    return rows, z.shape[0], p.mul_(T * _row_factor(s, z.shape[0]))


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    how = case["reduction"]
    if case["op"] == "distill":
        rows, count, g = _teacher_plain(s, s["logits"].float(), case["grads"])
        return {"loss": _reduced(rows, how, count),
                "grad": g.to(s["logits"].dtype) if case["grads"] else None}
    h, w = s["hidden"].float(), s["weight"].float()
    z = h @ w.t()
    form = _targets_plain if case["op"] == "linear" else _teacher_plain
    rows, count, g = form(s, z, case["grads"] != "none")
    return {"loss": _reduced(rows, how, count),
            "dhidden": (g @ w).to(s["hidden"].dtype) if case["grads"] != "none" else None,
            "dweight": (g.t() @ h).to(s["weight"].dtype) if case["grads"] == "both" else None}


def exact(case, seed):
    """The definition in 64 bits: p = softmax(z / T) row by row, the loss
    -sum_c y_c log p_c (+ sum y log y for a teacher), its gradient
    T (sum(y) p - y), y the target distribution as a dense matrix."""
    flops = work(case)["flops"] if case["op"] != "distill" else 0
    products = {"none": 1, "hidden": 2, "both": 3}.get(case["grads"], 1)
    if flops / products > 6e12:
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    linear = case["op"] != "distill"
    h, w = (s["hidden"].to(f64), s["weight"].to(f64)) if linear else (None, None)
    z = torch.mm(h, w.T) if linear else s["logits"].to(f64)
    B, C = z.shape
    T = case.get("temperature", 1.0)
    logp = torch.log_softmax(z / T, dim=1)
    del z
    y = torch.zeros_like(logp)
    r = torch.arange(B, device="cuda")
    if case["op"] == "linear":
        valid = s["targets"] != IGNORE
        y[r[valid], s["targets"][valid].long()] = 1.0
        entropy = torch.zeros(B, dtype=f64, device="cuda")
        n = max(1, int(valid.sum()))
    else:
        slots = s["idx"] >= 0
        t = (s["val"].to(f64) / T).masked_fill(~slots, -math.inf)
        ref = torch.logsumexp(t, 1) if s["lse"] is None else s["lse"].to(f64)
        logq = (t - ref[:, None]).masked_fill(~slots, 0.0)
        q = logq.exp().masked_fill(~slots, 0.0)
        y.scatter_add_(1, s["idx"].long().clamp(min=0), q)
        entropy = (q * logq).sum(1)
        n = B
    rows = T * T * (entropy - (y * logp).sum(1))
    loss = {"mean": rows.sum().reshape(1) / n, "sum": rows.sum().reshape(1),
            "none": rows}[case["reduction"]]
    out = {"loss": loss}
    keys = ("dhidden", "dweight") if linear else ("grad",)
    wanted = {"none": 0, "hidden": 1, "both": 2, True: 1, False: 0}[case["grads"]]
    if flops > 8e12 or not wanted:
        return dict(out, **{k: None for k in keys})
    up = torch.ones(1, dtype=f64, device="cuda") if s["scale"] is None else s["scale"].to(f64)
    up = up.reshape(-1, 1) * (T / n if case["reduction"] == "mean" else T)
    mass = y.sum(1, keepdim=True)
    g = (logp.exp_() * mass - y) * up
    if not linear:
        return dict(out, grad=g)
    return dict(out, dhidden=torch.mm(g, w),
                dweight=torch.mm(g.T, h) if wanted == 2 else None)
