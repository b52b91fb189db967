"""Inputs, the 64-bit reference and the error bounds of the loss operators' tests.

The reference is the losses' definition in float64 with torch's elementary
operations, on whatever device the inputs are on.

Bounds. Let u = eps/2 of the tensors' type, e = 2^-24. A logit is a sum of D
products in fp32 (three times as many for fp32 inputs, whose two fp16 parts each
lose at most e of a value and drop at most e of a product, 3 e together, or 2^-40
of the tensor's largest value where that is more): its error is at most
dz = (N D + 16) e sum|h||W|, N = 3 or 1, and 2^-40 (max|h| sum|W| + max|W| sum|h|)
for fp32. The log-sum-exp moves by at most the largest dz of the row plus the
roundings of its own sums, (V/64 + 64 + 40) e relative in the sum and a few e of
its value. One term of the logits' gradient is then off by |a| p (dz + dlse + 40 e)
before it is rounded once (u; in fp16 and in fp32's fp16 parts at least 2^-38 of
the largest upstream gradient, where the scaled form turns subnormal), and the
products over it add (N K + 16) e sum|g||x|, in fp32 also 2^-40 of the largest
|x| times sum|g|, before the result is rounded once more (u, and in fp16 2^-25
absolute).
"""
import math

import torch

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
E = 2.0 ** -24


def make(T, V, D, dtype, seed, device="cuda", ignored=0.2, k=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    c = {"hidden": torch.randn(T, D, generator=g).to(dt).to(device),
         "weight": (torch.randn(V, D, generator=g) * spread / math.sqrt(D)).to(dt).to(device),
         "up": ((torch.rand(T, generator=g) - 0.2) / max(1, T)).to(device)}
    dead = torch.rand(T, generator=g) < ignored
    if k == 0:
        y = torch.randint(0, V, (T,), generator=g)
        y[dead] = -100
        c["target"] = y.to(device)
    else:
        idx = torch.randint(0, V, (T, k), generator=g)  # with repeats when V is small
        idx[torch.rand(T, k, generator=g) < 0.15] = -1
        idx[dead] = -1
        c["index"] = idx.to(device)
        c["logit"] = (torch.randn(T, k, generator=g) * 3).to(device)
    return c


def reference(c, smoothing=0.0, z_loss=0.0, temperature=1.0, ignore_index=-100):
    """(loss, lse, dhidden, dweight, bounds) in float64; rows out of range get NaN losses."""
    dt = c["hidden"].dtype
    T, D = c["hidden"].shape
    V = c["weight"].shape[0]
    N = 3 if dt == torch.float32 else 1
    u = torch.finfo(dt).eps / 2
    tau = temperature
    if "target" in c:
        y = c["target"].long()
        bad = (y != ignore_index) & ((y < 0) | (y >= V))
        live = (y != ignore_index) & ~bad
    else:
        idx, tl = c["index"].long(), c["logit"].double()
        bad = (idx >= V).any(1)
        has = (idx >= 0) & (tl != -math.inf)
        live = has.any(1) & ~bad
    h = torch.where(live[:, None], c["hidden"].double(), 0.0)  # dead rows may hold anything
    w = c["weight"].double()
    up = torch.where(live, c["up"].double().expand(T), 0.0)
    z = h @ w.T / tau
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    want = torch.zeros_like(z)
    rows = torch.nonzero(live)[:, 0]
    if "target" in c:
        want[rows] += smoothing / V
        want[rows, y[rows]] += 1.0 - smoothing
        loss = lse - (want * z).sum(1) + z_loss * lse ** 2
        a = up * (1.0 + 2.0 * z_loss * lse)
        g = a[:, None] * p - up[:, None] * want
        loss_scale = 1.0
    else:
        t = torch.where(has & live[:, None], tl / tau, -math.inf)
        pk = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)
        logp = torch.where(pk > 0, torch.log(pk.clamp(min=1e-300)), 0.0)
        at = torch.where(idx >= 0, idx, 0).clamp(max=V - 1)
        want.scatter_add_(1, at, pk)
        loss = tau ** 2 * ((pk * logp).sum(1) - (want * z).sum(1) + lse)
        a = up * tau
        g = a[:, None] * (p - want)
        loss_scale = tau ** 2
    loss = torch.where(live, loss, 0.0)
    loss = torch.where(bad, math.nan, loss)
    lse = torch.where(live, lse, 0.0)
    # bounds
    f32 = dt == torch.float32
    dz = ((N * D + 16) * E) * (h.abs() @ w.abs().T) / tau
    if f32 and T:
        hmax, wmax = float(h.abs().max()), float(w.abs().max())
        dz = dz + 2.0 ** -40 / tau * (hmax * w.abs().sum(1)[None, :]
                                      + wmax * h.abs().sum(1)[:, None])
    top = dz.amax(1)
    zmax = z.abs().amax(1)
    dlse = top + (V / 64 + 104) * E + 4 * E * (lse.abs() + zmax)
    K = c["logit"].shape[1] if "logit" in c else 1
    dloss = loss_scale * (dlse + top + (16 + K) * E * (1 + zmax + lse.abs())
                          + 4 * E * (V if smoothing else 0) * smoothing) * (1 + 2 * z_loss * lse.abs()) \
        + z_loss * 4 * E * lse ** 2
    if smoothing:
        dloss = dloss + smoothing * (V / 64 + 80) * E * z.abs().mean(1)
    dp = a.abs()[:, None] * p * (dz + dlse[:, None] + 40 * E) \
        + 8 * E * (a.abs()[:, None] * (p + want) + up.abs()[:, None] * want)
    floor = up.abs().max() * tau * 2.0 ** -38 if dt != torch.bfloat16 and T else 0.0
    dg = dp + u * g.abs() * (3.0 if f32 else 1.0) + floor
    dg = torch.where(live[:, None], dg, 0.0)
    ga = g.abs()
    dh, dw = g @ w, g.T @ h
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    bh = dg @ w.abs() + (N * V + 16) * E * (ga @ w.abs())
    bw = dg.T @ h.abs() + (N * T + 16) * E * (ga.T @ h.abs())
    if f32 and T:
        bh = bh + 2.0 ** -40 * wmax * ga.sum(1)[:, None]
        bw = bw + 2.0 ** -40 * hmax * ga.sum(0)[:, None]
    bh = bh + u * (dh.abs() + bh) + tiny + 1e-37
    bw = bw + u * (dw.abs() + bw) + tiny + 1e-37
    bounds = {"loss": dloss + 1e-37, "lse": dlse + 1e-37, "dh": bh, "dw": bw}
    return loss, lse, dh, dw, bounds


def check(name, got, ref, bound):
    got = got.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaNs differ"
    d = torch.where(nan, 0.0, (got - ref).abs())
    b = torch.where(nan, 1.0, bound.expand_as(d))
    worst = float((d / b).max()) if d.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound (largest error {float(d.max()):.3g})"
    return worst
