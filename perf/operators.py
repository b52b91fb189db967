"""The loss operators' measured cases: a language model's head with its loss, over real ranges.

Two operators, each as its loss alone ("eval") and as a training step's loss with the gradients of
both factors ("train"):
  xent     softmax cross entropy of hidden @ weight.T against one target per token
  distill  the divergence of the softmax of hidden @ weight.T from a teacher's top-K logits
`run` computes them in plain torch operations in fp32, or (own) through the package.
"""
import math

import torch

own = False

IGNORE = -100
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _case(name, op, train, tokens, vocab, dim, dtype, ignored=0.0, k=0, temperature=1.0,
          smoothing=0.0, z_loss=0.0, scale=1.0):
    c = {"op": op, "train": train, "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype,
         "ignored": ignored, "k": k, "temperature": temperature, "smoothing": smoothing,
         "z_loss": z_loss, "scale": scale}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # scoring one continuation token: the smallest call, one row of hidden states
        _case("xent eval 1 token", "xent", False, 1, 32000, 2048, "bf16"),
        # perplexity of two thousand tokens under a GPT-2-small-shaped head (odd vocabulary)
        _case("xent eval gpt2 bf16", "xent", False, 2047, 50257, 768, "bf16", ignored=0.01),
        # a short fine-tuning example whose prompt is masked: a few dozen live rows, a large head
        _case("xent train 40 tokens", "xent", True, 40, 131072, 2048, "bf16", ignored=0.3),
        # one worker's micro-batch under the GPT-2-small-shaped head, full fp32 mode
        _case("xent train gpt2 fp32", "xent", True, 1024, 50257, 768, "fp32"),
        # the same head in bf16 mixed precision, a long micro-batch with ragged length
        _case("xent train gpt2 bf16", "xent", True, 4095, 50257, 768, "bf16", ignored=0.02),
        # fp16 mixed precision: loss scaling, label smoothing, z-loss
        _case("xent train fp16", "xent", True, 1000, 32000, 2048, "fp16", smoothing=0.1,
              z_loss=1e-4, scale=1024.0),
        # an 8B-model-sized head and a full micro-batch, the largest step
        _case("xent train 8k tokens", "xent", True, 8192, 131072, 4096, "bf16", ignored=0.02),
        # instruction tuning: most of the batch is prompt, only the answers are learned from
        _case("xent train masked", "xent", True, 4096, 65536, 2048, "bf16", ignored=0.6),
        # checking a student against a handful of stored teacher rows
        _case("distill eval 16 tokens", "distill", False, 16, 50257, 1024, "bf16", k=8,
              temperature=2.0),
        # a distillation step from 64 stored teacher logits per token
        _case("distill train k64", "distill", True, 4096, 131072, 2048, "bf16", ignored=0.02, k=64,
              temperature=2.0),
        # a small student in fp16 mixed precision, odd sizes, loss scaling
        _case("distill train fp16", "distill", True, 513, 32003, 1024, "fp16", k=20,
              temperature=1.0, scale=1024.0),
        # full fp32 mode, many teacher entries
        _case("distill train fp32", "distill", True, 256, 50257, 768, "fp32", k=100,
              temperature=4.0),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["xent", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    train = rng.random() < 0.7
    tokens, vocab = log_int(1, 8192), log_int(2000, 131072)
    dim = log_int(64, 4096)
    if rng.random() < 0.8:  # widths are mostly whole multiples of 64, sometimes anything
        dim = max(64, dim // 64 * 64)
    if dtype == "fp32":  # 4-byte weights stay within the largest listed weight's bytes
        vocab = min(vocab, 65536)
    ignored = rng.choice([0.0, 0.0, 0.02, 0.3, 0.7])
    scale = 1024.0 if dtype == "fp16" else 1.0
    if op == "xent":
        return _case(None, op, train, tokens, vocab, dim, dtype, ignored,
                     smoothing=rng.choice([0.0, 0.0, 0.1]), z_loss=rng.choice([0.0, 0.0, 1e-4]),
                     scale=scale)
    return _case(None, op, train, tokens, vocab, dim, dtype, ignored, k=log_int(1, 128),
                 temperature=rng.choice([1.0, 2.0, 4.0]), scale=scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, V, D, K = case["tokens"], case["vocab"], case["dim"], case["k"]
    dt = _DTYPES[case["dtype"]]

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    # logits of spread 1.28 around the background, as a head of width 4096 and deviation 0.02 gives
    weight = torch.empty(V, D, dtype=dt, device="cuda")
    weight.normal_(0.0, 1.28 / math.sqrt(D), generator=g)
    dead = rand(T) < case["ignored"]
    if T > 1 and case["ignored"] == 0.0:
        dead[:] = False
    s = {"case": dict(case), "weight": weight}
    if case["op"] == "xent":
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        first = target
        s["target"] = torch.where(dead, torch.full_like(target, IGNORE), target)
    else:
        # K different entries per row, best first; one row in 16 has fewer, dead rows have none
        base = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        step = 1 + (rand(T, 1) * (V // K - 1)).long()
        k = torch.arange(K, device="cuda")[None, :]
        index = (base + k * step) % V
        first = index[:, 0]
        count = torch.where(rand(T, 1) < 1 / 16, 1 + (rand(T, 1) * K).long().clamp(max=K - 1),
                            torch.full((T, 1), K, device="cuda"))
        count = torch.where(dead[:, None], torch.zeros_like(count), count)
        s["index"] = torch.where(k < count, index, torch.full_like(index, -1)).int()
        # a teacher's sorted logits: a steep head and a long tail
        fall = torch.cumsum(-torch.log(rand(T, K).clamp(min=1e-6)) * 1.5 / (1.0 + 0.2 * k), 1)
        tdt = dt if case["dtype"] == "bf16" else torch.float32
        s["teacher"] = (18.0 + 2.0 * rand(T, 1) - fall).to(tdt)
    # the student knows something: the (first) target's logit is raised by 0 to 15
    hidden = torch.empty(T, D, device="cuda").normal_(generator=g)
    to = weight[first].float()
    norm2 = (to * to).sum(1, keepdim=True).clamp(min=1e-6)
    hidden += to * (15.0 * rand(T, 1) / norm2)
    s["hidden"] = hidden.to(dt)
    live = (~dead).sum().clamp(min=1).float()
    s["dloss"] = (case["scale"] / live).expand(T).contiguous()  # the mean over live tokens
    return s


def _plain(s):
    c = s["case"]
    h, w = s["hidden"].float(), s["weight"].float()
    T, V = c["tokens"], c["vocab"]
    tau = c["temperature"]
    z = h @ w.t()
    if tau != 1.0:
        z *= 1.0 / tau
    top = z.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
    zero = torch.zeros_like(lse)
    if c["op"] == "xent":
        eps, zl = c["smoothing"], c["z_loss"]
        live = s["target"] != IGNORE
        at = torch.where(live, s["target"], torch.zeros_like(s["target"]))[:, None]
        loss = lse - (1.0 - eps) * torch.gather(z, 1, at)[:, 0]
        if eps:
            loss = loss - (eps / V) * z.sum(1)
        if zl:
            loss = loss + zl * lse * lse
        part = torch.full((T, 1), 1.0 - eps, device=z.device)
    else:
        valid = s["index"] >= 0
        live = valid.any(1)
        at = torch.where(valid, s["index"], torch.zeros_like(s["index"])).long()
        t = torch.where(valid, s["teacher"].float() / tau, torch.full_like(z[:, :1], -1e30))
        e = torch.exp(t - t.amax(1, keepdim=True)) * valid
        total = e.sum(1, keepdim=True).clamp(min=1e-30)
        part = e / total
        logp = t - t.amax(1, keepdim=True) - torch.log(total)
        terms = torch.where(valid, part * (logp - torch.gather(z, 1, at)), torch.zeros_like(part))
        loss = tau * tau * (terms.sum(1) + lse)
    out = {"loss": torch.where(live, loss, zero), "lse": torch.where(live, lse, zero)}
    if c["train"]:
        grad = torch.exp(z.sub_(lse[:, None]))
        up = torch.where(live, s["dloss"], zero)
        if c["op"] == "xent":
            if c["z_loss"]:
                grad *= (1.0 + 2.0 * c["z_loss"] * lse)[:, None]
            if c["smoothing"]:
                grad -= c["smoothing"] / V
        else:
            up = up * tau
        grad.scatter_add_(1, at, -part)
        grad *= up[:, None]
        out["dhidden"] = (grad @ w).to(s["hidden"].dtype)
        out["dweight"] = (grad.t() @ h).to(s["weight"].dtype)
    return out


def run(state):
    if not own:
        return _plain(state)
    from zero_sharded_optimizer_amd import losses
    s, c = state, state["case"]
    if c["op"] == "xent":
        opt = {"ignore_index": IGNORE, "label_smoothing": c["smoothing"], "z_loss": c["z_loss"]}
        loss, saved = losses.linear_xent(s["hidden"], s["weight"], s["target"], **opt)
        out = {"loss": loss, "lse": saved.lse}
        if c["train"]:
            out["dhidden"], out["dweight"] = losses.linear_xent_grad(
                s["hidden"], s["weight"], s["target"], saved, s["dloss"], **opt)
    else:
        opt = {"temperature": c["temperature"]}
        loss, saved = losses.linear_distill(s["hidden"], s["weight"], s["index"], s["teacher"],
                                            **opt)
        out = {"loss": loss, "lse": saved.lse}
        if c["train"]:
            out["dhidden"], out["dweight"] = losses.linear_distill_grad(
                s["hidden"], s["weight"], s["index"], s["teacher"], saved, s["dloss"], **opt)
    return out


def work(case):
    """Each input once, each output once; the logits' product once, and with gradients the two
    products that they come from."""
    T, V, D, K = case["tokens"], case["vocab"], case["dim"], case["k"]
    size = 4 if case["dtype"] == "fp32" else 2
    moved = (T * D + V * D) * size + T * 8
    moved += T * 8 if case["op"] == "xent" else T * K * (4 + (2 if case["dtype"] == "bf16" else 4))
    flops = 2.0 * T * V * D
    if case["train"]:
        moved += (T * D + V * D) * size + T * 4
        flops *= 3
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    T, V, D = case["tokens"], case["vocab"], case["dim"]
    tau, eps, zl = case["temperature"], case["smoothing"], case["z_loss"]
    w = s["weight"].double()
    rows = 1024  # tokens at a time: the 64-bit logits of all of them would be large
    losses, lses, dhs = [], [], []
    dw = torch.zeros(V, D, dtype=torch.float64, device=w.device) if case["train"] else None
    for a in range(0, T, rows):
        b = min(T, a + rows)
        h = s["hidden"][a:b].double()
        z = torch.mm(h, w.t()) / tau
        lse = torch.logsumexp(z, dim=1)
        want = torch.zeros_like(z)  # the distribution that the softmax is pulled to
        if case["op"] == "xent":
            y = s["target"][a:b]
            live = y != IGNORE
            want += eps / V
            r = torch.nonzero(live)[:, 0]
            want[r, y[r]] += 1.0 - eps
            loss = (want * (lse[:, None] - z)).sum(1) + zl * lse ** 2
            pull, up = 1.0 + 2.0 * zl * lse, s["dloss"][a:b].double()
        else:
            idx = s["index"][a:b].long()
            live = (idx >= 0).any(1)
            t = s["teacher"][a:b].double() / tau
            p = torch.softmax(t.masked_fill(idx < 0, -math.inf), dim=1).nan_to_num(0.0)
            r, k = torch.nonzero(idx >= 0, as_tuple=True)
            want[r, idx[r, k]] = p[r, k]
            loss = tau ** 2 * (torch.xlogy(want, want) + want * (lse[:, None] - z)).sum(1)
            pull, up = torch.ones_like(lse), tau * s["dloss"][a:b].double()
        zero = torch.zeros_like(lse)
        losses.append(torch.where(live, loss, zero))
        lses.append(torch.where(live, lse, zero))
        if case["train"]:
            dz = torch.softmax(z, dim=1) * pull[:, None] - want
            dz = dz * torch.where(live, up, zero)[:, None]
            dhs.append(torch.mm(dz, w))
            dw += torch.mm(dz.t(), h)
    out = {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    if case["train"]:
        out["dhidden"], out["dweight"] = torch.cat(dhs), dw
    return out
