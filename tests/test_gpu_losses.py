"""The loss operators (zero_loss.h) on the GPU against their definition in
float64, at the sizes, masks, strides and types where they can go wrong."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from zero_sharded_optimizer_amd import losses  # noqa: E402
from loss_cases import DTYPES, check, make, reference  # noqa: E402


def say(*a):
    print(*a, flush=True)


def run(c, opt, **kw):
    """Loss and gradients of one case, with outputs pre-filled so that an element
    that is not written shows."""
    h, w = c["hidden"], c["weight"]
    dh = torch.full(h.shape, float("nan"), dtype=h.dtype, device=h.device)
    dw = torch.full(w.shape, float("nan"), dtype=w.dtype, device=w.device)
    if "target" in c:
        loss, saved = losses.linear_xent(h, w, c["target"], **opt)
        losses.linear_xent_grad(h, w, c["target"], saved, c["up"], dhidden=dh, dweight=dw, **opt,
                                **kw)
    else:
        loss, saved = losses.linear_distill(h, w, c["index"], c["logit"], **opt)
        losses.linear_distill_grad(h, w, c["index"], c["logit"], saved, c["up"], dhidden=dh,
                                   dweight=dw, **opt, **kw)
    return loss, saved, dh, dw


def ref_opt(opt):
    r = dict(opt)
    if "label_smoothing" in r:
        r["smoothing"] = r.pop("label_smoothing")
    return r


def verify(c, opt, **kw):
    loss, saved, dh, dw = run(c, opt, **kw)
    torch.cuda.synchronize()
    r_loss, r_lse, r_dh, r_dw, b = reference(c, **ref_opt(opt))
    worst = [check("loss", loss, r_loss, b["loss"]), check("lse", saved.lse, r_lse, b["lse"]),
             check("dhidden", dh, r_dh, b["dh"]), check("dweight", dw, r_dw, b["dw"])]
    say("  share of the bounds:", " ".join(f"{x:.2g}" for x in worst))
    return loss, saved, dh, dw


SHAPES = [(1, 1, 1), (1, 2, 3), (2, 33, 64), (3, 70, 8), (17, 300, 65), (64, 257, 96),
          (65, 64, 128), (130, 1000, 72), (257, 515, 320), (5, 4099, 40), (300, 129, 1),
          (31, 2049, 640)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_xent(shape, dtype):
    say(f"[case] xent {shape} {dtype}")
    verify(make(*shape, dtype, seed=sum(shape)), {})


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape,k", [((1, 1, 1), 1), ((2, 33, 64), 5), ((17, 300, 65), 16),
                                     ((64, 257, 96), 17), ((130, 1000, 72), 64),
                                     ((257, 515, 320), 100), ((9, 40, 24), 1024)], ids=str)
def test_distill(shape, k, dtype):
    say(f"[case] distill {shape} k={k} {dtype}")
    for tau in (1.0, 2.5):
        verify(make(*shape, dtype, seed=sum(shape) + k, k=k), {"temperature": tau})


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("opt", [{"label_smoothing": 0.1}, {"z_loss": 1e-3},
                                 {"label_smoothing": 0.3, "z_loss": 1e-2}], ids=str)
def test_xent_options(opt, dtype):
    say(f"[case] xent {opt} {dtype}")
    verify(make(100, 777, 136, dtype, seed=3), opt)


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("dtype,T,V", [("fp32", 16385, 6001), ("bf16", 70000, 4500),
                                       ("bf16", 70000, 4200), ("fp32", 1024, 50257),
                                       ("fp16", 1000, 33001), ("bf16", 250, 40000),
                                       ("fp32", 60, 40001)])
def test_several_pieces(op, dtype, T, V):
    """More tokens than one piece of the whole vocabulary holds; last pieces that
    end several tiles before the others do; and problems of one piece for each
    width of the logits' tiles."""
    say(f"[case] {op} pieces {T} x {V} {dtype}")
    c = make(T, V, 64, dtype, seed=5, k=0 if op == "xent" else 7)
    c["up"] = c["up"] * 100
    verify(c, {} if op == "xent" else {"temperature": 2.0})


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_wide_rows_and_few_tokens(op, dtype):
    """The vocabulary sum of dhidden split into runs."""
    say(f"[case] {op} split {dtype}")
    verify(make(3, 20011, 192, dtype, seed=6, k=0 if op == "xent" else 9), {})


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_empty_rows_may_hold_anything(op, dtype):
    say(f"[case] {op} garbage in empty rows {dtype}")
    c = make(77, 200, 64, dtype, seed=7, ignored=0.5, k=0 if op == "xent" else 4)
    dead = c["target"] == -100 if op == "xent" else (c["index"] < 0).all(1)
    assert dead.any() and not dead.all()
    at = torch.nonzero(dead)[:, 0]
    c["hidden"][at] = float("nan")
    c["hidden"][at[::2]] = float("inf")
    c["up"][at] = float("nan")
    if op == "distill":
        c["logit"][at] = float("nan")
    _, saved, dh, _ = verify(c, {})
    assert (dh[at] == 0).all() and (saved.lse[at] == 0).all()


@pytest.mark.parametrize("what", ["hidden", "upstream"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("tokens", [29, 77])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_live_row_that_is_not_finite_leaves_the_others(dtype, tokens, op, bad, what):
    """One element of one live row: the other rows' losses and dhidden stand as
    without it, at a scale of hidden and upstream that needs the operands' own."""
    say(f"[case] {op} {bad} in a live row's {what} {dtype} {tokens}")
    c = make(tokens, 300, 64, dtype, seed=12, k=0 if op == "xent" else 4)
    shift = 13 if dtype == "fp32" else 4
    c["hidden"] *= 2.0 ** -shift
    c["weight"] *= 2.0 ** shift
    c["up"] *= 2.0 ** -10
    live = c["target"] != -100 if op == "xent" else (c["index"] >= 0).any(1)
    row = int(torch.nonzero(live)[5, 0])
    opt = {"z_loss": 1e-3} if op == "xent" else {"temperature": 2.0}
    plain = {k: v.clone() for k, v in c.items()}
    plain["up"][row] = 0.0
    if what == "hidden":
        c["hidden"][row, 40] = bad
    else:
        c["up"][row] = bad
    loss, saved, dh, dw = run(c, opt)
    r_loss, r_lse, r_dh, _, b = reference(plain, **opt)
    keep = torch.arange(tokens, device="cuda") != row
    check("loss", loss[keep], r_loss[keep], b["loss"][keep])
    check("lse", saved.lse[keep], r_lse[keep], b["lse"][keep])
    check("dhidden", dh[keep], r_dh[keep], b["dh"][keep])
    assert not torch.isfinite(dh[row]).any() and not torch.isfinite(dw).all()
    if what == "hidden":
        assert not torch.isfinite(loss[row])


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_no_live_row(op):
    say(f"[case] {op} no live row")
    c = make(40, 300, 64, "bf16", seed=8, ignored=2.0, k=0 if op == "xent" else 3)
    c["hidden"].fill_(float("nan"))
    loss, saved, dh, dw = run(c, {})
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all() and (saved.lse == 0).all()


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_no_tokens(op):
    say(f"[case] {op} no tokens")
    c = make(0, 300, 64, "bf16", seed=8, k=0 if op == "xent" else 3)
    loss, saved, dh, dw = run(c, {})
    assert loss.numel() == 0 and dh.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("wide", [torch.int32, torch.int64])
def test_bad_targets_give_nan_and_no_gradient(wide):
    say(f"[case] bad targets {wide}")
    c = make(50, 200, 64, "bf16", seed=9)
    c["target"] = c["target"].to(wide)
    c["target"][3], c["target"][10], c["target"][20] = 200, -1, 2 ** 31 - 1
    loss, _, dh, _ = verify(c, {})
    assert torch.isnan(loss[[3, 10, 20]]).all() and (dh[[3, 10, 20]] == 0).all()
    c = make(50, 200, 64, "fp32", seed=9, k=5)
    c["index"] = c["index"].to(wide)
    c["index"][4, 2], c["index"][5, 0] = 200, 2 ** 31 - 1
    loss, _, dh, _ = verify(c, {"temperature": 2.0})
    assert torch.isnan(loss[[4, 5]]).all() and (dh[[4, 5]] == 0).all()


def test_ignore_index_inside_the_vocabulary():
    say("[case] ignore_index 0")
    c = make(50, 20, 64, "bf16", seed=10)
    c["target"][c["target"] == -100] = 0
    verify(c, {"ignore_index": 0})


def test_teacher_logits_of_minus_infinity_are_padding():
    say("[case] teacher -inf")
    c = make(30, 100, 64, "fp32", seed=11, k=6)
    c["logit"][:, 3] = -math.inf
    c["logit"][5] = -math.inf
    _, _, dh, _ = verify(c, {"temperature": 2.0})
    assert (dh[5] == 0).all()


@pytest.mark.parametrize("teacher", list(DTYPES))
def test_teacher_types_and_strides(teacher):
    say(f"[case] teacher {teacher}")
    c = make(33, 100, 64, "bf16", seed=12, k=11)
    wide = torch.zeros(33, 20, dtype=DTYPES[teacher], device="cuda")
    wide[:, 4:15] = c["logit"].to(DTYPES[teacher])
    c["logit"] = wide[:, 4:15]
    idx = torch.zeros(33, 13, dtype=torch.int32, device="cuda")
    idx[:, 1:12] = c["index"].int()
    c["index"] = idx[:, 1:12]
    verify(c, {"temperature": 2.0})


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("off", [0, 1, 4])
def test_strided_and_unaligned_tensors(dtype, off):
    """hidden a slice of wider rows, weight and dweight views of flat buffers at
    any element offset, dhidden beside hidden in one buffer."""
    say(f"[case] views {dtype} offset {off}")
    T, V, D = 70, 150, 128
    c = make(T, V, D, dtype, seed=13)
    dt = DTYPES[dtype]
    flat = torch.zeros(V * D + 64, dtype=dt, device="cuda")
    flat[off:off + V * D] = c["weight"].reshape(-1)
    c["weight"] = flat[off:off + V * D].view(V, D)
    both = torch.full((T, 2 * D + 24), float("nan"), dtype=dt, device="cuda")
    both[:, off:off + D] = c["hidden"]
    c["hidden"] = both[:, off:off + D]
    gflat = torch.full((V * D + 64,), 7.0, dtype=dt, device="cuda")
    dw = gflat[off:off + V * D].view(V, D)
    dh = both[:, off + D + 8:off + 2 * D + 8]
    loss, saved = losses.linear_xent(c["hidden"], c["weight"], c["target"])
    losses.linear_xent_grad(c["hidden"], c["weight"], c["target"], saved, c["up"], dhidden=dh,
                            dweight=dw)
    r_loss, _, r_dh, r_dw, b = reference(c)
    check("loss", loss, r_loss, b["loss"])
    check("dhidden", dh, r_dh, b["dh"])
    check("dweight", dw, r_dw, b["dw"])
    assert (gflat[:off] == 7).all() and (gflat[off + V * D:] == 7).all()
    assert torch.isnan(both[:, off + D:off + D + 8]).all()


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_one_gradient_alone_and_broadcast_upstream(op):
    say(f"[case] {op} one gradient")
    c = make(70, 150, 128, "bf16", seed=14, k=0 if op == "xent" else 5)
    c["up"] = torch.full((1,), 0.01, device="cuda").expand(70)
    _, saved, dh, dw = verify(c, {})
    fn, t = ((losses.linear_xent_grad, (c["target"],)) if op == "xent" else
             (losses.linear_distill_grad, (c["index"], c["logit"])))
    a, none = fn(c["hidden"], c["weight"], *t, saved, 0.01, need_dweight=False)
    assert none is None and torch.equal(a, dh)
    none, b = fn(c["hidden"], c["weight"], *t, saved, c["up"][:1], need_dhidden=False)
    assert none is None and torch.equal(b, dw)


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_the_same_call_gives_the_same_bits_on_any_stream(op):
    say(f"[case] {op} repeat, streams")
    c = make(200, 3000, 256, "bf16", seed=15, k=0 if op == "xent" else 8)
    one = run(c, {})
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        two = run(c, {})
    s.synchronize()
    for x, y in zip((one[0], one[1].lse, *one[2:]), (two[0], two[1].lse, *two[2:])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_captured_into_a_graph(op):
    say(f"[case] {op} graph")
    a = make(90, 500, 128, "bf16", seed=16, k=0 if op == "xent" else 8)
    b = make(90, 500, 128, "bf16", seed=17, ignored=0.6, k=0 if op == "xent" else 8)
    want = [run(a, {}), run(b, {})]
    static = {k: v.clone() for k, v in a.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(static, {})
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(static, {})
    for i in (0, 1, 0, 1, 1):
        for k, v in (a, b)[i].items():
            static[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        run((a, b)[1 - i], {})  # the program's own eager work in between
        for x, y in zip((out[0], out[1].lse, *out[2:]),
                        (want[i][0], want[i][1].lse, *want[i][2:])):
            assert torch.equal(x, y)


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_gradient_against_differences(op):
    """Central differences of the loss along each row's gradient, tilted by a
    random direction. With step s the loss's own error (its bound, summed over
    rows) enters as that over s, and the third derivative, at most 2 |dz|^3 a row
    for a softmax (|dz| the largest change of a logit per unit step), as s^2 / 6."""
    say(f"[case] {op} differences")
    c = make(24, 90, 48, "fp32", seed=18, k=0 if op == "xent" else 6)
    c["up"] = torch.full((24,), 0.1, device="cuda")
    opt = {"z_loss": 1e-3, "label_smoothing": 0.1} if op == "xent" else {"temperature": 1.5}
    _, _, dh, dw = run(c, opt)
    up = c["up"].double()
    g = torch.Generator().manual_seed(19)
    tau = opt.get("temperature", 1.0)
    s = 2.0 ** -6
    for which, grad in (("hidden", dh), ("weight", dw)):
        tilt = torch.randn(c[which].shape, generator=g).cuda()
        d = grad / grad.norm(dim=1, keepdim=True).clamp(min=1e-20) \
            + 0.3 * tilt / tilt.norm(dim=1, keepdim=True)
        ends = []
        for sign in (1, -1):
            m = dict(c)
            m[which] = c[which] + sign * s * d
            ends.append(float((up * run(m, opt)[0].double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * s)
        noise = float((up * reference(c, **ref_opt(opt))[4]["loss"]).sum()) * 2 / s
        if which == "hidden":
            dz = (d.double() @ c["weight"].double().T).abs().amax(1) / tau
        else:
            dz = (c["hidden"].double() @ d.double().T).abs().amax(1) / tau
        live = (c["target"] != -100) if op == "xent" else (c["index"] >= 0).any(1)
        curve = s * s / 6 * float((up * live * 2 * tau * tau * dz ** 3).sum()) * 1.1
        # the moved inputs are rounded: 2^-24 of their size, felt over a step of 2 s
        moved = float((grad.double().abs() * c[which].double().abs()).sum()) * 2.0 ** -24 / s
        got = float((grad.double() * d.double()).sum())
        tol = noise + curve + moved
        say(f"  {which}: {got:.6g} against {slope:.6g}, tolerance {tol:.2g}")
        assert tol < 0.2 * abs(got)
        assert abs(got - slope) <= tol


def test_extreme_logits():
    """Probabilities of one and zero, and logits around +-200."""
    say("[case] extreme logits")
    for dtype in DTYPES:
        c = make(40, 300, 64, dtype, seed=20, spread=60.0)
        verify(c, {})


def test_gradients_land_in_a_worker_buffer_and_step():
    """Both losses as one model's step: each logical worker's head gradient is
    written straight into its flat gradient buffer, and the sharded step's
    averaged gradient is the mean of what the formula gives."""
    from zero_sharded_optimizer_amd.optimizer import ZeroOptimizer
    say("[case] losses into the sharded step")
    g = torch.Generator().manual_seed(21)
    body = torch.nn.Linear(24, 64, bias=False)
    head = torch.nn.Parameter(torch.randn(301, 64, generator=g) * 0.1)
    with torch.no_grad():
        body.weight.copy_(torch.randn(64, 24, generator=g) * 0.2)
    body, head = body.cuda(), torch.nn.Parameter(head.detach().cuda())
    zo = ZeroOptimizer([body.weight, head], 2, 1, precision="fp32", lr=1e-2)
    zo.zero_grad()
    total = torch.zeros(301, 64, dtype=torch.float64, device="cuda")
    for k in range(2):
        x = torch.randn(30, 24, generator=g).cuda()
        h = body(x)
        c = make(30, 301, 64, "fp32", seed=22 + k, k=0 if k == 0 else 4)
        c["hidden"], c["weight"] = h.detach(), head.detach()
        c["up"] = torch.full((30,), 1 / 30, device="cuda")
        gb, gh = zo.worker_grads(k)
        if k == 0:
            _, saved = losses.linear_xent(h.detach(), head.detach(), c["target"])
            dh, _ = losses.linear_xent_grad(h.detach(), head.detach(), c["target"], saved, 1 / 30,
                                            dweight=gh)
        else:
            _, saved = losses.linear_distill(h.detach(), head.detach(), c["index"], c["logit"])
            dh, _ = losses.linear_distill_grad(h.detach(), head.detach(), c["index"], c["logit"],
                                               saved, 1 / 30, dweight=gh)
        body.weight.grad = None
        h.backward(dh)
        gb.copy_(body.weight.grad)
        _, _, _, dw, b = reference(c)
        check("head gradient", gh, dw, b["dw"])
        total += gh.double()
    before = head.detach().clone()
    zo.step()
    mean = zo.averaged_grad()[body.weight.numel():].view(301, 64).double()
    assert float((mean - total / 2).abs().max()) <= 2.0 ** -22 * float(total.abs().max())
    assert not torch.equal(before, head.detach())


@pytest.mark.parametrize("precision", ["fp32", "bf16", "fp16"])
def test_example_learns(precision):
    """The example's both losses fall by more than half: gradients of the wrong sign,
    scale or row would not do that."""
    import os
    import sys
    say(f"[case] example {precision}")
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    sys.path.insert(0, at)
    try:
        import train_lm_head
    finally:
        sys.path.remove(at)
    first, last = train_lm_head.train(steps=120, precision=precision, vocab=211)
    say("  ", first, last)
    for name in first:
        assert math.isfinite(last[name]) and last[name] < first[name] / 2, (first, last)


def test_weight_of_more_than_2_to_the_31_elements():
    """Offsets beyond 32 bits in the weight and its gradient, targets at both ends."""
    say("[case] 530000 x 4096")
    V, D, T = 530000, 4096, 5
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    w.normal_(0.0, 1.5 / math.sqrt(D), generator=torch.Generator("cuda").manual_seed(23))
    h = torch.randn(T, D, generator=torch.Generator().manual_seed(24)).bfloat16().cuda()
    c = {"hidden": h, "weight": w, "up": torch.full((T,), 0.2, device="cuda"),
         "target": torch.tensor([V - 1, 0, V // 2, -100, V - 129]).cuda()}
    loss, saved, dh, dw = run(c, {})
    # the same rows in small pieces: only the sums over the vocabulary join them
    z = torch.cat([h.double() @ x.double().T for x in w.split(1 << 16)], 1)
    lse = torch.logsumexp(z, 1)
    live = c["target"] >= 0
    g = torch.softmax(z, 1) * 0.2 * live[:, None]
    rows = torch.nonzero(live)[:, 0]
    g[rows, c["target"][rows]] -= 0.2
    want = torch.where(live, lse - z[torch.arange(T), c["target"].clamp(min=0)], 0.0)
    # |z| < 10, each off by (D + 16) 2^-24 of sum|h||w| < 70; the sum as in loss_cases
    assert float((loss - want).abs().max()) <= 2 * (D + 16) * 2.0 ** -24 * 70 \
        + (V / 64 + 200) * 2.0 ** -24
    u, slack = 2.0 ** -8, 2 * (D + V / 64 + 300) * 2.0 ** -24 * 70
    at = 0
    r_dh = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    b_dh = torch.zeros_like(r_dh)
    for x, gx in zip(w.split(1 << 16), g.split(1 << 16, dim=1)):
        r_dh += gx @ x.double()
        b_dh += gx.abs() @ x.double().abs()
        r_dw, b_dw = gx.T @ h.double(), gx.T.abs() @ h.double().abs()
        d = (dw[at:at + x.shape[0]].double() - r_dw).abs()
        assert bool((d <= u * r_dw.abs() + (u * (1 + u) + slack) * b_dw + 1e-37).all()), at
        at += x.shape[0]
    d = (dh.double() - r_dh).abs()
    assert bool((d <= u * r_dh.abs() + (u * (1 + u) + slack + V * 2.0 ** -24) * b_dh).all())
