"""The loss operators' fp32 heads are fp32 throughout: every value keeps its 24 bits
whatever else stands in its tensor, so the bounds here have no share of a tensor's
largest value in them (tests/loss_cases.py allows one).

Bounds, with e = 2^-24. fp32 operands go through the product in parts whose dropped
products are at most 3 e of a product, and D products are summed in fp32: a logit is
off by at most dz = (3 D + 16) e sum|h||W|. The sum of the exponentials moves by at most
what it is with every logit off by its own dz, and by (V/64 + 104) e of itself; lse
is rounded a few times by its own size and that of the largest logit, which the
exponentials are taken relative to. An entry of the logits' gradient moves by what its
probability does with the logit and the lse off by these, 40 e of it, and a few e of
its parts; its parts lose at most 3 e of it. Sums of K products add (3 K + 16) e of the sum of
their magnitudes, and the result is rounded once.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from loss_cases import make  # noqa: E402
from test_gpu_losses import run, say  # noqa: E402

E = 2.0 ** -24
TINY = 1e-37  # results and parts this near fp32's smallest normal value are subnormal


def exact(c, temperature=1.0):
    """name -> (value, bound) in float64."""
    h, w = c["hidden"].double(), c["weight"].double()
    T, D = h.shape
    V = w.shape[0]
    z = h @ w.T / temperature
    dz = (3 * D + 16) * E * (h.abs() @ w.abs().T) / temperature
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    top = z.amax(1)
    share = torch.exp(z + dz - lse[:, None])
    dlse = torch.log(share.sum(1)) + (V / 64 + 104) * E + 4 * E * (lse.abs() + top.abs())
    want = torch.zeros_like(z)
    if "target" in c:
        live = c["target"] >= 0
        want[torch.nonzero(live)[:, 0], c["target"][live]] = 1.0
        entropy, K = torch.zeros_like(lse), 1
    else:
        live = (c["index"] >= 0).any(1)
        pk = torch.softmax(torch.where(c["index"] >= 0, c["logit"].double() / temperature,
                                       -math.inf), 1).nan_to_num(0.0)
        want.scatter_add_(1, c["index"].clamp(min=0), pk)
        entropy, K = torch.xlogy(pk, pk).sum(1), c["index"].shape[1]
    seen = torch.where(want > 0, z.abs(), 0.0).amax(1)
    loss = temperature ** 2 * (entropy + lse - (want * z).sum(1))
    dloss = temperature ** 2 * (dlse + (want * dz).sum(1)
                                + (16 + K) * E * (1 + seen + lse.abs() + top.abs()))
    a = torch.where(live, c["up"].double().expand(T) * temperature, 0.0)[:, None]
    g = a * (p - want)
    dg = a.abs() * (torch.exp(z + dz - lse[:, None] + dlse[:, None]) - p + 40 * E * p) \
        + 8 * E * a.abs() * (p + want) + 3 * E * g.abs()
    dg = torch.where(live[:, None], dg, 0.0)
    out = {"loss": (torch.where(live, loss, 0.0), dloss),
           "lse": (torch.where(live, lse, 0.0), dlse)}
    for name, x, gx, dx in (("dhidden", w, g, dg), ("dweight", h, g.T, dg.T)):
        r = gx @ x
        b = dx @ x.abs() + (3 * gx.shape[1] + 16) * E * (gx.abs() @ x.abs())
        out[name] = (r, b + E * (r.abs() + b) + TINY)
    return out


def verify(c, opt=None, rows=None):
    """`rows`: the tokens whose results are looked at (dweight then is not)."""
    opt = opt or {}
    loss, saved, dh, dw = run(c, opt)
    torch.cuda.synchronize()
    got = {"loss": loss, "lse": saved.lse, "dhidden": dh, "dweight": dw}
    for name, (value, bound) in exact(c, **opt).items():
        if rows is not None:
            if name == "dweight":
                continue
            got[name], value, bound = got[name][rows], value[rows], bound[rows]
        off = (got[name].double() - value).abs()
        assert torch.isfinite(got[name]).all(), f"{name} is not finite"
        worst = float((off / bound).max())
        say(f"  {name}: {worst:.2g} of its bound")
        assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"


OPS = [("xent", {}), ("distill", {"temperature": 2.0})]


@pytest.mark.parametrize("op,opt", OPS, ids=[o for o, _ in OPS])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("power", [27, 34, 60])
@pytest.mark.parametrize("which", ["hidden", "weight"])
def test_a_large_finite_row_leaves_the_others(which, power, T, op, opt):
    say(f"[case] {op} {T} tokens, a row of {which} times 2^{power}")
    c = make(T, 301, 64, "fp32", seed=40, k=0 if op == "xent" else 4)
    live = c["target"] >= 0 if op == "xent" else (c["index"] >= 0).any(1)
    c[which][int(torch.nonzero(live)[3, 0])] *= 2.0 ** power
    verify(c, opt)


@pytest.mark.parametrize("op,opt", OPS, ids=[o for o, _ in OPS])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("apart", [25.0, 60.0])
def test_gradients_of_rare_entries(apart, T, op, opt):
    """Half of the vocabulary is `apart` below the other in every row's logits, and no
    row's target: its probabilities are all that its rows of dweight are made of."""
    say(f"[case] {op} {T} tokens, half of the vocabulary {apart} below")
    c = make(T, 301, 64, "fp32", seed=41, k=0 if op == "xent" else 4)
    c["hidden"][:, 0] = 1.0
    c["weight"][:, 0] = 0.0
    c["weight"][150:, 0] = -apart * opt.get("temperature", 1.0)
    for name in ("target", "index"):
        if name in c:
            c[name] = torch.where(c[name] >= 150, c[name] - 150, c[name]).clamp(max=149)
    verify(c, opt)


@pytest.mark.parametrize("op,opt", OPS, ids=[o for o, _ in OPS])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("span", [30, 70])
def test_rows_of_small_upstream_keep_their_gradients(span, T, op, opt):
    say(f"[case] {op} {T} tokens, upstreams over 2^{span}")
    c = make(T, 301, 64, "fp32", seed=42, k=0 if op == "xent" else 4)
    c["up"] = 2.0 ** -(torch.arange(T, device="cuda") * 7 % (span + 1)).float()
    verify(c, opt)


@pytest.mark.parametrize("op,opt", OPS, ids=[o for o, _ in OPS])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("powers", [(-75, -75), (-60, 60), (60, -60), (95, -95), (-20, -100),
                                    (-105, -20)], ids=str)
def test_any_magnitude(powers, T, op, opt):
    """A vocabulary that is no multiple of a tile, so that some of the last one is
    masked, under logits that are ordinary or all zero."""
    say(f"[case] {op} {T} tokens, hidden and weight times 2^{powers}")
    c = make(T, 301, 64, "fp32", seed=43, k=0 if op == "xent" else 4)
    c["hidden"] *= 2.0 ** powers[0]
    c["weight"] *= 2.0 ** powers[1]
    verify(c, opt)


@pytest.mark.parametrize("op,opt", OPS, ids=[o for o, _ in OPS])
@pytest.mark.parametrize("T", [40, 150])
def test_a_row_of_zeros_beside_rows_that_overflow(T, op, opt):
    """Its logits are all zero, whatever the others' are: loss and dhidden are those of
    equal probabilities."""
    say(f"[case] {op} {T} tokens, a row of zeros, the others' logits infinite")
    c = make(T, 301, 64, "fp32", seed=44, k=0 if op == "xent" else 4)
    live = c["target"] >= 0 if op == "xent" else (c["index"] >= 0).any(1)
    row = torch.nonzero(live)[5, 0]
    c["hidden"] *= 2.0 ** 85
    c["weight"] *= 2.0 ** 85
    c["hidden"][row] = 0.0
    # the reference of that row alone: the others' overflow in float32, not in float64
    one = {k: v.clone() for k, v in c.items()}
    one["hidden"][:] = 0.0
    loss, saved, dh, _ = run(c, opt)
    got = {"loss": loss, "lse": saved.lse, "dhidden": dh}
    for name, x in got.items():
        value, bound = exact(one, **opt)[name]
        assert bool(((x[row].double() - value[row]).abs() <= bound[row]).all()), name


@pytest.mark.parametrize("T", [40, 150])
def test_the_largest_finite_values(T):
    """Values that 8 bits would round to infinity, met by zeros in the other factor."""
    say(f"[case] {T} tokens, values of fp32's maximum")
    c = make(T, 301, 64, "fp32", seed=45)
    c["hidden"][:, 3] = 0.0
    c["weight"][::3, 3] = 3.4028234663852886e38
    loss, saved = run(c, {})[:2]
    for name, x in (("loss", loss), ("lse", saved.lse)):
        value, bound = exact(c)[name]
        assert bool(((x.double() - value).abs() <= bound).all()), name
