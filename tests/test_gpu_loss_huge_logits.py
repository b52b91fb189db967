"""The loss operators where single logits are far beyond what an exponential takes:
losses are finite and right to their logits' own rounding, and no gradient is infinite."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from loss_cases import DTYPES, make  # noqa: E402
from test_gpu_losses import run, say  # noqa: E402

E = 2.0 ** -24


@pytest.mark.parametrize("op,opt", [("xent", {}), ("distill", {"temperature": 2.0})],
                         ids=["xent", "distill"])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("dtype,power", [("bf16", 22), ("bf16", 34), ("bf16", 60), ("fp32", 22),
                                         ("fp32", 34), ("fp32", 60), ("fp16", 14)], ids=str)
def test_one_row_of_huge_logits(dtype, power, T, op, opt):
    """Every number that enters the loss is of the row's largest logit's size at most, and
    is rounded some D times by that size: (4 D + 64) 2^-24 of it, at the temperature. fp16's row is
    large by both factors."""
    say(f"[case] {op} {dtype} {T} tokens, a row's logits times 2^{power}")
    c = make(T, 301, 64, dtype, seed=50, k=0 if op == "xent" else 4)
    if dtype == "fp16":
        c["weight"] *= 2.0 ** 14
        c["hidden"] *= 2.0 ** -14
    live = c["target"] >= 0 if op == "xent" else (c["index"] >= 0).any(1)
    row = int(torch.nonzero(live)[3, 0])
    if dtype == "fp16":
        c["hidden"][row] *= 2.0 ** 14
    c["hidden"][row] *= 2.0 ** power
    loss, saved, dh, dw = run(c, opt)
    tau = opt.get("temperature", 1.0)
    h, w = c["hidden"][row].double(), c["weight"].double()
    z = w @ h / tau
    lse = torch.logsumexp(z, 0)
    if op == "xent":
        want = lse - z[c["target"][row]]
    else:
        ok = c["index"][row] >= 0
        t = c["logit"][row][ok].double() / tau
        p = torch.softmax(t, 0)
        want = tau ** 2 * (torch.xlogy(p, p).sum() + lse - (p * z[c["index"][row][ok]]).sum())
    size = float((w.abs() @ h.abs()).max()) / tau
    bound = (4 * 64 + 64) * E * size * tau ** 2
    say(f"  loss {float(loss[row]):.6g}, exact {float(want):.6g}, bound {bound:.2g}")
    assert torch.isfinite(loss).all() and torch.isfinite(saved.lse).all()
    assert abs(float(loss[row]) - float(want)) <= bound
    assert abs(float(saved.lse[row]) - float(lse)) <= bound
    assert torch.isfinite(dh).all()
    if dtype != "fp16":
        assert torch.isfinite(dw).all()
    # probabilities and the target's share are at most 1 each
    cap = 2.02 * tau * float(c["up"].abs().max()) * float(w.abs().sum(0).max())
    assert float(dh[row].abs().max()) <= cap
