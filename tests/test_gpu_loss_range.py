"""The loss operators' gradients where one factor is near the end of its type's range
and the result is not: nothing on the way there may overflow."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from loss_cases import make  # noqa: E402
from test_gpu_losses import say, verify  # noqa: E402


@pytest.mark.parametrize("op,opt", [("xent", {}), ("distill", {"temperature": 2.0})],
                         ids=["xent", "distill"])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("power", [116, -116])
def test_gradients_by_large_factors(power, dtype, T, op, opt):
    """dhidden is made of the weight's size, dweight of hidden's: both within 2^120 here."""
    say(f"[case] {op} {dtype} {T} tokens, weight times 2^{power}, hidden the inverse")
    c = make(T, 301, 64, dtype, seed=60, k=0 if op == "xent" else 4)
    c["weight"] *= 2.0 ** power
    c["hidden"] *= 2.0 ** -power
    verify(c, opt)
