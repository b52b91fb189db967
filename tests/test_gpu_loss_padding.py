"""Teacher entries that are padding by their logit: what the header says of padding holds
for them, also where the same index stands in the row once more."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from loss_cases import DTYPES, make  # noqa: E402
from test_gpu_losses import say, verify  # noqa: E402


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T", [40, 150])
def test_saved_logits_of_padding_are_zero(T, dtype):
    say(f"[case] padding by -inf {dtype} {T}")
    c = make(T, 300, 64, dtype, seed=70, ignored=0.0, k=6)
    c["index"] = c["index"].clamp(min=0)
    c["logit"][:, 1] = -math.inf
    c["index"][::2, 1] = c["index"][::2, 4]    # padding beside the same index with a share
    c["index"][1::4, 5] = -1                   # padding by index, whatever its logit
    c["logit"][1::4, 5] = math.nan
    c["logit"][7] = -math.inf                  # an empty row
    padding = (c["index"] < 0) | (c["logit"] == -math.inf)
    c["logit"] = torch.where(c["index"] < 0, 0.0, c["logit"])
    _, saved, dh, _ = verify(c, {"temperature": 2.0})
    assert bool((saved.logit[padding] == 0).all())
    z = c["hidden"].double() @ c["weight"].double().T
    want = torch.gather(z, 1, c["index"].clamp(min=0))
    assert bool(((saved.logit - want).abs()[~padding] < 1e-4).all())
    assert bool((dh[7] == 0).all())
