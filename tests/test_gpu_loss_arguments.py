"""The loss operators' stream and workspace arguments, and widths from 4096 up."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import zero_sharded_optimizer_amd as z  # noqa: E402
from zero_sharded_optimizer_amd import losses  # noqa: E402
from loss_cases import DTYPES, make  # noqa: E402
from test_gpu_losses import run, say, verify  # noqa: E402


def both(c, workspaces=(None, None), stream=None):
    """Loss and gradients of a case, with the given workspaces and stream; new outputs."""
    h, w = c["hidden"], c["weight"]
    if "target" in c:
        loss, saved = losses.linear_xent(h, w, c["target"], workspace=workspaces[0], stream=stream)
        dh, dw = losses.linear_xent_grad(h, w, c["target"], saved, c["up"],
                                         workspace=workspaces[1], stream=stream)
    else:
        loss, saved = losses.linear_distill(h, w, c["index"], c["logit"], workspace=workspaces[0],
                                            stream=stream)
        dh, dw = losses.linear_distill_grad(h, w, c["index"], c["logit"], saved, c["up"],
                                            workspace=workspaces[1], stream=stream)
    return [loss, saved.lse, dh, dw]


CASES = [(T, dtype, op) for T in (40, 300) for dtype in DTYPES for op in ("xent", "distill")]


@pytest.mark.parametrize("T,dtype,op", CASES, ids=str)
def test_given_streams(T, dtype, op):
    """A stream object or its handle: the work and the outputs' memory are that stream's."""
    say(f"[case] stream {T} {dtype} {op}")
    c = make(T, 1003, 128, dtype, seed=80, k=0 if op == "xent" else 5)
    want = both(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(3):  # memory given back is taken again, in that stream's order
            got = both(c, stream=stream)
        assert torch.cuda.current_stream() != s
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,dtype,op", CASES, ids=str)
def test_given_workspaces(T, dtype, op):
    """One buffer for both calls, whatever it holds; nothing beyond the bytes asked for is
    touched, and less is refused."""
    say(f"[case] workspace {T} {dtype} {op}")
    c = make(T, 1003, 128, dtype, seed=81, k=0 if op == "xent" else 5)
    want = both(c)
    need = [losses.loss_workspace_bytes(c["hidden"], c["weight"], g) for g in (False, True)]
    buf = torch.full((max(need) + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    for _ in range(2):
        got = both(c, (buf[:need[0]], buf[:need[1]]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((buf[max(need):] == 0xFF).all())
        buf[:max(need)] = 0xFF
    for ws in ((buf[:need[0] - 1], None), (None, buf[:need[1] - 1]), (buf[16:], None)):
        with pytest.raises(z.ZeroError, match="workspace"):
            both(c, ws)
    for ws in (buf.cpu(), buf[::2], 7):
        with pytest.raises(ValueError, match="workspace"):
            both(c, (ws, None))


def test_a_stream_of_another_kind_is_refused():
    say("[case] other device's stream")
    c = make(8, 30, 64, "bf16", seed=82)

    class Elsewhere:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream is on"):
        both(c, stream=Elsewhere())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,V,D,op", [(3, 300, 65536, "xent"), (70, 500, 65536, "distill"),
                                      (300, 1000, 8200, "xent"), (20, 700, 12289, "distill"),
                                      (130, 600, 5001, "xent")], ids=str)
def test_wide_heads(T, V, D, op, dtype):
    say(f"[case] wide {T} x {V} x {D} {op} {dtype}")
    verify(make(T, V, D, dtype, seed=83, k=0 if op == "xent" else 6), {})


@pytest.mark.parametrize("dtype,T,V,D,op", [("fp32", 40, 6001, 20000, "xent"),
                                            ("fp32", 300, 9001, 11000, "distill"),
                                            ("bf16", 20, 7001, 65528, "xent"),
                                            ("fp16", 70000, 4500, 72, "distill")], ids=str)
def test_several_pieces_of_wide_heads(dtype, T, V, D, op):
    """Pieces cut by the packed weights' size, and a packed weight with many tokens."""
    say(f"[case] pieces {T} x {V} x {D} {op} {dtype}")
    c = make(T, V, D, dtype, seed=84, k=0 if op == "xent" else 6)
    need = losses.loss_workspace_bytes(c["hidden"], c["weight"], True)
    c["up"] = c["up"] * min(100.0, math.sqrt(T))
    verify(c, {})
    planes = 3 if dtype == "fp32" else 1
    if D > 1000:
        assert need < planes * 2 * V * D  # less than the whole weight: several pieces


@pytest.mark.parametrize("T,dtype,op", [c for c in CASES if c[1] != "bf16"], ids=str)
def test_captured_into_a_graph(T, dtype, op):
    """Replays on two sets of inputs, with eager work and synchronizations between them,
    give the eager calls' bits; which rows take part changes from one to the other."""
    say(f"[case] graph {T} {dtype} {op}")
    k = 0 if op == "xent" else 5
    sets = [make(T, 1003, 128, dtype, seed=85 + i, ignored=0.2 + 0.5 * i, k=k) for i in (0, 1)]
    want = [run(c, {}) for c in sets]
    static = {name: x.clone() for name, x in sets[0].items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(static, {})
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(static, {})
    for i in (0, 1, 0, 1, 1):
        for name, x in sets[i].items():
            static[name].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        run(sets[1 - i], {})
        for x, y in zip((out[0], out[1].lse, *out[2:]), (want[i][0], want[i][1].lse, *want[i][2:])):
            assert torch.equal(x, y)
