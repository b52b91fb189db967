"""The loss operators' host side, on the CPU: refusals, workspace sizes, and the
tests' 64-bit reference against torch's own cross entropy and KL divergence."""
import ctypes as C
import math

import pytest
import torch

from zero_sharded_optimizer_amd import _abi, losses
from loss_cases import make, reference

lib = _abi.load()
A = 0x7F0000000000  # addresses that are only looked at: every call here is refused or empty
MiB = 1 << 20


def head(**kw):
    d = dict(tokens=8, vocab=100, dim=64, hidden=A, hidden_stride=64, weight=A + 16 * MiB,
             weight_stride=64, dtype=_abi.ZERO_LOSS_BF16, reserved=0)
    d.update(kw)
    return _abi.zero_head(**d)


def xent(**kw):
    d = dict(target=A + 32 * MiB, index_dtype=_abi.ZERO_INDEX_I64, reserved=0, ignore_index=-100,
             label_smoothing=0.0, z_loss=0.0)
    d.update(kw)
    return _abi.zero_xent_params(**d)


def distill(**kw):
    d = dict(index=A + 32 * MiB, logit=A + 48 * MiB, index_stride=4, logit_stride=4, k=4,
             index_dtype=_abi.ZERO_INDEX_I32, logit_dtype=_abi.ZERO_LOSS_F32, reserved=0,
             temperature=2.0)
    d.update(kw)
    return _abi.zero_distill_params(**d)


def grads(**kw):
    d = dict(upstream=A + 64 * MiB, upstream_stride=1, dhidden=A + 80 * MiB, dhidden_stride=64,
             dweight=A + 96 * MiB, dweight_stride=64)
    d.update(kw)
    return _abi.zero_head_grads(**d)


LOSS, LSE, LOGIT, WS = A + 112 * MiB, A + 128 * MiB, A + 144 * MiB, A + 1024 * MiB
BIG = 1 << 40


def refused(st, words):
    assert st == _abi.ZERO_EINVAL
    assert words in lib.zero_last_error().decode(), lib.zero_last_error().decode()


def call_xent(h, p, loss=LOSS, lse=LSE, ws=WS, n=BIG):
    return lib.zero_linear_xent(C.byref(h), C.byref(p), loss, lse, ws, n, None)


def call_xent_grad(h, p, g, lse=LSE, ws=WS, n=BIG):
    return lib.zero_linear_xent_grad(C.byref(h), C.byref(p), lse, C.byref(g), ws, n, None)


def call_distill(h, p, loss=LOSS, lse=LSE, logit=LOGIT, ws=WS, n=BIG):
    return lib.zero_linear_distill(C.byref(h), C.byref(p), loss, lse, logit, ws, n, None)


def call_distill_grad(h, p, g, lse=LSE, logit=LOGIT, ws=WS, n=BIG):
    return lib.zero_linear_distill_grad(C.byref(h), C.byref(p), lse, logit, C.byref(g), ws, n,
                                        None)


@pytest.mark.parametrize("kw,words", [
    (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 20) + 1), "tokens"), (dict(vocab=0), "vocab"),
    (dict(vocab=(1 << 24) + 1), "vocab"), (dict(dim=0), "dim"), (dict(dim=(1 << 16) + 1), "dim"),
    (dict(hidden_stride=63), "hidden_stride"), (dict(weight_stride=63), "weight_stride"),
    (dict(weight_stride=(1 << 32) + 1), "weight_stride"), (dict(hidden=None), "hidden is NULL"),
    (dict(weight=None), "weight is NULL"), (dict(hidden=A + 1), "aligned"),
    (dict(weight=A + 1), "aligned"), (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"),
    (dict(reserved=1), "reserved")], ids=str)
def test_head_refusals(kw, words):
    h = head(**kw)
    out = C.c_size_t()
    refused(lib.zero_loss_workspace_bytes(C.byref(h), 1, C.byref(out)), words)
    refused(call_xent(h, xent()), words)
    refused(call_xent_grad(h, xent(), grads()), words)
    refused(call_distill(h, distill()), words)
    refused(call_distill_grad(h, distill(), grads()), words)


@pytest.mark.parametrize("kw,words", [
    (dict(target=None), "target is NULL"), (dict(target=A + 4), "aligned"),
    (dict(index_dtype=2), "index_dtype"), (dict(label_smoothing=1.0), "label_smoothing"),
    (dict(label_smoothing=-0.1), "label_smoothing"),
    (dict(label_smoothing=math.nan), "label_smoothing"), (dict(z_loss=-1.0), "z_loss"),
    (dict(z_loss=math.inf), "z_loss"), (dict(z_loss=1e39), "z_loss"),
    (dict(label_smoothing=1.0 - 2.0 ** -40), "label_smoothing"),
    (dict(reserved=1), "reserved")], ids=str)
def test_xent_refusals(kw, words):
    refused(call_xent(head(), xent(**kw)), words)
    refused(call_xent_grad(head(), xent(**kw), grads()), words)


@pytest.mark.parametrize("kw,words", [
    (dict(index=None), "NULL"), (dict(logit=None), "NULL"), (dict(index=A + 2), "aligned"),
    (dict(logit=A + 2), "aligned"), (dict(k=0), "k must be"), (dict(k=1025), "k must be"),
    (dict(index_stride=3), "index_stride"), (dict(logit_stride=3), "logit_stride"),
    (dict(index_dtype=7), "index_dtype"), (dict(logit_dtype=7), "logit_dtype"),
    (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
    (dict(temperature=math.nan), "temperature"), (dict(temperature=1e-60), "temperature"),
    (dict(reserved=1), "reserved")], ids=str)
def test_distill_refusals(kw, words):
    refused(call_distill(head(), distill(**kw)), words)
    refused(call_distill_grad(head(), distill(**kw), grads()), words)


@pytest.mark.parametrize("kw,words", [
    (dict(dhidden=None, dweight=None), "both NULL"), (dict(upstream=None), "upstream is NULL"),
    (dict(upstream=A + 2), "upstream"), (dict(upstream_stride=-1), "upstream_stride"),
    (dict(dhidden=A + 1), "aligned"), (dict(dweight=A + 1), "aligned"),
    (dict(dhidden_stride=63), "dhidden_stride"), (dict(dweight_stride=63), "dweight_stride"),
    (dict(dhidden=A), "dhidden overlaps hidden"), (dict(dweight=A + 16 * MiB), "overlaps weight"),
    (dict(dweight=A + 80 * MiB + 512), "overlaps"), (dict(dweight=LSE), "overlaps lse"),
    (dict(dweight=A + 64 * MiB), "overlaps upstream"),
    (dict(dhidden=A + 32 * MiB), "overlaps"), (dict(dhidden=WS + 4096), "overlaps")], ids=str)
def test_gradient_refusals(kw, words):
    refused(call_xent_grad(head(), xent(), grads(**kw)), words)
    refused(call_distill_grad(head(), distill(), grads(**kw)), words)


def test_null_structs_outputs_and_workspace():
    h, p, q, g = head(), xent(), distill(), grads()
    refused(lib.zero_linear_xent(None, C.byref(p), LOSS, LSE, WS, BIG, None), "head is NULL")
    refused(lib.zero_linear_xent(C.byref(h), None, LOSS, LSE, WS, BIG, None), "params is NULL")
    refused(lib.zero_linear_distill(C.byref(h), None, LOSS, LSE, LOGIT, WS, BIG, None), "params")
    refused(lib.zero_linear_xent_grad(C.byref(h), C.byref(p), LSE, None, WS, BIG, None), "grads")
    refused(lib.zero_loss_workspace_bytes(C.byref(h), 0, None), "bytes is NULL")
    for kw, words in ((dict(loss=None), "loss"), (dict(lse=None), "lse"), (dict(ws=None), "works"),
                      (dict(ws=WS + 16), "256-byte"), (dict(n=1000), "workspace holds"),
                      (dict(loss=LSE + 8), "overlaps"), (dict(lse=A + 32 * MiB), "overlaps target"),
                      (dict(loss=LOSS + 2), "aligned"), (dict(ws=A & ~255), "overlaps")):
        refused(call_xent(h, p, **kw), words)
    refused(call_distill(h, q, logit=None), "logit is NULL")
    refused(call_distill(h, q, logit=LOSS), "overlaps")
    refused(call_distill_grad(h, q, g, logit=None), "logit is NULL")
    refused(call_xent_grad(h, p, g, lse=None), "lse is NULL")
    refused(call_xent_grad(h, p, g, n=1000), "workspace holds")


def test_interleaved_columns_do_not_overlap():
    """dhidden beside hidden in one pitched buffer passes that check and is
    refused only for the workspace, which is looked at before it."""
    h = head(hidden=A, hidden_stride=160)
    refused(call_xent_grad(h, xent(), grads(dhidden=A + 80 * 2, dhidden_stride=160,
                                            dweight=A + 16 * MiB)), "dweight overlaps weight")
    refused(call_xent_grad(h, xent(), grads(dhidden=A + 60 * 2, dhidden_stride=160)),
            "dhidden overlaps hidden")
    # the last columns of a row against the first of the next
    refused(call_xent_grad(h, xent(), grads(dhidden=A + 100 * 2, dhidden_stride=160)),
            "dhidden overlaps hidden")


def test_empty_calls_touch_nothing():
    h = head(tokens=0, hidden=None)
    assert call_xent(h, xent(target=None), None, None, None, 0) == _abi.ZERO_OK
    assert call_distill(h, distill(index=None, logit=None), None, None, None, None, 0) \
        == _abi.ZERO_OK


def test_workspace_is_far_below_the_logits():
    """8192 tokens x 131072: the logits would be 4 GiB in fp32."""
    out = C.c_size_t()
    h = head(tokens=8192, vocab=131072, dim=4096, hidden_stride=4096, weight_stride=4096)
    assert lib.zero_loss_workspace_bytes(C.byref(h), 0, C.byref(out)) == _abi.ZERO_OK
    assert out.value < 512 * MiB
    assert lib.zero_loss_workspace_bytes(C.byref(h), 1, C.byref(out)) == _abi.ZERO_OK
    assert out.value < 1024 * MiB


def test_python_refuses_host_tensors_and_wrong_shapes():
    c = make(4, 10, 8, "bf16", seed=0, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        losses.linear_xent(c["hidden"], c["weight"], c["target"])
    with pytest.raises(TypeError):
        losses.linear_xent(None, c["weight"], c["target"])
    with pytest.raises(ValueError, match="GPU"):
        losses.linear_distill(c["hidden"], c["weight"], c["target"][:, None], c["hidden"][:, :1])


@pytest.mark.parametrize("smoothing", [0.0, 0.2])
def test_reference_xent_is_torchs(smoothing):
    c = make(20, 30, 16, "fp32", seed=1, device="cpu")
    h = c["hidden"].double().requires_grad_()
    w = c["weight"].double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(h @ w.T, c["target"], reduction="none",
                                             label_smoothing=smoothing)
    (loss * c["up"].double()).sum().backward()
    r = reference(c, smoothing=smoothing)
    assert torch.allclose(r[0], loss.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(r[2], h.grad, rtol=1e-11, atol=1e-13)
    assert torch.allclose(r[3], w.grad, rtol=1e-11, atol=1e-13)


def test_reference_distill_is_torchs():
    c = make(20, 30, 16, "fp32", seed=2, device="cpu", ignored=0.0, k=6)
    c["index"] = torch.stack([torch.randperm(30, generator=torch.Generator().manual_seed(i))[:6]
                              for i in range(20)])
    h = c["hidden"].double().requires_grad_()
    w = c["weight"].double().requires_grad_()
    tau = 2.0
    p = torch.softmax(c["logit"].double() / tau, 1)
    q = torch.log_softmax(h @ w.T / tau, 1).gather(1, c["index"])
    loss = tau ** 2 * torch.nn.functional.kl_div(q, p, reduction="none").sum(1)
    (loss * c["up"].double()).sum().backward()
    r = reference(c, temperature=tau)
    assert torch.allclose(r[0], loss.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(r[2], h.grad, rtol=1e-11, atol=1e-13)
    assert torch.allclose(r[3], w.grad, rtol=1e-11, atol=1e-13)


def test_host_layer_under_sanitizers(tmp_path):
    """zero_loss_abi.cpp with stub launchers over random shapes
    (tests/sanitize/loss_driver.cpp), with AddressSanitizer and
    UndefinedBehaviorSanitizer."""
    import os
    from test_sanitizers import ROOT, _build_and_run
    csrc = os.path.join(ROOT, "zero_sharded_optimizer_amd", "csrc")
    out = _build_and_run(tmp_path, "loss_driver",
                         [os.path.join(ROOT, "tests", "sanitize", "loss_driver.cpp"),
                          os.path.join(csrc, "zero_loss_abi.cpp"),
                          os.path.join(csrc, "zero_abi.cpp")],
                         includes=[os.path.join(ROOT, "include"), csrc])
    assert "0 failures" in out


def test_header_is_plain_c(tmp_path):
    import os
    import shutil
    import subprocess
    from test_sanitizers import ROOT
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    src = tmp_path / "h.c"
    src.write_text('#include "zero_loss.h"\nint main(void) { return sizeof(zero_head) != 64 || '
                   'sizeof(zero_xent_params) != 40 || sizeof(zero_distill_params) != 56 || '
                   'sizeof(zero_head_grads) != 48; }\n')
    exe = str(tmp_path / "h")
    r = subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror",
                        f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe]).returncode == 0
    for c_type, size in ((_abi.zero_head, 64), (_abi.zero_xent_params, 40),
                         (_abi.zero_distill_params, 56), (_abi.zero_head_grads, 48)):
        assert C.sizeof(c_type) == size
