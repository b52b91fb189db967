"""Arguments of the loss operators whose double is in range and whose float is not, on
the CPU: what the kernels compute with is what is checked."""
import ctypes as C
import math
import os

import pytest

from zero_sharded_optimizer_amd import _abi
from test_sanitizers import ROOT, _build_and_run
from test_loss_host import call_distill, call_distill_grad, distill, grads, head, refused

lib = _abi.load()


@pytest.mark.parametrize("t", [1e39, 1e30, 1.9e19, 1.0e-19, 1e-30, 4e-39, math.inf])
def test_temperatures_out_of_range(t):
    refused(call_distill(head(), distill(temperature=t)), "temperature")
    refused(call_distill_grad(head(), distill(temperature=t), grads()), "temperature")


@pytest.mark.parametrize("t", [1.8e19, 1.1e-19, 0.5, 100.0])
def test_temperatures_in_range(t):
    """Looked at before the workspace, which is too small here."""
    refused(call_distill(head(), distill(temperature=t), n=1000), "workspace holds")
    refused(call_distill_grad(head(), distill(temperature=t), grads(), n=1000), "workspace holds")


def test_plans_under_sanitizers(tmp_path):
    """zero_loss_abi.cpp with stub launchers (tests/sanitize/loss_plan_driver.cpp), with
    AddressSanitizer and UndefinedBehaviorSanitizer: distillation's entry points, and the
    tiles and launches of every plan."""
    csrc = os.path.join(ROOT, "zero_sharded_optimizer_amd", "csrc")
    out = _build_and_run(tmp_path, "loss_plan_driver",
                         [os.path.join(ROOT, "tests", "sanitize", "loss_plan_driver.cpp"),
                          os.path.join(csrc, "zero_loss_abi.cpp"),
                          os.path.join(csrc, "zero_abi.cpp")],
                         includes=[os.path.join(ROOT, "include"), csrc])
    assert "0 failures" in out
