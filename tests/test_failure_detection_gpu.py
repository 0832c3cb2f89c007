"""Failure detection without faulting the GPU.

Every wait inside the tensor-core prefill is bounded.  A test switch, read by the
library when it loads, makes the MMA issuer of the process's first tensor-core call
withhold one completion, so the waits behind it run out after a short limit: the
kernel must record a timeout in its workspace (read back as LIGER_ERR_TIMEOUT, with
the site of the first wait that gave up), drain, free its tensor memory and return --
and the CUDA context must stay usable for a normal call right after.  The switch is
set in a child process so that it never reaches the other tests."""
import pytest

from tests import child_scenarios

pytestmark = pytest.mark.gpu


def test_bounded_wait_reports_timeout_and_context_survives(cuda_device):
    out = child_scenarios.run("stall_then_recover", child_scenarios.STALL_ENV)
    assert "timeout reported" in out


def test_cached_attention_reports_timeouts_and_context_survives(cuda_device):
    """The same for the cached attention, whose first two calls never announce the first CTA's first tile."""
    out = child_scenarios.run("cached_stall", {**child_scenarios.STALL_ENV, "LIGER_TEST_INJECT_STALL": "2"})
    assert "cached attention timeouts reported" in out
