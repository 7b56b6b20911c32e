"""The bounded waits give up by the limit they are given, and no sooner."""
import time

import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("timeout_us", [1000, 50000, 300000])
def test_every_wait_gives_up_at_its_limit(timeout_us):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_selftest_bounded_wait(status, timeout_us=100)  # the kernel's load is not timed
    torch.cuda.synchronize()
    status.zero_()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    pkv.pkv_selftest_bounded_wait(status, timeout_us=timeout_us)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    # all three at once: their limit, and what a launch and a poll may add
    assert timeout_us * 1e-6 * 0.98 <= took <= timeout_us * 1e-6 + 0.2
    assert pkv.pkv_read_status(status) == pkv.PKV_DEV_TIMEOUT
