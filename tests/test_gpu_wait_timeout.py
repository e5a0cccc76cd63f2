"""The bounded wait of a whole warp: when some lanes find the phase complete and others give up, all give up (the
self-test reports BLINK_DEVICE_FLAG otherwise), and the library's kernels run on as before."""
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [1, 100, 20000])
def test_a_warp_gives_up_together(limit_us):
    ws = blink.new_workspace(256, "cuda")
    assert blink.blink_selftest_wait_timeout(limit_us, ws) == blink.BLINK_DEVICE_TIMEOUT
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    h = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    r = blink.blink_token_logprobs(h, torch.zeros(500, 64, dtype=torch.bfloat16, device="cuda"), top=2)
    assert r["top_ids"].tolist() == [[0, 1]] * 3
