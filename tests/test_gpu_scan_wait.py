"""The gated recurrence's wait for its neighbours' maps ends after its limit, is
reported, and leaves the context usable."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_scan_wait_timeout_reports_and_context_survives():
    import video_vit_encoder_gb300 as jg
    from video_vit_encoder_gb300._lib import ERR_ARG, ERR_DEVICE_TIMEOUT
    gv = torch.randn(1, 2000, 128, device="cuda")
    want = jg.gated_scan_fwd(gv)
    assert jg.selftest_scan_wait_timeout(200) == ERR_DEVICE_TIMEOUT
    jg.ops_sync()      # reported once
    for a, b in zip(jg.gated_scan_fwd(gv), want):
        assert torch.equal(a, b)
    assert jg.selftest_scan_wait_timeout(0) == ERR_ARG
    jg.ops_sync()
