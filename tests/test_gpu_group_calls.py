"""Calls of the ragged-group entry points beside other work on the device."""
import pytest
import torch

import swiglu_fp8_activation_gb300 as sgq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_wait_timeouts_waits_for_every_stream():
    """A stream that does not block the default one still runs when the count is asked for."""
    sgq.wait_timeouts()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)           # some 0.2 s of the device's clock
    assert not st.query()
    assert sgq.wait_timeouts() == 0
    assert st.query()
