"""Windows of any size, without a GPU: one beyond every sequence is none, up to the largest number that the call takes and beyond it; and
the workspace of calls that are refused."""
import pytest
import torch

import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import cache


@pytest.mark.parametrize("fmt,code", [("none", 3), ("per_token", 2)])
@pytest.mark.parametrize("window", [1 << 31, (1 << 62) + 1, (1 << 63) - 130, (1 << 63) - 64, (1 << 63) - 2, (1 << 63) - 1])
def test_a_window_beyond_every_sequence_is_none(sgq_lib, fmt, code, window):
    ws = cache._lib().sgq_attention_workspace_bytes
    for sizes in ((2, 8, 4, 64, 6250, 16), (1, 8, 8, 128, 1 << 20, 64), (3, 8, 2, 256, 2, 16)):
        assert ws(code, *sizes, window) == ws(code, *sizes, 0)
        assert sgq.attention_workspace_bytes(fmt, *sizes, window) == ws(code, *sizes, 0)


def test_windows_no_64_bits_hold(sgq_lib):
    want = sgq.attention_workspace_bytes("none", 2, 8, 4, 64, 6250, 16)
    assert want > 0
    for window in (1 << 63, (1 << 64) + 5, 1 << 70):
        assert sgq.attention_workspace_bytes("none", 2, 8, 4, 64, 6250, 16, window) == want
    q, c = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(8, 4, 16, 64, dtype=torch.bfloat16)
    table, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for window in (-1, -(1 << 63), -(1 << 64) + 5):
        assert sgq.attention_workspace_bytes("none", 2, 8, 4, 64, 6250, 16, window) == 0
        with pytest.raises(sgq.SgqError, match="window"):
            sgq.paged_attention(q, c, c.clone(), table, n, window=window)


def test_calls_that_are_refused_have_no_workspace(sgq_lib):
    """Formats that a cache does not have, heads whose rows are no whole pieces."""
    ws = cache._lib().sgq_attention_workspace_bytes
    sizes = (2, 8, 4)
    assert ws(3, *sizes, 72, 6250, 16, 0) > 0 and ws(2, *sizes, 80, 6250, 16, 0) > 0
    for fmt in (-1, 0, 1, 4, 7):
        assert ws(fmt, *sizes, 64, 6250, 16, 0) == 0
    for fmt, D in ((3, 60), (3, 4), (3, 0), (2, 72), (2, 8), (3, 264), (2, 272)):
        assert ws(fmt, *sizes, D, 6250, 16, 0) == 0
