"""Calls of the ragged-group entry points beside other work on the device."""
import pytest
import torch

import group_ref as ref
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


@pytest.mark.parametrize("used", [1, 8, 600])
@pytest.mark.parametrize("T", [512, 513, 2000])
def test_lora_with_most_adapters_not_in_use(T, used):
    """The slots of a batch on a table of 600 adapters, on either side of the step from one form to the other."""
    G, R, K, N = 600, 16, 136, 264
    r = ref.gen(T + used)
    ids = torch.randperm(G, generator=r)[:used][torch.randint(0, used, (T,), generator=r)].to(torch.int32)
    x, y = torch.randn(T, K, generator=r).to(torch.bfloat16), torch.randn(T, N, generator=r).to(torch.bfloat16)
    a, b = (torch.randn(G, R, K, generator=r) / 8).to(torch.bfloat16), torch.randn(G, N, R, generator=r).to(torch.bfloat16)
    off, rows, slots = ref.group_rows(ids.view(T, 1), G)
    assert (sgq.lora_workspace_bytes(T, G, R) == 0) == (T <= 512)
    res, tol = ref.lora(x, a, b, y, off, rows, slots.view(-1), None, T)
    dx, da, db, dy, doff, drows, dslots = [t.to(DEV) for t in (x, a, b, y, off, rows, slots)]
    ref.check(sgq.lora_add(dx, da, db, dy, doff, rows=drows, slots=dslots).cpu(), res, tol)
