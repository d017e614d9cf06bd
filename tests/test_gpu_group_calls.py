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


@pytest.mark.parametrize("R", [64, 128])
def test_lora_with_the_largest_table_of_adapters(R):
    G, T, K, N = 1024, 700, 72, 392
    r = ref.gen(R)
    ids = torch.where(torch.rand(T, generator=r) < 0.5, 1023, torch.randint(-1, G, (T,), generator=r)).to(torch.int32)
    x, y = torch.randn(T, K, generator=r).to(torch.bfloat16), torch.randn(T, N, generator=r).to(torch.bfloat16)
    a, b = (torch.randn(G, R, K, generator=r) / 8).to(torch.bfloat16), torch.randn(G, N, R, generator=r).to(torch.bfloat16)
    off, rows, slots = ref.group_rows(ids.view(T, 1), G)
    res, tol = ref.lora(x, a, b, y, off, rows, slots.view(-1), None, T)
    dx, da, db, dy, doff, drows, dslots = [t.to(DEV) for t in (x, a, b, y, off, rows, slots)]
    ref.check(sgq.lora_add(dx, da, db, dy, doff, rows=drows, slots=dslots).cpu(), res, tol)


@pytest.mark.parametrize("fmt", ["mxfp8", "block128", "per_token", "none"])
@pytest.mark.parametrize("T", [9, 400])
def test_experts_of_one_rank(T, fmt):
    """Ids of 32 experts of which 8 to 11 are here: most slots belong to no group, and the sum passes over them."""
    k, G, N, K = 4, 4, 200, 256
    r = ref.gen(T)
    ids = torch.stack([torch.randperm(32, generator=r)[:k] for _ in range(T)]).to(torch.int32) - 8
    off, rows, slots = ref.group_rows(ids, G)
    S = T * k
    x, xs, w, ws = ref.operands(fmt, T, G, N, K, T)
    want, tol = ref.grouped_gemm(fmt, x, xs, w, ws, off, rows, S, torch.zeros(S, N), torch.bfloat16)
    laid = ref.swizzled(ws) if fmt == "mxfp8" else ws
    dx, dxs, dw, dws = [None if t is None else t.to(DEV) for t in (x, xs, w, laid)]
    o, rw, sl = sgq.group_rows(ids.to(DEV), G)
    out = torch.full((S, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    sgq.grouped_gemm(dx, dw, o, fmt=fmt, x_scale=dxs, w_scale=dws, rows=rw, out=out)
    n = int(off[-1])
    assert torch.equal(o.cpu(), off) and torch.equal(sl.cpu(), slots) and n < S
    ref.check(out[:n].cpu(), want[:n], tol[:n], fmt)
    assert out[n:].isnan().all()
    weights = torch.rand(T, k, generator=r)
    res, tol = ref.combine(out.cpu(), slots, weights, torch.bfloat16)
    ref.check(sgq.combine_rows(out, sl, weights.to(DEV)).cpu(), res, tol)


@pytest.mark.parametrize("a,b", [(254, 0), (0, 254), (0, 0), (0, 117), (117, 0), (60, 57), (60, 54), (0, 127), (254, 120), (254, 121), (254, 254)])
def test_mxfp8_scales_at_the_ends_of_their_range(a, b):
    """128 terms 2^(a + b - 254) of one sign: the sum rounded once, subnormal results too, infinity beyond the type's range."""
    one = torch.full((1,), 0x38, dtype=torch.uint8, device=DEV)              # 1.0
    x, w = one.expand(8, 128).contiguous(), one.expand(1, 64, 128).contiguous()
    xs = torch.full((8, 4), a, dtype=torch.uint8, device=DEV)
    ws = torch.full((1, 128, 4), b, dtype=torch.uint8, device=DEV)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    want = torch.tensor(2.0 ** (a + b - 254 + 7), dtype=torch.float64).to(torch.bfloat16)
    for negative in (False, True):
        got = sgq.grouped_gemm(x | (0x80 if negative else 0), w, off, x_scale=xs, w_scale=ws).cpu()
        assert (got == (-want if negative else want)).all()
