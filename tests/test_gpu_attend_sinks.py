"""paged_attention's sinks at the ends of 32 bits: where a sequence has no token the answer is zeros and lse the sink itself; a sink
above every logit takes all the weight, one below it none."""
import math

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16
KINDS = [("none", BF16), ("none", F16), ("per_token", BF16), ("per_token", F16)]
MOST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("form", ["clusters", "one CTA", "shares"])
def test_sinks_at_the_ends_of_32_bits(fmt, dtype, form):
    sinks = torch.tensor([-math.inf, -MOST, -3.0e38, -2.1e38, -1.0e30, -87.3, 0.1, 1.0e30, 2.0e38, 2.5e38, MOST, 1.7])
    lengths, heads, P, D = [0, 40, 0, 700, 1] if form != "one CTA" else [0, 40, 0, 30, 1], 2, 16, 64
    table, pages = ref.table_of(lengths, P)
    k, v, ks, vs = ref.pool(fmt, pages, heads, P, D, dtype, 0)
    q = torch.randn(5, len(sinks), D, generator=ref.gen(1)).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n, sinks=sinks)
    if form == "shares":
        table = torch.nn.functional.pad(table, (0, 4000), value=-1)
    assert (sgq.attention_workspace_bytes(fmt, 5, len(sinks), heads, D, table.shape[1], P) > 0) == (form == "shares")
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out, lse = sgq.paged_attention(*map(on, (q, k, v, table, n)), fmt=fmt, k_scale=on(ks), v_scale=on(vs), sinks=on(sinks), lse=True)
    out, lse = out.cpu(), lse.cpu()
    assert torch.equal(lse[n == 0], sinks.expand(2, -1))
    some = n > 0
    assert torch.isfinite(lse[some]).all()
    ref.check(lse[some], wl[some], tl[some], "lse")
    ref.check(out, want, tol, "out")
