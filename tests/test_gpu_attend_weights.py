"""paged_attention where one token stands far above many: what the many weigh together is in the answer, not only
in the total.

Tolerance. A weight enters its product as fp16 (bf16 beside a bf16 cache) in one or two parts. Where it is subnormal it is
off by half of fp16's last step, 2^-25, and the largest weight that a warp has met is at 2^5 or above: so by 2^-30
of the largest, here 1, for each token. The rest is what the parts lose of each weight, 2^-11 (one fp16 part: half of eps, 2^-10), 2^-21
(two, of 2^-22) or 2^-17 (two of bf16, of 2^-18), 2^-18 of everything for logits of at most
2^5 in 32 bits, exp2 and the sums of equal numbers, and the rounding of the result."""
import math

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16
KINDS = [("none", BF16), ("none", F16), ("per_token", BF16), ("per_token", F16)]


@pytest.mark.parametrize("fmt,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nats,n", [(13.0, 4096), (16.0, 32768), (17.5, 32768), (20.0, 131072)])
def test_many_small_weights_behind_a_large_one(fmt, dtype, D, nats, n):
    """Every 16th of the first 128 tokens, one at least for each warp of the CTA that takes them, `nats` above all others; the values of those are 0
    and of the others 1, so that the answer is what the small weights come to. One CTA, or two, sums them all."""
    P = 64
    pages = n // P
    high = torch.arange(0, 128, 16)
    k, v = torch.zeros(2, pages, 1, P, D)
    v.fill_(1.0)
    k[high // P, 0, high % P, 0], v[high // P, 0, high % P] = 1.0, 0.0
    ks = vs = None
    if fmt == "none":
        k, v = k.to(dtype), v.to(dtype)
    else:
        k, v = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (k, v))
        ks, vs = torch.ones(2, pages, 1, P, device=DEV)
    q = torch.zeros(1, 1, D, dtype=dtype)
    q[..., 0] = nats
    table = torch.arange(pages, dtype=torch.int32).view(1, -1)
    assert sgq.attention_workspace_bytes(fmt, 1, 1, 1, D, pages, P) > 0 or n < 8192
    many, few = float(n - len(high)), float(len(high))
    total = many * math.exp(-nats) + few
    want = torch.full((1, 1, D), many * math.exp(-nats) / total, dtype=torch.float64)
    parts = {("none", BF16): 2.0 ** -17, ("none", F16): 2.0 ** -21, ("per_token", BF16): 2.0 ** -11, ("per_token", F16): 2.0 ** -21}[fmt, dtype]
    floor = 0.0 if (fmt, dtype) == ("none", BF16) else 2.0 ** -30
    tol = want * (parts + 2.0 ** -18) + floor * many / total
    tol = tol + ref.rounding(want + tol, dtype)
    binding.set_sm_budget(1)
    try:
        out, lse = sgq.paged_attention(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), fmt=fmt, k_scale=ks,
                                       v_scale=vs, scale=1.0, lse=True)
    finally:
        binding.set_sm_budget(0)
    assert abs(lse.item() - nats - math.log(total)) <= 2.0 ** -18 * 20
    ref.check(out.cpu(), want, tol)
