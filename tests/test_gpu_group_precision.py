"""How many bits the products over ragged groups keep: long sums of
grouped_gemm in every plan (group_ref.py derives what is allowed;
test_group_ref.py shows on the CPU that fewer bits fail)."""
import pytest
import torch

import group_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FMTS = ["mxfp8", "block128", "per_token", "none"]


@pytest.mark.parametrize("K", [1024, 4480, 8192])
@pytest.mark.parametrize("sizes,N,sms", [([33], 264, 0), ([40, 60] * 4, 520, 3), ([300, 150], 392, 2)],
                         ids=["few tiles", "narrow tiles", "wide tiles"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows in order", "gathered"])
@pytest.mark.parametrize("fmt", FMTS)
def test_long_sums_are_held_in_fp32(fmt, gather, sizes, N, sms, K):
    S = sum(sizes)
    off = torch.cumsum(torch.tensor([0] + sizes), 0).to(torch.int32)
    x, xs, w, ws = ref.operands(fmt, S, len(sizes), N, K, K + S)
    rows = torch.randperm(S, generator=ref.gen(S)).to(torch.int32) if gather else None
    res, tol = ref.grouped_gemm(fmt, x, xs, w, ws, off, rows, S, torch.zeros(S, N), torch.bfloat16)
    laid = ref.swizzled(ws) if fmt == "mxfp8" else ws
    dx, dxs, dw, dws, doff, drows = [None if t is None else t.to(DEV) for t in (x, xs, w, laid, off, rows)]
    binding.set_sm_budget(sms)
    try:
        got = sgq.grouped_gemm(dx, dw, doff, fmt=fmt, x_scale=dxs, w_scale=dws, rows=drows).cpu()
    finally:
        binding.set_sm_budget(0)
    ref.check(got, res, tol, fmt)
    limit = ref.misrounded_limit(res, ref.spread(fmt, x, xs, w, ws, off, rows, S), K, torch.bfloat16)
    assert ref.misrounded(got, res) <= limit, (ref.misrounded(got, res), limit)
