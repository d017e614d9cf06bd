"""How many bits the products over ragged groups keep: long sums of
grouped_gemm in every plan, and lora_add's factor v in both of its forms
(group_ref.py derives what is allowed; test_group_ref.py shows on the CPU that
fewer bits fail)."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("few", [False, True], ids=["many slots an adapter", "few slots an adapter"])
def test_lora_keeps_v_in_fp32(few, R, dtype):
    """v whose last bits alone reach y, in sums that are exact in fp32: y is the result rounded once, bit for bit."""
    T, N, K = 300, 264, 64
    x, a, b, res = ref.exact_lora(T, R, N, K, dtype, R)
    G = 1
    if few:
        T = min(128, 8192 // R)
        G, x, res = (T * R + 127) // 128, x[:T].contiguous(), res[:T]
    off = torch.tensor([0] + [T] * G, dtype=torch.int32)
    assert (sgq.lora_workspace_bytes(T, G, R) == 0) == few
    y = torch.zeros(T, N, dtype=dtype, device=DEV)
    sgq.lora_add(x.to(DEV), a.expand(G, R, K).contiguous().to(DEV), b.expand(G, N, R).contiguous().to(DEV), y, off.to(DEV))
    assert torch.equal(y.cpu(), res.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [40, 128])
def test_lora_many_tiles_a_cta(R, dtype):
    """Two CTAs that walk over many sets of slots and columns of each: every set's v stays until its last product."""
    T, N, K = 1500, 1160, 64
    x, a, b, res = ref.exact_lora(T, R, N, K, dtype, R + 1)
    off = torch.tensor([0, 400, 401, 401, T], dtype=torch.int32)
    y = torch.zeros(T, N, dtype=dtype, device=DEV)
    dx, da, db, doff = x.to(DEV), a.expand(4, R, K).contiguous().to(DEV), b.expand(4, N, R).contiguous().to(DEV), off.to(DEV)
    binding.set_sm_budget(2)
    try:
        sgq.lora_add(dx, da, db, y, doff)
    finally:
        binding.set_sm_budget(0)
    assert torch.equal(y.cpu(), res.to(dtype))
