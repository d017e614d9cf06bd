"""The checks of the ragged-group operators' precision (group_ref.py) on the
CPU: results whose sums or factors are kept in too few bits fail them."""
import pytest
import torch

import group_ref as ref

FMTS = ["mxfp8", "block128", "per_token", "none"]


def held(v, bits):
    """v rounded to `bits` significant bits."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 2 ** bits), e - bits)


@pytest.mark.parametrize("K", [1024, 4480, 8192])
@pytest.mark.parametrize("fmt", FMTS)
def test_sums_in_few_bits_are_found(fmt, K):
    S, N = 33, 264
    x, xs, w, ws = ref.operands(fmt, S, 1, N, K, K)
    off = torch.tensor([0, S])
    res, tol = ref.grouped_gemm(fmt, x, xs, w, ws, off, None, S, torch.zeros(S, N), torch.bfloat16)
    size = ref.spread(fmt, x, xs, w, ws, off, None, S)
    limit = ref.misrounded_limit(res, size, K, torch.bfloat16)
    xv, wv = ref.values(fmt, x, xs), ref.values(fmt, w[0], None if ws is None else ws[0], N)
    for bits in (24, 12, 11, 8):
        run = torch.zeros(S, N, dtype=torch.float64)
        for k in range(0, K, 128):
            run = held(run + xv[:, k:k + 128] @ wv[:, k:k + 128].T, bits)
        share = ref.misrounded(run.to(torch.bfloat16), res)
        assert (share > limit) == (bits < 24), (bits, share, limit)
    # eight parts of K, each rounded to 16 bits before they are added
    parts = [held(p, 11) for p in ((xv[:, i * K // 8:(i + 1) * K // 8] @ wv[:, i * K // 8:(i + 1) * K // 8].T) for i in range(8))]
    assert ref.misrounded(sum(parts).to(torch.bfloat16), res) > limit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [8, 24, 64, 72, 128])
def test_factors_in_few_bits_are_found(R, dtype):
    x, a, b, res = ref.exact_lora(20, R, 136, 64, dtype, R)
    xv, av, bv = x.double(), a[0].double(), b[0].double()
    v = xv @ av.T
    assert torch.equal(v @ bv.T, res) and torch.equal(v, v.float().double())
    assert float(v[:, :-2].abs().max()) < 128 and float(res.abs().max()) > 0
    want = res.to(dtype)
    digits = torch.finfo(dtype).bits - (8 if dtype == torch.bfloat16 else 5)      # significant bits of the type
    one = held(v, digits)
    two = one + held(v - one, digits)
    for few in (one, two) if dtype == torch.bfloat16 else (one,):
        assert float(((few @ bv.T).to(dtype) != want).double().mean()) > 0.2
