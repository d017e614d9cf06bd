"""paged_attention over E4M3 rows whose scales lie far apart, at logits that are alike or far apart: the
softmax's total counts every row, whatever the row of v is scaled by. Against the plain 64-bit form, with the
tolerances derived in cache_ref.py."""
import math

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16
P, D, HEADS, GROUP = 16, 64, 2, 4


def rows(lengths, dtype, seed, k_size, v_scale):
    """A cache for sequences of these lengths in which token t's k codes are multiplied by k_size(t) and its v scale is v_scale(t)
    (0: a row of zeros); (table, k, v, k_scale, v_scale)."""
    table, pages = ref.table_of(lengths, P, seed=seed)
    k, v, ks, vs = ref.pool("per_token", pages, HEADS, P, D, dtype, seed)
    for b, n in enumerate(lengths):
        for t in range(n):
            at = (table[b, t // P].item(), slice(None), t % P)
            ks[at] *= k_size(t)
            vs[at] = v_scale(t)
            if v_scale(t) == 0:
                v[at] = 0
    return table, k, v, ks, vs


def calls(q, k, v, ks, vs, table, n):
    """(out, lse) by clusters that take an item each, by shares of all CTAs and by shares of a few."""
    on = lambda *ts: [t.to(DEV) for t in ts]  # noqa: E731
    dq, dk, dv, dks, dvs, dt, dn = on(q, k, v, ks, vs, table, n)
    wide = torch.nn.functional.pad(dt, (0, -(-60000 // P)), value=-1)
    kw = dict(fmt="per_token", k_scale=dks, v_scale=dvs, lse=True)
    assert sgq.attention_workspace_bytes("per_token", len(n), q.shape[1], HEADS, D, table.shape[1], P) == 0
    assert sgq.attention_workspace_bytes("per_token", len(n), q.shape[1], HEADS, D, wide.shape[1], P) > 0
    yield "clusters", *(t.cpu() for t in sgq.paged_attention(dq, dk, dv, dt, dn, **kw))
    yield "shares", *(t.cpu() for t in sgq.paged_attention(dq, dk, dv, wide, dn, **kw))
    binding.set_sm_budget(1)
    try:
        yield "few shares", *(t.cpu() for t in sgq.paged_attention(dq, dk, dv, wide, dn, **kw))
    finally:
        binding.set_sm_budget(0)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_zeros_at_logits_far_above_the_others(dtype):
    """Rows of v of zeros, whose scale is 0, 84 to 88 nats above ordinary rows before them: they are the total, and the answer is
    what the others weigh beside them, e^-84 of 448 at most."""
    lengths, low = [700, 400], 200
    table, k, v, ks, vs = rows(lengths, dtype, 1, lambda t: 0.0 if t < low else 1.0, lambda t: 1.0 if t < low else 0.0)
    k[:] = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8)                   # each row the same: logits of 0, or of sum(q) * scale
    ks[:] = (ks > 0).float()
    q = torch.zeros(2, HEADS * GROUP, D)
    q[..., 0] = torch.linspace(84.0, 88.0, HEADS * GROUP)
    q = q.to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    at = q[..., 0].double()                                                              # q * 8 below, scale 1/8
    for form, out, lse in calls(q * 8, k, v, ks, vs, table, n):
        want = at + (n.double() - low).log().view(2, 1)
        assert torch.isfinite(lse).all(), form
        # x in units of log2, the total's sums and log2: 2^-20 of the size
        ref.check(lse, want, 2.0 ** -20 * want, form)
        assert (out.double().abs() <= 448 * math.exp(-84.0)).all(), form


CUTS = [(2.0 ** -60, 2.0 ** 68), (0.0, 2.0 ** 40), (0.0, 2.0 ** 98), (2.0 ** -99, 2.0 ** 99), (2.0 ** 99, 2.0 ** -99), (2.0 ** 60, 0.0)]


@pytest.mark.parametrize("first,then", CUTS)
@pytest.mark.parametrize("order", ["cut", "tiles"])
def test_totals_where_scales_lie_far_apart(first, then, order):
    """Half of the rows, or every second tile of them, scaled by one and the others by the other, at logits that are alike: out and
    lse count both."""
    lengths = [700, 130, 300]
    which = (lambda t: t < 300) if order == "cut" else (lambda t: t // 128 % 2 == 0)
    table, k, v, ks, vs = rows(lengths, BF16, 2, lambda t: 1.0, lambda t: first if which(t) else then)
    q = (torch.randn(3, HEADS * GROUP, D, generator=ref.gen(3)) * 0.2).to(BF16)
    n = torch.tensor(lengths, dtype=torch.int32)
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n)
    for form, out, lse in calls(q, k, v, ks, vs, table, n):
        ref.check(lse, wl, tl, f"{form} lse")
        ref.check(out, want, tol, form)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("small", [2.0 ** -120, 2.0 ** -100, 0.0])
def test_totals_beside_rows_of_next_to_nothing(dtype, small):
    """Rows whose scale is near the end of 32 bits, as cache_write leaves them, before ordinary ones."""
    lengths = [700, 130, 300]
    table, k, v, ks, vs = rows(lengths, dtype, 4, lambda t: 1.0, lambda t: small if t % 300 < 150 else 0.01)
    q = torch.randn(3, HEADS * GROUP, D, generator=ref.gen(5)).to(dtype)
    n = torch.tensor(lengths, dtype=torch.int32)
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n)
    for form, out, lse in calls(q, k, v, ks, vs, table, n):
        ref.check(lse, wl, tl, f"{form} lse")
        ref.check(out, want, tol, form)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -120, 2.0 ** -130, 2.0 ** -140])
def test_rows_of_next_to_nothing_alone(scale):
    """Down to subnormal scales: the answer is the rows' mean, to bf16's last step."""
    lengths = [700, 130, 300]
    table, k, v, ks, vs = rows(lengths, BF16, 6, lambda t: 1.0, lambda t: scale)
    q = torch.randn(3, HEADS * GROUP, D, generator=ref.gen(7)).to(BF16)
    n = torch.tensor(lengths, dtype=torch.int32)
    want, tol, wl, tl = ref.attention(q, k, v, ks, vs, table, n)
    for form, out, lse in calls(q, k, v, ks, vs, table, n):
        ref.check(lse, wl, tl, f"{form} lse")
        ref.check(out, want, tol, form)


def test_small_rows_that_cache_write_leaves():
    """Rows of v of every size down to bf16's subnormals, written and attended: scales as small as a subnormal number's."""
    T = 400
    r = ref.gen(8)
    k = torch.randn(T, HEADS, D, generator=r).to(BF16)
    v = (torch.randn(T, HEADS, D, generator=r) * torch.exp2(torch.linspace(-133, -90, T)).view(T, 1, 1)).to(BF16)
    v[7] = 0
    pages = -(-T // P)
    kc, vc = torch.zeros(2, pages, HEADS, P, D, dtype=torch.uint8, device=DEV)
    ks, vs = torch.zeros(2, pages, HEADS, P, device=DEV)
    sgq.cache_write(k.to(DEV), v.to(DEV), kc, vc, torch.arange(T, device=DEV), fmt="per_token", k_scale=ks, v_scale=vs)
    assert 0 < vs[vs > 0].min() < 2.0 ** -130
    table, n = torch.arange(pages, dtype=torch.int32).view(1, -1), torch.tensor([T], dtype=torch.int32)
    q = torch.randn(1, HEADS * GROUP, D, generator=r).to(BF16)
    for some in (T, 40):                                                                 # with larger rows among them, and without
        n[0] = some
        want, tol, wl, tl = ref.attention(q, kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), table, n)
        for form, out, lse in calls(q, kc, vc, ks, vs, table, n):
            ref.check(lse, wl, tl, f"{form} lse")
            ref.check(out, want, tol, form)
