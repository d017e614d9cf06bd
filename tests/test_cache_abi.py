"""The paged cache's entry points (include/sgq_cache.h) without a GPU: exports,
host checks with the documented status before anything is launched (fake,
never dereferenced pointers), the Python entry points' refusals, and the frequencies."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import cache

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgq_cache.h")
OK, INVALID, UNSUPPORTED, MISALIGNED, LAUNCH = 0, 1, 2, 3, 4
FP16, INTERLEAVED, INVERSE = 1 << 5, 1 << 6, 1 << 7
BF16 = torch.bfloat16
STEP = 1 << 36


def P(i, off=0):
    return (1 << 44) + i * STEP + off


def test_exports_and_constants(sgq_lib):
    with open(HEADER) as f:
        text = f.read()
    names = re.findall(r"^(?:int|int64_t)\s+(\w+)\(", text, flags=re.M)
    assert {"rope", "cache_write", "cache_read", "paged_attention", "sgq_attention_workspace_bytes"} == set(names)
    for n in names:
        assert hasattr(sgq_lib, n), n
    value = lambda n: int(re.search(rf"#define {n}\s+(\d+)", text).group(1))  # noqa: E731
    assert (value("SGQ_MAX_HEAD"), value("SGQ_MAX_HEADS"), value("SGQ_MAX_PAGE"), value("SGQ_MAX_SEQUENCES")) == \
        (sgq.MAX_HEAD, sgq.MAX_HEADS, sgq.MAX_PAGE, sgq.MAX_SEQUENCES)
    shift = lambda n: 1 << int(re.search(rf"#define {n}\s+\(1u << (\d+)\)", text).group(1))  # noqa: E731
    assert shift("SGQ_F_ROPE_INTERLEAVED") == cache.F_ROPE_INTERLEAVED and shift("SGQ_F_ROPE_INVERSE") == cache.F_ROPE_INVERSE


@pytest.fixture
def L(sgq_lib):
    return cache._lib()


def refused(st):
    assert st != LAUNCH, "a fake-pointer call passed the host checks"
    return st


def heads(p=P(0), H=4, ts=256, hs=64):
    return C.byref(cache.Heads(p, H, ts, hs))


def turn(R=64, freqs=P(20), pos=P(21), pb=8, factor=1.0):
    return C.byref(cache.Rope(R, freqs, pos, pb, factor))


def kv(pages=8, size=16, H=4, D=64, ps=4096, hs=1024, ts=64, k=P(10), v=P(11), ks=None, vs=None):
    return C.byref(cache.KvCache(pages, size, H, D, ps, hs, ts, k, v, ks, vs))


def rope(L, flags=0, T=8, D=64, r=None, x=None, out=None):
    return refused(L.rope(flags, T, D, r or turn(), x or heads(), out or heads(P(1)), None))


def test_rope_refusals(L):
    assert rope(L, T=0, x=heads(None)) == OK
    assert refused(L.rope(0, 8, 64, None, heads(), heads(P(1)), None)) == INVALID
    assert refused(L.rope(0, 8, 64, turn(), None, heads(P(1)), None)) == INVALID
    assert rope(L, flags=1) == INVALID
    assert rope(L, T=-1) == INVALID
    assert rope(L, T=1 << 31) == INVALID
    assert rope(L, D=60) == UNSUPPORTED
    assert rope(L, D=264) == UNSUPPORTED
    assert rope(L, D=0) == INVALID
    assert rope(L, r=turn(R=24)) == UNSUPPORTED
    assert rope(L, r=turn(R=80)) == UNSUPPORTED          # beyond D
    assert rope(L, r=turn(R=0)) == INVALID
    assert rope(L, r=turn(pb=2)) == INVALID
    assert rope(L, r=turn(factor=math.inf)) == INVALID
    assert rope(L, r=turn(factor=math.nan)) == INVALID
    assert rope(L, r=turn(freqs=None)) == INVALID
    assert rope(L, r=turn(pos=None)) == INVALID
    assert rope(L, r=turn(freqs=P(20, 4))) == MISALIGNED
    assert rope(L, r=turn(pos=P(20, 4))) == MISALIGNED
    assert rope(L, x=heads(None)) == INVALID
    assert rope(L, x=heads(H=0)) == INVALID
    assert rope(L, x=heads(H=5)) == INVALID              # not as many as out
    assert rope(L, x=heads(H=1025), out=heads(P(1), H=1025, ts=1025 * 64)) == UNSUPPORTED
    assert rope(L, x=heads(ts=-256)) == INVALID
    assert rope(L, x=heads(ts=1 << 60)) == INVALID
    assert rope(L, x=heads(ts=260)) == MISALIGNED
    assert rope(L, x=heads(hs=68)) == MISALIGNED
    assert rope(L, x=heads(P(0, 8))) == MISALIGNED
    assert rope(L, out=heads(P(1, 8))) == MISALIGNED
    assert rope(L, out=heads(P(1), ts=128)) == INVALID   # its tokens share addresses
    assert rope(L, out=heads(P(1), hs=32, ts=512)) == INVALID
    assert rope(L, out=heads(P(0, 64))) == INVALID       # not in place, not apart
    assert rope(L, out=heads(P(0), ts=512)) == INVALID   # in place at other strides
    assert rope(L, x=heads(ts=512), out=heads(P(0, 448), ts=512)) == INVALID     # the last head's rows meet x's
    assert rope(L, out=heads(P(20))) == INVALID
    assert rope(L, out=heads(P(21, 16))) == INVALID


def write(L, fmt=3, flags=0, T=8, c=None, r=None, q=None, qo=None, k=None, v=None, slots=P(5), sb=4):
    return refused(L.cache_write(fmt, flags, T, c or kv(), r, q, qo, k or heads(P(0)), v or heads(P(1)), slots, sb, None))


def fp8(**kw):
    return kv(**{"ks": P(12), "vs": P(13), **kw})


def test_cache_refusals(L):
    """What cache_write, cache_read and paged_attention refuse of a cache."""
    calls = {"write": lambda c, fmt: write(L, fmt=fmt, c=c),
             "read": lambda c, fmt: refused(L.cache_read(fmt, 0, 8, c, P(5), 4, P(6), P(7), None)),
             "attend": lambda c, fmt: refused(L.paged_attention(fmt, 0, 2, c, heads(P(0), H=8, ts=512), P(1), 4, P(2), 1.0, 0, None, P(3), None, P(4), None))}
    for name, call in calls.items():
        no = lambda want, c, fmt=3: call(c, fmt) == want or pytest.fail(name)  # noqa: E731
        for fmt in (0, 1, 4, -1):
            no(INVALID, kv(), fmt)
        no(INVALID, kv(pages=0))
        no(INVALID, kv(pages=-1))
        no(INVALID, kv(pages=1 << 31))
        no(INVALID, kv(size=0))
        no(UNSUPPORTED, kv(size=65537))
        no(INVALID, kv(H=0))
        no(UNSUPPORTED, kv(H=1025))
        no(UNSUPPORTED, kv(D=60))
        no(UNSUPPORTED, kv(D=264))
        no(UNSUPPORTED, fp8(D=56), 2)
        no(INVALID, kv(k=None))
        no(INVALID, kv(v=None))
        no(INVALID, kv(ks=P(12), vs=P(13)))              # scales with 16-bit rows
        no(INVALID, kv(ks=P(12), vs=None), 2)
        no(INVALID, kv(ks=None, vs=P(13)), 2)
        no(MISALIGNED, kv(k=P(10, 8)))
        no(MISALIGNED, kv(ps=4100))
        no(MISALIGNED, kv(ts=68, hs=2048, ps=8192))
        no(MISALIGNED, fp8(ts=72, hs=2048, ps=8192), 2)  # 16-byte rows of codes
        no(MISALIGNED, fp8(ks=P(12, 2)), 2)
        no(INVALID, kv(ps=-4096))
        no(INVALID, kv(ps=1 << 60))
        no(UNSUPPORTED, kv(ps=1 << 39))                  # 2^40 bytes
        no(INVALID, kv(hs=512))                          # rows share addresses
        no(INVALID, kv(ts=32))
        no(INVALID, kv(v=P(10)))
        no(INVALID, kv(v=P(10, 4096)))                   # v begins inside k's pages
        no(INVALID, fp8(vs=P(12, 16)), 2)
        no(INVALID, fp8(ks=P(10, 64)), 2)


def test_cache_write_refusals(L):
    assert write(L, T=0, k=heads(None)) == OK
    assert refused(L.cache_write(3, 0, 8, None, None, None, None, heads(P(0)), heads(P(1)), P(5), 4, None)) == INVALID
    assert write(L, flags=INVERSE) == INVALID
    assert write(L, flags=INTERLEAVED) == INVALID        # without rope
    assert write(L, T=-1) == INVALID
    assert write(L, T=1 << 31) == INVALID
    assert write(L, sb=2) == INVALID
    assert write(L, slots=None) == INVALID
    assert write(L, slots=P(5, 2)) == MISALIGNED
    assert write(L, slots=P(5, 4), sb=8) == MISALIGNED
    assert write(L, q=heads(P(2)), qo=heads(P(3))) == INVALID                # without rope
    assert write(L, r=turn(), q=heads(P(2))) == INVALID                      # without q_out
    assert write(L, r=turn(), qo=heads(P(2))) == INVALID
    assert write(L, r=turn(), q=heads(P(2), H=5, ts=512), qo=heads(P(3))) == INVALID
    assert write(L, r=turn(R=80)) == UNSUPPORTED
    assert write(L, k=heads(P(0), H=3)) == INVALID       # not the cache's heads
    assert write(L, v=heads(P(1), H=8, ts=512)) == INVALID
    assert write(L, k=heads(P(0), hs=60)) == MISALIGNED
    assert write(L, k=heads(P(10, 1024))) == INVALID     # inside the cache
    assert write(L, v=heads(P(11))) == INVALID
    assert write(L, slots=P(10, 16)) == INVALID
    assert write(L, fmt=2, c=fp8(), slots=P(13)) == INVALID
    assert write(L, r=turn(), q=heads(P(2)), qo=heads(P(10))) == INVALID
    assert write(L, r=turn(), q=heads(P(11)), qo=heads(P(3))) == INVALID
    assert write(L, r=turn(freqs=P(10))) == INVALID
    assert write(L, r=turn(), q=heads(P(2)), qo=heads(P(0))) == INVALID      # over k
    assert write(L, r=turn(), q=heads(P(2)), qo=heads(P(5))) == INVALID      # over the slots
    assert write(L, r=turn(), q=heads(P(2)), qo=heads(P(2, 128))) == INVALID
    # q_out's last head over k's first, in one projection's rows
    part = lambda off: heads(P(2, off * 2), ts=1024)  # noqa: E731
    assert write(L, r=turn(), q=part(0), qo=part(192), k=part(256), v=part(512)) == INVALID


def test_read_refusals(L):
    read = lambda fmt=3, flags=0, S=8, c=None, slots=P(5), sb=4, k=P(6), v=P(7): refused(L.cache_read(fmt, flags, S, c or kv(), slots, sb, k, v, None))  # noqa: E731
    assert read(S=0, slots=None, k=None, v=None) == OK
    assert read(flags=INTERLEAVED) == INVALID
    assert read(S=-1) == INVALID
    assert read(S=1 << 31) == INVALID
    assert read(sb=1) == INVALID
    assert read(slots=None) == INVALID
    assert read(k=None, v=None) == INVALID
    assert read(k=P(6, 8)) == MISALIGNED
    assert read(slots=P(5, 1)) == MISALIGNED
    assert read(k=P(10)) == INVALID
    assert read(v=P(11, 128)) == INVALID
    assert read(k=P(5)) == INVALID
    assert read(v=P(6, 16)) == INVALID
    assert read(fmt=2, c=fp8(), v=P(12)) == INVALID


def test_attention_refusals(L):
    def att(fmt=3, flags=0, B=2, c=None, q=None, t=P(1), width=6250, n=P(2), scale=1.0, window=0, sinks=None, out=P(3), lse=None, ws=P(4)):
        return refused(L.paged_attention(fmt, flags, B, c or kv(), q or heads(P(0), H=8, ts=512), t, width, n, scale, window, sinks, out, lse, ws, None))
    assert att(B=0, q=heads(None), out=None) == OK
    assert att(flags=INTERLEAVED) == INVALID
    assert att(B=-1) == INVALID
    assert att(B=65537) == UNSUPPORTED
    assert att(width=-1) == INVALID
    assert att(width=1 << 28) == UNSUPPORTED             # 2^32 tokens
    assert att(window=-1) == INVALID
    assert att(scale=math.nan) == INVALID
    assert att(scale=math.inf) == INVALID
    assert att(q=heads(P(0), H=6, ts=512)) == INVALID    # not a multiple of the cache's heads
    assert att(q=heads(P(0), H=2, ts=512)) == INVALID
    assert att(q=heads(P(0), H=2048, ts=2048 * 64)) == UNSUPPORTED
    for kw in ("t", "n", "out", "ws"):
        assert att(**{kw: None}) == INVALID, kw
    assert att(q=heads(P(0, 8), H=8, ts=512)) == MISALIGNED
    for kw, off in (("t", 2), ("n", 2), ("out", 8), ("ws", 8), ("lse", 2), ("sinks", 1)):
        assert att(**{kw: P(6, off)}) == MISALIGNED, kw
    for i in (0, 1, 2, 10, 11, 14):
        assert att(sinks=P(14), out=P(i)) == INVALID, i
        assert att(sinks=P(14), lse=P(i)) == INVALID, i
        assert att(sinks=P(14), ws=P(i)) == INVALID, i
    assert att(lse=P(3)) == INVALID
    assert att(ws=P(3)) == INVALID
    assert att(fmt=2, c=fp8(), out=P(12)) == INVALID
    ws = L.sgq_attention_workspace_bytes
    assert ws(3, 2, 8, 4, 64, 4, 16, 0) == 0             # few tokens: one launch
    assert ws(3, 2, 8, 4, 64, 6250, 16, 0) > 0
    assert ws(3, 2, 8, 4, 64, 6250, 16, 100) == 0        # a short window
    assert ws(3, 64, 64, 8, 128, 10000, 16, 0) == ws(3, 128, 64, 8, 128, 20000, 16, 0)      # bounded by the CTAs
    for bad in ((0, 8, 4, 64, 6250, 16, 0), (2, 6, 4, 64, 6250, 16, 0), (2, 8, 4, 300, 6250, 16, 0), (2, 8, 4, 64, -1, 16, 0), (2, 8, 4, 64, 1 << 28, 16, 0),
                (2, 2048, 4, 64, 6250, 16, 0), (2, 8, 0, 64, 6250, 16, 0), (2, 8, 4, 64, 6250, 0, 0), (65537, 8, 4, 64, 6250, 16, 0), (2, 8, 4, 64, 6250, 16, -1),
                (65536, 1024, 1024, 64, 1 << 20, 16, 0)):
        assert ws(3, *bad) == 0, bad
    assert att(B=65536, width=1 << 20, q=heads(P(0), H=1024, ts=65536), c=kv(H=1024, ps=1 << 20)) == UNSUPPORTED        # 2^31 tiles
    assert sgq.attention_workspace_bytes("none", 2, 8, 4, 64, 6250, 16) == ws(3, 2, 8, 4, 64, 6250, 16, 0)


def bf(*shape):
    return torch.zeros(*shape, dtype=BF16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def i64(*shape):
    return torch.zeros(*shape, dtype=torch.int64)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_python_refusals():
    no = lambda f, *a, **k: pytest.raises(sgq.SgqError, f, *a, **k)  # noqa: E731
    x, f = bf(4, 2, 64), i64(32)
    no(sgq.rope, x, i64(4), f, layout="pairs")
    no(sgq.rope, x.float(), i64(4), f)
    no(sgq.rope, bf(4, 64), i64(4), f)
    no(sgq.rope, bf(4, 64, 2).transpose(1, 2), i64(4), f)
    no(sgq.rope, x, i64(3), f)
    no(sgq.rope, x, i64(4).float(), f)
    no(sgq.rope, x, i64(8)[::2], f)
    no(sgq.rope, x, i64(4), f.float())
    no(sgq.rope, x, i64(4), i64(32, 1))
    for factor in (math.inf, math.nan, -math.inf, 1e39):
        no(sgq.rope, x, i64(4), f, factor=factor)
    no(sgq.rope, x, i64(4), f)                                               # on the CPU
    c, s = bf(6, 2, 16, 64), i32(4)
    no(sgq.cache_write, x, x, c, c.clone(), s, fmt="mxfp8")
    no(sgq.cache_write, x, x, u8(6, 2, 16, 64), u8(6, 2, 16, 64), s)
    no(sgq.cache_write, x, x, c, bf(5, 2, 16, 64), s)
    no(sgq.cache_write, x, x, c, bf(6, 16, 2, 64).transpose(1, 2), s)        # other strides
    no(sgq.cache_write, x, x, bf(6, 16, 64), bf(6, 16, 64), s)
    no(sgq.cache_write, x, x, c.half(), c.half(), s)
    no(sgq.cache_write, x, x, c, c.clone(), s, k_scale=torch.zeros(6, 2, 16), v_scale=torch.zeros(6, 2, 16))
    no(sgq.cache_write, x, x, u8(6, 2, 16, 64), u8(6, 2, 16, 64), s, fmt="per_token")
    no(sgq.cache_write, x, x, u8(6, 2, 16, 64), u8(6, 2, 16, 64), s, fmt="per_token", k_scale=torch.zeros(6, 16, 2), v_scale=torch.zeros(6, 2, 16))
    no(sgq.cache_write, bf(4, 3, 64), bf(4, 3, 64), c, c.clone(), s)
    no(sgq.cache_write, x, x, c, c.clone(), i32(3))
    no(sgq.cache_write, x, x, c, c.clone(), s, positions=i64(4))
    no(sgq.cache_write, x, x, c, c.clone(), s, q=x)
    no(sgq.cache_write, x, x, c, c.clone(), s, q_out=x)
    no(sgq.cache_write, x, x, c, c.clone(), s, q=bf(3, 2, 64), positions=i64(4), freqs=f)
    no(sgq.cache_write, x, x, c, c.clone(), s)                               # on the CPU
    no(sgq.cache_read, c, c.clone(), i32(4, 1))
    no(sgq.cache_read, c, c.clone(), s, dtype=torch.float16)
    no(sgq.cache_read, c, c.clone(), s, k_out=bf(3, 2, 64))
    no(sgq.cache_read, c, c.clone(), s)                                      # on the CPU
    a = bf(3, 8, 64), c, c.clone(), i32(3, 5), i32(3)
    no(sgq.paged_attention, bf(3, 64), *a[1:])
    no(sgq.paged_attention, bf(3, 8, 32), *a[1:])
    no(sgq.paged_attention, *a[:3], i64(3, 5), i32(3))
    no(sgq.paged_attention, *a[:3], i32(5, 3), i32(3))
    no(sgq.paged_attention, *a[:3], i32(3, 5), i32(4))
    no(sgq.paged_attention, *a, sinks=torch.zeros(7))
    no(sgq.paged_attention, *a, out=bf(3, 8, 32))
    no(sgq.paged_attention, *a, lse=torch.zeros(3, 7))
    no(sgq.paged_attention, *a, workspace=u8(3))
    no(sgq.paged_attention, *a)                                              # on the CPU
    no(sgq.rope_frequencies, 24)
    no(sgq.rope_frequencies, 64, scaling="cubic")
    no(sgq.rope_frequencies, 64, scaling="yarn", stretch=4.0)                # no trained length
    no(sgq.rope_frequencies, 64, scaling="linear", stretch=0.5)


def test_frequencies():
    of = lambda t: [(v % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in t.tolist()]  # noqa: E731
    R, base = 64, 10000.0
    plain = [base ** (-2 * i / R) for i in range(R // 2)]
    t, factor = sgq.rope_frequencies(R, base, device="cpu")
    assert factor == 1.0 and t.dtype == torch.int64
    assert of(t) == pytest.approx(plain, rel=1e-14)
    assert of(sgq.rope_frequencies(R, base, scaling="linear", stretch=4.0, device="cpu")[0]) == pytest.approx([f / 4 for f in plain], rel=1e-14)
    ntk = of(sgq.rope_frequencies(R, base, scaling="ntk", stretch=4.0, device="cpu")[0])
    assert ntk[0] == pytest.approx(1.0) and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)
    t, factor = sgq.rope_frequencies(R, base, scaling="yarn", stretch=4.0, trained=4096, device="cpu")
    assert factor == pytest.approx(0.1 * math.log(4) + 1)
    for got, f in zip(of(t), plain):
        turned = 4096 * f / (2 * math.pi)
        if turned > 40:
            assert got == pytest.approx(f, rel=1e-12)
        elif turned < 0.8:
            assert got == pytest.approx(f / 4, rel=1e-12)
        else:
            assert f / 4 * (1 - 1e-12) <= got <= f * (1 + 1e-12)
    # f (1 - s) + f s: three roundings of 2^-53, and the turns' own
    assert of(sgq.rope_frequencies(R, base, scaling="yarn", stretch=1.0, trained=4096, device="cpu")[0]) == pytest.approx(plain, rel=2.0 ** -50)
    assert torch.equal(sgq.rope_turns(torch.tensor([math.pi, 2 * math.pi, 1.0]), device="cpu")[:2] >> 40, torch.tensor([-(1 << 63), 0]) >> 40)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_plain_rope_is_a_rotation(layout):
    x = torch.randn(5, 2, 48, generator=ref.gen(0), dtype=torch.float64)
    pos, freqs = torch.tensor([0, 1, 5, -7, 1 << 40]), ref.turns(32)
    y, _ = ref.rope(x, pos, freqs, layout, 1.0)
    assert torch.equal(y[0], x[0])
    assert y.square().sum().item() == pytest.approx(x.square().sum().item())
    back, _ = ref.rope(y, pos, freqs, layout, 1.0, True)
    assert torch.allclose(back, x, atol=1e-12)
    c, s = math.cos(ref.turns(32).tolist()[3] / 2.0 ** 64 * 2 * math.pi), math.sin(ref.turns(32).tolist()[3] / 2.0 ** 64 * 2 * math.pi)
    a, b = (3, 19) if layout == "half" else (6, 7)
    assert y[1, 0, a].item() == pytest.approx((x[1, 0, a] * c - x[1, 0, b] * s).item())
    assert y[1, 0, b].item() == pytest.approx((x[1, 0, a] * s + x[1, 0, b] * c).item())


def test_plain_attention_against_a_softmax():
    table, pages = ref.table_of([10, 0, 37], 8)
    k, v, _, _ = ref.pool("none", pages, 2, 8, 16, BF16, 0)
    q = torch.randn(3, 4, 16, generator=ref.gen(1)).to(BF16)
    out, tol, lse, _ = ref.attention(q, k, v, None, None, table, torch.tensor([10, 0, 37]))
    for b, n in ((0, 10), (2, 37)):
        rows = lambda c: torch.cat([c[int(p)] for p in table[b] if p >= 0], 1)[:, :n].double()  # noqa: E731
        x = torch.einsum("hgd,hnd->hgn", q[b].double().view(2, 2, 16), rows(k)) / 4
        assert torch.allclose(out[b].view(2, 2, 16), torch.softmax(x, -1) @ rows(v))
        assert torch.allclose(lse[b].view(2, 2), x.logsumexp(-1))
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
