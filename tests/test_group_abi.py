"""The ragged-group entry points (include/sgq_group.h) without a GPU: exports,
host checks with the documented status before anything is launched (fake,
never dereferenced pointers), and the Python entry points' refusals."""
import ctypes as C
import os
import re

import pytest
import torch

import group_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import grouped

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgq_group.h")
OK, INVALID, UNSUPPORTED, MISALIGNED, LAUNCH = 0, 1, 2, 3, 4
FP16 = 1 << 5
STEP = 1 << 36


def P(i, off=0):
    return C.c_void_p((1 << 44) + i * STEP + off)


def _text():
    with open(HEADER) as f:
        return f.read()


def test_exports_and_constants(sgq_lib):
    names = re.findall(r"^(?:int|int64_t)\s+(\w+)\(", _text(), flags=re.M)
    assert {"group_rows", "grouped_gemm", "combine_rows", "lora_add", "sgq_lora_workspace_bytes", "sgq_wait_timeouts"} == set(names)
    for n in names:
        assert hasattr(sgq_lib, n), n
    value = lambda n: int(re.search(rf"#define {n}\s+(\d+)", _text()).group(1))  # noqa: E731
    assert value("SGQ_MAX_GROUPS") == sgq.MAX_GROUPS
    assert value("SGQ_MAX_RANK") == sgq.MAX_RANK
    assert "#define SGQ_MAX_ROWS 0x7FFF0000" in _text()
    assert value("SGQ_FMT_16BIT") == sgq.GEMM_FORMATS["none"]
    assert {k: v for k, v in sgq.GEMM_FORMATS.items() if k != "none"} == sgq.FORMATS


@pytest.fixture
def L(sgq_lib):
    return grouped._lib()


def refused(st):
    assert st != LAUNCH, "a fake-pointer call passed the host checks"
    return st


def rows(L, idb=4, T=8, k=2, G=4, ids=P(0), off=P(1), r=P(2), s=P(3)):
    return refused(L.group_rows(idb, T, k, G, ids, off, r, s, None))


def test_group_rows_refusals(L):
    assert rows(L, idb=2) == INVALID
    assert rows(L, T=-1) == INVALID
    assert rows(L, k=0) == INVALID
    assert rows(L, G=0) == INVALID
    assert rows(L, T=1 << 30, k=2) == INVALID            # 2^31 ids
    assert rows(L, T=1 << 40, k=1 << 40) == INVALID
    assert rows(L, G=1025) == UNSUPPORTED
    for kw in ("ids", "off", "r"):
        assert rows(L, **{kw: None}) == INVALID, kw
    assert rows(L, T=0, off=None) == INVALID             # offsets are written even then
    assert rows(L, idb=8, ids=P(0, 4)) == MISALIGNED
    assert rows(L, r=P(2, 2)) == MISALIGNED
    assert rows(L, s=P(2, 60)) == INVALID                # the last of 16 rows
    assert rows(L, r=P(0, 16)) == INVALID
    assert rows(L, off=P(3, 4)) == INVALID


def gemm(L, fmt=0, flags=0, S=16, G=4, N=256, K=256, X=16, x=P(0), xs=P(1), w=P(2), ws=P(3), off=P(4), r=None, out=P(6)):
    return refused(L.grouped_gemm(fmt, flags, S, G, N, K, X, x, xs, w, ws, off, r, out, None))


def test_grouped_gemm_refusals(L):
    assert gemm(L, S=0, X=0, x=None, out=None) == OK     # nothing to do
    assert gemm(L, fmt=4) == INVALID
    assert gemm(L, fmt=-1) == INVALID
    assert gemm(L, flags=1) == INVALID
    assert gemm(L, S=-1) == INVALID
    assert gemm(L, S=1 << 31, X=1 << 31) == INVALID
    assert gemm(L, S=0x7FFF0001, X=0x7FFF0001) == INVALID
    assert gemm(L, X=1 << 31, r=P(5)) == INVALID
    assert gemm(L, G=0) == INVALID
    assert gemm(L, G=1025) == UNSUPPORTED
    assert gemm(L, N=0) == INVALID
    assert gemm(L, K=-32) == INVALID
    assert gemm(L, X=15) == INVALID                      # no rows: slot s is row s
    assert gemm(L, N=132) == UNSUPPORTED
    assert gemm(L, N=131072 + 8) == UNSUPPORTED
    assert gemm(L, K=131072 + 128) == UNSUPPORTED
    for fmt, K in ((0, 48), (1, 192), (2, 24), (3, 12)):
        kw = dict(xs=None, ws=None) if fmt == 3 else {}
        assert gemm(L, fmt=fmt, K=K, **kw) == UNSUPPORTED, fmt
    for kw in ("x", "xs", "w", "ws", "off", "out"):
        assert gemm(L, **{kw: None}) == INVALID, kw
    assert gemm(L, fmt=3) == INVALID                     # scales with 16-bit rows
    for kw in ("x", "w", "out"):
        assert gemm(L, **{kw: P(9, 8)}) == MISALIGNED, kw
    assert gemm(L, ws=P(3, 8)) == MISALIGNED
    assert gemm(L, fmt=1, xs=P(1, 2)) == MISALIGNED
    assert gemm(L, off=P(4, 1)) == MISALIGNED
    assert gemm(L, r=P(5, 2)) == MISALIGNED
    for i in range(6):
        assert gemm(L, r=P(5), out=P(i)) == INVALID, i


def comb(L, flags=0, T=8, k=2, S=16, N=64, y=P(0), s=P(1), w=P(2), out=P(3)):
    return refused(L.combine_rows(flags, T, k, S, N, y, s, w, out, None))


def test_combine_refusals(L):
    assert comb(L, T=0, y=None, out=None) == OK
    assert comb(L, flags=2) == INVALID
    assert comb(L, T=-1) == INVALID
    assert comb(L, k=0) == INVALID
    assert comb(L, T=1 << 30, k=4) == INVALID
    assert comb(L, S=-1) == INVALID
    assert comb(L, N=0) == INVALID
    assert comb(L, N=12) == UNSUPPORTED
    assert comb(L, N=131072 + 8) == UNSUPPORTED
    assert comb(L, T=1 << 24, k=1, N=131072, out=P(8)) == UNSUPPORTED     # 2^32 CTAs
    for kw in ("y", "s", "out"):
        assert comb(L, **{kw: None}) == INVALID, kw
    assert comb(L, y=P(0, 8)) == MISALIGNED
    assert comb(L, w=P(2, 2)) == MISALIGNED
    for i in range(3):
        assert comb(L, out=P(i)) == INVALID, i
    assert comb(L, out=P(0, 16 * 64 * 2 - 16)) == INVALID


def lora(L, flags=0, T=64, S=64, G=2, R=16, K=64, N=128, x=P(0), a=P(1), b=P(2), c=P(3), off=P(4), r=P(5), s=P(6), y=P(7), ws=P(8)):
    return refused(L.lora_add(flags, T, S, G, R, K, N, x, a, b, c, off, r, s, y, ws, None))


def test_lora_refusals(L):
    assert lora(L, S=0, x=None) == OK
    assert lora(L, T=0, x=None) == OK
    assert lora(L, flags=1) == INVALID
    assert lora(L, T=-1) == INVALID
    assert lora(L, S=1 << 31) == INVALID
    assert lora(L, G=0) == INVALID
    assert lora(L, G=1025) == UNSUPPORTED
    assert lora(L, R=0) == INVALID
    assert lora(L, R=12) == UNSUPPORTED
    assert lora(L, R=136) == UNSUPPORTED
    assert lora(L, K=60) == UNSUPPORTED
    assert lora(L, N=4) == UNSUPPORTED
    assert lora(L, r=None) == INVALID                    # rows and slots go together
    assert lora(L, s=None) == INVALID
    assert lora(L, S=4, r=None, s=None) == INVALID       # without rows, slot s is row s
    for kw in ("x", "a", "b", "off", "y", "ws"):
        assert lora(L, **{kw: None}) == INVALID, kw
    for kw in ("x", "a", "b", "y", "ws"):
        assert lora(L, **{kw: P(9, 8)}) == MISALIGNED, kw
    for i in range(7):
        assert lora(L, y=P(i)) == INVALID, i
        assert lora(L, ws=P(i)) == INVALID, i
    assert lora(L, ws=P(7)) == INVALID
    assert L.sgq_lora_workspace_bytes(64, 2, 16) == 64 * (16 * 4 + 16)
    assert L.sgq_lora_workspace_bytes(64, 2, 200) == 0
    assert L.sgq_lora_workspace_bytes(-1, 2, 8) == 0
    assert L.sgq_lora_workspace_bytes(64, 0, 8) == 0
    for S, G, R in ((1, 1, 8), (77, 4, 40), (64, 32, 16), (8, 1, 16), (9, 1, 16), (1 << 30, 1024, 128)):
        # what the Python lora_add allocates
        assert sgq.lora_workspace_bytes(S, G, R) == (0 if S * R <= 128 * G else S * (4 * R + 16))
    assert L.sgq_wait_timeouts(None) == INVALID


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_python_refusals():
    no = lambda f, *a, **k: pytest.raises(sgq.SgqError, f, *a, **k)  # noqa: E731
    no(sgq.group_rows, torch.zeros(4, 2), 4)                                    # float ids
    no(sgq.group_rows, i32(4, 2, 2), 4)
    no(sgq.group_rows, i32(4, 2), 0)
    no(sgq.group_rows, i32(4, 2), 1025)
    no(sgq.group_rows, i32(4, 0), 4)
    no(sgq.group_rows, i32(2, 4).t(), 4)                                        # strided
    no(sgq.group_rows, i32(4, 2), 4, offsets_out=i32(4))
    no(sgq.group_rows, i32(4, 2), 4)                                            # on the CPU
    off = i32(3)
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="fp4")
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="mxfp8")            # 16-bit rows
    no(sgq.grouped_gemm, u8(4, 64), u8(2, 32, 64), off)                         # scales missing
    no(sgq.grouped_gemm, u8(4, 64), u8(2, 32, 64), off, x_scale=u8(4, 2), w_scale=u8(2, 32, 2))   # w_scale not laid out
    no(sgq.grouped_gemm, u8(4, 48), u8(2, 32, 48), off, x_scale=u8(4, 1), w_scale=u8(2, 128, 4))  # K % 32
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none", x_scale=u8(4, 2))
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), i32(2), fmt="none")          # offsets too short
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off.long(), fmt="none")
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none", rows=i32(3).long())
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none", out_dtype=torch.float16)
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none", out=bf(4, 40))
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none", out_dtype=torch.float32)
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 72), off, fmt="none")
    no(sgq.grouped_gemm, bf(4, 64), bf(64, 64), off, fmt="none")
    no(sgq.grouped_gemm, bf(4, 64), bf(2, 32, 64), off, fmt="none")             # on the CPU
    no(sgq.combine_rows, bf(8, 64), i32(4, 2).long())
    no(sgq.combine_rows, bf(8, 64).float(), i32(4, 2))
    no(sgq.combine_rows, bf(8, 64), i32(4, 2), bf(4, 2))                        # weights are float32
    no(sgq.combine_rows, bf(8, 64), i32(4, 2), torch.zeros(4, 3))
    no(sgq.combine_rows, bf(8, 64), i32(8))
    no(sgq.combine_rows, bf(8, 64), i32(4, 2))                                  # on the CPU
    args = bf(4, 64), bf(2, 8, 64), bf(2, 32, 8), bf(4, 32), off
    no(sgq.lora_add, *args, rows=i32(4))                                        # rows without slots
    no(sgq.lora_add, *args, rows=i32(4), slots=i32(3))
    no(sgq.lora_add, *args, scaling=torch.zeros(3))
    no(sgq.lora_add, *args, workspace=u8(7))
    no(sgq.lora_add, args[0], args[1], bf(2, 8, 32), args[3], off)              # b transposed
    no(sgq.lora_add, args[0], args[1].half(), args[2], args[3], off)
    no(sgq.lora_add, *args)                                                     # on the CPU


def test_plain_group_rows_against_a_stable_sort():
    ids = torch.randint(-1, 5, (37, 3), generator=ref.gen(0)).to(torch.int32)
    offsets, rows_, slots = ref.group_rows(ids, 5)
    flat = ids.flatten()
    order = torch.sort(torch.where(flat < 0, 5, flat), stable=True).indices
    n = int((flat >= 0).sum())
    assert offsets[-1] == n
    assert torch.equal(rows_[:n].long(), order[:n] // 3)
    assert (rows_[n:] == -1).all()
    for i, v in enumerate(flat.tolist()):
        s = int(slots.flatten()[i])
        assert (s == -1) if v < 0 else (offsets[v] <= s < offsets[v + 1] and int(order[s]) == i)


def test_plain_ranges_hold_wild_offsets():
    assert ref.ranges(torch.tensor([-5, 3, 2, 900, 4]), 10) == [(0, 3), (3, 3), (3, 10), (10, 10)]


def test_plain_swizzle_matches_the_oracle():
    import numpy as np
    import oracle
    codes = torch.randint(0, 255, (1, 200, 7), generator=ref.gen(1)).to(torch.uint8)
    np.testing.assert_array_equal(ref.swizzled(codes)[0].numpy(), oracle.scale_layout("mxfp8", codes[0].numpy(), "swizzled"))


def test_lora_form_is_bounded_in_slots():
    """However many adapters are loaded, many slots take the tensor cores' form, with its workspace."""
    room = lambda S, R: S * (4 * R + 16)  # noqa: E731
    for R, most in ((8, 512), (16, 512), (24, 341), (64, 128), (128, 64)):
        assert sgq.lora_workspace_bytes(most, 1024, R) == 0
        assert sgq.lora_workspace_bytes(most + 1, 1024, R) == room(most + 1, R)
        assert sgq.lora_workspace_bytes(8192, 1024, R) == room(8192, R)
    assert sgq.lora_workspace_bytes(512, 64, 16) == 0
    assert sgq.lora_workspace_bytes(512, 63, 16) == room(512, 16)
