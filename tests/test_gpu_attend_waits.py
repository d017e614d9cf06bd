"""paged_attention where a wait runs out of time: the launch ends, is counted, and leaves what it has no part in as it
should be. A build of the same kernels whose waits are limited to milliseconds and in which one copy is never issued
(tests/cuda/attend_wait_check.cu), so that a barrier's phase stays open; nothing faults and nothing waits without a limit."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq
from swiglu_fp8_activation_gb300 import binding, cache

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
HEADS, D = 2, 64
NEVER, LATE = 1, 2


@pytest.fixture(scope="module")
def lib(sgq_lib):
    import __graft_entry__ as g
    out = os.path.join(ROOT, "_build", "libattend_wait_check.so")
    os.makedirs(os.path.dirname(out), exist_ok=True)
    src = [os.path.join(ROOT, "tests", "cuda", "attend_wait_check.cu"), os.path.join(g.CSRC, "sgq_cache_api.cu")]
    cmd = [g._nvcc(), *g.ARCH, "-O3", "-std=c++17", "-shared", "-cudart", "shared", "-Xcompiler", "-fPIC", "-I", g.CSRC, "-I", os.path.join(ROOT, "include"),
           "-Xlinker", "-Bsymbolic", "-Xlinker", f"-rpath={g._cuda_lib_dir(g._nvcc())}", "-o", out, *src, os.path.join(g.PKG, "libsgq.so")]
    subprocess.run(cmd, check=True)
    L = C.CDLL(out)
    L.paged_attention.restype, L.paged_attention.argtypes = C.c_int, cache._lib().paged_attention.argtypes
    L.check_limit.restype = C.c_longlong
    L.check_choose.argtypes = [C.c_int] * 4 + [C.c_longlong]
    L.check_spin.argtypes = [C.c_longlong, C.c_void_p]
    return L


def gave_up(lib):
    n = C.c_uint32(0)
    assert lib.check_gave_up(C.byref(n)) == 0
    return n.value


class Case:
    """Sequences of these lengths and a call of the build with short waits over them."""

    def __init__(self, lib, fmt, lengths, group, P, shares):
        self.lib, self.lengths, self.group = lib, lengths, group
        table, pages = ref.table_of(lengths, P)
        k, v, ks, vs = ref.pool(fmt, pages, HEADS, P, D, BF16, 0)
        q = torch.randn(len(lengths), HEADS * group, D, generator=ref.gen(1)).to(BF16)
        if shares:
            table = torch.nn.functional.pad(table, (0, -(-60000 // P)), value=-1)
        n = torch.tensor(lengths, dtype=torch.int32)
        self.q, self.k, self.v, self.ks, self.vs, self.table, self.n = (None if t is None else t.to(DEV) for t in (q, k, v, ks, vs, table, n))
        self.room = sgq.attention_workspace_bytes(fmt, len(lengths), HEADS * group, HEADS, D, table.shape[1], P)
        assert (self.room > 0) == shares
        self.code = cache.CACHE_FORMATS[fmt]
        self.cache = cache._cache(self.k, self.v, fmt, self.ks, self.vs, BF16)[0]
        self.plain = sgq.paged_attention(self.q, self.k, self.v, self.table, self.n, fmt=fmt, k_scale=self.ks, v_scale=self.vs)

    def run(self, mode=0, item=0, part=0, tile=0, cycles=0):
        assert self.lib.check_choose(mode, item, part, tile, cycles) == 0
        out = torch.zeros_like(self.q)
        ws = torch.empty(max(self.room, 16), dtype=torch.uint8, device=DEV)
        at = torch.cuda.current_stream().cuda_stream
        torch.cuda.synchronize()
        begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
        begin.record()
        st = self.lib.paged_attention(self.code, 0, len(self.lengths), self.cache, cache._heads(self.q, BF16, "q", self.q.shape), self.table.data_ptr(), self.table.shape[1],
                                      self.n.data_ptr(), D ** -0.5, 0, None, out.data_ptr(), None, ws.data_ptr() if self.room else None, at)
        assert st == 0
        end.record()
        torch.cuda.synchronize()
        self.ms = begin.elapsed_time(end)
        return out


def limits(lib, n):
    """Milliseconds that n limits of a wait take now."""
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
    begin.record()
    assert lib.check_spin(int(n * lib.check_limit()), torch.cuda.current_stream().cuda_stream) == 0
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end)


FORMS = [([60, 0, 64], False), ([500, 130, 64], False), ([2000, 0, 900, 1], False), ([3000, 129, 0, 700], True)]


@pytest.mark.parametrize("fmt,P", [("none", 16), ("none", 5), ("per_token", 16), ("per_token", 5)])
@pytest.mark.parametrize("lengths,shares", FORMS)
def test_a_copy_that_is_never_issued(lib, fmt, P, lengths, shares):
    """One part of a CTA's warps waits in vain, in its first tile, a later or the last, while the others are done: the launch ends, the CTA is
    counted once, items of other CTAs are right, and so is the next launch."""
    case = Case(lib, fmt, lengths, 4, P, shares)
    tokens = 128 if fmt == "per_token" else 64
    before = gave_up(lib)
    assert torch.equal(case.run(), case.plain) and gave_up(lib) == before
    for seq, head in ((0, 1), (2 if lengths[2] else 3, 0)):
        tiles = -(-lengths[seq] // tokens)
        for tile in sorted({0, tiles // 2, tiles - 1}):
            for part in range(4):
                count = gave_up(lib)
                out = case.run(NEVER, seq * HEADS + head, part, tile)
                assert gave_up(lib) == count + 1, (seq, tile, part)
                if not shares:
                    others = torch.ones(out.shape[:2], dtype=torch.bool)
                    others[seq, head * 4:head * 4 + 4] = False
                    assert torch.equal(out[others], case.plain[others]), (seq, tile, part)
    count = gave_up(lib)
    assert torch.equal(case.run(), case.plain) and gave_up(lib) == count


@pytest.mark.parametrize("P", [16, 5])
@pytest.mark.parametrize("lengths,shares", FORMS)
@pytest.mark.parametrize("mode", [NEVER, LATE])
def test_warps_that_share_a_part_of_the_tokens(lib, P, lengths, shares, mode):
    """Groups of 32 heads: two warps take a part's tokens, and one of them may have waited in vain for rows that the other
    sees landed, whether the tile has masked rows or not. (A late copy of one of a CTA's first tiles, that is: later ones keep both from going on.)"""
    case = Case(lib, "none", lengths, 32, P, shares)
    before = gave_up(lib)
    assert torch.equal(case.run(), case.plain) and gave_up(lib) == before
    tiles = -(-lengths[0] // 64)
    for tile in sorted({0, tiles // 2, tiles - 1}):
        for part in range(4):
            count = gave_up(lib)
            out = case.run(mode, 1, part, tile, lib.check_limit() * 3 // 2)
            more = gave_up(lib) - count
            assert more == 1 or (mode == LATE and tile > 0 and more == 0 and torch.equal(out, case.plain)), (tile, part)
    count = gave_up(lib)
    assert torch.equal(case.run(), case.plain) and gave_up(lib) == count


def test_the_last_copies_are_waited_for_and_no_others(lib):
    """A copy that lands half a limit after a wait for it has run out: the launch ends then, and waits for no phase that no copy ends."""
    for P in (16, 5):
        case = Case(lib, "none", [500, 130], 32, P, False)
        case.run()
        count = gave_up(lib)
        case.run(LATE, 1, 2, 0, lib.check_limit() * 3 // 2)
        assert gave_up(lib) == count + 1
        assert limits(lib, 1.0) < case.ms < limits(lib, 2.0)


@pytest.mark.parametrize("fmt", ["none", "per_token"])
def test_waits_end_soon_once_one_has_run_out(lib, fmt):
    """One CTA has hundreds of tiles ahead of it when its first one does not come: two limits, for the tile and for its copy, and no more."""
    binding.set_sm_budget(1)
    try:
        case = Case(lib, fmt, [60000], 8, 64, True)
        case.run()
        count = gave_up(lib)
        case.run(NEVER, 0, 1, 0)
        assert gave_up(lib) == count + 1
        assert limits(lib, 1.0) < case.ms < limits(lib, 2.5)
        assert torch.equal(case.run(), case.plain)
    finally:
        binding.set_sm_budget(0)
