"""Arguments of the serving calls that lie in one another's memory are refused (no GPU: every call
returns before a launch; the addresses are never dereferenced)."""
import ctypes

import pytest

from .test_serve_abi import lib, params  # noqa: F401  (lib: the fixture)

B, HKV, CAP, BUDGET, OUT = 2, 2, 100, 50, 60
BYTES = [2 * 128 // 8, 8, 2, 2, 3 * 128 // 8, 2, 4]  # of a record: d = 128, 3 bits, 64 projections


def blocks(sizes, start=1 << 30):
    """Addresses of blocks of these sizes, one right behind the other (16-byte aligned)."""
    at = [start]
    for n in sizes:
        at.append((at[-1] + n + 15) // 16 * 16)
    return at[:-1]


SOURCE, DEST = [B * HKV * CAP * n for n in BYTES], [B * HKV * OUT * n for n in BYTES]
NAMES = ([f"source {i}" for i in range(7)] + ["lens"] + [f"destination {i}" for i in range(7)] +
         ["kept", "out_lens", "scratch", "dev_status"])
SIZES = SOURCE + [4 * B] + DEST + [4 * B * HKV * BUDGET, 4 * B, 256, 4]


def evict(L, at):
    s, lens, d, (kept, out_lens, scratch, status) = at[:7], at[7], at[8:15], at[15:]
    return L.tq_evict(ctypes.byref(params(L)), B, HKV, lens, CAP, *s, BUDGET, 5, OUT, *d, kept, out_lens, scratch,
                      256, status, None)


@pytest.mark.parametrize("name", NAMES[8:])
def test_evict_refuses_what_it_writes_in_other_memory(lib, name):  # noqa: F811
    i = NAMES.index(name)
    for j, other in enumerate(NAMES):
        if j == i:
            continue
        for off in (0, (SIZES[j] - 1) // 16 * 16, -((SIZES[i] - 1) // 16 * 16)):
            at = blocks(SIZES)
            at[i] = at[j] + off  # from its first bytes, in its last ones, or up to its first ones
            assert evict(lib, at) == 1, (name, other, off)


ROWS = B * 4 * 128 * 2  # f16 queries of four heads
A_NAMES = (["workspace", "lens"] + [f"prefix {i}" for i in range(6)] + [f"own {i}" for i in range(6)] +
           ["q", "out", "scratch", "dev_status", "weights"])


def attend(L, sizes, at, weigh):
    ws, lens, pre, own, (q, out, scratch, status, weights) = at[0], at[1], at[2:8], at[8:14], at[14:]
    prm = params(L)
    prm.workspace = ws
    if weigh:
        return L.tq_attend_weigh(ctypes.byref(prm), q, 0, B, 4, HKV, 1, lens, CAP, *own, 0.0, weights, out, scratch,
                                 sizes[16], status, None)
    return L.tq_attend_shared(ctypes.byref(prm), q, 0, B, 4, HKV, 1, 70, *pre, lens, CAP, *own, 0.0, out, scratch,
                              sizes[16], status, None)


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("name", ["out", "scratch", "dev_status", "weights"])
def test_attention_refuses_what_it_writes_in_other_memory(lib, name, weigh):  # noqa: F811
    p = ctypes.byref(params(lib))
    need = (lib.tq_attend_weigh_scratch_bytes(p, 0, B, 4, HKV, 1, CAP) if weigh else
            lib.tq_attend_shared_scratch_bytes(p, 0, B, 4, HKV, 1, 70, CAP))
    sizes = ([lib.tq_workspace_bytes(128, 3, 64), 4 * B] + [HKV * 70 * n for n in BYTES[:6]] + SOURCE[:6] +
             [ROWS, ROWS, need, 4, 4 * B * HKV * CAP])
    i = A_NAMES.index(name)
    if name == "weights" and not weigh:
        return
    for j, other in enumerate(A_NAMES):
        unused = other.startswith("prefix") if weigh else other == "weights"
        if j == i or unused or (name == "out" and other == "q"):
            continue
        for off in (0, (sizes[j] - 1) // 16 * 16, -((sizes[i] - 1) // 16 * 16)):
            at = blocks(sizes)
            at[i] = at[j] + off
            assert attend(lib, sizes, at, weigh) == 1, (name, other, off)
