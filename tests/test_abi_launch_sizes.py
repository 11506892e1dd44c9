"""Host-only: the largest delta rule calls are those that the header names."""
import ctypes

import pytest

from selective_state_space_vjp_amd import binding as bd


def query(fn, desc):
    return getattr(bd.lib(), fn + "_workspace")(ctypes.byref(desc), ctypes.byref(ctypes.c_size_t(0)))


def chunk(batch, seqlen, H, HV, V, packed=0):
    return bd.DeltaChunkDesc(batch, seqlen, H, HV, 16, V, 1.0, bd.BF16, packed, 0)


@pytest.mark.parametrize("desc,ok", [
    (chunk(1, ((1 << 23) - 2) * 64, 1, 1, 16), True),            # (2^23 - 2 + 1) chunks
    (chunk(1, ((1 << 23) - 1) * 64, 1, 1, 16), False),
    (chunk(1, ((1 << 19) - 2) * 64, 16, 16, 16), True),
    (chunk(1, ((1 << 19) - 1) * 64, 16, 16, 16), False),
    (chunk(2, ((1 << 18) - 2) * 64, 16, 16, 16), True),
    (chunk(2, ((1 << 18) - 1) * 64, 16, 16, 16), False),
    (chunk(100, ((1 << 19) - 101) * 64, 16, 16, 16, 1), True),   # packed: one more chunk a sequence in all
    (chunk(100, ((1 << 19) - 100) * 64, 16, 16, 16, 1), False),
    (chunk(6710886 // 2 - 8, 0, 1, 1, 32), True),
    (chunk(6710886 // 2 - 7, 0, 1, 1, 32), False),
    (chunk((6710886 // 5 - 8) // 8, 16, 2, 8, 128), True),
    (chunk((6710886 // 5 - 8) // 8 + 1, 16, 2, 8, 128), False),
], ids=str)
def test_chunk_sizes(desc, ok):
    for fn in ("delta_chunk_fwd", "delta_chunk_bwd"):
        assert query(fn, desc) == (bd.OK if ok else bd.EUNSUPPORTED)


@pytest.mark.parametrize("batch,HV,V,ok", [
    ((1 << 23) - 1, 1, 64, True), (1 << 23, 1, 64, False),
    ((1 << 20) - 1, 8, 64, True), (1 << 20, 8, 64, False),
])
def test_step_sizes(batch, HV, V, ok):
    d = bd.DeltaStepDesc(batch, 1, 1, HV, 16, V, 1.0, bd.BF16, bd.GATE_PER_HEAD, 0)
    assert query("delta_step", d) == (bd.OK if ok else bd.EUNSUPPORTED)
