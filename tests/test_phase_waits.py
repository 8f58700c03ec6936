"""The waits of the persistent decode by parity, on a model of the barriers.

An mbarrier wait names a phase only by its parity. Asked for phase k while phase k - 1 is
still open it answers "complete" at once (phase k - 2 has the same parity), and asked for
phase k - 1 once phase k is complete as well it waits for phase k + 1. The decode's softmax
clears the rows past a partition's end in the V slot of tile j, after waiting for that tile.
Its P buffers (NP of them) prove that V tile j - NP has landed; the slot's previous tile is
j - NV. With NP > NV that tile may still be on its way, so the softmax first waits for the
value product that read it, on a barrier whose phases it has followed.
"""
import os
import re

import pytest

from paged_kv_cache_442_b200 import build as pa_build

NV, NP = 3, 4


def passes(completed, phase):
    """try_wait.parity on a barrier with `completed` phases behind it."""
    return (completed & 1) != (phase & 1)


def phases(ring, j, done):
    """Completed phases of tile j's slot when the tiles 0 .. done - 1 are done, in order."""
    return sum(t < done for t in range(j % ring, done + ring, ring) if t < done)


def guarded(j, landed, produced):
    """(does the guarded wait pass, is it right to) for V tiles 0 .. landed - 1 in shared
    memory and value products 0 .. produced - 1 done (each needs its tile)."""
    t = j - NV
    if t >= 0 and not passes(phases(NP, t, produced), t // NP):
        return False, True
    ok = passes(phases(NV, j, landed), j // NV)
    return ok, (not ok) or landed > j


@pytest.mark.parametrize("j", range(0, 24))
def test_the_guarded_wait_is_sound_and_ends(j):
    # tile j's P buffer was last read by tile j - NP: that product is done; tile j's own
    # product waits for the softmax, so at most j products are
    for produced in range(max(0, j - NP + 1), j + 1):
        for landed in range(produced, j + 2):
            if landed > produced + NV:      # a V slot is refilled once its product is done
                continue
            ok, right = guarded(j, landed, produced)
            assert right
            if produced > j - NV and landed > j:
                assert ok                   # nothing left to wait for


def test_a_bare_wait_is_not_sound():
    # V tile 4 of slot 1 still on its way: the wait for tile 7 passes all the same
    assert passes(phases(NV, 7, 4), 7 // NV)


def test_waiting_for_the_slot_s_previous_phase_may_never_end():
    # tiles 4 and 7 have both landed: phase 4 // NV asked for afterwards waits for tile 10
    assert not passes(phases(NV, 7, 8), 7 // NV - 1)


def test_the_kernel_guards_its_wait():
    src = open(os.path.join(pa_build.CSRC, "decode_tc.cu")).read()
    ring = dict(re.findall(r"constexpr int (N[PV]) = (\d+);", src))
    assert int(ring["NP"]) == NP and int(ring["NV"]) == NV
    at = src.index("failed |= !wait_or_abort(&v_full[vs]")
    assert re.search(r"t = j - NV;\s+failed \|= !wait_or_abort\(&pv_done\[t % NP\], \(t / NP\) & 1", src[at - 400:at])


def test_the_block_scale_decode_needs_no_guard():
    src = open(os.path.join(pa_build.CSRC, "decode_blockscale.cu")).read()
    assert "static_assert(NP <= NV" in src
