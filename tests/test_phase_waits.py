"""The waits of the persistent decode by parity, on a model of the barriers.

An mbarrier wait names a phase only by its parity: asked for phase k while phase k - 1 is
still open, it answers "complete" because phase k - 2 has the same parity. The decode's
softmax clears the rows past a partition's end in the V slot of tile j, after waiting for
that tile. Its P buffers (NP of them) prove that V tile j - NP has landed; the slot's
previous tile is j - NV. With NP > NV the previous tile may still be on its way, so the
wait needs the previous phase first.
"""
import os
import re

import pytest

from paged_kv_cache_442_b200 import build as pa_build

NV, NP = 3, 4


class Barrier:
    """Completed phases of one ring slot; wait(k) answers as try_wait.parity does."""

    def __init__(self, completed):
        self.completed = completed

    def passes(self, phase):
        return (self.completed & 1) != (phase & 1)


def landed_when_the_wait_passes(j, oldest_missing, waits):
    """Tile j's wait(s) while V tiles from `oldest_missing` on are still in flight: does
    every wait that passes mean that tile j has landed?"""
    slot_tiles = [t for t in range(j + 1) if t % NV == j % NV]
    done = sum(t < oldest_missing for t in slot_tiles)
    bar = Barrier(done)
    passed = all(bar.passes(ph) for ph in waits)
    return (not passed) or done == len(slot_tiles)


@pytest.mark.parametrize("j", range(NV, 24))
def test_waiting_for_the_previous_phase_first_is_sound(j):
    # pv_done of tile j - NP has been waited for: V tiles up to j - NP have landed
    for missing in range(max(0, j - NP + 1), j + 2):
        assert landed_when_the_wait_passes(j, missing, [j // NV - 1, j // NV])


def test_the_single_wait_is_not():
    assert not landed_when_the_wait_passes(7, 7 - NV, [7 // NV])


def test_the_kernel_waits_for_both_phases():
    src = open(os.path.join(pa_build.CSRC, "decode_tc.cu")).read()
    ring = dict(re.findall(r"constexpr int (N[PV]) = (\d+);", src))
    assert int(ring["NP"]) == NP and int(ring["NV"]) == NV
    waits = re.findall(r"failed \|= !wait_or_abort\(&v_full\[vs\], \(([^&]+)\) & 1", src)
    assert waits == ["(j / NV) - 1", "j / NV"]
