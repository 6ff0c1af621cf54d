"""The counting of finished tiles in the orthogonalisation's persistent kernel, as a discrete model on the CPU.

Every epilogue warp takes every tile: it waits for the tile's accumulator (two take turns; the next but one is
computed once all warps have released this one), releases it, stores its box and arrives on the tile's barrier of
a ring. Warp 0 also waits for that barrier's phase and then counts the tile for the CTAs that depend on it: by
then every warp must have stored. The search below walks every interleaving of three warps."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_grouped_gemm_fp32_b200", "csrc",
                      "orthogonalise.cu")


def ring_of_the_kernel():
    """Barriers that the kernel's epilogue warps arrive on in turn: the `stored` member of its shared memory."""
    text = open(SOURCE).read()
    smem = re.search(r"struct SmemO \{(.*?)\n\};", text, re.S).group(1)
    size = re.search(r"uint64_t stored(?:\[(\w+)\])?;", smem).group(1)
    if size is None:
        return 1
    return int(size) if size.isdigit() else int(re.search(rf"constexpr int {size} = (\d+);", text).group(1))


def counts_a_tile_early(ring, warps=3, tiles=7):
    """Whether some interleaving counts a tile that a warp has not stored."""
    WAIT, RELEASE, STORE, COUNT = range(4)
    start = tuple((0, WAIT) for _ in range(warps))
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        released = [t + (phase > RELEASE) for t, phase in state]      # tiles released, stored, by each warp
        stored = [t + (phase > STORE) for t, phase in state]
        for w, (t, phase) in enumerate(state):
            if t == tiles:
                continue
            if phase == WAIT:
                if t >= 2 and min(released) < t - 1:                  # accumulator t % 2 is not free yet
                    continue
                step = (t, RELEASE)
            elif phase == RELEASE:
                step = (t, STORE)
            elif phase == STORE:
                step = (t, COUNT) if w == 0 else (t + 1, WAIT)
            else:
                arrivals = sum(len(range(t % ring, s, ring)) for s in stored)
                if (arrivals // warps & 1) == (t // ring & 1):        # the phase of this parity has not completed
                    continue
                if min(stored) <= t:
                    return True
                step = (t + 1, WAIT)
            new = state[:w] + (step,) + state[w + 1:]
            if new not in seen:
                seen.add(new)
                todo.append(new)
    return False


@pytest.mark.parametrize("ring", [1, 2])
def test_the_model_finds_rings_that_are_too_small(ring):
    assert counts_a_tile_early(ring)


def test_no_tile_is_counted_before_every_warp_has_stored_it():
    assert not counts_a_tile_early(ring_of_the_kernel())
