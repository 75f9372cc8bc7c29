"""ep_expert_w4 clamps the offsets it reads on the device to the rows there are:
a model of the lookup on the CPU, over valid tables and others, then the
kernels with a table that ends past the rows."""
import numpy as np
import pytest
import torch

from tests.test_gpu_expert import make, run
from tests.test_gpu_expert_sums import check_sums

LANES = 64


def tiles_of(off, rows, height):
    """The tiles in the order of csrc/expert.hip's find_tile: lane i has E / 64
    neighbouring experts, its offsets clamped to the rows and against its own
    earlier ones; the lanes' tile counts are scanned."""
    E = len(off) - 1
    per = (E + LANES - 1) // LANES
    out = []
    for lane in range(LANES):
        o = [int(off[min(lane * per + j, E)]) for j in range(per + 1)]
        for j in range(per + 1):
            o[j] = min(max(o[j], o[j - 1] if j else 0), rows)
        for j in range(per):
            for i in range((o[j + 1] - o[j] + height - 1) // height):
                first = o[j] + i * height
                out.append((lane * per + j, first, min(height, o[j + 1] - first)))
    return out


@pytest.mark.parametrize("height", [8, 16, 64])
@pytest.mark.parametrize("E", [1, 3, 63, 64, 65, 200, 1024])
def test_lookup_stays_within_the_rows(E, height):
    g = np.random.default_rng(E)
    for trial in range(20):
        counts = g.integers(0, 1 + int(g.integers(1, 90)), E) * (g.random(E) < g.random())
        off = np.concatenate([[0], np.cumsum(counts)])
        n = int(off[-1])
        rows = n + int(g.integers(0, 4))
        tiles = tiles_of(off, rows, height)
        assert len(tiles) <= rows // height + min(rows, E)         # what is launched for
        seen = np.full(rows, -1)
        for e, first, count in tiles:
            assert count >= 1 and (seen[first:first + count] == -1).all()
            seen[first:first + count] = e
        assert np.array_equal(seen[:n], np.repeat(np.arange(E), counts)) and (seen[n:] == -1).all()
        # past the rows: as the table cut off there
        less = int(g.integers(0, n + 1))
        assert tiles_of(off, less, height) == tiles_of(np.minimum(off, less), less, height)
        # anything else (negative, falling, huge) names existing experts and rows only
        bad = g.integers(-2**31, 2**31, E + 1) if trial % 2 else g.integers(-5, 2 * rows + 5, E + 1)
        for e, first, count in tiles_of(bad, rows, height):
            assert 0 <= e < E and first >= 0 and count >= 1 and first + count <= rows


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("counts", [[1, 0, 2, 0, 0, 1], [9, 18, 0, 40], [60, 0, 150, 30]])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
def test_offsets_past_the_rows(counts, fp8, act):
    """The last experts' rows end where the rows do."""
    print("expert offsets %s fp8=%s %s" % (counts, fp8, act), flush=True)
    s = make(counts, 384, 72, act, fp8, seed=5, spare=3)
    rows = s["xv"].shape[0]
    s["off"][-1] += 100                                # rows + 97
    out = run(s, 72, act, fp8)
    s["off"] = np.minimum(s["off"], rows)
    assert torch.equal(run(s, 72, act, fp8), out)
    check_sums(s, out, act)
