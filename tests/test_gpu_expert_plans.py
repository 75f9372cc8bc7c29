"""Every kernel that ep_expert_w4 chooses from, against its definition in 64
bits: the cases name the kernel they are meant for, and the library's own rule
(csrc/expert_plan.h, compiled here for the CPU) has to choose it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import opsref
from tests.test_gpu_expert import run
from tests.test_gpu_expert_sums import check_sums

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WRAPPER = """
#include "expert_plan.h"
extern "C" void plan(int fp8, int silu, int rows, int cols, int outs, int E, long long* p)
{
    const ep::ExpertPlan x = ep::expert_plan(fp8, silu, rows, cols, outs, E);
    p[0] = x.tiles; p[1] = x.rows; p[2] = x.split; p[3] = x.groups; p[4] = x.parts; p[5] = x.workgroups;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(WRAPPER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "combine_ep_layout_05_amd", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))

    def f(fp8, act, rows, cols, outs, E):
        p = (ctypes.c_longlong * 6)()
        lib.plan(int(fp8), int(act == "silu_mul"), rows, cols, outs, E, p)
        return dict(zip(("tiles", "rows", "split", "groups", "parts", "workgroups"), p))
    return f


SPARE = 3          # rows behind the batch; they count in the rule as masked entries do
# kernel, fp8, act, cols, outs, rows per expert
CASES = {}
for act, many, wide, wider in (("none", 1032, 8200, 12296), ("silu_mul", 520, 4104, 6152)):
    for fp8 in (True, False):
        t = ("fp8_" if fp8 else "bf16_") + act
        few = "stream8" if fp8 else "stream16"                  # up to 2 rows per expert
        # one wave per group: many experts of 0 to 2 rows; 19 blocks: a second, clamped window of
        # scales; few experts of many rows
        CASES["one_wave_" + t] = (few, 1, fp8, act, 384, many, [0, 1, 2, 1, 0, 1, 2, 0, 1, 2] * 15)
        CASES["one_wave_second_window_" + t] = (few, 1, fp8, act, 2432, wide,
                                                [0] * 5 + [1, 0, 9, 0, 0, 3] + [0] * 5)
        CASES["one_wave_deep_" + t] = ("stream16", 1, fp8, act, 384, wider, [40, 20, 35, 25])
        # four waves per group, each with more than 16 blocks: even and odd
        CASES["four_waves_second_window_" + t] = (few, 4, fp8, act, 8448, 40, [1, 0, 2, 0, 0, 1])
        CASES["four_waves_second_window_odd_" + t] = ("stream16", 4, fp8, act, 8576, 72, [17, 0, 5])
        # more row tiles than run together, in several groups of weight rows
        CASES["chunks_" + t] = ("tiles", 0, fp8, act, 384, 600 if act == "none" else 328,
                                [900, 0, 700, 650, 77, 3, 128, 64])
        # long columns, an odd and an even number of blocks; tiles of every number of row groups
        CASES["tiles_long_odd_" + t] = ("tiles", 0, fp8, act, 2176, 3400 if act == "none" else 1704,
                                        [0, 130, 0, 0, 65, 1, 17, 48] + [0] * 32)
        CASES["tiles_long_" + t] = ("tiles", 0, fp8, act, 2304, 3400 if act == "none" else 1704,
                                    [33, 0, 0, 64, 0, 2, 0, 81] + [0] * 32)


def make(fp8, act, cols, outs, counts, seed):
    g = np.random.default_rng(seed)
    E, n, blocks = len(counts), int(sum(counts)) + SPARE, cols // 128
    N = 2 * outs if act == "silu_mul" else outs
    s = dict(off=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
             codes=g.integers(0, 256, size=(E, N, cols // 2), dtype=np.uint8),
             scales=(g.uniform(0.5, 1.5, size=(E, N, blocks)) * 0.4 / np.sqrt(cols)).astype(np.float32))
    if fp8:
        by = g.integers(0, 0x69, size=(n, cols), dtype=np.uint8)
        s["x"] = by | g.integers(0, 2, size=by.shape, dtype=np.uint8) << 7
        s["xs"] = g.uniform(0.005, 0.02, size=(n, blocks)).astype(np.float32)
        s["xv"] = opsref.e4m3(s["x"]) * np.repeat(s["xs"].astype(np.float64), 128, axis=1)
    else:
        t = torch.from_numpy(g.standard_normal((n, cols)).astype(np.float32)).to(torch.bfloat16)
        s["x"], s["xs"], s["xv"] = t, None, t.double().numpy()
    return s


def form(p):
    return ("tiles" if p["tiles"] else "stream%d" % p["rows"], p["split"])


@pytest.mark.parametrize("name", sorted(CASES))
def test_cases_reach_their_kernels(plan, name):
    kernel, split, fp8, act, cols, outs, counts = CASES[name]
    p = plan(fp8, act, sum(counts) + SPARE, cols, outs, len(counts))
    assert form(p) == (kernel, split), p
    blocks = cols // 128
    if "second_window" in name:              # blocks of the first wave, in pairs
        assert ((blocks + 1) // 2 + split - 1) // split * 2 > 16
    if "chunks" in name:
        assert sum((c + 63) // 64 for c in counts) > 32 and p["groups"] > 1
    elif split == 1:
        assert outs % (64 if act == "none" else 32) != 0         # a ragged last group


@pytest.mark.parametrize("fp8", [True, False])
def test_choice_by_rows_and_workgroups(plan, fp8):
    """The rule at measured points (gate and up of 2048, 4096 columns: 16 groups
    per expert): few rows or few workgroups stream, and where the workgroups
    of tiles come close to filling the GPU the choice does not jump."""
    def tiles(E, per_expert, cols=4096, outs=2048, act="silu_mul"):
        return bool(plan(fp8, act, E * per_expert, cols, outs, E)["tiles"])
    for E, stream, tile in ((1, 512, 1024), (4, 128, 256), (8, 32, 128), (16, 16, 32), (24, 4, 16),
                            (31, 2, 4), (32, 1, 2), (256, 1, 2)):
        assert not tiles(E, stream) and tiles(E, tile), E
    first = [next(r for r in range(1, 5000) if tiles(E, r)) for E in range(1, 40)]
    assert first == sorted(first, reverse=True)                # more workgroups, fewer rows
    assert first[30] <= first[31] + 1                          # 31 and 32 experts
    assert not tiles(18, 16, 1024, 7168, "none") and tiles(18, 64, 1024, 7168, "none")
    assert not tiles(64, 16, 1024, 256) and tiles(64, 64, 1024, 256)
    # no overflow at the largest sizes the call takes
    assert plan(fp8, "none", 2**31 - 1, 2**23, 8, 1024)["tiles"]
    assert plan(fp8, "none", 2**31 - 1, 2**23, 8, 1)["workgroups"] > 0


def test_every_kernel_is_reached():
    reached = {(c[0], c[1], c[2], c[3]) for c in CASES.values()}
    for act in ("none", "silu_mul"):
        for split in (1, 4):
            assert {("stream8", split, True, act), ("stream16", split, True, act),
                    ("stream16", split, False, act)} <= reached
        assert {("tiles", 0, True, act), ("tiles", 0, False, act)} <= reached


def test_launch_limits(plan):
    """Sizes that ep.h says are taken have launches below 2^32 threads; where the
    launch is larger the call refuses."""
    import combine_ep_layout_05_amd as ep
    fake = ctypes.c_void_p(0x10000)                    # never dereferenced: refused before

    def rc(payload, rows, cols, E, outs, act):
        return ep._lib.ep_expert_w4(fake, fake, payload, rows, cols, fake, E, fake, fake, outs, act,
                                    fake, None)
    g = np.random.default_rng(0)
    over = under = 0
    for _ in range(4000):
        rows, E = int(2 ** g.uniform(0, 31)) - 1, int(2 ** g.uniform(0, 10.01))
        outs, cols = int(2 ** g.uniform(3, 26)) // 8 * 8, 128 * int(2 ** g.uniform(0, 9))
        fp8, silu = bool(g.integers(2)), int(g.integers(2))
        threads = plan(fp8, "silu_mul" if silu else "none", rows, cols, outs, E)["workgroups"] * 256
        m = min(rows, E)
        taken = (rows // 64 + m + 32) * (outs + 256) < 2 ** (32 - silu) and \
            (rows // 8 + m) * (outs + 64) < 2 ** (30 - silu)
        if taken:
            assert threads < 2 ** 32
            under += 1
        if threads >= 2 ** 32:
            assert rc(0 if fp8 else 1, rows, cols, E, outs, silu) == -1
            over += 1
    assert over > 200 and under > 200
    # streaming, 4 waves per group: refused well below 2^38 elements of output
    p = plan(True, "none", 1024, 4096, 1 << 20, 1024)
    assert not p["tiles"] and p["workgroups"] * 256 >= 2 ** 32
    assert rc(0, 1024, 4096, 1024, 1 << 20, 0) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_products(name):
    kernel, split, fp8, act, cols, outs, counts = CASES[name]
    print("expert plan %s: %s/%d C=%d D=%d" % (name, kernel, split, cols, outs), flush=True)
    s = make(fp8, act, cols, outs, counts, seed=cols + outs)
    check_sums(s, run(s, outs, act, fp8), act)
