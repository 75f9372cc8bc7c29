"""ep_expert_w4 holds its sums in 32 bits whatever the rows' type: small
products beside large ones that cancel, where a sum in fewer bits would drop
them; and the same values give the same bits as fp8 and as bf16 rows."""
import numpy as np
import pytest
import torch

from tests import opsref
from tests.test_gpu_expert import make, run

# rows per expert: up to 2048 columns "stream" and "stream_deep" take the streaming kernel, "tiles"
# the tile kernel; with more all of them stream (test_gpu_expert_plans has long columns on tiles)
COUNTS = {"stream": [0, 1, 3, 0, 1, 0, 0, 2, 0, 1], "stream_deep": [7, 8, 9, 0, 33],
          "tiles": [70, 1, 0, 130], "tiles_one": [300]}


def small_beside_large(counts, cols, outs, fp8, seed):
    """Rows whose every block holds one +448 and one -448, under equal codes of
    value 1, and otherwise values below 0.25 in steps of 2^-9.

    Every product is a multiple of 2^-10, and the magnitudes of a row's products
    add up to less than 2 * 448 + 126 * 0.25 * 6 = 1085 per block, below 2^14 for
    up to 15 blocks: any partial sum, in whatever order, is a multiple of 2^-10
    below 2^14, which 24 bits hold exactly.  With scales of 1 an fp32 sum is
    therefore exact, and the output its one rounding to bf16."""
    g = np.random.default_rng(seed)
    n, blocks = int(sum(counts)) + 3, cols // 128
    assert blocks <= 15
    by = g.integers(0, 0x28, size=(n, blocks, 128)).astype(np.uint8)      # 0 .. 0.234
    by |= (g.integers(0, 2, size=by.shape) << 7).astype(np.uint8)
    at = np.stack([g.permutation(128)[:2] for _ in range(blocks)])
    E = len(counts)
    code = g.integers(0, 16, size=(E, outs, blocks, 128)).astype(np.uint8)
    for b in range(blocks):
        by[:, b, at[b, 0]], by[:, b, at[b, 1]] = 0x7E, 0xFE               # +448, -448
        code[:, :, b, at[b, 0]] = code[:, :, b, at[b, 1]] = 2             # both times 1
    by, code = by.reshape(n, cols), code.reshape(E, outs, cols)
    s = dict(off=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
             codes=code[:, :, 0::2] | code[:, :, 1::2] << 4,
             scales=np.ones((E, outs, blocks), np.float32), xv=opsref.e4m3(by))
    if fp8:
        s["x"], s["xs"] = by, np.ones((n, blocks), np.float32)
    else:
        s["x"], s["xs"] = torch.from_numpy(s["xv"].astype(np.float32)).to(torch.bfloat16), None
    return s


def test_the_inputs_need_the_bits():
    """On the CPU: dropping what lies below 2^-14 of the largest product of 16
    changes the outputs, so the tests below tell such a sum from one in 32 bits."""
    s = small_beside_large([4], 384, 16, True, 1)
    want, _, _ = opsref.expert(s["xv"][:4], s["off"], s["codes"], s["scales"], "none")
    w = np.empty((16, 384))
    w[:, 0::2], w[:, 1::2] = opsref.E2M1[s["codes"][0] & 15], opsref.E2M1[s["codes"][0] >> 4]
    p = (s["xv"][:4, None, :] * w).reshape(4, 16, 24, 16)
    step = 2.0 ** (np.floor(np.log2(abs(p).max(-1, keepdims=True))) - 14)
    cut = (np.trunc(p / step) * step).sum((2, 3))
    assert (abs(cut - want) > 2.0 ** -8 * abs(want)).mean() > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("cols,outs", [(128, 8), (384, 72), (640, 200), (1920, 264)])
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_small_products_beside_large_ones(counts, cols, outs):
    for fp8 in (True, False):
        print("sums %s C=%d D=%d fp8=%s" % (counts, cols, outs, fp8), flush=True)
        s = small_beside_large(COUNTS[counts], cols, outs, fp8, seed=cols)
        n = int(s["off"][-1])
        acc, _, _ = opsref.expert(s["xv"][:n], s["off"], s["codes"], s["scales"], "none")
        want = torch.from_numpy(acc).to(torch.float32).to(torch.bfloat16)       # acc is exact in fp32
        got = run(s, outs, "none", fp8).cpu()
        assert torch.equal(got[:n] + 0.0, want + 0.0)                            # (-0 and +0 alike)


def check_sums(s, out, act):
    """Sums in 32 bits, whatever the rows' type.  fp8 rows: values below 2 and
    values from 2 on are summed apart, 16 products at a time in fixed point, which
    is exact: e4m3 values below 2 times e2m1 values are multiples of 2^-10 below
    2^3.5, those from 2 on multiples of 2^-3 below 2^11.4, both within 2^-14 of the
    power of two below the largest.  A sum of 16 fits 24 bits.  At most 16 of these
    (bf16 rows: 128 products) are added in fp32 per block, then one scale product
    and one addition per block, and 8 more joins, each off by at most one step
    (2^-23, a truncated addition included); SiLU has slope at most 1.1 and is
    computed within (|g| + 8) steps; the result is rounded to bf16 once (2^-8)."""
    n, blocks = int(s["off"][-1]), s["scales"].shape[2]
    want, acc, mag = opsref.expert(s["xv"][:n], s["off"], s["codes"], s["scales"], act)
    got = out[:n].double().cpu().numpy()
    d = ((16 if s.get("xs") is not None else 128) + 2 * blocks + 8) * 2.0 ** -23 * mag
    if act == "silu_mul":
        D = want.shape[1]
        g, u, dg, du = acc[:, :D], acc[:, D:], d[:, :D], d[:, D:]
        sg = abs(g / (1 + np.exp(-g)))
        d = 1.1 * dg * (abs(u) + du) + (sg + 1.1 * dg) * du + (abs(g) + 8) * 2.0 ** -23 * sg * abs(u)
    bound = d * (1 + 2.0 ** -8) + 2.0 ** -8 * abs(want) + 2.0 ** -126
    bad = ~(abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(),
                           got[bad][:5].tolist(), want[bad][:5].tolist())
    assert bool((out[n:] == -7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("cols,outs", [(128, 40), (896, 136), (2176, 72)])
def test_fp8_sums_within_32_bits(counts, cols, outs, act):
    """Half of the values below 0.12, and pairs of +-448 that cancel."""
    print("fp8 sums %s C=%d D=%d %s" % (counts, cols, outs, act), flush=True)
    s = make(COUNTS[counts], cols, outs, act, True, seed=cols + 1)
    g = np.random.default_rng(3)
    # every fourth column pair cancels: +-448 under equal codes
    for c in range(0, cols, 8):
        s["x"][:, c], s["x"][:, c + 1] = 0x7E, 0xFE
        low = s["codes"][:, :, c // 2] & 15
        s["codes"][:, :, c // 2] = low | low << 4
    small = g.random(s["x"].shape) < 0.5
    s["x"] = np.where(small & ((s["x"] & 127) < 0x7E), s["x"] & 0x9F, s["x"])    # below 0.12
    s["xv"] = opsref.e4m3(s["x"]) * np.repeat(s["xs"].astype(np.float64), 128, axis=1)
    check_sums(s, run(s, outs, act, True), act)
