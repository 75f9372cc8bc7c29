"""ep_expert_w4 against its definition in 64 bits: both row types and both
epilogues, one row to many rows per expert, empty experts, ragged sizes, every
code, rows past the batch; and the serving step route -> layout and dispatch
-> experts -> combine, eager and replayed."""
import numpy as np
import pytest
import torch

from tests import opsref

pytestmark = pytest.mark.gpu


def ep_():
    import combine_ep_layout_05_amd as ep
    return ep


def bits(a):
    return torch.from_numpy(a).cuda()


def make(counts, cols, outs, act, fp8, seed, spare=3):
    """Rows laid out expert by expert (`spare` rows behind the last), weights,
    outputs filled with a pattern."""
    g = np.random.default_rng(seed)
    E, n = len(counts), int(sum(counts)) + spare
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    N = 2 * outs if act == "silu_mul" else outs
    s = dict(off=off, codes=g.integers(0, 256, size=(E, N, cols // 2)).astype(np.uint8),
             scales=(g.uniform(0.5, 1.5, size=(E, N, cols // 128)) * 0.4 / np.sqrt(cols)).astype(np.float32))
    if fp8:
        by = g.integers(0, 256, size=(n, cols)).astype(np.uint8)
        by[(by & 127) == 127] = 0x3A                   # no NaN
        by[(by & 127) > 0x68] -= 0x20                  # mostly of moderate size
        s["x"] = by
        s["xs"] = g.uniform(0.005, 0.02, size=(n, cols // 128)).astype(np.float32)
        s["xv"] = opsref.e4m3(by) * np.repeat(s["xs"].astype(np.float64), 128, axis=1)
    else:
        t = torch.from_numpy(g.standard_normal((n, cols)).astype(np.float32)).to(torch.bfloat16)
        s["x"], s["xs"], s["xv"] = t, None, t.double().numpy()
    return s


def run(s, outs, act, fp8):
    ep = ep_()
    x = bits(s["x"]) if fp8 else s["x"].cuda()
    out = torch.full((x.shape[0], outs), -7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_w4(x, bits(s["xs"]) if fp8 else None, bits(s["off"]), bits(s["codes"]),
                    bits(s["scales"]), out, act=act)
    torch.cuda.synchronize()
    return out


def check(s, out, act):
    """fp32 sums: the products of a block are exact or rounded once, at most 128 additions within
    a block, one scale product and one addition per block, each off by at most one step (2^-23,
    a truncated addition included); silu has slope at most 1.1 and is computed within
    (|g| + 8) steps; the result is rounded to bf16 once (2^-8).

    fp8 rows: the matrix instruction adds the 16 products of a lane's 16 bytes in fixed point, in
    steps of 2^-14 of the power of two below the largest product, dropping what is smaller (read off
    the instruction: next to 2^16, 14.06 counts as 12 and 7.03 as 0; between groups it adds in
    fp32).  So each of a block's 128 products is off by less than 2^-14 of the largest, which is at
    most max|x| * max|w| over the block."""
    n = int(s["off"][-1])
    want, acc, mag = opsref.expert(s["xv"][:n], s["off"], s["codes"], s["scales"], act)
    got = out[:n].double().cpu().numpy()
    blocks = s["scales"].shape[2]
    d = (128 + 2 * blocks + 8) * 2.0 ** -23 * mag
    if s.get("xs") is not None:
        xm = abs(s["xv"][:n]).reshape(n, blocks, 128).max(2)
        for e in range(len(s["off"]) - 1):
            a, b = int(s["off"][e]), int(s["off"][e + 1])
            d[a:b] += 128 * 2.0 ** -14 * xm[a:b] @ (6.0 * s["scales"][e].T)
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


COUNTS = {
    "one_row": [0, 1, 0],
    "one_each": [1] * 9,
    "ragged": [0, 3, 16, 17, 0, 1, 40, 2, 33, 0, 0, 5],
    "single_expert": [70],
    "one_large": [1, 0, 300, 2],
    "last_only": [0] * 40 + [2],
    "many_experts": ([0, 1, 0, 2] * 256),
    "ragged_large": [0, 130, 64, 65, 0, 1, 700, 2, 33, 0, 0, 15],
    "many_larger": ([0, 11, 1, 24] * 256),
}


@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("cols,outs", [(128, 8), (384, 72), (640, 40), (896, 264), (1152, 24), (1280, 200)])
def test_products(counts, cols, outs, act, fp8):
    if counts in ("many_experts", "many_larger") and cols > 128:
        pytest.skip("covered by the small size")
    print("expert %s C=%d D=%d %s fp8=%s" % (counts, cols, outs, act, fp8), flush=True)
    s = make(COUNTS[counts], cols, outs, act, fp8, seed=cols + outs)
    check(s, run(s, outs, act, fp8), act)


@pytest.mark.parametrize("fp8,cols,outs,act,counts", [
    (True, 7168, 512, "silu_mul", [2, 0, 5, 1]), (False, 2048, 1032, "none", [7, 130, 0, 1]),
    (False, 6144, 264, "silu_mul", [1, 1, 20]), (True, 2560, 2000, "none", [129, 64, 63, 128]),
])
def test_products_large(fp8, cols, outs, act, counts):
    print("expert large C=%d D=%d %s fp8=%s" % (cols, outs, act, fp8), flush=True)
    s = make(counts, cols, outs, act, fp8, seed=cols)
    check(s, run(s, outs, act, fp8), act)


@pytest.mark.parametrize("fp8", [True, False])
def test_every_code_at_every_column(fp8):
    """One-hot rows pick single weights: output = code value * scale exactly
    (bf16 holds both), for each of a block's 128 columns."""
    cols, outs = 256, 64
    g = np.random.default_rng(2)
    codes = g.integers(0, 256, size=(1, outs, cols // 2)).astype(np.uint8)
    scales = (2.0 ** g.integers(-3, 4, size=(1, outs, 2))).astype(np.float32)
    eye = np.eye(cols)
    s = dict(off=np.array([0, cols], np.int32), codes=codes, scales=scales)
    if fp8:
        s["x"], s["xs"] = (eye * 0x38).astype(np.uint8), np.full((cols, 2), 2.0, np.float32)   # 0x38 = 1.0
        factor = 2.0
    else:
        s["x"], s["xs"] = torch.from_numpy(eye.astype(np.float32)).to(torch.bfloat16), None
        factor = 1.0
    out = run(s, outs, "none", fp8).double().cpu().numpy()
    w = np.empty((outs, cols))
    w[:, 0::2], w[:, 1::2] = opsref.E2M1[codes[0] & 15], opsref.E2M1[codes[0] >> 4]
    want = (w * np.repeat(scales[0], 128, axis=1)).T * factor
    np.testing.assert_array_equal(out, want)


@pytest.mark.parametrize("fp8", [True, False])
def test_unused_rows_and_experts_are_not_read_into_results(fp8):
    """NaN in the rows behind the batch and in the scales of experts without
    rows, and offsets past the rows, change nothing."""
    s = make([0, 5, 0, 18, 0], 256, 40, "silu_mul", fp8, seed=3)
    ref = run(s, 40, "silu_mul", fp8)
    s["scales"][[0, 2, 4]] = np.nan
    if fp8:
        s["x"][23:] = 0x7F
        s["xs"][23:] = np.nan
    else:
        s["x"][23:] = float("nan")
    assert torch.equal(run(s, 40, "silu_mul", fp8), ref)


@pytest.mark.parametrize("fp8", [True, False])
def test_special_rows_stay_apart(fp8):
    """A row with a NaN or a zero scale changes no other row."""
    s = make([20, 3], 256, 24, "none", fp8, seed=9)
    ref = run(s, 24, "none", fp8)
    if fp8:
        s["xs"][4, 1], s["x"][7, 3], s["xs"][9] = np.nan, 0x7F, 0.0
    else:
        s["x"][4, 200], s["x"][7, 3], s["x"][9] = float("nan"), float("inf"), 0.0
    out = run(s, 24, "none", fp8)
    same = [r for r in range(23) if r not in (4, 7, 9)]
    assert torch.equal(out[same], ref[same])
    assert bool(out[4].isnan().all()) and bool((out[9] == 0).all())
    assert not bool(torch.isfinite(out[7].float()).any()) or not fp8


def test_no_rows():
    ep = ep_()
    s = make([0, 0, 0], 128, 16, "none", True, seed=1, spare=4)
    assert bool((run(s, 16, "none", True) == -7.0).all())
    z = lambda *sh, dt=torch.uint8: torch.zeros(*sh, dtype=dt, device="cuda")
    ep.ep_expert_w4(z(0, 128), z(0, 1, dt=torch.float32), bits(s["off"]), bits(s["codes"]),
                    bits(s["scales"]), z(0, 16, dt=torch.bfloat16))
    torch.cuda.synchronize()


def serving(T, H, I, E, K, payload, seed):
    ep = ep_()
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = ep.EpBuffers(T, H, K, E, 4, payload=payload)
    w_up = torch.randn(E, 2 * I, H, device="cuda", generator=g) * H ** -0.5
    w_down = torch.randn(E, H, I, device="cuda", generator=g) * I ** -0.5
    experts = ep.EpExpertsW4(T, K, *ep.w4_quantise(w_up), *ep.w4_quantise(w_down))
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda", generator=g)
    return ep, b, experts, x, logits


@pytest.mark.parametrize("payload", ["fp8", "bf16"])
@pytest.mark.parametrize("T,H,I,E,K", [(1, 512, 256, 16, 4), (5, 1024, 128, 8, 8), (70, 256, 384, 12, 3)])
def test_serving_step(T, H, I, E, K, payload):
    """route -> layout and dispatch -> experts -> combine; each product checked
    on what the step before it left."""
    print("serving T=%d H=%d I=%d E=%d K=%d %s" % (T, H, I, E, K, payload), flush=True)
    ep, b, experts, x, logits = serving(T, H, I, E, K, payload, T)
    logits[:, 2] = -float("inf")
    idx, w = b.route(logits, scale=1.5)
    b.layout_dispatch(idx, x)
    experts.mid.fill_(-7.0)
    experts.out.fill_(-7.0)
    y = experts(b)
    out = b.combine(y, w)
    torch.cuda.synchronize()
    off = b.expert_offset.cpu().numpy()
    fp8 = payload == "fp8"
    if fp8:
        xv = opsref.e4m3(b.recv_x.cpu().numpy()) * np.repeat(b.recv_scales.double().cpu().numpy(), 128, 1)
    else:
        xv = b.recv_x.double().cpu().numpy()
    check(dict(off=off, codes=experts.w_up.cpu().numpy(), scales=experts.s_up.cpu().numpy(), xv=xv,
               xs=b.recv_scales),
          experts.mid, "silu_mul")
    check(dict(off=off, codes=experts.w_down.cpu().numpy(), scales=experts.s_down.cpu().numpy(),
               xv=experts.mid.double().cpu().numpy()), experts.out, "none")
    rid, rw, _ = opsref.route(logits.double().cpu().numpy(), K, "softmax", None, True, 1.5)
    assert np.array_equal(idx.cpu().numpy(), rid)
    row = b.row_of_pair.long().reshape(T, K)
    terms = w.double()[:, :, None] * y.double()[row]
    bound = 2.0 ** -8 * terms.sum(1).abs() + (K + 1) * 2.0 ** -24 * terms.abs().sum(1)
    assert bool(((out.double() - terms.sum(1)).abs() <= bound * (1 + 2.0 ** -8)).all())


@pytest.mark.parametrize("T,E,K,payload", [(6, 16, 4, "fp8"), (200, 4, 2, "fp8"), (200, 4, 2, "bf16")])
def test_serving_step_captured(T, E, K, payload):
    """The whole step in one graph, replayed on new tokens; and two of them on
    two streams at once, each with its own buffers."""
    steps = [serving(T, 512, 256, E, K, payload, 3), serving(T, 512, 256, E, K, payload, 4)]
    graphs = []
    for ep, b, experts, x, logits in steps:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        ep.ep_graph_begin(s)
        idx, w = b.route(logits, stream=s)
        b.layout_dispatch(idx, x, stream=s)
        b.combine(experts(b, stream=s), w, stream=s)
        graphs.append((ep.ep_graph_end(s), s))
    for i in range(4):
        for ep, b, experts, x, logits in steps:
            x.copy_(torch.randn_like(x))
            logits.copy_(torch.randn_like(logits))
            if i == 2:
                logits[3] = -float("inf")          # a padding token: no expert, output 0
        torch.cuda.synchronize()
        for g, s in graphs:
            g.launch(s)
        torch.cuda.synchronize()
        got = [b.out.clone() for _, b, *_ in steps]
        for (ep, b, experts, x, logits), o in zip(steps, got):
            idx, w = b.route(logits)
            b.layout_dispatch(idx, x)
            assert torch.equal(b.combine(experts(b), w), o)
            if i == 2:
                assert bool((o[3] == 0).all())
        torch.cuda.synchronize()
    for g, _ in graphs:
        g.destroy()
