"""Gradients of dispatch and combine (ep_dispatch_backward,
ep_combine_backward): bit for bit where the definition fixes every rounding,
against 64 bits where a sum's order is the kernel's; masked entries, repeated
experts, rows nobody names, odd widths, one token; against torch's gradients
of the whole layout-dispatch-combine path."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

CASES = [  # T, H, E, K, share of masked entries
    (1, 8, 4, 1, 0.0), (1, 7168, 256, 8, 0.0), (4, 6144, 256, 8, 0.0), (3, 520, 16, 16, 0.3),
    (5, 1032, 8, 6, 0.5), (128, 7168, 288, 8, 0.0), (257, 2056, 64, 3, 0.1), (64, 1024, 2, 2, 0.9),
    (1021, 1032, 64, 6, 0.05), (2, 16392, 4, 2, 0.0),
    # rows of 64 MiB and more (nontemporal accesses): wide, narrow, few; more pairs than workgroups
    (2100, 2056, 64, 8, 0.1), (5500, 1032, 64, 6, 0.1), (512, 16392, 16, 4, 0.1), (70000, 8, 16, 16, 0.1),
]


def ep_():
    import combine_ep_layout_05_amd as ep
    return ep


def setup(T, H, E, K, masked, seed=0):
    """Buffers with a batch laid out; repeated experts in a token are allowed."""
    ep = ep_()
    g = np.random.default_rng(seed)
    idx = g.integers(0, E, size=(T, K)).astype(np.int32)
    idx[g.random((T, K)) < masked] = -1
    if T > 2 and masked:
        idx[T // 2] = -1
    P = 2 if E % 2 == 0 else 1
    b = ep.EpBuffers(T, H, K, E, P, payload="bf16")
    b.layout(torch.from_numpy(idx).cuda())
    tg = torch.Generator(device="cuda").manual_seed(seed)
    n = T * K
    mk = lambda r: torch.randn(r, H, device="cuda", generator=tg, dtype=torch.bfloat16)
    w = torch.rand(T, K, device="cuda", generator=tg)
    torch.cuda.synchronize()
    return ep, b, mk(T), mk(n), w


@pytest.mark.parametrize("T,H,E,K,masked", CASES)
def test_combine_backward(T, H, E, K, masked):
    print("combine_backward T=%d H=%d E=%d K=%d masked=%g" % (T, H, E, K, masked), flush=True)
    ep, b, go, y, w = setup(T, H, E, K, masked)
    row = b.row_of_pair.long()
    put = row >= 0
    y[~torch.zeros(T * K, dtype=torch.bool, device="cuda").index_fill_(0, row[put], True)] = float("nan")
    gy = torch.full((T * K, H), -3.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((T, K), float("nan"), device="cuda")
    b.combine_backward(go, y, w, gy, gw)
    torch.cuda.synchronize()
    tok = torch.arange(T * K, device="cuda")[put] // K
    want = torch.full_like(gy, -3.0)
    want[row[put]] = (w.reshape(-1)[put][:, None] * go.float()[tok]).to(torch.bfloat16)
    assert torch.equal(gy.view(torch.int16), want.view(torch.int16))
    terms = go.double()[tok] * y[row[put]].double()
    ref = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    ref[put], mag[put] = terms.sum(1), terms.abs().sum(1)
    # a lane adds at most H/256 + 8 products, then 6 + 16 joins; each off by half a step
    bound = (H / 256 + 32) * 2.0 ** -24 * mag
    assert bool(((gw.reshape(-1).double() - ref).abs() <= bound).all())
    assert bool((gw.reshape(-1)[~put] == 0).all())


@pytest.mark.parametrize("T,H,E,K,masked", CASES)
def test_dispatch_backward(T, H, E, K, masked):
    print("dispatch_backward T=%d H=%d E=%d K=%d masked=%g" % (T, H, E, K, masked), flush=True)
    ep, b, _, y, _ = setup(T, H, E, K, masked, seed=1)
    row = b.row_of_pair.long().reshape(T, K)
    got = b.dispatch_backward(y)
    torch.cuda.synchronize()
    acc = torch.zeros(T, H, device="cuda")
    for k in range(K):
        acc = torch.where((row[:, k] >= 0)[:, None], acc + y.float()[row[:, k].clamp_min(0)], acc)
    assert torch.equal(got.view(torch.int16), acc.to(torch.bfloat16).view(torch.int16))


def test_special_values_stay_in_their_rows():
    """Infinities and NaN in one token's gradient or one row reach only the
    values that the formula names."""
    ep, b, go, y, w = setup(6, 256, 8, 3, 0.0, seed=4)
    go[2, 7] = float("inf")
    row = b.row_of_pair.reshape(6, 3)
    y[int(row[4, 1]), 9] = float("nan")
    gy, gw = b.combine_backward(go, y, w)
    gx = b.dispatch_backward(y)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(gy.float())
    assert int(bad.sum()) == 3 and bool(bad[row[2].long(), 7].all())
    assert (~torch.isfinite(gw)).nonzero().tolist() == [[2, 0], [2, 1], [2, 2], [4, 1]]
    assert (~torch.isfinite(gx.float())).nonzero().tolist() == [[4, 9]]


def test_dedup_dispatch_backward():
    """K = P over the couples' rows: the gradient of the dedup dispatch."""
    ep = ep_()
    T, H, K, E, P = 37, 768, 8, 32, 8
    g = np.random.default_rng(8)
    idx = torch.from_numpy(g.integers(-1, E, size=(T, K)).astype(np.int32)).cuda()
    d = ep.EpDedupBuffers(T, H, K, E, P, payload="bf16")
    d.layout(idx)
    rows = torch.randn(T * P, H, device="cuda").to(torch.bfloat16)
    gx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_dispatch_backward(rows, d.tp_row, gx)
    torch.cuda.synchronize()
    r = d.tp_row.long().reshape(T, P)
    acc = torch.zeros(T, H, device="cuda")
    for p in range(P):
        acc = torch.where((r[:, p] >= 0)[:, None], acc + rows.float()[r[:, p].clamp_min(0)], acc)
    assert torch.equal(gx, acc.to(torch.bfloat16))


@pytest.mark.parametrize("fp8", [False, True])
def test_whole_path_against_autograd(fp8):
    """route -> dispatch -> a gain per expert -> combine, and back: grad of the
    logits and of x against torch's gradients of the same path in 64 bits.

    The path rounds to bf16 once in the experts' rows, once in each receive
    row's gradient (twice with the gain), once in grad_x, each off by half a
    step (2^-8) of its value; the fp32 steps in between add less than one more.
    grad_w is a dot product of bf16 rows that carry one such rounding."""
    ep = ep_()
    T, H, E, K = 48, 512, 16, 4
    g = torch.Generator(device="cuda").manual_seed(77)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda", generator=g)
    gain = torch.rand(E, H, device="cuda", generator=g) + 0.5
    go = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    b = ep.EpBuffers(T, H, K, E, 4, payload="fp8" if fp8 else "bf16")
    idx, w = b.route(logits)
    b.layout_dispatch(idx, x)
    n = T * K
    rows = b.recv_x.view(torch.float8_e4m3fn).float().reshape(n, -1, 128) * b.recv_scales[..., None] \
        if fp8 else b.recv_x.float()
    rows = rows.reshape(n, H)
    pair = b.src_pair.long()
    gains = gain[idx.reshape(-1)[pair].long()]
    y = (rows * gains).to(torch.bfloat16)
    b.combine(y, w)
    gy, gw = b.combine_backward(go, y, w)
    gx = b.dispatch_backward((gy.float() * gains).to(torch.bfloat16))
    gl = torch.empty_like(logits)
    ep.ep_route_backward(logits, idx, gw, gl)
    torch.cuda.synchronize()

    xd = x.double().requires_grad_()
    ld = logits.double().requires_grad_()
    wd = torch.softmax(torch.gather(ld, 1, idx.long()), 1)
    tok = torch.arange(n, device="cuda") // K
    seen = rows[b.row_of_pair.long()].double() if fp8 else xd[tok]
    if fp8:                                        # straight through the rounding
        seen = seen + xd[tok] - xd[tok].detach()
    ye = gain[idx.reshape(-1).long()].double() * seen
    out = (wd.reshape(-1)[:, None] * ye).reshape(T, K, H).sum(1)
    out.backward(go.double())
    step = 2.0 ** -8
    terms = (wd.detach().reshape(-1)[:, None] * gain[idx.reshape(-1).long()].double()
             * go.double()[tok]).abs().reshape(T, K, H).sum(1)
    assert bool(((gx.double() - xd.grad).abs() <= 4 * step * terms).all())
    # |error of gw| <= step * sum |go * y|; the logits' gradient is linear in gw with factors
    # q_k (delta - q_j), at most q_k each
    mag = (ye.detach().abs() * go.double()[tok].abs()).sum(1).reshape(T, K)
    lim = 2 * step * (wd.detach() * mag + wd.detach() * (wd.detach() * mag).sum(1, keepdim=True))
    err = torch.gather((gl.double() - ld.grad).abs(), 1, idx.long())
    assert bool((err <= lim).all())
    rest = torch.ones_like(gl).scatter_(1, idx.long(), 0.0)
    assert bool((gl * rest == 0).all())


def test_combine_backward_against_differences():
    """<go, combine(y + h v, w + h u)> - <go, combine(y, w)> is bilinear in y
    and w, evaluated in 64 bits from the formula the forward kernel meets bit
    for bit elsewhere: the central difference is exact up to its rounding, and
    the gradients enter with their own (bf16: half a step per element)."""
    ep, b, go, y, w = setup(9, 264, 8, 3, 0.2, seed=6)
    row = b.row_of_pair.long().reshape(9, 3)
    ok = (row >= 0)[:, :, None]
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(y.shape, device="cuda", generator=g, dtype=torch.float64)
    u = torch.randn(w.shape, device="cuda", generator=g, dtype=torch.float64)

    def f(yy, ww):
        sel = torch.where(ok, yy[row.clamp_min(0)], 0.0)
        return ((ww[:, :, None] * sel).sum(1) * go.double()).sum()
    h = 1e-3
    diff = (f(y.double() + h * v, w.double() + h * u) - f(y.double() - h * v, w.double() - h * u)) / (2 * h)
    gy, gw = b.combine_backward(go, y, w)
    along = (gy.double() * v).sum() + (gw.double() * u).sum()
    tol = 2.0 ** -8 * (gy.double() * v).abs().sum() + 1e-4 * (gw.double() * u).abs().sum() + 1e-6
    assert float((diff - along).abs()) <= float(tol)


def test_gradients_graph_replays():
    """Both gradients captured together, replayed on fresh inputs with eager
    work in between: every replay equals the eager result."""
    ep, b, go, y, w = setup(64, 2048, 32, 8, 0.1, seed=3)
    gy, gw = torch.zeros_like(y), torch.empty_like(w)
    gx = torch.empty_like(go)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    ep.ep_graph_begin(s)
    b.combine_backward(go, y, w, gy, gw, stream=s)
    b.dispatch_backward(gy, gx, stream=s)
    graph = ep.ep_graph_end(s)
    for i in range(4):
        go.copy_(torch.randn_like(go))
        w.copy_(torch.rand_like(w))
        torch.cuda.synchronize()
        graph.launch(s)
        torch.cuda.synchronize()
        ey, ew = b.combine_backward(go, y, w)
        ex = b.dispatch_backward(ey)
        torch.cuda.synchronize()
        assert torch.equal(gy, ey) and torch.equal(gw, ew) and torch.equal(gx, ex)
    graph.destroy()


def test_batch_below_the_capacity():
    """Gradients of n < T tokens use the first rows of the buffers only."""
    ep = ep_()
    b = ep.EpBuffers(50, 512, 4, 8, 2, payload="bf16")
    idx = torch.randint(0, 8, (11, 4), dtype=torch.int32, device="cuda")
    b.layout(idx)
    go = torch.randn(11, 512, device="cuda").to(torch.bfloat16)
    y = torch.randn(44, 512, device="cuda").to(torch.bfloat16)
    w = torch.rand(11, 4, device="cuda")
    gy, gw = b.combine_backward(go, y, w)
    gx = b.dispatch_backward(gy)
    torch.cuda.synchronize()
    assert gy.shape == (44, 512) and gw.shape == (11, 4) and gx.shape == (11, 512)
    row = b.row_of_pair[:44].long()
    want = (w.reshape(-1)[:, None] * go.float().repeat_interleave(4, 0)).to(torch.bfloat16)
    assert torch.equal(gy[row], want)
    with pytest.raises(ValueError, match="tokens"):
        b.combine_backward(go[:10], y, w)


def test_missing_outputs_on_a_stream_beside_a_busy_one():
    """Outputs that the call allocates are filled on its own stream: work that
    is still queued on the current stream neither delays the fill until after
    the kernel nor uses the same memory."""
    ep, b, go, y, w = setup(64, 2048, 32, 8, 0.2, seed=12)
    ey, ew = b.combine_backward(go, y, w)
    ex = b.dispatch_backward(ey)
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            a @ a                                     # tens of milliseconds on the current stream
        gone = torch.full_like(y, 5.0)                # and memory it still writes when freed
        del gone
        gy, gw = b.combine_backward(go, y, w, stream=s)
        gx = b.dispatch_backward(gy, stream=s)
        s.synchronize()
        got = [t.clone() for t in (gy, gw, gx)]       # on the current stream, after all of its work
        torch.cuda.synchronize()
        for t, e in zip(got, (ey, ew, ex)):
            assert torch.equal(t, e)


def test_dedup_combine_backward():
    """ep_combine_backward is the gradient of the two dedup levels together:
    against torch's gradients, in 64 bits, of the partials and their sum, over
    the tables of the dedup layout.  (Tokens with several experts of one
    partition, masked entries and a token without any.)"""
    ep = ep_()
    T, H, K, E, P = 41, 520, 8, 32, 8
    g = np.random.default_rng(18)
    idx_h = g.integers(-1, E, size=(T, K)).astype(np.int32)
    idx_h[7] = -1
    idx = torch.from_numpy(idx_h).cuda()
    b = ep.EpBuffers(T, H, K, E, P, payload="bf16")
    d = ep.EpDedupBuffers(T, H, K, E, P, payload="bf16")
    b.layout(idx)
    d.layout(idx)
    tg = torch.Generator(device="cuda").manual_seed(3)
    go, y = (torch.randn(r, H, device="cuda", generator=tg, dtype=torch.bfloat16) for r in (T, T * K))
    w = torch.rand(T, K, device="cuda", generator=tg)
    d.combine_partial(y, b.row_of_pair, w)
    out = d.combine_reduce()
    gy, gw = b.combine_backward(go, y, w)
    torch.cuda.synchronize()

    row = b.row_of_pair.long().reshape(T, K)
    assert int((row >= 0).sum()) > int((d.tp_row >= 0).sum()) > T       # shared copies
    yd, wd = y.double().requires_grad_(), w.double().requires_grad_()
    terms = wd[:, :, None] * yd[row.clamp_min(0)]
    bit = 1 << torch.arange(K, device="cuda")
    in_part = (d.kmask.reshape(T, P, 1) & bit) != 0                     # [T, P, K]
    in_part &= (d.tp_row.reshape(T, P, 1) >= 0) & (row >= 0)[:, None]
    partial = torch.where(in_part[..., None], terms[:, None], 0.0).sum(2)
    ref = partial.sum(1)
    # forward: each partial rounded to bf16, then their sum (half a step, 2^-8 each)
    lim = 2.0 ** -8 * (partial.abs().sum(1) + ref.abs()) * (1 + 2.0 ** -7) + 1e-30
    assert bool(((out.double() - ref).abs() <= lim).all())
    ref.backward(go.double())
    # bf16 rows: one fp32 product, rounded; weights: H/256 + 32 additions of fp32 terms
    assert bool(((gy.double() - yd.grad).abs() <= (2.0 ** -8 + 2.0 ** -23) * yd.grad.abs()).all())
    mag = (go.double()[:, None].abs() * y.double()[row.clamp_min(0)].abs()).sum(2)
    assert bool(((gw.double() - wd.grad).abs() <= (H / 256 + 32) * 2.0 ** -24 * mag).all())
    assert bool((gw[row < 0] == 0).all())
