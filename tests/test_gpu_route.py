"""ep_route and ep_route_backward against their definitions in 64 bits: types,
sizes from one token and one expert to the limits, ties, switched-off experts,
rows with nothing left, infinities and NaN; the gradient against the formula
and against differences of the kernel's own weights."""
import numpy as np
import pytest
import torch

from tests import opsref

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24                       # half a step of fp32, relative


def ep_():
    import combine_ep_layout_05_amd as ep
    return ep


def run(l, K, bias=None, **kw):
    ep = ep_()
    T = l.shape[0]
    ids = torch.full((T, K), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), 1e30, device="cuda")
    ep.ep_route(l, ids, w, bias=bias, **kw)
    torch.cuda.synchronize()
    return ids, w


def tolerance(l, E):
    """Relative error of a weight: the exponent's argument l - m is rounded
    (its size times half a step), exp and the division are within a few steps,
    the sum of E terms is at most E/64 + 10 additions deep; the same again for
    the terms of the sum.  The range counts up to 104, where exp is 0."""
    fin = l[np.isfinite(l)]
    rng = min(float(fin.max() - fin.min()), 104.0) if fin.size else 0.0
    return (2 * rng + E / 64 + 26) * EPS


def make(T, E, seed, dtype, spread=1.5):
    g = np.random.default_rng(seed)
    l = torch.from_numpy((spread * g.standard_normal((T, E))).astype(np.float32)).to(dtype)
    return l.cuda()


MODES = [("softmax", True, False), ("softmax", False, False), ("sigmoid", True, False),
         ("sigmoid", False, False), ("sigmoid", True, True), ("sigmoid", False, True)]
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 16, 16), (4, 256, 8), (5, 65, 2), (128, 288, 8), (7, 129, 6),
          (33, 257, 4), (9, 511, 16), (130, 1024, 8), (2, 1000, 1), (1027, 100, 3),
          # 16 lanes per token: aligned rows, rows of odd length, tokens left over in the last wave
          (4096, 128, 8), (4099, 37, 16), (4097, 256, 2), (5003, 250, 6), (4098, 16, 1),
          (8195, 128, 8), (8193, 61, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm,biased", MODES)
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_route(T, E, K, score, renorm, biased, dtype):
    print("route T=%d E=%d K=%d %s renorm=%s bias=%s %s" % (T, E, K, score, renorm, biased, dtype),
          flush=True)
    l = make(T, E, T * 1000 + E, dtype)
    bias = None
    if biased:
        bias = torch.from_numpy((0.2 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)).cuda()
    ids, w = run(l, K, bias, score=score, renorm=renorm, scale=2.5)
    ln = l.double().cpu().numpy()
    rid, rw, _ = opsref.route(ln, K, score, None if bias is None else bias.double().cpu().numpy(),
                              renorm, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=tolerance(ln, E), atol=2.0 ** -126)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_take_the_lowest_index(score):
    """Few distinct values, both zeros among them: equal logits are chosen in
    index order, across lanes and across one lane's registers."""
    g = np.random.default_rng(5)
    l = torch.from_numpy(g.integers(-2, 3, size=(64, 300)).astype(np.float32))
    l[::2][l[::2] == 0] = -0.0
    l[5] = 0.0
    l[6] = torch.finfo(torch.float32).min
    ids, w = run(l.cuda(), 16, score=score)
    rid, rw, _ = opsref.route(l.double().numpy(), 16, score, None, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5, atol=2.0 ** -126)
    assert ids[5].tolist() == list(range(16)) and ids[6].tolist() == list(range(16))


def test_equal_scores_under_a_bias():
    """Equal logits and equal biases tie exactly; a bias of -inf switches an
    expert off, one of +inf puts it first."""
    l = torch.zeros(3, 130).cuda()
    bias = torch.zeros(130)
    bias[[3, 70]] = 0.5
    bias[0], bias[129] = -float("inf"), float("inf")
    bias[1] = float("nan")
    ids, w = run(l, 5, bias.cuda(), score="sigmoid", renorm=True)
    assert ids.cpu().tolist() == [[129, 3, 70, 2, 4]] * 3
    assert torch.equal(w.cpu(), torch.full((3, 5), 0.2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm,biased", MODES)
def test_masked_rows(score, renorm, biased, dtype):
    """Experts switched off by -inf: rows with fewer than K left get -1 and
    weight 0 behind them, rows with none get only those; the type's lowest
    value is an ordinary logit."""
    T, E, K = 40, 96, 8
    l = make(T, E, 11, dtype)
    g = np.random.default_rng(12)
    for t in range(T):
        off = g.permutation(E)[:E - (t % 11)]
        l[t, torch.from_numpy(off).cuda()] = -float("inf")
    l[3] = -float("inf")
    l[4] = torch.finfo(dtype).min
    l[5, 3] = torch.finfo(dtype).min
    bias = torch.linspace(-0.2, 0.2, E).cuda() if biased else None
    ids, w = run(l, K, bias, score=score, renorm=renorm)
    ln = l.double().cpu().numpy()
    rid, rw, _ = opsref.route(ln, K, score, None if bias is None else bias.double().cpu().numpy(),
                              renorm, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    # where every choice underflows (sigmoid of the lowest value) the weights are 0 on both sides
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=(2 * 104 + 30) * EPS, atol=2.0 ** -126)
    assert (ids[3] == -1).all() and (w[3] == 0).all()


def test_infinite_and_nan_logits():
    l = make(6, 70, 3, torch.float32)
    l[0, 5] = float("inf")                       # takes the whole softmax
    l[1, [2, 66]] = float("inf")                 # shared
    l[2, 9] = float("nan")                       # not chosen, reported in the weights
    l[3] = float("nan")                          # nothing to choose
    ids, w = run(l, 4, renorm=False)
    assert ids[0, 0] == 5 and w[0].tolist() == [1, 0, 0, 0]
    assert ids[1, :2].tolist() == [2, 66] and w[1].tolist() == [0.5, 0.5, 0, 0]
    assert 9 not in ids[2].tolist() and (ids[2] >= 0).all() and w[2].isnan().all()
    assert (ids[3] == -1).all() and (w[3] == 0).all()
    ids5, w5 = run(l[4:].contiguous(), 4, renorm=False)
    assert torch.equal(ids5, ids[4:]) and torch.equal(w5, w[4:])     # the other rows are untouched


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_route_backward(T, E, K, score, renorm, dtype):
    print("route_backward T=%d E=%d K=%d %s renorm=%s %s" % (T, E, K, score, renorm, dtype),
          flush=True)
    ep = ep_()
    l = make(T, E, T + 7 * E, dtype)
    if E > 20:
        l[:, 1::9] = -float("inf")
    if T > 2:
        l[1] = -float("inf")
    ids, _ = run(l, K, score=score, renorm=renorm)
    g = torch.from_numpy(np.random.default_rng(9).standard_normal((T, K)).astype(np.float32)).cuda()
    g[ids < 0] = float("nan")                    # gradients of masked entries are not used
    out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    ep.ep_route_backward(l, ids, g, out, score=score, renorm=renorm, scale=2.5)
    torch.cuda.synchronize()
    ln = l.double().cpu().numpy()
    want, size = opsref.route_grad(ln, ids.cpu().numpy(), g.double().cpu().numpy(), score, renorm, 2.5)
    got = out.double().cpu().numpy()
    half = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0
    # every factor carries the weights' relative error, the differences that of their larger terms
    bound = 3 * tolerance(ln, E) * size + half * abs(want) + 2.0 ** -126
    assert np.all(abs(got - want) <= bound), float((abs(got - want) / bound).max())


def test_route_backward_repeated_and_foreign_ids():
    """An expert named twice gets both terms; ids outside 0..E-1 take no part."""
    ep = ep_()
    l = make(4, 70, 21, torch.float32)
    ids = torch.tensor([[3, 3, 69, -1], [0, 70, 1, 2], [5, 5, 5, 5], [-1, -9, 2**31 - 1, 70]],
                       dtype=torch.int32).cuda()
    g = torch.tensor([[1.0, -2.0, 0.5, 9.0], [1, 1, 1, -1], [1, 2, 3, 4], [1, 2, 3, 4]]).cuda()
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        out = torch.empty_like(l)
        ep.ep_route_backward(l, ids, g, out, score=score, renorm=renorm)
        want, size = opsref.route_grad(l.double().cpu().numpy(), ids.cpu().numpy(),
                                       g.double().cpu().numpy(), score, renorm, 1.0)
        bound = 3 * tolerance(l.cpu().numpy(), 70) * size + 2.0 ** -126
        assert np.all(abs(out.double().cpu().numpy() - want) <= bound), (score, renorm)
        assert (out[3] == 0).all()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_backward_against_differences(score, renorm):
    """sum(g * w) along a direction v: (f(l + h v) - f(l - h v)) / 2h of the
    kernel's own weights.  With |v| <= 1 per element and |g| <= 1 the third
    derivative of K weights is at most 8 K, so the quotient is off by at most
    8 K h^2 / 6; each weight (at most 1) is off by `tolerance`, K of them on
    either side, over 2h."""
    ep = ep_()
    T, E, K, h = 64, 96, 6, 2.0 ** -6
    rng = np.random.default_rng(33)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    l = (l * 64).round() / 64                    # l +- h v is exact
    # the choice must not change within h: its experts stand clear of the rest
    top = l.topk(K, dim=1).indices
    l.scatter_add_(1, top, (1.0 + torch.arange(K, 0, -1).float() / 8).expand(T, K))
    v = torch.from_numpy(rng.integers(-1, 2, size=(T, E)).astype(np.float32))
    g = torch.from_numpy(rng.uniform(-1, 1, size=(T, K)).astype(np.float32)).cuda()
    kw = dict(score=score, renorm=renorm)
    ids, _ = run(l.cuda(), K, **kw)
    i1, w1 = run((l + h * v).cuda(), K, **kw)
    i0, w0 = run((l - h * v).cuda(), K, **kw)
    # compare by expert: the order within the choice may differ
    def by_expert(i, w):
        return torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, i.long(), w.double())
    gd = by_expert(ids, g)
    assert torch.equal(i1.sort(1).values, ids.sort(1).values)
    assert torch.equal(i0.sort(1).values, ids.sort(1).values)
    diff = (gd * (by_expert(i1, w1) - by_expert(i0, w0))).sum(1) / (2 * h)
    out = torch.empty(T, E, device="cuda")
    ep.ep_route_backward(l.cuda(), ids, g, out, **kw)
    along = (out.double() * v.cuda().double()).sum(1)
    tol = 8 * K * h * h / 6 + K * tolerance(l.numpy(), E) / h
    assert float((diff - along).abs().max()) <= tol


def test_route_graph_replays_and_streams():
    """Captured on a side stream, replayed with eager work between: every
    replay equals the eager result of its inputs."""
    ep = ep_()
    T, E, K = 128, 288, 8
    l = make(T, E, 1, torch.float32)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    g = torch.randn(T, K, device="cuda")
    gl = torch.empty_like(l)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    ep.ep_graph_begin(s)
    ep.ep_route(l, ids, w, stream=s)
    ep.ep_route_backward(l, ids, g, gl, stream=s)
    graph = ep.ep_graph_end(s)
    for i in range(4):
        l.copy_(make(T, E, 50 + i, torch.float32))
        torch.cuda.synchronize()
        graph.launch(s)
        torch.cuda.synchronize()
        eid, ew = run(l, K)
        egl = torch.empty_like(l)
        ep.ep_route_backward(l, eid, g, egl)
        torch.cuda.synchronize()
        assert torch.equal(ids, eid) and torch.equal(w, ew) and torch.equal(gl, egl)
    graph.destroy()


def test_more_tokens_than_the_grid_holds():
    """2^24 + 5 tokens of two experts: the waves stride over the tokens."""
    ep = ep_()
    T = (1 << 24) + 5
    l = torch.randn(T, 2, device="cuda")
    ids, w = run(l, 1)
    assert torch.equal(ids[:, 0].long(), (l[:, 1] > l[:, 0]).long())
    assert bool((w == 1).all())
    gl = torch.empty_like(l)
    ep.ep_route_backward(l, ids, torch.ones_like(w), gl, renorm=False)
    p = torch.softmax(l.double(), 1).gather(1, ids.long())
    want = (p * (1 - p)).expand(T, 2) * torch.where(torch.arange(2, device="cuda")[None] == ids, 1.0, -1.0)
    # the weights' relative error (a range below 16), once per factor
    assert bool(((gl.double() - want).abs() <= 3 * (2 * 16 + 26) * EPS * 2 * p).all())
