"""ep_route and ep_route_backward with 16 lanes per token (4096 tokens and more,
up to 256 experts): four tokens share a wave, and what one of them holds --
switched-off experts, none left, infinities, NaN, ties -- stays its own."""
import numpy as np
import pytest
import torch

from tests import opsref
from tests.test_gpu_route import EPS, MODES, make, run, tolerance

pytestmark = pytest.mark.gpu

T = 4099                               # the last wave has three tokens
FULL, PARTLY, NONE, NAN = range(4)


def states(n):
    """Every state beside every other in a wave of four, in every place."""
    t = np.arange(n)
    return (t + t // 4 + t // 16) % 4


def mixed(n, E, dtype, seed):
    l = make(n, E, seed, dtype).float().cpu()
    g = np.random.default_rng(seed)
    st = states(n)
    off = torch.from_numpy(g.random((n, E)) < g.choice([0.3, 0.9, 0.97], size=(n, 1)))
    l[torch.from_numpy((st == PARTLY) | (st == NAN))[:, None] & off] = -float("inf")
    l[torch.from_numpy(st == NONE)] = -float("inf")
    for t in np.nonzero(st == NAN)[0]:
        l[t, int(g.integers(E))] = float("nan")
    return l.to(dtype).cuda(), st


def reference(l, K, score, bias, renorm, scale):
    return opsref.route(l.double().cpu().numpy(), K, score,
                        None if bias is None else bias.double().cpu().numpy(), renorm, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm,biased", MODES)
@pytest.mark.parametrize("E,K", [(96, 8), (250, 6), (256, 16), (13, 13)])
def test_states_beside_each_other(E, K, score, renorm, biased, dtype):
    print("narrow E=%d K=%d %s renorm=%s bias=%s %s" % (E, K, score, renorm, biased, dtype), flush=True)
    l, st = mixed(T, E, dtype, E + K)
    bias = torch.linspace(-0.2, 0.2, E).cuda() if biased else None
    kw = dict(score=score, renorm=renorm, scale=1.5)
    ids, w = run(l, K, bias, **kw)
    rid, rw, _ = reference(l, K, score, bias, renorm, 1.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    ln = l.double().cpu().numpy()
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=tolerance(ln, E), atol=2.0 ** -126, equal_nan=True)
    none = torch.from_numpy(st == NONE).cuda()
    assert bool((ids[none] == -1).all()) and bool((w[none] == 0).all())
    # the tokens beside a NaN: bit for bit as without it
    nan = torch.from_numpy(st == NAN).cuda()
    clean = torch.where(torch.isnan(l) & nan[:, None], torch.zeros_like(l), l)
    ids2, w2 = run(clean, K, bias, **kw)
    assert torch.equal(ids[~nan], ids2[~nan]) and torch.equal(w[~nan], w2[~nan])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [96, 250])
def test_ties_take_the_lowest_index(score, E, dtype):
    g = np.random.default_rng(5)
    l = torch.from_numpy(g.integers(-2, 3, size=(T, E)).astype(np.float32))
    l[::2][l[::2] == 0] = -0.0
    l[5::7] = 0.0
    l[6::7] = float(torch.finfo(dtype).min)
    ids, w = run(l.to(dtype).cuda(), 16, score=score)
    rid, rw, _ = opsref.route(l.to(dtype).double().numpy(), 16, score, None, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=(2 * 4 + 30) * EPS, atol=2.0 ** -126)
    want = torch.arange(16, dtype=torch.int32).expand(T, 16)
    assert torch.equal(ids.cpu()[5::7], want[5::7]) and torch.equal(ids.cpu()[6::7], want[6::7])


@pytest.mark.parametrize("E", [96, 250])
def test_infinite_biases(E):
    l = torch.zeros(T, E).cuda()
    l[1::4] = 1.0
    l[2::4] = -float("inf")
    bias = torch.zeros(E)
    bias[[3, 70]] = 0.5
    bias[0], bias[E - 1] = -float("inf"), float("inf")
    bias[1] = float("nan")
    ids, w = run(l, 5, bias.cuda(), score="sigmoid", renorm=True)
    want = torch.tensor([[E - 1, 3, 70, 2, 4]], dtype=torch.int32).repeat(T, 1)
    weight = torch.full((T, 5), 0.2)
    want[2::4], weight[2::4] = -1, 0.0
    assert torch.equal(ids.cpu(), want)
    # five equal weights over their sum: each addition and the division half a step
    np.testing.assert_allclose(w.cpu().numpy(), weight.numpy(), rtol=6 * EPS)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_logits(dtype):
    l = make(T, 70, 3, dtype)
    l[0::4, 5] = float("inf")                    # takes the whole softmax
    l[1::4, 2] = l[1::4, 66] = float("inf")      # shared
    l[3::4] = float("nan")                       # nothing to choose
    ids, w = run(l, 4, renorm=False)
    assert bool((ids[0::4, 0] == 5).all())
    assert torch.equal(w[0::4], torch.tensor([[1.0, 0, 0, 0]], device="cuda").expand_as(w[0::4]))
    assert torch.equal(ids[1::4, :2], torch.tensor([[2, 66]], device="cuda").int().expand_as(ids[1::4, :2]))
    assert torch.equal(w[1::4], torch.tensor([[0.5, 0.5, 0, 0]], device="cuda").expand_as(w[1::4]))
    assert bool((ids[3::4] == -1).all()) and bool((w[3::4] == 0).all())
    rid, rw, _ = reference(l[2::4], 4, "softmax", None, False, 1.0)
    np.testing.assert_array_equal(ids[2::4].cpu().numpy(), rid)
    np.testing.assert_allclose(w[2::4].cpu().numpy(), rw, atol=2.0 ** -126,
                               rtol=tolerance(l[2::4].double().cpu().numpy(), 70))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
@pytest.mark.parametrize("E,K", [(96, 8), (61, 16), (128, 6)])
def test_gradients_beside_each_other(E, K, score, renorm, dtype):
    """The same states under ep_route_backward (8192 tokens and more, rows of up to
    512 bytes).  A NaN logit makes its own row's gradient NaN where the weights
    are sums over the row, and no other row's."""
    import combine_ep_layout_05_amd as ep
    n = 8195
    print("narrow backward E=%d K=%d %s renorm=%s %s" % (E, K, score, renorm, dtype), flush=True)
    l, st = mixed(n, E, dtype, E + 3)
    ids, _ = run(l, K, score=score, renorm=renorm)
    g = torch.from_numpy(np.random.default_rng(9).standard_normal((n, K)).astype(np.float32)).cuda()
    g[ids < 0] = float("nan")                    # gradients of masked entries are not used
    out = torch.full((n, E), float("nan"), dtype=dtype, device="cuda")
    ep.ep_route_backward(l, ids, g, out, score=score, renorm=renorm, scale=2.5)
    torch.cuda.synchronize()
    keep = st != NAN
    ln = l.double().cpu().numpy()[keep]
    want, size = opsref.route_grad(ln, ids.cpu().numpy()[keep], g.double().cpu().numpy()[keep],
                                   score, renorm, 2.5)
    got = out.double().cpu().numpy()
    half = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0
    bound = 3 * tolerance(ln, E) * size + half * abs(want) + 2.0 ** -126
    assert np.all(abs(got[keep] - want) <= bound), float((abs(got[keep] - want) / bound).max())
    assert (got[st == NONE] == 0).all()
    if score == "softmax" and not renorm:        # rows with a choice and a NaN in the sum
        some = (st == NAN) & (ids >= 0).any(1).cpu().numpy()
        assert np.isnan(got[some]).any(1).all()
