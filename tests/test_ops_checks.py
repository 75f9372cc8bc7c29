"""CPU checks of the router, gradient and expert-product entry points: every
refusal of the C calls and of the binding, made before anything reaches a GPU,
and the layout of 4-bit weights."""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_layout_05_amd as ep
from tests import opsref

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)   # never dereferenced
NONE = None


def lib():
    return ep._lib


def test_route_refusals():
    f = lib().ep_route
    ok = [FAKE, 0, 4, 256, 8, 0, NONE, 1, 1.0, FAKE, FAKE, NONE]

    def rc(**over):
        a = list(ok)
        for i, v in over.items():
            a[int(i[1:])] = v
        return f(*a)
    assert rc(_1=2) == -1 and rc(_5=2) == -1 and rc(_7=2) == -1      # dtype, score, renorm
    assert rc(_8=float("nan")) == -1 and rc(_8=float("inf")) == -1   # scale
    assert rc(_6=FAKE) == -1                                         # bias with softmax
    assert rc(_5=1, _6=ODD) == -1                                    # misaligned bias
    assert rc(_2=-1) == -1 and rc(_4=0) == -1 and rc(_4=17) == -1
    assert rc(_3=1025) == -1 and rc(_3=0) == -1 and rc(_3=7) == -1   # E; K > E
    assert rc(_2=1 << 28) == -1                                      # T*K >= 2^31
    for i in (0, 9, 10):
        assert rc(**{"_%d" % i: NONE}) == -1 and rc(**{"_%d" % i: ODD}) == -1
    assert f(NONE, 1, 0, 256, 8, 0, NONE, 0, 1.0, NONE, NONE, NONE) == 0      # empty batch


def test_route_backward_refusals():
    f = lib().ep_route_backward
    ok = [FAKE, 1, 4, 256, 8, 1, 1, 1.0, FAKE, FAKE, FAKE, NONE]

    def rc(**over):
        a = list(ok)
        for i, v in over.items():
            a[int(i[1:])] = v
        return f(*a)
    assert rc(_1=-1) == -1 and rc(_5=-1) == -1 and rc(_6=-1) == -1 and rc(_7=float("inf")) == -1
    assert rc(_2=-1) == -1 and rc(_4=17) == -1 and rc(_3=4) == -1 and rc(_3=1025) == -1
    for i in (0, 8, 9, 10):
        assert rc(**{"_%d" % i: NONE}) == -1 and rc(**{"_%d" % i: ODD}) == -1
    assert f(NONE, 0, 0, 8, 8, 0, 0, 1.0, NONE, NONE, NONE, NONE) == 0


def test_gradient_refusals():
    f, g = lib().ep_combine_backward, lib().ep_dispatch_backward
    ok = [FAKE, FAKE, FAKE, FAKE, 4, 1024, 8, FAKE, FAKE, NONE]
    for i, v in ((4, -1), (5, 0), (5, 1001), (6, 0), (6, 17), (4, 1 << 28)):
        a = list(ok)
        a[i] = v
        assert f(*a) == -1, (i, v)
    for i in (0, 1, 2, 3, 7, 8):
        for v in (NONE, ODD):
            a = list(ok)
            a[i] = v
            assert f(*a) == -1, (i, v)
    assert f(NONE, NONE, NONE, NONE, 0, 1024, 8, NONE, NONE, NONE) == 0
    ok = [FAKE, FAKE, 4, 1024, 8, FAKE, NONE]
    for i, v in ((2, -1), (3, 0), (3, 1001), (4, 0), (4, 17), (2, 1 << 28)):
        a = list(ok)
        a[i] = v
        assert g(*a) == -1, (i, v)
    for i in (0, 1, 5):
        for v in (NONE, ODD):
            a = list(ok)
            a[i] = v
            assert g(*a) == -1, (i, v)
    assert g(NONE, NONE, 0, 1024, 8, NONE, NONE) == 0


def test_expert_refusals():
    f = lib().ep_expert_w4
    ok = [FAKE, FAKE, 0, 64, 1024, FAKE, 16, FAKE, FAKE, 512, 1, FAKE, NONE]

    def rc(**over):
        a = list(ok)
        for i, v in over.items():
            a[int(i[1:])] = v
        return f(*a)
    assert rc(_2=7) == -2                                            # payload
    assert rc(_10=2) == -1 and rc(_3=-1) == -1                       # act, rows
    assert rc(_4=0) == -1 and rc(_4=1000) == -1 and rc(_9=0) == -1 and rc(_9=12) == -1
    assert rc(_6=0) == -1 and rc(_6=1025) == -1
    assert rc(_3=2**31 - 1) == -1                                    # grid limit
    assert rc(_4=1 << 24) == -1 and rc(_9=1 << 30) == -1             # offset limits
    assert rc(_4=1 << 20, _9=1 << 15) == -1
    for i in (0, 1, 5, 7, 8, 11):
        assert rc(**{"_%d" % i: NONE}) == -1 and rc(**{"_%d" % i: ODD}) == -1
    assert rc(_0=ctypes.c_void_p(0x10008)) == -1 and rc(_7=ctypes.c_void_p(0x10008)) == -1
    assert f(NONE, NONE, 1, 0, 1024, NONE, 16, NONE, NONE, 512, 0, NONE, NONE) == 0


def test_binding_refusals():
    i32 = dict(dtype=torch.int32)
    bf = dict(dtype=torch.bfloat16)
    l, idx, w = torch.zeros(4, 32), torch.zeros(4, 8, **i32), torch.zeros(4, 8)
    for args, kw, exc, word in [
            ((l, idx, w), {}, ValueError, "device tensor"),
            ((l.half(), idx, w), {}, TypeError, "dtype"),
            ((l, idx.long(), w), {}, TypeError, "dtype"),
            ((l, idx, w.double()), {}, TypeError, "dtype"),
            ((l[0], idx, w), {}, ValueError, "logits"),
            ((l, idx[:3], w), {}, ValueError, "topk_idx"),
            ((l, idx, w[:, :7]), {}, ValueError, "topk_w"),
            ((l, idx, w), dict(score="top"), ValueError, "score"),
            ((l, idx, w), dict(score="sigmoid", bias=torch.zeros(31)), ValueError, "bias"),
            ((l, idx, w), dict(score="sigmoid", bias=torch.zeros(32).half()), TypeError, "dtype")]:
        with pytest.raises(exc, match=word):
            ep.ep_route(*args, **kw)
    with pytest.raises(TypeError):
        ep.ep_route_backward(l, idx, w, l.bfloat16())
    with pytest.raises(ValueError, match="grad_logits"):
        ep.ep_route_backward(l, idx, w, l[:3])
    with pytest.raises(ValueError, match="grad_topk_w"):
        ep.ep_route_backward(l, idx, w[:3], l.clone())
    go, y, rop = torch.zeros(4, 256, **bf), torch.zeros(32, 256, **bf), torch.zeros(32, **i32)
    gy, gw = torch.zeros(32, 256, **bf), torch.zeros(4, 8)
    for over, word in [(dict(go=go[:3]), "grad_out"), (dict(y=y[:31]), "expert_out"),
                       (dict(rop=rop[:31]), "row_of_pair"), (dict(gy=gy[:, :248]), "grad_expert_out"),
                       (dict(gw=gw[:3]), "grad_topk_w"), ({}, "device tensor")]:
        d = dict(go=go, y=y, rop=rop, w=w, gy=gy, gw=gw)
        d.update(over)
        with pytest.raises(ValueError, match=word):
            ep.ep_combine_backward(d["go"], d["y"], d["rop"], d["w"], d["gy"], d["gw"])
    with pytest.raises(ValueError, match="row_of_pair"):
        ep.ep_dispatch_backward(gy, rop[:31], go)
    with pytest.raises(ValueError, match="grad_recv"):
        ep.ep_dispatch_backward(gy[:31], rop, go)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_dispatch_backward(gy, rop, go)


def test_expert_binding_refusals():
    u8 = dict(dtype=torch.uint8)
    d = dict(x=torch.zeros(6, 256, **u8), xs=torch.zeros(6, 2), off=torch.zeros(4, dtype=torch.int32),
             w=torch.zeros(3, 32, 128, **u8), ws=torch.zeros(3, 32, 2),
             out=torch.zeros(6, 16, dtype=torch.bfloat16), act="silu_mul")

    def call(**over):
        a = dict(d, **over)
        ep.ep_expert_w4(a["x"], a["xs"], a["off"], a["w"], a["ws"], a["out"], act=a["act"])
    for over, exc, word in [
            ({}, ValueError, "device tensor"), (dict(act="none"), ValueError, "w:"),
            (dict(act="gelu"), ValueError, "act"), (dict(xs=None), ValueError, "x_scales"),
            (dict(xs=d["xs"][:5]), ValueError, "x_scales"), (dict(off=d["off"][:3]), ValueError, "expert_offset"),
            (dict(w=d["w"][:, :31]), ValueError, "w:"), (dict(ws=d["ws"][:, :, :1]), ValueError, "w_scales"),
            (dict(out=d["out"][:5]), ValueError, "out"), (dict(x=torch.zeros(6, 256)), TypeError, "dtype"),
            (dict(x=torch.zeros(6, 256, dtype=torch.bfloat16)), ValueError, "x_scales"),
            (dict(w=d["w"].int()), TypeError, "dtype"), (dict(off=d["off"].long()), TypeError, "dtype")]:
        with pytest.raises(exc, match=word):
            call(**over)


def test_experts_class_refusals():
    w_up, s_up = ep.w4_quantise(torch.randn(3, 256, 384))
    w_dn, s_dn = ep.w4_quantise(torch.randn(3, 384, 128))
    e = ep.EpExpertsW4(4, 2, w_up, s_up, w_dn, s_dn)
    assert (e.E, e.H, e.I) == (3, 384, 128) and e.out.shape == (8, 384)
    for bad in ((w_up[:, :255], s_up, w_dn, s_dn), (w_up, s_up[:, :, :2], w_dn, s_dn),
                (w_up, s_up, w_dn[:2], s_dn[:2]), (w_up, s_up, w_dn, s_dn[:, :5])):
        with pytest.raises(ValueError):
            ep.EpExpertsW4(4, 2, *bad)
    b = ep.EpBuffers(4, 384, 2, 3, 1, device="cpu")
    with pytest.raises(ValueError, match="device tensor"):
        e(b)
    with pytest.raises(ValueError, match="buffers"):
        e(ep.EpBuffers(4, 256, 2, 3, 1, device="cpu"))
    with pytest.raises(ValueError, match="logits"):
        b.route(torch.zeros(5, 3))
    with pytest.raises(ValueError, match="tokens"):
        b.combine_backward(torch.zeros(3, 384), torch.zeros(8, 384), torch.zeros(4, 2))


def test_w4_quantise():
    """Codes are the nearest e2m1 values (ties to the even code), found here by
    search over the values; signs, zero blocks and the low nibble first."""
    g = np.random.default_rng(0)
    w = g.standard_normal((5, 256)).astype(np.float32)
    w[1, :128] = 0.0
    w[2, :128] = 0.0
    w[2, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]      # scale 1: every midpoint
    codes, scales = ep.w4_quantise(torch.from_numpy(w))
    assert codes.dtype == torch.uint8 and codes.shape == (5, 128) and scales.shape == (5, 2)
    c = np.empty((5, 256), np.int64)
    c[:, 0::2], c[:, 1::2] = codes.numpy() & 15, codes.numpy() >> 4
    s = scales.numpy()
    np.testing.assert_array_equal(s, abs(w.reshape(5, 2, 128)).max(2) / np.float32(6))
    q = (w / np.repeat(np.where(s > 0, s, 1), 128, axis=1)).astype(np.float64)
    dist = abs(abs(q)[..., None] - opsref.E2M1[:8])
    best = dist == dist.min(-1, keepdims=True)
    even = best & (np.arange(8) % 2 == 0)
    want = np.where(even.any(-1), even.argmax(-1), best.argmax(-1))
    np.testing.assert_array_equal(c & 7, want)
    np.testing.assert_array_equal((c >> 3)[q != 0], (q < 0)[q != 0])
    assert (c[1, :128] & 7 == 0).all() and s[1, 0] == 0
    with pytest.raises(ValueError):
        ep.w4_quantise(torch.zeros(2, 100))
    two = ep.w4_quantise(torch.from_numpy(w).reshape(1, 5, 256).bfloat16())
    assert two[0].shape == (1, 5, 128)


def test_reference_gradients_match_differences():
    """The 64-bit formulas the GPU tests compare with, against central
    differences of the 64-bit weights (steps of 1e-5: an error of about h^2 plus
    2^-52 / h, far below 1e-8)."""
    g = np.random.default_rng(1)
    T, E, K, h = 5, 12, 4, 1e-5
    l = g.standard_normal((T, E))
    l[1, 3] = -np.inf
    up = g.standard_normal((T, K))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _, _ = opsref.route(l, K, score, None, renorm, 1.7)
            grad, _ = opsref.route_grad(l, ids, up, score, renorm, 1.7)
            for e in range(E):
                d = np.zeros(E)
                d[e] = h
                hi, a, _ = opsref.route(l + d, K, score, None, renorm, 1.7)
                lo, b, _ = opsref.route(l - d, K, score, None, renorm, 1.7)
                assert np.array_equal(hi, ids) and np.array_equal(lo, ids)
                np.testing.assert_allclose((up * (a - b)).sum(1) / (2 * h), grad[:, e], atol=1e-8)


class FakeTensor:
    """What the pointer check of a call looks at, on a made-up device."""

    def __init__(self, device, contiguous=True):
        self.index, self.contiguous, self.device = device, contiguous, "cuda:%d" % device

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096


def test_tensors_of_other_devices_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, there = FakeTensor(0), FakeTensor(1)
    with pytest.raises(ValueError, match="cuda:0 and cuda:1"):
        ep._ptrs(None, here, None, there)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        ep._ptrs(None, there, there)
    with pytest.raises(ValueError, match="contiguous"):
        ep._ptrs(None, here, FakeTensor(0, contiguous=False))

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 77
    with pytest.raises(ValueError, match="stream"):
        ep._ptrs(Stream, here)
    Stream.device = torch.device("cuda", 0)
    assert ep._ptrs(Stream, here, None) == ([4096, None], 77)


@pytest.mark.parametrize("shape", [(), (127,), (4, 129)])
def test_quantise_refuses_partial_blocks(shape):
    with pytest.raises(ValueError, match="multiple of 128"):
        ep.w4_quantise(torch.zeros(shape))


class FakeStream:
    device, cuda_stream = torch.device("cuda", 0), 99


@pytest.fixture
def fake_streams(monkeypatch):
    """A current stream `here` and torch.cuda.stream as a record of which one
    is current; `made` lists (maker, stream it ran under)."""
    here, made, now = FakeStream(), [], []
    now.append(here)

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            now.append(self.s)

        def __exit__(self, *exc):
            now.pop()
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: made.append(("record", s)))
    for name in ("zeros_like", "empty_like", "empty", "zeros"):
        def maker(*a, _f=getattr(torch, name), _n=name, **kw):
            made.append((_n, now[-1]))
            return _f(*a, **kw)
        monkeypatch.setattr(torch, name, maker)
    for name in ("ep_combine_backward", "ep_dispatch_backward"):
        monkeypatch.setattr(ep, name, lambda *a, _n=name: made.append((_n, a[-1])))
    return here, made


def test_missing_outputs_are_made_on_the_calls_stream(fake_streams, monkeypatch):
    """The fill of an output and its memory belong to the stream that the
    kernel runs on: on another they are not ordered with it."""
    here, made = fake_streams
    b = ep.EpBuffers(4, 384, 2, 3, 1, device="cpu")
    go, y, w = torch.ones(4, 384), torch.ones(8, 384), torch.ones(4, 2)
    s = FakeStream()
    del made[:]
    b.combine_backward(go, y, w, stream=s)
    b.dispatch_backward(y, stream=s)
    assert [m for m in made if m[0] != "record"] == [
        ("zeros_like", s), ("empty_like", s), ("ep_combine_backward", s),
        ("empty", s), ("ep_dispatch_backward", s)]
    assert [m for m in made if m[0] == "record"] == [("record", here)] * 3
    del made[:]
    b.combine_backward(go, y, w)
    b.dispatch_backward(y)
    assert [m[1] for m in made if not m[0].startswith("ep_")] == [here] * 3
    # captured on a stream that torch's allocator knows nothing of: refused, not made
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    del made[:]
    for call in (lambda: b.combine_backward(go, y, w, stream=s),
                 lambda: b.combine_backward(go, y, w, torch.ones_like(y), stream=s),
                 lambda: b.dispatch_backward(y, stream=s)):
        with pytest.raises(ValueError, match="outputs must be given"):
            call()
    assert not [m for m in made if m[0].startswith("ep_") or m[0] in ("empty", "zeros_like", "empty_like")
                and m[1] is s]


def test_quantise_works_in_pieces(monkeypatch):
    """Large weights are laid out piece by piece, with the same result: no
    intermediate (of 8 bytes per weight) is as large as the weight."""
    w = torch.randn(3, 37, 384)
    assert w.numel() <= ep._W4_PIECE
    whole = ep.w4_quantise(w)
    largest = []
    bucketize = torch.bucketize
    monkeypatch.setattr(torch, "bucketize",
                        lambda q, *a, **kw: largest.append(q.numel()) or bucketize(q, *a, **kw))
    for piece in (1, 384, 5000):                       # a row at least, and pieces that end inside
        monkeypatch.setattr(ep, "_W4_PIECE", piece)
        del largest[:]
        codes, scales = ep.w4_quantise(w)
        assert torch.equal(codes, whole[0]) and torch.equal(scales, whole[1])
        assert max(largest) <= max(piece, 384) and sum(largest) == w.numel()
    view = torch.randn(384, 6).t()                     # not contiguous
    assert torch.equal(ep.w4_quantise(view)[0], ep.w4_quantise(view.contiguous())[0])
    empty = ep.w4_quantise(torch.zeros(0, 5, 256))
    assert empty[0].shape == (0, 5, 128) and empty[1].shape == (0, 5, 2)
