"""CPU tests of the operators between token ids and the expert layer: every refusal is
made before anything reaches the GPU, by the C entry points (with pointers that must
not be followed) and by the Python checks; the oracle's gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

import newton_schulz_gram_amd as nsg
from oracle import layer_oracle as ref

P16 = 0x10000  # an aligned address that no call may follow
OK, ARG, DTYPE, SHAPE, WORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def embedding(ids=P16, bits=64, T=4, W=P16, dt=1, V=10, C=8, ld=8, scale=1.0, out=P16):
    return nsg.lib().nsg_embedding(ids, bits, T, W, dt, V, C, ld, scale, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=16), DTYPE), (dict(dt=3), DTYPE), (dict(dt=-1), DTYPE), (dict(T=-1), SHAPE), (dict(T=(1 << 25) + 1), SHAPE),
    (dict(V=-1), SHAPE), (dict(V=(1 << 20) + 1), SHAPE), (dict(C=-1), SHAPE), (dict(C=70000, ld=70000), SHAPE), (dict(ld=7), SHAPE),
    (dict(ld=(1 << 31) + 1), SHAPE), (dict(ids=None), ARG), (dict(ids=P16 + 4), ARG), (dict(ids=P16 + 2, bits=32), ARG),
    (dict(W=None), ARG), (dict(W=P16 + 1), ARG), (dict(dt=2, W=P16 + 2), ARG), (dict(out=None), ARG), (dict(out=P16 + 1), ARG),
    (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(T=0, ids=None, out=None), OK), (dict(C=0, ld=0), OK),
])
def test_embedding_refusals(kw, code):
    assert embedding(**kw) == code


def embedding_backward(dout=P16, dt=1, T=4, C=8, ld=8, ids=P16, bits=64, V=10, scale=1.0, dW=P16, odt=1, acc=0, ws=P16, n=1 << 30):
    return nsg.lib().nsg_embedding_backward(dout, dt, T, C, ld, ids, bits, V, scale, dW, odt, acc, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=8), DTYPE), (dict(dt=4), DTYPE), (dict(odt=3), DTYPE), (dict(T=-1), SHAPE), (dict(T=(1 << 25) + 1), SHAPE),
    (dict(V=-1), SHAPE), (dict(V=(1 << 20) + 1), SHAPE), (dict(C=70000, ld=70000), SHAPE), (dict(ld=7), SHAPE), (dict(acc=2), ARG),
    (dict(scale=NAN), ARG), (dict(dout=None), ARG), (dict(dout=P16 + 1), ARG), (dict(ids=None), ARG), (dict(ids=P16 + 4), ARG),
    (dict(dW=None), ARG), (dict(dW=P16 + 1), ARG), (dict(odt=2, dW=P16 + 2), ARG), (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE),
    (dict(ws=P16 + 8), WORKSPACE), (dict(V=0), OK), (dict(C=0, ld=0), OK), (dict(T=0, acc=1), OK),
])
def test_embedding_backward_refusals(kw, code):
    assert embedding_backward(**kw) == code


def layer_norm(x=P16, dt=1, R=4, C=8, ld=8, w=P16, b=P16, wdt=2, eps=1e-5, y=P16, stats=P16):
    return nsg.lib().nsg_layer_norm(x, dt, R, C, ld, w, b, wdt, eps, y, stats, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), DTYPE), (dict(wdt=4), DTYPE), (dict(R=-1), SHAPE), (dict(R=(1 << 25) + 1), SHAPE), (dict(C=0, ld=0), SHAPE),
    (dict(C=65537, ld=65537), SHAPE), (dict(ld=7), SHAPE), (dict(eps=-1e-5), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG),
    (dict(x=None), ARG), (dict(y=None), ARG), (dict(stats=None), ARG), (dict(x=P16 + 1), ARG), (dict(y=P16 + 1), ARG),
    (dict(w=P16 + 2), ARG), (dict(b=P16 + 2), ARG), (dict(stats=P16 + 2), ARG), (dict(R=0), OK), (dict(R=0, C=0, ld=0), OK),
])
def test_layer_norm_refusals(kw, code):
    assert layer_norm(**kw) == code


def layer_norm_backward(dy=P16, lddy=8, x=P16, ldx=8, dt=1, R=4, C=8, stats=P16, w=P16, wdt=2, dx=P16, dw=P16, db=P16, ws=P16,
                        n=1 << 30):
    return nsg.lib().nsg_layer_norm_backward(dy, lddy, x, ldx, dt, R, C, stats, w, wdt, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), DTYPE), (dict(wdt=-1), DTYPE), (dict(R=-1), SHAPE), (dict(C=0, lddy=0, ldx=0), SHAPE), (dict(lddy=7), SHAPE),
    (dict(ldx=7), SHAPE), (dict(dy=None), ARG), (dict(x=None), ARG), (dict(stats=None), ARG), (dict(dx=None), ARG),
    (dict(dy=P16 + 1), ARG), (dict(x=P16 + 1), ARG), (dict(dx=P16 + 1), ARG), (dict(w=P16 + 2), ARG), (dict(dw=P16 + 2), ARG),
    (dict(db=P16 + 2), ARG), (dict(stats=P16 + 1), ARG), (dict(ws=None), WORKSPACE), (dict(ws=None, db=None), WORKSPACE),
    (dict(n=16), WORKSPACE), (dict(ws=P16 + 4), WORKSPACE), (dict(R=0, dw=None, db=None), OK), (dict(R=0, C=0, lddy=0, ldx=0), OK),
])
def test_layer_norm_backward_refusals(kw, code):
    assert layer_norm_backward(**kw) == code


def route(l=P16, dt=1, T=4, E=8, ld=8, k=2, score=0, bias=None, mask=None, norm=1, scale=1.0, ids=P16, w=P16, counts=P16, probs=P16,
          loss=P16, ws=P16, n=1 << 30):
    return nsg.lib().nsg_expert_route(l, dt, T, E, ld, k, score, bias, mask, norm, scale, ids, w, counts, probs, loss, ws, n, None)


ROUTER_REFUSALS = [
    (dict(dt=3), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 25), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE),
    (dict(k=0), SHAPE), (dict(k=9), SHAPE), (dict(E=100, ld=100, k=65), SHAPE), (dict(ld=7), SHAPE), (dict(score=2), ARG), (dict(norm=2), ARG),
    (dict(scale=NAN), ARG), (dict(l=None), ARG), (dict(l=P16 + 1), ARG), (dict(ids=None), ARG), (dict(ids=P16 + 2), ARG),
    (dict(counts=P16 + 2), ARG),
]


@pytest.mark.parametrize("kw,code", ROUTER_REFUSALS + [
    (dict(w=None), ARG), (dict(w=P16 + 2), ARG), (dict(bias=P16 + 2), ARG), (dict(counts=None), ARG), (dict(probs=None), ARG),
    (dict(loss=None), ARG), (dict(probs=P16 + 2), ARG), (dict(loss=P16 + 2), ARG), (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE),
    (dict(ws=P16 + 4), WORKSPACE), (dict(T=0, counts=None, probs=None, loss=None), OK),
])
def test_route_refusals(kw, code):
    assert route(**kw) == code


def route_backward(l=P16, dt=1, T=4, E=8, ld=8, k=2, score=0, norm=1, scale=1.0, ids=P16, dw=P16, counts=P16, balance=1.0, dloss=None,
                   dl=P16):
    return nsg.lib().nsg_expert_route_backward(l, dt, T, E, ld, k, score, norm, scale, ids, dw, counts, balance, dloss, dl, None)


@pytest.mark.parametrize("kw,code", ROUTER_REFUSALS + [
    (dict(dw=P16 + 2), ARG), (dict(balance=INF), ARG), (dict(dloss=P16 + 2), ARG), (dict(dloss=P16, counts=None), ARG),
    (dict(dl=None), ARG), (dict(dl=P16 + 1), ARG), (dict(T=0), OK),
])
def test_route_backward_refusals(kw, code):
    assert route_backward(**kw) == code


def test_workspace_sizes():
    assert nsg.embedding_backward_workspace_size(0, 10, 8) == 0
    assert nsg.embedding_backward_workspace_size(5, 0, 8) == 0
    assert nsg.embedding_backward_workspace_size(100, 1000, 64) >= 4 * 4 * 100
    assert nsg.layer_norm_backward_workspace_size(0, 8) == 0
    assert nsg.layer_norm_backward_workspace_size(5, 8) > 0
    assert nsg.expert_route_workspace_size(0, 8) == 0
    assert nsg.expert_route_workspace_size(5, 8) > 0
    L = nsg.lib()
    n = ctypes.c_size_t(0)
    assert L.nsg_embedding_backward_workspace_size(1, 1, 1, None) == ARG
    assert L.nsg_layer_norm_backward_workspace_size(1, 1, None) == ARG
    assert L.nsg_expert_route_workspace_size(1, 1, None) == ARG
    assert L.nsg_embedding_backward_workspace_size(1, 1 << 21, 1, ctypes.byref(n)) == SHAPE
    assert L.nsg_layer_norm_backward_workspace_size(-1, 1, ctypes.byref(n)) == SHAPE
    assert L.nsg_expert_route_workspace_size(1, 2000, ctypes.byref(n)) == SHAPE


def test_no_cpu_path():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: nsg.embedding(ids, x), lambda: nsg.embedding_backward(x, ids[:, 0].contiguous(), 3), lambda: nsg.layer_norm(x),
                 lambda: nsg.layer_norm_backward(x, x, torch.zeros(2, 4)), lambda: nsg.expert_route(x, 2),
                 lambda: nsg.expert_route_backward(x, ids)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def slope(f, a, g, h=1e-5):
    """The difference of f along a random direction, and g's."""
    d = np.random.default_rng(1).standard_normal(a.shape)
    return (f(a + h * d) - f(a - h * d)) / (2 * h), (g * d).sum()


def test_oracle_layer_norm_gradients():
    g = np.random.default_rng(0)
    x, w, b, u = g.standard_normal((5, 37)), g.standard_normal(37), g.standard_normal(37), g.standard_normal((5, 37))
    _, mean, rstd = ref.layer_norm(x, w, b, 1e-3)
    dx, dw, db = ref.layer_norm_backward(u, x, mean, rstd, w)
    for f, a, d in ((lambda v: (ref.layer_norm(v, w, b, 1e-3)[0] * u).sum(), x, dx), (lambda v: (ref.layer_norm(x, v, b, 1e-3)[0] * u).sum(), w, dw),
                    (lambda v: (ref.layer_norm(x, w, v, 1e-3)[0] * u).sum(), b, db)):
        assert np.allclose(*slope(f, a, d), rtol=1e-7, atol=1e-7)


def test_oracle_embedding_gradient():
    g = np.random.default_rng(0)
    W, ids, u = g.standard_normal((6, 5)), np.array([[1, 1, -1], [5, 6, 1]]), g.standard_normal((2, 3, 5))
    dW, _, n = ref.embedding_backward(u, ids, 6, 3.0)
    assert np.allclose(*slope(lambda v: (ref.embedding(ids, v, 3.0) * u).sum(), W, dW), rtol=1e-8)
    assert n.tolist() == [0, 3, 0, 0, 0, 1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_router_gradients(score, normalize):
    g = np.random.default_rng(0)
    l, dw = g.standard_normal((9, 12)), g.standard_normal((9, 3))
    ids = ref.choose(l, 3, score, mask=np.arange(9) % 4 != 0)
    counts, _, _ = ref.balance(l, ids, score, 3)
    dl, size = ref.route_backward(l, ids, dw, score, normalize, 1.7, counts, 0.3)
    assert (np.abs(dl) <= size * (1 + 1e-12)).all()

    def loss(v):
        keep = (ids >= 0).any(1)
        probs = ref.shares(v[keep], score).sum(0) / counts[-1]
        return (ref.weights(v, ids, score, normalize, 1.7) * dw).sum() + 0.3 * 12 / (3 * counts[-1]) * (counts[:-1] * probs).sum()

    assert np.allclose(*slope(loss, l, dl), rtol=1e-6, atol=1e-9)


def test_oracle_choice_of_ties_and_masks():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, 0.0, np.nan]])
    assert ref.choose(l, 3, "softmax").tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 2]]
    assert ref.choose(l[:1], 2, "sigmoid", bias=np.array([2.0, 0.0, 0.1, 9.0])).tolist() == [[0, 2]]
