"""GPU tests of the operators between token ids and the expert layer against the fp64
oracle: the embedding, layer norm, the router with its balance loss, their gradients.

Tolerances count roundings, u = 2^-24 for fp32 and half(t) = eps / 2 for an output's
type, whose subnormal numbers are multiples of step(t):
  embedding   one product: (u + half(t)) |v|
  its gradient  n sums and one product: ((n + 2) u) sum |scale d|, then half(t) |v|;
              with accumulate one more sum
  layer norm  D: the most additions that an element passes through in a row's sums.  A
              lane adds at most 64 elements, 6 steps join the lanes, 16 the waves: 86.
              The mean is off by (D + 2) u mean|x|, the differences from it by u each,
              what that leaves of the mean by (D + 4) u mean|d| <= (D + 4) u / rstd; the
              variance by (D + 8) u of itself, rstd by half as much and 4 u more:
              u (|w| (D + 4) + |w xh| (D / 2 + 12) + 3 |y|), then half(t) |y|
  its gradient  g is off by u, xh by 2 u, mean g by (D + 3) u mean|g|, mean(g xh) by
              (D + 7) u mean|g xh|: rstd u ((D + 6) mean|g| + |xh| (D + 12) mean|g xh|
              + 6 |g|), then half(t) |dx|; weights' gradients: (R + 6) u sum of sizes
  router      exp is taken as within 2 u, its argument l - top is off by u |l - top|:
              scores are off by (a + 4) u with a the largest |l - top|, sums of them
              by 22 u more (16 in a lane, 6 steps) or k u: (2 a + k + 40) u of a weight or
              probability; probs and the loss N u more; gradients (4 a + 2 k + 80) u
              of the sum of the sizes of their terms, then half(t)
"""
import numpy as np
import pytest
import torch

import newton_schulz_gram_amd as nsg
from oracle import layer_oracle as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
D = 86


def half(t):
    return torch.finfo(t).eps / 2


def step(t):
    return torch.finfo(t).tiny * torch.finfo(t).eps


def f64(t):
    return t.detach().cpu().double().numpy()


def normal(shape, dt, seed, scale=1.0, shift=0.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy((scale * g.standard_normal(shape) + shift).astype(np.float32)).to(DT[dt]).cuda()


def close(got, want, tol, what=""):
    """|got - want| <= tol + the rounding to got's type."""
    t = got.dtype
    assert tuple(got.shape) == np.shape(want), what
    g = f64(got)
    bad = ~(np.abs(g - want) <= tol + half(t) * (np.abs(want) + tol) + step(t))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), g[bad][:3], np.asarray(want)[bad][:3])


def pitched(x, extra, offset=0):
    """The same matrix in rows `extra` elements longer, from `offset` elements on."""
    R, C = x.shape
    room = torch.full((R * (C + extra) + offset,), float("nan"), dtype=x.dtype, device=x.device)
    v = room[offset:].view(R, C + extra)[:, :C]
    v.copy_(x)
    return v


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
def token_ids(shape, V, seed, wide=True, drop=0.1):
    """Ids of which some are met often; some are none."""
    g = np.random.default_rng(seed)
    ids = np.minimum(np.asarray(V * g.random(shape) ** 3).astype(np.int64), V - 1)
    ids = np.where(g.random(shape) < drop, -1, ids)
    if ids.size > 3:
        ids.reshape(-1)[1] = V
        ids.reshape(-1)[2] = -2 ** 40 if wide else -2 ** 31
        ids.reshape(-1)[3] = 2 ** 40 if wide else 2 ** 31 - 1
    return torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape,V,C", [((0,), 5, 8), ((1,), 1, 1), ((7,), 17, 3), ((3, 5), 1000, 130), ((2, 2, 9), 40, 513),
                                       ((1000,), 333, 1024), ((5,), 9, 4097), ((), 4, 64), ((64,), 100, 65536)])
def test_embedding(dt, shape, V, C):
    W = normal((V, C), dt, seed=V + C)
    for wide in (True, False):
        ids = token_ids(shape, V, seed=V, wide=wide)
        for scale in (1.0, 27.712812):
            want = ref.embedding(ids.cpu().numpy(), f64(W), float(np.float32(scale)))
            close(nsg.embedding(ids, W, scale), want, U * np.abs(want))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("extra,offset", [(8, 0), (5, 0), (8, 1), (3, 3)])
def test_embedding_of_pitched_rows(dt, extra, offset):
    W = normal((50, 264), dt, seed=3)
    ids = token_ids((77,), 50, seed=4)
    assert torch.equal(nsg.embedding(ids, pitched(W, extra, offset), 1.5), nsg.embedding(ids, W, 1.5))


def test_embedding_of_ids_that_are_all_none():
    W = torch.full((4, 40), float("nan"), device="cuda")
    assert torch.equal(nsg.embedding(torch.full((6,), -1, device="cuda"), W), torch.zeros(6, 40, device="cuda"))
    assert nsg.embedding(torch.tensor([0], device="cuda"), torch.empty(0, 40, device="cuda")).eq(0).all()


def embedding_gradient(dout, ids, V, scale, got, old=None):
    scale = float(np.float32(scale))
    want, size, n = ref.embedding_backward(f64(dout), ids.cpu().numpy(), V, scale)
    tol = (n[:, None] + 2) * U * size
    if old is not None:
        want, tol = want + old, tol + U * (np.abs(old) + size)
    close(got, want, tol)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,V,C", [(0, 5, 8), (1, 1, 1), (8, 2, 3), (9, 1024, 40), (1000, 1025, 130), (1024, 1, 65),
                                   (4096, 500, 300), (16384, 32003, 24), (16385, 32003, 24), (33, 1 << 20, 5), (3001, 7, 2060)])
def test_embedding_backward(dt, T, V, C):
    for wide in (True, False):
        ids = token_ids((T,), V, seed=T + V, wide=wide)
        dout = normal((T, C), dt, seed=T + C)
        embedding_gradient(dout, ids, V, 1.5, nsg.embedding_backward(dout, ids, V, 1.5))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("odt", list(DT))
def test_embedding_backward_into_another_type(dt, odt):
    T, V, C = 2500, 300, 200
    ids, dout = token_ids((T,), V, seed=1), normal((T, C), dt, seed=2)
    out = torch.full((V, C), float("nan"), dtype=DT[odt], device="cuda")
    assert nsg.embedding_backward(dout, ids, V, out=out) is out
    embedding_gradient(dout, ids, V, 1.0, out)
    old = normal((V, C), odt, seed=5)
    out = old.clone()
    nsg.embedding_backward(dout, ids, V, out=out, accumulate=True)
    embedding_gradient(dout, ids, V, 1.0, out, f64(old))


def test_embedding_backward_leaves_rows_without_tokens_alone():
    ids = torch.tensor([3, 3, -1, 9, 7], device="cuda")
    out = torch.full((10, 33), float("nan"), device="cuda")
    out[3] = out[7] = 1
    nsg.embedding_backward(torch.ones(5, 33, device="cuda"), ids, 10, out=out, accumulate=True)
    assert out[3].eq(3).all() and out[7].eq(2).all()
    assert out[[0, 1, 2, 4, 5, 6, 8]].isnan().all()  # and 9 holds a NaN plus one
    nsg.embedding_backward(torch.ones(0, 33, device="cuda"), ids[:0], 10, out=out, accumulate=True)
    assert out[3].eq(3).all()
    assert nsg.embedding_backward(torch.ones(0, 33, device="cuda"), ids[:0], 10).eq(0).all()


@pytest.mark.parametrize("T", [5, 63, 64, 65, 1000, 20000])
@pytest.mark.parametrize("fill", [0, 11, -1])
def test_embedding_backward_of_one_token(T, fill):
    """A run over every chunk, or no run."""
    ids = torch.full((T,), fill, device="cuda")
    dout = normal((T, 40), "f32", seed=T)
    embedding_gradient(dout, ids, 12, 2.0, nsg.embedding_backward(dout, ids, 12, 2.0))


@pytest.mark.parametrize("T", [70000, 600001])
def test_embedding_backward_of_many_tokens(T):
    """Runs of every length, over chunks of several lengths, and a sort whose workgroups read their ids twice."""
    V, C = 50000, 6
    ids = token_ids((T,), V, seed=T)
    ids[T // 2:T // 2 + 9000] = 4321
    dout = normal((T, C), "bf16", seed=T)
    got = nsg.embedding_backward(dout, ids, V, out=torch.empty(V, C, device="cuda"))
    embedding_gradient(dout, ids, V, 1.0, got)
    assert torch.equal(got, nsg.embedding_backward(dout, ids, V, out=torch.empty(V, C, device="cuda")))


def test_embedding_backward_layouts():
    """Batched ids, rows with a pitch, outputs and inputs off any boundary."""
    ids = token_ids((6, 50), 70, seed=1)
    dout = normal((6, 50, 136), "bf16", seed=2)
    want = nsg.embedding_backward(dout, ids, 70)
    flat = dout.view(300, 136)
    for extra, offset in ((8, 0), (3, 0), (8, 1)):
        assert torch.equal(nsg.embedding_backward(pitched(flat, extra, offset), ids.view(-1), 70), want)
    room = torch.full((70 * 136 + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[1:-2].view(70, 136)
    nsg.embedding_backward(dout, ids, 70, out=out)
    assert torch.equal(out, want) and room[0] == 7 and room[-2:].eq(7).all()


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
WIDTHS = [1, 2, 3, 8, 63, 64, 65, 256, 257, 512, 513, 1000, 1024, 2048, 2050, 4096, 4100, 8192, 11008, 16384, 16385, 32768, 40001,
          65536]


def norm_case(R, C, dt, wdt, seed, shift=0.0, scale=1.0):
    x = normal((R, C), dt, seed, scale, shift)
    w = normal((C,), wdt, seed + 1, 0.3, 1.0)
    b = normal((C,), wdt, seed + 2, 0.3)
    return x, w, b


def check_norm(x, w, b, eps, y, stats):
    xd = f64(x)
    wd, bd = (None if t is None else f64(t) for t in (w, b))
    eps = float(np.float32(eps))
    want, mean, rstd = ref.layer_norm(xd, wd, bd, eps)
    mtol = (D + 2) * U * np.abs(xd).mean(1) + U * np.abs(mean)
    close(stats[0], mean, mtol, "mean")
    close(stats[1], rstd, (D / 2 + 12) * U * rstd, "rstd")
    xh = np.abs((xd - mean[:, None]) * rstd[:, None])
    ws = 1.0 if wd is None else np.abs(wd)
    close(y, want, U * (ws * (D + 4) + ws * xh * (D / 2 + 12) + 3 * np.abs(want)), "y")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("C", WIDTHS)
def test_layer_norm(dt, C):
    for R, wdt in ((1, "f32"), (7, dt), (67 if C < 5000 else 5, "f32")):
        x, w, b = norm_case(R, C, dt, wdt, seed=R + C)
        check_norm(x, w, b, 1e-5, *nsg.layer_norm(x, w, b, 1e-5))


@pytest.mark.parametrize("dt", list(DT))
def test_layer_norm_without_weights_and_of_other_shapes(dt):
    x, w, b = norm_case(30, 200, dt, "bf16", seed=1)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_norm(x, ww, bb, 1e-3, *nsg.layer_norm(x, ww, bb, eps=1e-3))
    y, stats = nsg.layer_norm(x, w, b)
    y3, s3 = nsg.layer_norm(x.view(5, 6, 200), w, b)
    assert torch.equal(y3.view(30, 200), y) and torch.equal(stats, s3)
    for extra, offset in ((8, 0), (5, 0), (8, 1)):
        yp, sp = nsg.layer_norm(pitched(x, extra, offset), w, b)
        assert torch.equal(yp, y) and torch.equal(sp, stats)
    y0, s0 = nsg.layer_norm(x[:0], w, b)
    assert y0.shape == (0, 200) and s0.shape == (2, 0)


@pytest.mark.parametrize("C", [64, 1000, 4096, 20000, 65536])
@pytest.mark.parametrize("shift,scale", [(1000.0, 1.0), (-3.0, 1e-3), (0.0, 1e6), (0.0, 1e-6)])
def test_layer_norm_of_large_means_and_small_spreads(C, shift, scale):
    x, w, b = norm_case(9, C, "f32", "f32", seed=C, shift=shift, scale=scale)
    check_norm(x, w, b, 1e-12, *nsg.layer_norm(x, w, b, 1e-12))


@pytest.mark.parametrize("C", [3, 300, 4096, 16384, 20000])
@pytest.mark.parametrize("scale", [1e-18, 1e16])
def test_layer_norm_at_the_ends_of_its_range(C, scale):
    """Squares of 1e-36 (above 2^-126), and of 1e32, whose sum is below 2^128; no eps."""
    x, w, b = norm_case(9, C, "f32", "f32", seed=C, scale=scale)
    y, stats = nsg.layer_norm(x, w, b, 0.0)
    check_norm(x, w, b, 0.0, y, stats)
    dy = normal((9, C), "f32", seed=1)
    check_norm_gradient(dy, x, stats, w, *nsg.layer_norm_backward(dy, x, stats, w))


def test_layer_norm_of_constant_and_non_finite_rows():
    x = torch.full((6, 300), 3.5, device="cuda")
    x[1] = normal((300,), "f32", seed=1)
    x[2, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    y, stats = nsg.layer_norm(x, eps=1e-5)
    assert y[0].eq(0).all() and y[5].eq(0).all() and stats[0, 0] == 3.5
    assert abs(stats[1, 0].item() - 1e-5 ** -0.5) < 1e-4
    assert y[1].isfinite().all() and y[2:5].isnan().all(1).all()


def check_norm_gradient(dy, x, stats, w, dx, dw, db):
    d, xd, (mean, rstd) = f64(dy), f64(x), f64(stats)
    wd = None if w is None else f64(w)
    R, C = xd.shape
    want = ref.layer_norm_backward(d, xd, mean, rstd, wd)
    xh = np.abs((xd - mean[:, None]) * rstd[:, None])
    g = np.abs(d if wd is None else d * wd)
    mg, mgx = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    close(dx, want[0], rstd[:, None] * U * ((D + 6) * mg + xh * (D + 12) * mgx + 6 * g), "dx")
    if dw is not None:
        close(dw, want[1], (R + 6) * U * (np.abs(d) * xh).sum(0), "dweight")
    if db is not None:
        close(db, want[2], (R + 6) * U * np.abs(d).sum(0), "dbias")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("C", WIDTHS)
def test_layer_norm_backward(dt, C):
    for R, wdt in ((1, "f32"), (7, dt), (600 if C < 1100 else 67 if C < 5000 else 5, "f32")):
        x, w, b = norm_case(R, C, dt, wdt, seed=R + C)
        dy = normal((R, C), dt, seed=R + C + 9, scale=0.1)
        _, stats = nsg.layer_norm(x, w, b)
        dx, dw, db = nsg.layer_norm_backward(dy, x, stats, w)
        assert dw.dtype == db.dtype == w.dtype
        check_norm_gradient(dy, x, stats, w, dx, dw, db)


@pytest.mark.parametrize("R,C", [(20000, 64), (5003, 1250), (300, 8192), (2600, 513)])
def test_layer_norm_backward_of_many_rows(R, C):
    x, w, b = norm_case(R, C, "bf16", "f32", seed=R)
    dy = normal((R, C), "bf16", seed=R + 1)
    _, stats = nsg.layer_norm(x, w, b)
    got = nsg.layer_norm_backward(dy, x, stats, w)
    check_norm_gradient(dy, x, stats, w, *got)
    for a, b2 in zip(got, nsg.layer_norm_backward(dy, x, stats, w)):
        assert torch.equal(a, b2)


@pytest.mark.parametrize("C", [200, 20000])
def test_layer_norm_backward_parts_and_layouts(C):
    x, w, b = norm_case(30, C, "bf16", "bf16", seed=1)
    dy = normal((30, C), "bf16", seed=4)
    _, stats = nsg.layer_norm(x, w, b)
    dx, dw, db = nsg.layer_norm_backward(dy, x, stats, w)
    for wg, bg in ((True, False), (False, True), (False, False)):
        got = nsg.layer_norm_backward(dy, x, stats, w, weight_grad=wg, bias_grad=bg)
        assert torch.equal(got[0], dx)
        assert (got[1] is None) != wg and (got[2] is None) != bg
        assert (not wg or torch.equal(got[1], dw)) and (not bg or torch.equal(got[2], db))
    plain = nsg.layer_norm_backward(dy, x, stats)
    assert plain[1].dtype == torch.float32
    check_norm_gradient(dy, x, stats, None, *plain)
    got = nsg.layer_norm_backward(dy.view(5, 6, C), x.view(5, 6, C), stats, w)
    assert torch.equal(got[0].view(30, C), dx) and torch.equal(got[1], dw)
    got = nsg.layer_norm_backward(pitched(dy, 3, 1), pitched(x, 8), stats, w)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    got = nsg.layer_norm_backward(dy[:0], x[:0], stats[:, :0].contiguous(), w)
    assert got[0].shape == (0, C) and got[1].eq(0).all() and got[2].eq(0).all()


def test_layer_norm_gradient_against_differences():
    """The chain of both calls: the loss sum(y u) changes by dx . h along any direction h."""
    R, C = 11, 300
    x, w, b = norm_case(R, C, "f32", "f32", seed=8)
    u = normal((R, C), "f32", seed=9)
    _, stats = nsg.layer_norm(x, w, b)
    got = [f64(t) for t in nsg.layer_norm_backward(u, x, stats, w)]
    loss = lambda xd, wd, bd: (ref.layer_norm(xd, wd, bd)[0] * f64(u)).sum()  # noqa: E731
    args, g = [f64(t) for t in (x, w, b)], np.random.default_rng(10)
    for i in range(3):
        h = g.standard_normal(args[i].shape)
        up, down = ([a + s * 1e-5 * h if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        slope = (loss(*up) - loss(*down)) / 2e-5
        # fp32 gradients: about D u of the sum of the sizes; differences: 1e-10 of the loss's third derivative
        assert abs(slope - (got[i] * h).sum()) <= 1e-4 * (1 + np.abs(got[i] * h).sum() ** 0.5), i


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
def router_case(T, E, dt, seed, spread=1.5):
    g = np.random.default_rng(seed)
    l = spread * g.standard_normal((T, E)) + 0.5 * g.standard_normal(E)
    return torch.from_numpy(l.astype(np.float32)).to(DT[dt]).cuda()


def spread_of(l):
    f = l[np.isfinite(l)]
    return float(np.abs(f).max() * 2) if f.size else 0.0


def check_route(logits, k, score, normalize, scale, got, bias=None, mask=None, balance=False):
    l = f64(logits)
    ids = ref.choose(l, k, score, None if bias is None else f64(bias), None if mask is None else mask.cpu().numpy())
    assert np.array_equal(got.ids.cpu().numpy(), ids)
    want = ref.weights(l, ids, score, normalize, float(np.float32(scale)))
    a = spread_of(l)
    close(got.weights, want, (2 * a + k + 40) * U * np.abs(want), "weights")
    if not balance:
        assert got.counts is None and got.probs is None and got.loss is None
        return ids
    counts, probs, loss = ref.balance(l, ids, score, k)
    assert np.array_equal(got.counts.cpu().numpy(), counts)
    N = counts[-1]
    close(got.probs, probs, (2 * a + 40 + N) * U * probs, "probs")
    close(got.loss, loss, (2 * a + 60 + N + l.shape[1]) * U * loss, "loss")
    return ids


ROUTERS = [(1, 1, 1), (3, 2, 1), (17, 4, 4), (1000, 5, 3), (65, 16, 16), (33, 17, 2), (500, 60, 4), (129, 64, 64), (77, 65, 6),
           (300, 128, 8), (31, 200, 33), (1030, 256, 8), (5, 300, 1), (200, 512, 10), (64, 1000, 64), (41, 1024, 8)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", ROUTERS)
def test_route(dt, score, T, E, k):
    logits = router_case(T, E, dt, seed=T + E)
    g = np.random.default_rng(E)
    bias = torch.from_numpy((0.2 * g.standard_normal(E)).astype(np.float32)).cuda()
    mask = torch.from_numpy(g.random(T) < 0.8).cuda()
    for normalize, scale in ((True, 1.0), (False, 2.5)):
        kw = dict(score=score, normalize=normalize, scale=scale)
        check_route(logits, k, score, normalize, scale, nsg.expert_route(logits, k, **kw))
        check_route(logits, k, score, normalize, scale, nsg.expert_route(logits, k, bias=bias, balance=True, **kw), bias=bias,
                    balance=True)
        check_route(logits, k, score, normalize, scale, nsg.expert_route(logits, k, mask=mask, balance=True, **kw), mask=mask,
                    balance=True)


@pytest.mark.parametrize("T,E,k", [(20000, 64, 6), (9001, 512, 8), (70001, 8, 2)])
def test_route_of_many_tokens(T, E, k):
    logits = router_case(T, E, "bf16", seed=T)
    got = nsg.expert_route(logits, k, balance=True)
    check_route(logits, k, "softmax", True, 1.0, got, balance=True)
    for a, b in zip(got, nsg.expert_route(logits, k, balance=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E", [7, 64, 256, 700])
def test_route_of_equal_logits(score, bias, E):
    """Ties go to the lower index; few different values, zeros of both signs among them."""
    g = np.random.default_rng(E)
    l = torch.from_numpy(g.choice([-0.0, 0.0, 1.0, -2.0], size=(50, E)).astype(np.float32)).cuda()
    l[0] = 0
    b = torch.zeros(E, device="cuda") if bias else None
    k = min(E, 9)
    check_route(l, k, score, True, 1.0, nsg.expert_route(l, k, score=score, bias=b, balance=True), bias=b, balance=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E", [6, 60, 256, 1000])
def test_route_of_masked_experts(score, bias, E):
    """-inf and the type's lowest value among the logits; rows with fewer finite ones than k, and none."""
    g = np.random.default_rng(E + 1)
    l = router_case(40, E, "f32", seed=E)
    l[torch.from_numpy(g.random((40, E)) < 0.5).cuda()] = -float("inf")
    l[3] = -float("inf")
    l[4], l[4, E // 2] = -float("inf"), -50.0
    l[5] = torch.finfo(torch.float32).min
    l[6], l[6, E - 1] = torch.finfo(torch.float32).min, 1.0
    b = torch.from_numpy((0.2 * g.standard_normal(E)).astype(np.float32)).cuda() if bias else None
    if bias:
        b[E - 2] = -float("inf")
    for normalize in (True, False):
        got = nsg.expert_route(l, 4, score=score, bias=b, balance=True, normalize=normalize)
        lr = l.clone()
        lr[5:7] = lr[5:7].clamp(min=-1e4)  # as far from the rest in fp64
        ids = ref.choose(f64(l), 4, score, None if b is None else f64(b))
        assert np.array_equal(got.ids.cpu().numpy(), ids)
        assert (got.ids[3] == -1).all() and (got.weights[3] == 0).all()
        w = ref.weights(f64(lr), ids, score, normalize, 1.0)
        if score == "sigmoid" and normalize:
            w[5] = np.where(ids[5] >= 0, 1 / max(1, (ids[5] >= 0).sum()), 0)
        rows = [i for i in range(40) if i != 5] if score == "sigmoid" else list(range(40))
        close(got.weights[rows], w[rows], (2 * 60 + 44) * U * np.abs(w[rows]), "weights")
        counts, probs, loss = ref.balance(f64(lr), ids, score, 4)
        assert np.array_equal(got.counts.cpu().numpy(), counts) and counts[E] <= 39
        close(got.probs, probs, (2 * 60 + 80) * U * probs + 1e-30, "probs")


def test_route_of_nothing():
    l = torch.empty(0, 12, device="cuda")
    got = nsg.expert_route(l, 3, balance=True)
    assert got.ids.shape == (0, 3) and got.counts.eq(0).all() and got.probs.eq(0).all() and got.loss == 0
    l = torch.full((5, 12), -float("inf"), device="cuda")
    got = nsg.expert_route(l, 3, balance=True)
    assert got.ids.eq(-1).all() and got.weights.eq(0).all() and got.counts.eq(0).all() and got.loss == 0
    got = nsg.expert_route(torch.zeros(5, 12, device="cuda"), 3, mask=torch.zeros(5, dtype=torch.bool, device="cuda"), balance=True)
    assert got.ids.eq(-1).all() and got.weights.eq(0).all() and got.counts.eq(0).all() and got.loss == 0
    dl = nsg.expert_route_backward(l, got.ids, torch.ones(5, 3, device="cuda"), counts=got.counts)
    assert dl.eq(0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_non_finite_logits(score):
    l = router_case(6, 40, "f32", seed=1)
    l[1, 5], l[2, 6], l[3] = float("nan"), float("inf"), float("nan")
    got = nsg.expert_route(l, 3, score=score, balance=True)
    ids = got.ids.cpu()
    assert (ids[1] != 5).all() and (ids[1] >= 0).all() and ids[2, 0] == 6 and ids[3].eq(-1).all()
    assert got.weights[1:3].isnan().all() == (score == "softmax") and got.weights[3].eq(0).all()
    assert got.weights[[0, 4, 5]].isfinite().all() and got.counts[40] == 5
    assert got.loss.isnan()
    if score == "sigmoid":
        assert got.weights[1:3].isfinite().all()


@pytest.mark.parametrize("dt", list(DT))
def test_route_layouts_and_masks_of_bytes(dt):
    l = router_case(90, 60, dt, seed=2)
    mask = torch.arange(90, device="cuda") % 3 != 0
    want = nsg.expert_route(l, 4, mask=mask, balance=True)
    dw = normal((90, 4), "f32", seed=3)
    grad = nsg.expert_route_backward(l, want.ids, dw, counts=want.counts)
    for extra, offset in ((4, 0), (3, 0), (8, 1)):
        v = pitched(l, extra, offset)
        got = nsg.expert_route(v, 4, mask=mask.to(torch.uint8), balance=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(nsg.expert_route_backward(v, want.ids, dw, counts=want.counts), grad)


def test_route_with_far_scores_in_the_choice():
    """A bias may choose experts whose scores are nothing beside the largest: their weights add up to 1 all the same."""
    l = torch.tensor([[0.0, -200.0, -201.0, 5.0]], device="cuda")
    b = torch.tensor([0.0, 4.0, 4.0, 0.0], device="cuda")
    for score in ("softmax", "sigmoid"):
        got = nsg.expert_route(l, 2, score=score, bias=b)
        assert got.ids.tolist() == [[1, 2]]
        want = ref.weights(f64(l), np.array([[1, 2]]), score, True, 1.0)
        close(got.weights, want, (2 * 400 + 44) * U * want)


def check_route_gradient(logits, ids, dw, score, normalize, scale, got, counts=None, coef=1.0):
    l = f64(logits)
    want, size = ref.route_backward(l, ids.cpu().numpy(), None if dw is None else f64(dw), score, normalize,
                                    float(np.float32(scale)), None if counts is None else counts.cpu().numpy(), coef)
    close(got, want, (4 * spread_of(l) + 2 * ids.shape[1] + 80) * U * size, "dlogits")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", ROUTERS)
def test_route_backward(dt, score, T, E, k):
    logits = router_case(T, E, dt, seed=T + E)
    mask = torch.from_numpy(np.random.default_rng(E).random(T) < 0.8).cuda()
    dw = normal((T, k), "f32", seed=k)
    dloss = torch.full((), 4096.0, device="cuda")
    for normalize, scale in ((True, 1.0), (False, 2.5)):
        kw = dict(score=score, normalize=normalize, scale=scale)
        r = nsg.expert_route(logits, k, mask=mask, balance=True, **kw)
        got = nsg.expert_route_backward(logits, r.ids, dw, **kw)
        check_route_gradient(logits, r.ids, dw, score, normalize, scale, got)
        got = nsg.expert_route_backward(logits, r.ids, dw, counts=r.counts, balance=0.5, dloss=dloss, **kw)
        check_route_gradient(logits, r.ids, dw, score, normalize, scale, got, r.counts, 2048.0)
        got = nsg.expert_route_backward(logits, r.ids, None, counts=r.counts, balance=1024.0, **kw)
        check_route_gradient(logits, r.ids, None, score, normalize, scale, got, r.counts, 1024.0)


def test_route_backward_of_many_tokens():
    logits = router_case(70001, 8, "f32", seed=5)
    r = nsg.expert_route(logits, 2, balance=True)
    dw = normal((70001, 2), "f32", seed=6)
    got = nsg.expert_route_backward(logits, r.ids, dw, counts=r.counts, balance=1e5)
    check_route_gradient(logits, r.ids, dw, "softmax", True, 1.0, got, r.counts, 1e5)
    assert torch.equal(got, nsg.expert_route_backward(logits, r.ids, dw, counts=r.counts, balance=1e5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward_of_masked_experts(score, normalize):
    """Gradients are finite, and zero at logits of -inf; ids that are no expert count as none."""
    l = router_case(40, 60, "f32", seed=7)
    l[torch.from_numpy(np.random.default_rng(8).random((40, 60)) < 0.5).cuda()] = -float("inf")
    l[3] = -float("inf")
    kw = dict(score=score, normalize=normalize)
    r = nsg.expert_route(l, 4, balance=True, **kw)
    ids = r.ids.clone()
    ids[9, 1], ids[10, 0], ids[11] = 60, -2 ** 31, 2 ** 31 - 1
    dw = normal((40, 4), "f32", seed=9)
    got = nsg.expert_route_backward(l, ids, dw, counts=r.counts, balance=100.0, **kw)
    assert got.isfinite().all() and got[l == -float("inf")].eq(0).all() and got[11].eq(0).all()
    ids = torch.where((ids >= 0) & (ids < 60), ids, -1)
    assert torch.equal(got, nsg.expert_route_backward(l, ids, dw, counts=r.counts, balance=100.0, **kw))
    with np.errstate(all="ignore"):
        want, size = ref.route_backward(f64(l.clamp(min=-1e4)), ids.cpu().numpy(), f64(dw), score, normalize, 1.0,
                                        r.counts.cpu().numpy(), 100.0)
    close(got, want, (4 * 20 + 88) * U * size, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_against_differences(score, normalize):
    T, E, k = 13, 24, 3
    logits = router_case(T, E, "f32", seed=11)
    r = nsg.expert_route(logits, k, score=score, normalize=normalize, scale=2.0, balance=True)
    dw = normal((T, k), "f32", seed=12)
    got = f64(nsg.expert_route_backward(logits, r.ids, dw, score=score, normalize=normalize, scale=2.0, counts=r.counts, balance=3.0))
    ids, counts = r.ids.cpu().numpy(), r.counts.cpu().numpy()

    def loss(l):
        N = counts[E]
        probs = ref.shares(l, score).sum(0) / N
        return (ref.weights(l, ids, score, normalize, 2.0) * f64(dw)).sum() + 3.0 * E / (k * N) * (counts[:E] * probs).sum()

    l = f64(logits)
    for seed in range(4):
        h = np.random.default_rng(seed).standard_normal(l.shape)
        slope = (loss(l + 1e-5 * h) - loss(l - 1e-5 * h)) / 2e-5
        assert abs(slope - (got * h).sum()) <= 2e-5 * np.abs(got * h).sum() + 1e-8
