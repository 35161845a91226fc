"""GPU tests of the operators between token ids and the expert layer as a training step
uses them: together with the expert layer, on other streams, captured into graphs, with
workspaces of the caller's, with offsets past 32 bits, at the ends of their limits."""
import numpy as np
import pytest
import torch

import newton_schulz_gram_amd as nsg
from oracle import layer_oracle as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rand(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def integers(hi, shape, seed, lo=0, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def same(a, b):
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x, y)


def every_call(seed, dtype=torch.bfloat16, T=300, V=500, C=264, E=60, k=4):
    """Inputs, and a function that makes each call once and returns all outputs."""
    ids, W = integers(V, (T,), seed, lo=-3), rand((V, C), seed + 1, dtype)
    gamma, beta = rand((C,), seed + 2), rand((C,), seed + 3)
    dy, logits = rand((T, C), seed + 4, dtype), rand((T, E), seed + 5, dtype)
    bias, dw = rand((E,), seed + 6, scale=0.1), rand((T, k), seed + 7)
    mask = rand((T,), seed + 8) > -1
    dloss = torch.full((), 3.0, device="cuda")

    def run(ws=(None,) * 3):
        x = nsg.embedding(ids, W, 1.5)
        y, stats = nsg.layer_norm(x, gamma, beta)
        dx, dg, db = nsg.layer_norm_backward(dy, x, stats, gamma, workspace=ws[0])
        dW = nsg.embedding_backward(dx, ids, V, 1.5, workspace=ws[1])
        r = nsg.expert_route(logits, k, score="sigmoid", bias=bias, mask=mask, balance=True, workspace=ws[2])
        dl = nsg.expert_route_backward(logits, r.ids, dw, score="sigmoid", counts=r.counts, balance=0.5, dloss=dloss)
        return (x, y, stats, dx, dg, db, dW, *r, dl)

    inputs = (ids, W, gamma, beta, dy, logits, bias, dw, mask)
    need = (nsg.layer_norm_backward_workspace_size(T, C), nsg.embedding_backward_workspace_size(T, V, C),
            nsg.expert_route_workspace_size(T, E))
    return inputs, run, need


def test_workspaces_of_the_caller():
    """Exactly as large as needed, larger, and full of anything; nothing behind their end is written."""
    _, run, need = every_call(1)
    want = run()
    for fill in (0, 255):
        rooms = [torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda") for n in need]
        same(run([r[:n] for r, n in zip(rooms, need)]), want)
        for r in rooms:
            assert r[-64:].eq(fill).all()
    big = [torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda") for n in need]
    same(run(big), want)
    # one that is too small is not used
    small = [torch.full((max(n - 1, 0),), 5, dtype=torch.uint8, device="cuda") for n in need]
    same(run(small), want)
    assert all(s.eq(5).all() for s in small)


def test_workspaces_refused():
    _, run, need = every_call(2)
    with pytest.raises(ValueError):
        run([torch.empty(need[0], dtype=torch.uint8), None, None])
    with pytest.raises(nsg.NSGError):  # off its 16-byte boundary
        run([torch.empty(need[0] + 16, dtype=torch.uint8, device="cuda")[8:], None, None])


def test_on_other_streams():
    """Work follows the current stream: inputs that another kernel of that stream is still writing."""
    inputs, run, _ = every_call(3)
    want = run()
    torch.cuda.synchronize()
    copies = [t.clone() for t in inputs]
    side = torch.cuda.Stream()
    busy = rand((4096, 4096), 9)
    with torch.cuda.stream(side):
        for t in inputs:
            t.zero_()
        for _ in range(8):
            busy @ busy
        for t, c in zip(inputs, copies):
            t.copy_(c)
        got = run()
    side.synchronize()
    same(got, want)


def test_two_streams_at_once():
    runs = [every_call(10 + i)[1] for i in range(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        got = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(r())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        same(g, w)


@pytest.mark.parametrize("T,V,C,E", [(300, 500, 264, 60), (20000, 3000, 40, 512), (2100, 100, 1250, 8)])
def test_graph_replays(T, V, C, E):
    """Captured once, replayed on new inputs with eager work in between, with other graphs' replays too."""
    inputs, run, _ = every_call(20, T=T, V=V, C=C, E=E)
    others, run2, _ = every_call(40, T=T, V=V, C=C, E=E)
    fresh = [[t.clone() for t in every_call(60 + i, T=T, V=V, C=C, E=E)[0]] for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        run2()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for fn in (run, run2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fn()
        graphs.append((g, out))
    for i in range(4):
        for t, f in zip(inputs, fresh[i % 2]):
            t.copy_(f)
        for t, f in zip(others, fresh[(i + 1) % 2]):
            t.copy_(f)
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in out] for _, out in graphs]
        same(got[0], run())
        same(got[1], run2())
        rand((64, 64), i) @ rand((64, 64), i + 1)


def test_refusals_of_gpu_tensors():
    x, ids = rand((6, 40), 1), integers(6, (6,), 2)
    r = nsg.expert_route(x, 3, balance=True)
    y, stats = nsg.layer_norm(x)
    bad = [
        lambda: nsg.embedding(ids.float(), x), lambda: nsg.embedding(ids.cpu(), x), lambda: nsg.embedding(ids, x.t()),
        lambda: nsg.embedding(ids, x[0]), lambda: nsg.embedding(ids, x.double()), lambda: nsg.embedding(ids.repeat(2)[::2], x),
        lambda: nsg.embedding_backward(x, ids[:5], 9), lambda: nsg.embedding_backward(x, ids, 9, accumulate=True),
        lambda: nsg.embedding_backward(x, ids, 9, out=x), lambda: nsg.embedding_backward(x.t().contiguous().t(), ids, 9),
        lambda: nsg.embedding_backward(x, ids, 9, out=torch.empty(9, 80, device="cuda")[:, :40]),
        lambda: nsg.embedding_backward(x.expand(3, 6, 40), ids.expand(3, 6).contiguous(), 9),
        lambda: nsg.layer_norm(x.t()), lambda: nsg.layer_norm(x[0]), lambda: nsg.layer_norm(x, x[0, :39]),
        lambda: nsg.layer_norm(x, x[0], x[0].half()), lambda: nsg.layer_norm(x, x[0].double()), lambda: nsg.layer_norm(x, x[0].cpu()),
        lambda: nsg.layer_norm(x[:, :1].expand(6, 40)), lambda: nsg.layer_norm(x.unsqueeze(1).expand(6, 2, 40)),
        lambda: nsg.layer_norm_backward(x.half(), x, stats), lambda: nsg.layer_norm_backward(x[:5], x, stats),
        lambda: nsg.layer_norm_backward(x, x, stats[:1]), lambda: nsg.layer_norm_backward(x, x, stats.double()),
        lambda: nsg.layer_norm_backward(x, x, stats, x[0, :3]), lambda: nsg.layer_norm_backward(x, x, stats.cpu()),
        lambda: nsg.expert_route(x, 0), lambda: nsg.expert_route(x, 41), lambda: nsg.expert_route(x, 2, score="tanh"),
        lambda: nsg.expert_route(x, 2, bias=x[0, :5]), lambda: nsg.expert_route(x, 2, bias=x[0].half()),
        lambda: nsg.expert_route(x, 2, mask=ids), lambda: nsg.expert_route(x, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda")),
        lambda: nsg.expert_route(x[0], 2), lambda: nsg.expert_route(x.t(), 2),
        lambda: nsg.expert_route_backward(x, r.ids.long()), lambda: nsg.expert_route_backward(x, r.ids[:5]),
        lambda: nsg.expert_route_backward(x, r.ids, r.weights[:, :2]), lambda: nsg.expert_route_backward(x, r.ids, r.weights.half()),
        lambda: nsg.expert_route_backward(x, r.ids, r.weights, counts=r.counts[:-1]),
        lambda: nsg.expert_route_backward(x, r.ids, r.weights, dloss=r.loss),
        lambda: nsg.expert_route_backward(x, r.ids, r.weights, counts=r.counts, dloss=r.probs),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: nsg.embedding(ids, x, float("nan")), lambda: nsg.layer_norm(x, eps=-1.0),
                 lambda: nsg.layer_norm(x[:, :0]), lambda: nsg.expert_route(rand((2, 1025), 3), 2),
                 lambda: nsg.expert_route(x, 2, scale=float("inf")), lambda: nsg.embedding_backward(x, ids, -1),
                 lambda: nsg.embedding_backward(x, ids, (1 << 20) + 1)):
        with pytest.raises((nsg.NSGError, RuntimeError)):
            call()


# ---------------------------------------------------------------------------
# together with the expert layer
# ---------------------------------------------------------------------------
def test_a_layer_of_experts_from_token_ids_and_back():
    """embedding -> layer norm -> router -> sort, dispatch, experts, combine, and every gradient,
    in fp32 against autograd in 64 bits.

    The tolerance: sums of at most 400 terms in each of the 8 stages between an input and the
    last gradient, each off by 400 u of the sum of its terms' sizes; these cancel to no less than
    a tenth here: 8 * 400 u * 10 = 2e-3 of a gradient's norm at worst, and a tenth of that
    holds for errors that do not all have one sign."""
    B, S, V, C, F, E, k = 3, 70, 90, 96, 40, 12, 3
    T = B * S
    ids = integers(V, (B, S), 1)
    ids[:, -7:] = -1  # padding
    mask = (ids >= 0).view(-1)
    W, gamma, beta = rand((V, C), 2), 1 + 0.1 * rand((C,), 3), 0.1 * rand((C,), 4)
    Wr, We = 0.3 * rand((E, C), 5), 0.2 * rand((E, F, C), 6)
    bias, dout = 0.05 * rand((E,), 7), rand((T, F), 8)

    x = nsg.embedding(ids, W, 2.0)
    y, stats = nsg.layer_norm(x, gamma, beta)
    flat = y.view(T, C)
    logits = flat @ Wr.t()
    r = nsg.expert_route(logits, k, bias=bias, mask=mask, scale=1.5, balance=True)
    plan = nsg.expert_sort(r.ids, E)
    rows = nsg.expert_dispatch(flat, plan)
    cut = plan.offsets.tolist()
    z = torch.zeros(T * k, F, device="cuda")
    for e in range(E):
        z[cut[e]:cut[e + 1]] = rows[cut[e]:cut[e + 1]] @ We[e].t()
    out = nsg.expert_combine(z, plan, r.weights)
    assert out[~mask].eq(0).all() and cut[E] == k * int(mask.sum())

    dz, dw = nsg.expert_combine_backward(dout, z, plan, r.weights)
    drows, dWe = torch.zeros_like(rows), torch.zeros_like(We)
    for e in range(E):
        drows[cut[e]:cut[e + 1]] = dz[cut[e]:cut[e + 1]] @ We[e]
        dWe[e] = dz[cut[e]:cut[e + 1]].t() @ rows[cut[e]:cut[e + 1]]
    dl = nsg.expert_route_backward(logits, r.ids, dw, scale=1.5, counts=r.counts, balance=5.0)
    dflat = nsg.expert_combine(drows, plan) + dl @ Wr
    dx, dgamma, dbeta = nsg.layer_norm_backward(dflat.view(B, S, C), x, stats, gamma)
    dW = nsg.embedding_backward(dx, ids, V, 2.0)

    p = [t.double().cpu().requires_grad_() for t in (W, gamma, beta, Wr, We)]
    i = ids.view(-1).cpu()
    keep = i >= 0
    xr = torch.where(keep[:, None], 2.0 * p[0][i.clamp(min=0)], 0.0)
    yr = torch.nn.functional.layer_norm(xr, (C,), p[1], p[2], 1e-5)
    s = torch.softmax(yr @ p[3].t(), 1)
    ch = torch.topk(s + bias.double().cpu(), k, dim=1).indices
    assert torch.equal(torch.where(keep[:, None], ch, -1).int(), r.ids.cpu())
    w = s.gather(1, ch)
    w = 1.5 * w / w.sum(1, keepdim=True) * keep[:, None]
    outr = sum(w[:, j, None] * torch.einsum("tc,tfc->tf", yr, p[4][ch[:, j]]) for j in range(k))
    N = int(keep.sum())
    counts = torch.bincount(ch[keep].reshape(-1), minlength=E)
    loss = E / (k * N) * (counts.double() * (s[keep].sum(0) / N)).sum()
    assert torch.equal(torch.cat([counts, torch.tensor([N])]).int(), r.counts.cpu())
    assert abs(r.loss.item() - loss.item()) <= 1e-5
    want = torch.autograd.grad((outr * dout.double().cpu()).sum() + 5.0 * loss, p)
    for got, exp, name in zip((dW, dgamma, dbeta, dl.t() @ flat, dWe), want, ("embedding", "gamma", "beta", "router", "experts")):
        assert (got.double().cpu() - exp).norm() <= 2e-4 * exp.norm(), name
    assert (out.double().cpu() - outr).norm() <= 2e-4 * outr.norm()


def test_a_training_step_with_fp8_experts():
    """The same path in bf16 with the 8-bit products and the Muon step: twice, bit for bit, and finite."""
    T, V, C, F, E, k = 512, 1000, 256, 128, 16, 4
    ids = integers(V, (T,), 1, lo=-2, dtype=torch.int32)

    def step():
        W, gamma, beta = (rand(s, 2 + i, torch.bfloat16) for i, s in enumerate(((V, C), (C,), (C,))))
        Wr, We = rand((E, C), 5, torch.bfloat16, 0.1), rand((E, F, C), 6, torch.bfloat16, 0.05)
        M, dout = torch.zeros(E, F, C, device="cuda"), rand((T, F), 7, torch.bfloat16, 0.1)
        x = nsg.embedding(ids, W, 16.0)
        h, stats = nsg.layer_norm(x, gamma, beta)
        logits = h @ Wr.t()
        r = nsg.expert_route(logits, k, score="sigmoid", mask=ids >= 0, balance=True)
        plan = nsg.expert_sort(r.ids, E)
        hq, (wq, ws, wtq, wts) = nsg.quantize_fp8(h), nsg.quantize_fp8(We, block="tile", transposed=True)
        y = nsg.expert_gemm_fp8(*hq, wq, ws, plan.offsets, rows=plan.tokens)
        out = nsg.expert_combine(y, plan, r.weights)
        e5m2 = torch.float8_e5m2
        dy, dw = nsg.expert_combine_backward(dout, y, plan, r.weights)
        dh = nsg.expert_combine(nsg.expert_gemm_fp8(*nsg.quantize_fp8(dy, dtype=e5m2), wtq, wts, plan.offsets), plan)
        dWe = nsg.expert_wgrad_fp8(*nsg.quantize_fp8_columns(dy, plan.offsets, dtype=e5m2),
                                   *nsg.quantize_fp8_columns(h, plan.offsets, rows=plan.tokens), plan.offsets)
        dl = nsg.expert_route_backward(logits, r.ids, dw, score="sigmoid", counts=r.counts, balance=0.01)
        dx, dgamma, dbeta = nsg.layer_norm_backward(dh + dl @ Wr, x, stats, gamma)
        dW = nsg.embedding_backward(dx, ids, V, 16.0, out=torch.empty(V, C, device="cuda"))
        nsg.muon_step(We, M, dWe, mu=0.95, lr=0.02, seed=3)
        return out, *r, dl, dx, dgamma, dbeta, dW, We, M

    a, b = step(), step()
    same(a, b)
    assert all(t.float().isfinite().all() for t in a)
    assert a[0][ids < 0].eq(0).all() and a[9][0].ne(0).any()


def test_ids_that_leave_an_expert_empty_and_the_same_index_twice():
    """ids of the caller's own for the gradient: equal experts of a token add up."""
    l = rand((5, 20), 1)
    ids = torch.tensor([[3, 3], [3, 4], [-1, 19], [0, 0], [7, -5]], dtype=torch.int32, device="cuda")
    dw = rand((5, 2), 2)
    got = nsg.expert_route_backward(l, ids, dw, normalize=False).double().cpu()
    s = l.double().cpu().requires_grad_()
    p, e = torch.softmax(s, 1), ids.cpu().long()
    total = (p.gather(1, e.clamp(min=0)) * dw.double().cpu() * ((e >= 0) & (e < 20))).sum()
    want = torch.autograd.grad(total, s)[0]
    assert (got - want).abs().max() <= 200 * U


# ---------------------------------------------------------------------------
# large sizes
# ---------------------------------------------------------------------------
def test_embedding_offsets_past_32_bits():
    V, C = 1 << 20, 2304  # 2.4e9 elements
    W = torch.zeros(V, C, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, V - 1, 932067, 932068, 5, V], device="cuda")
    rows = rand((5, C), 1, torch.bfloat16)
    W[ids[:5]] = rows
    out = nsg.embedding(ids, W)
    assert torch.equal(out[:5], rows) and out[5].eq(0).all()
    del W
    dW = nsg.embedding_backward(out, ids, V)
    assert torch.equal(dW[ids[:5]], rows)
    assert int(dW.count_nonzero(1).ne(0).sum()) == 5
    nsg.embedding_backward(out, ids, V, out=dW, accumulate=True)
    assert torch.equal(dW[ids[:5]], (rows.float() * 2).bfloat16())


@pytest.mark.parametrize("C", [3, 64, 260, 1030])
@pytest.mark.parametrize("lengths", ["one id", "half of them", "around 16 parts", "around 32 parts", "many long ones"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_of_ids_that_come_often(C, lengths, accumulate):
    """Runs of equal ids over few and many chunks of the sorted list (of 8 tokens or more),
    whole numbers whose sums are exact in fp32 in any order."""
    n = {"one id": [30000],
         "half of them": [1] * 9000 + [15000] + [3] * 2000,
         "around 16 parts": [8 * k + d for k in range(13, 21) for d in (-1, 0, 1, 5)] * 5 + [1, 0, 2],
         "around 32 parts": [8 * k + d for k in range(29, 37) for d in (-1, 0, 1, 5)] * 3 + [1, 0, 2],
         "many long ones": [2000, 0, 1, 1999, 2001] * 4 + [513] * 7}[lengths]
    ids = torch.arange(len(n)).repeat_interleave(torch.tensor(n))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(5))].cuda()
    dout = integers(4, (len(ids), C), 6, lo=-4).to(torch.bfloat16)
    out = integers(100, (len(n), C), 7, lo=-100).float()
    want = out.double().cpu() if accumulate else torch.zeros(len(n), C, dtype=torch.float64)
    want.index_add_(0, ids.cpu(), dout.double().cpu(), alpha=2)
    got = nsg.embedding_backward(dout, ids, len(n), scale=2.0, out=out, accumulate=accumulate)
    assert torch.equal(got.double().cpu(), want)


def test_embedding_of_many_rows():
    """Output and dout past 32-bit offsets."""
    T, V, C = 700_000, 50, 4096
    W = rand((V, C), 1, torch.bfloat16)
    ids = integers(V, (T,), 2, dtype=torch.int32)
    out = nsg.embedding(ids, W)
    for a in (0, 524_287, T - 3):
        assert torch.equal(out[a:a + 3], W[ids[a:a + 3].long()])
    dW = nsg.embedding_backward(out, ids, V, out=torch.empty(V, C, device="cuda"))
    n = torch.bincount(ids, minlength=V).double()[:, None]
    want = n * W.double()
    # n sums in chunks of 64 and their joins: at most 64 + n / 64 additions of numbers of one size
    assert ((dW.double() - want).abs() <= (66 + n / 64) * U * want.abs()).all()


def test_layer_norm_offsets_past_32_bits():
    R, C = 540_000, 4096
    x = rand((R, C), 1, torch.bfloat16)
    y, stats = nsg.layer_norm(x)
    dx, dw, db = nsg.layer_norm_backward(x, x, stats)
    for a in (0, 524_287, R - 9):
        part, s = nsg.layer_norm(x[a:a + 9])
        assert torch.equal(part, y[a:a + 9]) and torch.equal(s, stats[:, a:a + 9])
        assert torch.equal(nsg.layer_norm_backward(x[a:a + 9], x[a:a + 9], s)[0], dx[a:a + 9])
    assert dw.isfinite().all() and (db.double() - x.sum(0, dtype=torch.float64)).abs().max() <= R * U * x.abs().double().sum(0).max()


@pytest.mark.parametrize("E", [256, 1024])
def test_router_offsets_past_32_bits(E):
    T, k = (1 << 31) // E + 4000, 2
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    for a in range(0, T, 1 << 20):
        l[a:a + (1 << 20)] = rand((min(1 << 20, T - a), E), a, torch.bfloat16)
    r = nsg.expert_route(l, k, balance=True)
    assert r.counts[E] == T and r.counts[:E].sum() == T * k
    g = nsg.expert_route_backward(l, r.ids, r.weights)
    for a in (0, T - 4100, T - 9):
        part = nsg.expert_route(l[a:a + 9], k)
        assert torch.equal(part.ids, r.ids[a:a + 9]) and torch.equal(part.weights, r.weights[a:a + 9])
        want = nsg.expert_route_backward(l[a:a + 9], part.ids, part.weights).float()
        assert (g[a:a + 9].float() - want).abs().max() <= 2 ** -8 * want.abs().max()


def test_long_pitches():
    """Rows far apart: offsets of the pitch times the row past 32 bits."""
    R, C, ld = 5, 70, (1 << 29) + 64
    room = torch.zeros((R - 1) * ld + C, dtype=torch.bfloat16, device="cuda")
    v = room.as_strided((R, C), (ld, 1))
    x = rand((R, C), 1, torch.bfloat16)
    v.copy_(x)
    same(nsg.layer_norm(v), nsg.layer_norm(x))
    _, stats = nsg.layer_norm(x)
    same(nsg.layer_norm_backward(v, v, stats), nsg.layer_norm_backward(x, x, stats))
    same(nsg.expert_route(v, 3, balance=True), nsg.expert_route(x, 3, balance=True))
    ids = torch.tensor([4, 0, 3], device="cuda")
    assert torch.equal(nsg.embedding(ids, v), nsg.embedding(ids, x))
    ids = torch.tensor([1, 0, 1, 2, 2], device="cuda")
    assert torch.equal(nsg.embedding_backward(v, ids, 4), nsg.embedding_backward(x, ids, 4))


def test_a_vocabulary_and_a_choice_at_their_limits():
    ids = torch.tensor([(1 << 20) - 1, 1 << 20, 0], device="cuda")
    d = rand((3, 2), 1)
    dW = nsg.embedding_backward(d, ids, 1 << 20)
    assert torch.equal(dW[-1], d[0]) and torch.equal(dW[0], d[2]) and int(dW.count_nonzero()) == 4
    l = rand((70, 1024), 2)
    r = nsg.expert_route(l, 64, balance=True)
    assert np.array_equal(r.ids.cpu().numpy(), ref.choose(l.double().cpu().numpy(), 64, "softmax"))
    b = rand((1024,), 3, scale=1e-7)  # keys that only 64 bits tell apart
    flat = torch.zeros(70, 1024, device="cuda")
    for k in (1, 5, 63, 64):
        r = nsg.expert_route(flat, k, score="sigmoid", bias=b)
        assert np.array_equal(r.ids.cpu().numpy(), ref.choose(flat.double().cpu().numpy(), k, "sigmoid", b.double().cpu().numpy())), k


@pytest.mark.parametrize("E", [12, 60, 128, 200, 512, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biased_scores_that_nearly_meet(E, score):
    """Pairs, runs and whole rows of keys a few roundings of fp32 apart: the order is that of 64 bits."""
    g = np.random.default_rng(E)
    T, k = 64, min(E, 8)
    l = g.standard_normal((T, E)).astype(np.float32)
    s = ref.scores(l.astype(np.float64), score)
    # the bias brings each score of row 0 next to a level that neighbours share
    level = np.repeat(g.standard_normal(E // 4 + 1), 4)[:E] * 1e-3
    b = (level + 0.5 - s[0] + 1e-8 * g.standard_normal(E)).astype(np.float32)
    l[1:40] = l[0] + 1e-6 * g.standard_normal((39, E)).astype(np.float32)
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(b).cuda()
    for kk in (1, k):
        r = nsg.expert_route(lt, kk, score=score, bias=bt)
        assert np.array_equal(r.ids.cpu().numpy(), ref.choose(l.astype(np.float64), kk, score, b.astype(np.float64)))


@pytest.mark.parametrize("E", [2, 12, 16, 60, 128, 200, 256, 512, 1000])
@pytest.mark.parametrize("kind,bias", [("last bits", False), ("few values", False), ("few values", True), ("all equal", False),
                                       ("all equal", True), ("zeros of both signs", False), ("zeros of both signs", True),
                                       ("ends of the range", False)])
def test_logits_that_differ_by_little(E, kind, bias):
    """The k largest in their exact order, equal ones by index: fp32 logits in their last bits,
    and 16-bit ones of few values; with a bias of zeros the order of softmax's scores is theirs."""
    T, k = 700, min(E, 11)
    g = torch.Generator().manual_seed(E)
    at = torch.randint(0, {"last bits": 1 << 9, "few values": 7}.get(kind, 2), (T, E), generator=g)
    sign = torch.randint(0, 2, (T, 1), generator=g) * 2.0 - 1
    if kind == "last bits":
        l = sign * (1.5 + at * 2.0 ** -23)
    elif kind == "few values":
        l = (sign * at * 0.5).bfloat16()
    elif kind == "all equal":
        l = torch.full((T, E), -3.25).to(torch.float16)
    elif kind == "zeros of both signs":
        l = torch.where(at > 0, 0.0, -0.0)
    else:
        l = torch.tensor([3.4e38, 1e-45, 0.0, -1e-45, -3.4e38, 3.4028234e38, -3.4028234e38])[torch.randint(0, 7, (T, E), generator=g)]
    l = l.cuda()
    r = nsg.expert_route(l, k, normalize=True, bias=torch.zeros(E, device="cuda") if bias else None)
    x = l.double().cpu().numpy() + 0.0
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    assert np.array_equal(r.ids.cpu().numpy(), order)
    if kind != "ends of the range":
        v = np.exp(np.take_along_axis(x, order, 1) - x.max(1, keepdims=True))
        # exponentials within 3 of 2^-24 and of their arguments (at most 3), their sum, the quotient
        assert np.allclose(r.weights.cpu().numpy(), v / v.sum(1, keepdims=True), rtol=(2 * (3 + 3) + k + 4) * U, atol=0)


@pytest.mark.parametrize("E", [8, 60, 256, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T", [50, 3000])
def test_gradients_of_weights_that_are_none(E, score, normalize, T):
    """A token with fewer experts than k: what stands where its ids are -1 is not read, be it NaN."""
    k = 5
    l, dw = rand((T, E), 50), rand((T, k), 51)
    few = integers(k + 2, (T, 1), 52)
    l = torch.where(l.argsort(1, descending=True).argsort(1) < few, l, -float("inf"))
    r = nsg.expert_route(l, k, score=score, normalize=normalize, balance=True)
    none = r.ids < 0
    assert none.any() and not none.all()
    grads = [nsg.expert_route_backward(l, r.ids, torch.where(none, v, dw), score=score, normalize=normalize, counts=r.counts)
             for v in (0.0, float("nan"), float("inf"))]
    assert grads[0].isfinite().all()
    same(grads[1:], [grads[0]] * 2)


@pytest.mark.parametrize("E", [16, 64, 65, 128, 200, 256, 257, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("near", [False, True])
def test_as_many_choices_as_can_be(E, score, near):
    """k = 64 or all experts, with a bias and the balance loss: the largest launches in shared memory."""
    T, k = 600, min(E, 64)
    l, b = rand((T, E), 60), rand((E,), 61, scale=1e-7 if near else 0.1)
    if near:  # a quarter of the tokens: keys that only 64 bits tell apart
        l[::4] = 0.25
    r = nsg.expert_route(l, k, score=score, bias=b, balance=True)
    x = l.double().cpu().numpy()
    ids = r.ids.cpu().numpy()
    assert np.array_equal(ids, ref.choose(x, k, score, b.double().cpu().numpy()))
    counts = r.counts.cpu().numpy()
    assert np.array_equal(counts[:-1], np.bincount(ids.ravel(), minlength=E)) and counts[-1] == T
    if k == E:
        assert (counts[:-1] == T).all()


@pytest.mark.parametrize("E", [3, 16, 60, 128, 256, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T", [77, 3001])
def test_what_padded_tokens_hold(E, score, bias, T):
    """Whatever stands in a token that does not count, all results are those of zeros there."""
    k = min(E, 4)
    l, dw, mask = rand((T, E), 70, torch.bfloat16), rand((T, k), 71), integers(5, (T,), 72) > 0
    b = rand((E,), 73, scale=0.1) if bias else None
    want = None
    for v in (0.0, float("nan"), float("inf"), -float("inf"), 3e38):
        x = torch.where(mask[:, None], l, v)
        g = torch.where(mask[:, None], dw, v)
        r = nsg.expert_route(x, k, score=score, bias=b, mask=mask, balance=True)
        got = (*r, nsg.expert_route_backward(x, r.ids, g, score=score, counts=r.counts))
        assert r.ids[~mask].eq(-1).all() and got[-1][~mask].eq(0).all() and r.loss.isfinite() and got[-1].isfinite().all()
        want = want or got
        same(got, want)
        ids = torch.where(mask, integers(50, (T,), 74), -1)
        dW = nsg.embedding_backward(torch.where(mask[:, None], l, v), ids, 50)
        assert dW.isfinite().all()


@pytest.mark.parametrize("E", [8, 60, 128, 256, 512, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [50, 2500])
def test_logits_that_are_not_finite_in_tokens_that_count(E, score, bias, dtype, T):
    """What a NaN or an infinity does to its own token, in the choice, the weights, the loss and the
    gradient; and that it does nothing to the other tokens."""
    k, inf, nan = 4, float("inf"), float("nan")
    clean = rand((T, E), 80, dtype)
    l = clean.clone()
    l[3, E // 2] = nan
    l[5, E - 1] = inf
    l[7] = nan
    l[9, 0], l[9, E - 2] = nan, inf
    l[11, 1:] = nan  # one expert left
    l[13] = -inf
    l[13, 2], l[13, 5] = 1.0, nan  # one expert left, of those that are finite
    l[T - 1, 1] = l[T - 1, E - 3] = inf
    l[T - 2, ::2] = nan
    special = torch.tensor([3, 5, 7, 9, 11, 13, T - 1, T - 2], device="cuda")
    infs = torch.tensor([5, 9, T - 1], device="cuda")  # rows with +inf
    ours = torch.ones(T, dtype=torch.bool, device="cuda")
    ours[special] = False
    b = rand((E,), 81, scale=0.1) if bias else None
    x = l.double().cpu().numpy()
    ids = ref.choose(x, k, score, None if b is None else b.double().cpu().numpy())
    chosen = torch.from_numpy(ids >= 0).cuda()
    dw = rand((T, k), 82)
    for normalize in (True, False):
        kw = dict(score=score, normalize=normalize)
        r, plain = nsg.expert_route(l, k, bias=b, balance=True, **kw), nsg.expert_route(clean, k, bias=b, **kw)
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        assert torch.equal(r.ids, nsg.expert_route(l, k, bias=b, **kw).ids)
        assert torch.equal(r.weights[ours], plain.weights[ours])
        w = r.weights[special]
        assert w[~chosen[special]].eq(0).all()
        if score == "softmax":
            assert w[chosen[special]].isnan().all()
        else:
            want = torch.from_numpy(ref.weights(np.where(np.isnan(x), -inf, x), ids, score, normalize, 1.0)).cuda()[special]
            a = 2 * clean.double().abs().max().item()  # of logits, as of the differences that are taken of them
            assert ((w.double() - want).abs() <= (2 * a + k + 40) * U * want).all()
        # the loss: tokens with a choice whose scores' sum is a NaN (softmax of an infinity too)
        some = chosen.any(1)
        assert r.counts[E] == int(some.sum())
        bad = torch.isnan(l).any(1)
        if score == "softmax":
            bad[infs] = True
        assert bool(r.probs.isnan().all()) == bool(r.loss.isnan()) == bool((bad & some).any())
        assert bool((bad & some).any()) != (score == "softmax" and bias)  # there a NaN leaves a token no choice

        for counts in (None, r.counts):
            got = nsg.expert_route_backward(l, r.ids, dw, counts=counts, balance=3.0, **kw)
            want = nsg.expert_route_backward(clean, r.ids, dw, counts=counts, balance=3.0, **kw)
            assert torch.equal(got[ours], want[ours]) and got[ours].isfinite().all()
            assert got[~some].eq(0).all()
            rows = got[special]
            hit = (bad & some)[special]
            if counts is not None:  # p is a NaN in all of the token
                assert rows[hit].isnan().all() and rows[~hit].isfinite().all()
            elif score == "sigmoid":  # the chosen's scores are finite
                assert rows.isfinite().all()
            elif normalize:  # the chosen's weights are NaN
                at = torch.where(chosen, r.ids, 0).long()
                assert torch.gather(got, 1, at)[chosen & (bad & some)[:, None]].isnan().all()
            else:  # softmax: each logit is in each score
                assert rows[hit].isnan().all()


@pytest.mark.parametrize("E", [8, 60, 128, 256, 512, 1000])
@pytest.mark.parametrize("T", [50, 3000])
@pytest.mark.parametrize("level", [-15.0, -40.0, -58.0, -200.0])
@pytest.mark.parametrize("size", [1.0, 1e-19, 1e-30])
def test_small_gradients_of_small_sigmoid_scores(E, T, level, size):
    """Normalised weights and the balance loss of a token whose scores are all small: the shares that
    they are made of are not, so the gradient is as exact as any other's, however small it is.

    The tolerance of the router's gradient: (4 a + 2 k + 80) u of the sum of its terms' sizes, a the
    largest |l| that an exponential is taken of; then fp32's own rounding, and of numbers below
    2^-126 its step."""
    k = min(E, 6)
    l, dw = level + 0.5 * rand((T, E), 90), size * rand((T, k), 91)
    r = nsg.expert_route(l, k, score="sigmoid", balance=True)
    x, ids, counts = l.double().cpu().numpy(), r.ids.cpu().numpy(), r.counts.cpu().numpy()
    d = dw.double().cpu().numpy()
    a = np.abs(x).max()
    for dweights, c, coef in ((dw, None, 0.0), (None, r.counts, size), (dw, r.counts, size)):
        got = nsg.expert_route_backward(l, r.ids, dweights, score="sigmoid", counts=c, balance=coef).double().cpu().numpy()
        want, terms = ref.route_backward(x, ids, None if dweights is None else d, "sigmoid", True, 1.0,
                                         None if c is None else counts, float(np.float32(coef)))
        tol = (4 * a + 2 * k + 80) * U * terms
        bad = ~(np.abs(got - want) <= tol + U * np.abs(want) + 2.0 ** -126)
        assert not bad.any(), (int(bad.sum()), got[bad][:3], want[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("E", [12, 16, 60, 128, 200, 256, 512, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_biases_of_any_size(E, score, dtype):
    """Infinities, NaN, numbers beside which scores are nothing, and numbers that are nothing beside them."""
    l = rand((300, E), 95, dtype)
    b = rand((E,), 96, scale=0.1)
    for i, v in enumerate((float("inf"), -float("inf"), 1e30, float("nan"), -1e30, 1e-40)):
        b[i::11] = v
    x, bd = l.double().cpu().numpy(), b.double().cpu().numpy()
    a = 2 * np.abs(x).max()
    for k in sorted({1, 3, min(E, 8), min(E, 31), min(E, 64)}):
        for normalize in (True, False):
            r = nsg.expert_route(l, k, score=score, bias=b, normalize=normalize)
            ids = ref.choose(x, k, score, bd)
            assert np.array_equal(r.ids.cpu().numpy(), ids), k
            want = ref.weights(x, ids, score, normalize, 1.0)
            assert (np.abs(r.weights.double().cpu().numpy() - want) <= (2 * a + k + 40) * U * want).all(), k


@pytest.mark.parametrize("E", [8, 60, 128, 256, 512, 1000])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("level", [-15.0, -40.0, -58.0, -200.0])
@pytest.mark.parametrize("scale", [1e30, -1e15, 1.0, 1e-30])
def test_weights_of_any_scale_of_small_sigmoid_scores(E, bias, level, scale):
    """Normalised weights are shares of the scale, whatever the scores are."""
    T, k = 200, min(E, 6)
    l = level + 0.5 * rand((T, E), 97)
    b = rand((E,), 98, scale=0.1) if bias else None
    x = l.double().cpu().numpy()
    r = nsg.expert_route(l, k, score="sigmoid", bias=b, scale=scale)
    ids = ref.choose(x, k, "sigmoid", None if b is None else b.double().cpu().numpy())
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    want = ref.weights(x, ids, "sigmoid", True, float(np.float32(scale)))
    # a: the largest |l| that an exponential is taken of
    assert (np.abs(r.weights.double().cpu().numpy() - want) <= (2 * np.abs(x).max() + k + 40) * U * np.abs(want)).all()


def test_embedding_of_more_rows_than_a_workgroup_each_can_take():
    """More than 2^23 rows of several parts: four rows to a workgroup, parts in the grid's second direction."""
    T, V, C = (1 << 23) + 77, 100, 1030
    W = rand((V, C), 1, torch.bfloat16)
    ids = integers(V, (T,), 2, lo=-1, dtype=torch.int32)
    out = nsg.embedding(ids, W)
    for a in range(0, T, 1 << 20):
        i = ids[a:a + (1 << 20)].long()
        assert torch.equal(out[a:a + (1 << 20)], torch.where((i >= 0)[:, None], W[i.clamp(min=0)], 0)), a
