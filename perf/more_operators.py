"""The operators between token ids and the expert layer, as they are measured.

What a training step runs before expert_sort, and its gradients after it: the
embedding of token ids, layer norm, and the router with its balance loss.

With `own` false, run() computes them from elementary torch operations in
32 bits (scores that are compared with a bias on them in 64); with `own` true
it calls the library.

  embed       out[t] = scale W[ids[t]]; zeros for an id outside 0 .. V - 1
  embed grad  dW[v] = scale sum of dout[t] over the tokens with ids[t] = v
  norm        y = (x - mean) rstd gamma + beta, rstd = 1 / sqrt(var + eps);
              stats [2, R] = mean, rstd
  norm grad   dx, dgamma, dbeta
  route       s = softmax(l) or sigmoid(l).  A token's k choices are its largest
              logits, with a bias its largest s + bias; equal ones go to the lower
              index; -inf and masked tokens give none (id -1, weight 0).  weights
              = scale s, divided by their sum where normalised.  With the balance
              loss also counts [E + 1] (choices of each expert, tokens with a
              choice, N), probs [E] (the mean over those tokens of s / sum s) and
              loss = E / (k N) sum_e counts[e] probs[e]
  route grad  dl for the weights' gradient and balance x dloss of the loss, whose
              counts are constants
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-5
BALANCE = 0.01


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # eight sequences decoding: one id each
        dict(name="embed 8", kind="embed", T=8, V=128000, C=4096, ids=64, scale=64.0, dtype="bf16"),
        # a training batch of 16384 tokens, its last sequences padded
        dict(name="embed 16384", kind="embed", T=16384, V=128000, C=4096, ids=64, scale=1.0, dtype="bf16", pad=0.03),
        # a short batch of uneven length over a small vocabulary, gradients in fp32
        dict(name="embed grad 4099", kind="embed_grad", T=4099, V=32003, C=768, ids=32, scale=27.7, dtype="f32", pad=0.1),
        # a training batch over a large vocabulary: text, so that a few tokens are a tenth of it
        dict(name="embed grad 65536", kind="embed_grad", T=65536, V=128000, C=4096, ids=64, scale=1.0, dtype="bf16"),
        # four sequences decoding
        dict(name="norm 4", kind="norm", R=4, C=4096, dtype="bf16", w="bf16", bias=True),
        # a training batch in front of the expert layer
        dict(name="norm 16384", kind="norm", R=16384, C=4096, dtype="bf16", w="f32", bias=True),
        # uneven sides in fp32: a short batch of a small model
        dict(name="norm grad 1003 x 1250", kind="norm_grad", R=1003, C=1250, dtype="f32", w="f32", bias=True),
        # the training batch's way back
        dict(name="norm grad 16384", kind="norm_grad", R=16384, C=4096, dtype="bf16", w="f32", bias=True),
        # 32 sequences decoding through the router of 512 fine-grained experts
        dict(name="route 32", kind="route", T=32, E=512, k=8, score="softmax", dtype="f32", normalize=True, scale=1.0,
             bias=False, balance=False),
        # a training batch, padded: sigmoid scores, a bias that balances the choice, the balance loss
        dict(name="route 16384 biased", kind="route", T=16384, E=256, k=8, score="sigmoid", dtype="bf16", normalize=True,
             scale=2.5, bias=True, balance=True, pad=0.03),
        # a training batch's way back through 512 experts: gradients of the weights and of the balance loss
        dict(name="route grad 16384", kind="route_grad", T=16384, E=512, k=8, score="softmax", dtype="bf16",
             normalize=True, scale=1.0, bias=False, balance=True),
        # few experts, probabilities as weights, no balance loss
        dict(name="route grad 4099", kind="route_grad", T=4099, E=60, k=4, score="softmax", dtype="f32",
             normalize=False, scale=1.0, bias=False, balance=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: mostly a multiple of 64, sometimes any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(lo, n // 64 * 64)


def draw(rng):
    kind = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "route", "route", "route_grad", "route_grad"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("embed", "embed_grad"):
        C = _width(rng, 64, 8192)
        most = 2 if dt == "f32" else 1
        return dict(kind=kind, T=_log(rng, 1, min(65536, 260_000_000 // (most * C))),
                    V=_log(rng, 1000, min(260_000, 500_000_000 // (most * C))), C=C, ids=rng.choice([32, 64]),
                    scale=rng.choice([1.0, math.sqrt(C)]), dtype=dt, pad=rng.choice([0.0, 0.0, 0.1]))
    if kind in ("norm", "norm_grad"):
        C = _width(rng, 64, 16384)
        return dict(kind=kind, R=_log(rng, 1, min(32768, 60_000_000 // (C * (2 if dt == "f32" else 1)))), C=C, dtype=dt,
                    w=rng.choice(["f32", dt]), bias=rng.choice([True, True, False]))
    E = rng.choice([4, 8, 60, 64, 128, 160, 256, 384, 512])
    bias = rng.choice([True, False]) if kind == "route" else False
    return dict(kind=kind, T=_log(rng, 1, 7_000_000 // E), E=E, k=rng.choice([k for k in (1, 2, 4, 6, 8) if k <= E]),
                score=rng.choice(["softmax", "softmax", "sigmoid"]), dtype=dt, normalize=rng.choice([True, True, False]),
                scale=rng.choice([1.0, 2.5]), bias=bias, balance=rng.choice([True, True, False]),
                pad=rng.choice([0.0, 0.0, 0.1]))


def _size(dt):
    return torch.empty((), dtype=DT[dt]).element_size()


def _frequencies(V):
    """How often each token of a vocabulary is met in text: about one over its rank."""
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
    return p / p.sum()


def work(case):
    c = case
    kind = c["kind"]
    s = _size(c["dtype"])
    if kind == "embed":  # each row that is met once
        met = float((1 - (1 - _frequencies(c["V"])) ** c["T"]).sum())
        return {"bytes": (met + c["T"]) * c["C"] * s + c["T"] * c["ids"] // 8, "flops": c["T"] * c["C"]}
    if kind == "embed_grad":
        return {"bytes": (c["T"] + c["V"]) * c["C"] * s + c["T"] * c["ids"] // 8, "flops": 2 * c["T"] * c["C"]}
    if kind == "norm":
        w = c["C"] * _size(c["w"]) * (2 if c["bias"] else 1)
        return {"bytes": 2 * c["R"] * c["C"] * s + w + 8 * c["R"], "flops": 8 * c["R"] * c["C"]}
    if kind == "norm_grad":
        w = c["C"] * _size(c["w"]) * (3 if c["bias"] else 2)
        return {"bytes": 3 * c["R"] * c["C"] * s + w + 8 * c["R"], "flops": 14 * c["R"] * c["C"]}
    n = c["T"] * c["E"]
    if kind == "route":
        return {"bytes": n * s + 8 * c["T"] * c["k"] + (8 * c["E"] if c["balance"] else 0), "flops": 10 * n}
    return {"bytes": 2 * n * s + 8 * c["T"] * c["k"] + (4 * c["E"] if c["balance"] else 0), "flops": 12 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, shape, dt):
    """Normal values with a spread of channel sizes and of row means."""
    x = torch.randn(shape, generator=g, device=DEV)
    c = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEV))
    return (x * c + 0.3 * torch.randn((shape[0], 1), generator=g, device=DEV)).to(DT[dt])


def _padded(g, n, pad):
    """Which of n tokens count: the ends of sequences of 512 at most, a share `pad` of all, do not."""
    at = torch.arange(n, device=DEV)
    length = min(512, n)
    ends = length * (1 - 2 * pad * torch.rand(-(-n // length), generator=g, device=DEV))
    return at % length < ends[at // length]


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind = c["kind"]
    pad = c.get("pad", 0.0)
    if kind in ("embed", "embed_grad"):
        T, V, C = c["T"], c["V"], c["C"]
        cut = _frequencies(V).cumsum(0).to(DEV)
        ids = torch.searchsorted(cut, torch.rand(T, generator=g, device=DEV, dtype=torch.float64)).clamp_(max=V - 1)
        if pad:
            ids = torch.where(_padded(g, T, pad), ids, -1)
        ids = ids.to(torch.int32 if c["ids"] == 32 else torch.int64)
        if kind == "embed":
            return dict(case=c, ids=ids, W=(0.02 * torch.randn((V, C), generator=g, device=DEV)).to(DT[c["dtype"]]))
        return dict(case=c, ids=ids, dout=(0.1 * torch.randn((T, C), generator=g, device=DEV)).to(DT[c["dtype"]]))
    if kind in ("norm", "norm_grad"):
        R, C = c["R"], c["C"]
        s = dict(case=c, x=_activations(g, (R, C), c["dtype"]),
                 gamma=(1 + 0.1 * torch.randn(C, generator=g, device=DEV)).to(DT[c["w"]]),
                 beta=(0.1 * torch.randn(C, generator=g, device=DEV)).to(DT[c["w"]]) if c["bias"] else None)
        if kind == "norm_grad":
            s["stats"] = _norm(s["x"], s["gamma"], s["beta"])[1]
            s["dy"] = (0.1 * torch.randn((R, C), generator=g, device=DEV)).to(DT[c["dtype"]])
        return s
    T, E, k = c["T"], c["E"], c["k"]
    popular = 0.5 * torch.randn(E, generator=g, device=DEV)
    s = dict(case=c, logits=(1.2 * torch.randn((T, E), generator=g, device=DEV) + popular).to(DT[c["dtype"]]),
             bias=-0.1 * popular if c["bias"] else None, mask=_padded(g, T, pad) if pad else None)
    if kind == "route_grad":
        routing = _route(s)
        s["ids"], s["counts"] = routing[0], routing[2] if c["balance"] else None
        s["dw"] = 0.1 * torch.randn((T, k), generator=g, device=DEV)
        # what a scaled loss passes down; fp16 gradients need a large one
        s["dloss"] = torch.full((), 65536.0 if c["dtype"] == "f16" else 1.0, device=DEV) if c["balance"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _embed(W, ids, scale):
    there = (ids >= 0) & (ids < W.shape[0])
    rows = W[torch.where(there, ids, 0).long()].float() * scale
    return torch.where(there[:, None], rows, 0.0).to(W.dtype)


def _embed_grad(dout, ids, V, scale):
    there = (ids >= 0) & (ids < V)
    at = torch.where(there, ids, V).long()  # row V takes what belongs nowhere
    dW = torch.zeros((V + 1, dout.shape[1]), device=dout.device).index_add_(0, at, dout.float())
    return (dW[:V] * scale).to(dout.dtype)


def _norm(x, gamma, beta):
    f = x.float()
    mean = f.mean(1, keepdim=True)
    d = f - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return y.to(x.dtype), torch.cat([mean, rstd], dim=1).t().contiguous()


def _norm_grad(dy, x, stats, gamma, bias):
    mean, rstd = stats[0][:, None], stats[1][:, None]
    d, xh = dy.float(), (x.float() - mean) * rstd
    g = d * gamma.float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dbeta = d.sum(0).to(gamma.dtype) if bias else None
    return dx.to(x.dtype), (d * xh).sum(0).to(gamma.dtype), dbeta


def _scores(l, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _choose(key, k):
    """The k largest of each row, one after the other: the first of equal ones; -1 where none is left."""
    ids = []
    for j in range(k):
        at = key.argmax(1, keepdim=True)
        ids.append(torch.where(torch.gather(key, 1, at) > -math.inf, at, -1))
        if j + 1 < k:
            key = key.scatter(1, at, -math.inf)
    return torch.cat(ids, dim=1)


def _route(state):
    c, l, bias, mask = state["case"], state["logits"], state["bias"], state["mask"]
    T, E = l.shape
    k = c["k"]
    f = l.float()
    s = _scores(f, c["score"])
    # a bias leads to scores next to each other: compared in 64 bits
    key = f if bias is None else _scores(l.double(), c["score"]) + bias.double()
    if mask is not None:
        key = torch.where(mask[:, None], key, -math.inf)
    ids = _choose(key, k)
    there = ids >= 0
    w = torch.where(there, torch.gather(s, 1, ids.clamp(min=0)), 0.0)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = w * c["scale"]
    if not c["balance"]:
        return ids.to(torch.int32), w
    some = there.any(1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
    counts.scatter_add_(0, torch.where(there, ids, E).reshape(-1), there.reshape(-1).long())
    N = some.sum()
    counts[E] = N
    p = torch.where(some[:, None], s / s.sum(1, keepdim=True), 0.0)
    probs = p.sum(0) / N.clamp(min=1)
    loss = (counts[:E].float() * probs).sum() * (E / k) / N.clamp(min=1)
    return ids.to(torch.int32), w, counts.to(torch.int32), probs, loss


def _route_grad(state):
    c, l, ids, dw, counts = state["case"], state["logits"], state["ids"].long(), state["dw"], state["counts"]
    T, E = l.shape
    s = _scores(l.float(), c["score"])
    there = ids >= 0
    at = ids.clamp(min=0)
    sj = torch.where(there, torch.gather(s, 1, at), 0.0)
    g = torch.where(there, dw * c["scale"], 0.0)
    if c["normalize"]:
        total = sj.sum(1, keepdim=True)
        wj = sj / torch.where(total > 0, total, 1.0)
        d = wj * (g - (g * wj).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - sj)
        dl = torch.zeros((T, E), device=l.device).scatter_add_(1, at, d)
    elif c["score"] == "sigmoid":
        dl = torch.zeros((T, E), device=l.device).scatter_add_(1, at, g * sj * (1 - sj))
    else:
        full = torch.zeros((T, E), device=l.device).scatter_add_(1, at, g)
        dl = s * (full - (g * sj).sum(1, keepdim=True))
    if counts is not None:
        N = counts[E].clamp(min=1).double()
        coef = (state["dloss"].double() * BALANCE * E / c["k"] / N / N * counts[:E]).float()
        p = s / s.sum(1, keepdim=True)
        b = p * (coef - (p * coef).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            b = b * (1 - s)
        dl = dl + torch.where(there.any(1, keepdim=True), b, 0.0)
    return dl.to(l.dtype)


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    kind = c["kind"]
    if kind == "embed":
        return _embed(state["W"], state["ids"], c["scale"])
    if kind == "embed_grad":
        return _embed_grad(state["dout"], state["ids"], c["V"], c["scale"])
    if kind == "norm":
        return _norm(state["x"], state["gamma"], state["beta"])
    if kind == "norm_grad":
        return _norm_grad(state["dy"], state["x"], state["stats"], state["gamma"], c["bias"])
    return _route(state) if kind == "route" else _route_grad(state)


def _run_own(state):
    import newton_schulz_gram_amd as nsg

    c = state["case"]
    kind = c["kind"]
    if kind == "embed":
        return nsg.embedding(state["ids"], state["W"], scale=c["scale"])
    if kind == "embed_grad":
        return nsg.embedding_backward(state["dout"], state["ids"], c["V"], scale=c["scale"])
    if kind == "norm":
        return nsg.layer_norm(state["x"], state["gamma"], state["beta"], eps=EPS)
    if kind == "norm_grad":
        return nsg.layer_norm_backward(state["dy"], state["x"], state["stats"], state["gamma"], bias_grad=c["bias"])
    if kind == "route":
        out = nsg.expert_route(state["logits"], c["k"], score=c["score"], bias=state["bias"], mask=state["mask"],
                               normalize=c["normalize"], scale=c["scale"], balance=c["balance"])
        return tuple(out) if c["balance"] else (out.ids, out.weights)
    return nsg.expert_route_backward(state["logits"], state["ids"], state["dw"], score=c["score"],
                                     normalize=c["normalize"], scale=c["scale"], counts=state["counts"],
                                     balance=BALANCE, dloss=state["dloss"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_routing(l, ids, c):
    """Weights [T, k] and the tokens' shares p [T, E] of chosen experts ids (-1: none), differentiable."""
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
    chosen = torch.zeros_like(s)
    for j in range(ids.shape[1]):
        chosen = chosen + torch.nn.functional.one_hot(ids[:, j].clamp(min=0), s.shape[1]) * (ids[:, j, None] >= 0)
    w = s / (s * chosen).sum(1, keepdim=True).clamp(min=1e-300) if c["normalize"] else s
    w = c["scale"] * w.gather(1, ids.clamp(min=0)) * (ids >= 0)
    return w, s / s.sum(1, keepdim=True)


def _exact_loss(p, counts, c):
    n = max(int(counts[-1]), 1)
    return c["E"] / (c["k"] * n) * (counts[:-1].double() * p.sum(0) / n).sum()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "embed":
        out = torch.zeros((c["T"], c["C"]), dtype=torch.float64, device=DEV)
        there = torch.nonzero((s["ids"] >= 0) & (s["ids"] < c["V"]))[:, 0]
        out[there] = s["W"][s["ids"][there].long()].double() * c["scale"]
        return out
    if kind == "embed_grad":
        dW = torch.zeros((c["V"], c["C"]), dtype=torch.float64, device=DEV)
        there = torch.nonzero((s["ids"] >= 0) & (s["ids"] < c["V"]))[:, 0]
        dW.index_put_((s["ids"][there].long(),), s["dout"][there].double(), accumulate=True)
        return dW.mul_(c["scale"])
    if kind in ("norm", "norm_grad"):
        x = s["x"].double().requires_grad_()
        gamma = s["gamma"].double().requires_grad_()
        beta = torch.zeros(c["C"], dtype=torch.float64, device=DEV) if s["beta"] is None else s["beta"].double()
        beta.requires_grad_()
        y = torch.nn.functional.layer_norm(x, (c["C"],), gamma, beta, EPS)
        if kind == "norm":
            var, mean = torch.var_mean(x.detach(), dim=1, correction=0)
            return y.detach(), torch.stack([mean, torch.rsqrt(var + EPS)])
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        return dx, dgamma, dbeta if c["bias"] else None
    l = s["logits"].double()
    if kind == "route":
        key = l if s["bias"] is None else \
            (torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)) + s["bias"].double()
        order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
        ids = order if s["mask"] is None else torch.where(s["mask"][:, None], order, -1)
        w, p = _exact_routing(l, ids, c)
        if not c["balance"]:
            return ids.to(torch.int32), w
        counts = torch.bincount(ids[ids >= 0], minlength=c["E"])
        counts = torch.cat([counts, (ids[:, :1] >= 0).sum().reshape(1)])
        p = p * (ids[:, :1] >= 0)
        return ids.to(torch.int32), w, counts.to(torch.int32), p.sum(0) / max(int(counts[-1]), 1), _exact_loss(p, counts, c)
    l.requires_grad_()
    ids = s["ids"].long()
    w, p = _exact_routing(l, ids, c)
    total = (w * s["dw"].double()).sum()
    if s["counts"] is not None:
        total = total + s["dloss"].double() * BALANCE * _exact_loss(p * (ids >= 0).any(1, keepdim=True), s["counts"], c)
    return torch.autograd.grad(total, l)[0]
