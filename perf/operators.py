"""The expert layer's operators around a Muon step, as they are measured.

A layer of experts (or one plain linear layer) whose weight bucket [E, N, K] the
Muon step updates: tokens sorted by expert and brought back with their router
weights, operands quantised to 8 bit floating point with one scale for each
block of 128, the products of such operands (plain, batched, by expert), and
the product that gives the bucket [E, N, K] of weight gradients which
muon_step takes.

With `own` false, run() computes them from elementary torch operations in
32 bits; with `own` true it calls the library.

Layouts that both share (K is the contraction, Kp = K rounded up to 128):
  operand   q [B, R, Kp] float8 (zeros behind K), scale fp32 [B, Kp/128, R] (one
            for 128 elements of a row) or [B, Kp/128, ceil(R/128)] (one for a
            128 x 128 tile)
  plan      offsets [E + 1]: sorted rows offsets[e] .. offsets[e + 1] are expert
            e's; rows [T, k]: the sorted row of each (token, choice), -1 if it was
            dropped; tokens [T k]: the token in each sorted row, -1 behind the last
  columns   qt [C, cap] float8: the rows of expert e become columns, each expert's
            starting at a multiple of 128, zeros behind its last; cap =
            128 (P // 128 + E) for P rows; scale fp32 [cap/128, C]
"""
import math

import torch

own = False

BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TINY = 2.0 ** -126  # the smallest scale: an fp32 number whose inverse is one too
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one prompt batch of an uneven length through the router of 512 fine-grained
        # experts (the 512 x 2048 x 512 bucket), some choices dropped at capacity
        dict(name="gather 4099 x 8", kind="gather", T=4099, k=8, E=512, C=2048, dtype="bf16", drop=0.01),
        # one token while serving: its eight experts' answers summed
        dict(name="return 1 x 8", kind="return", T=1, k=8, E=512, C=2048, dtype="bf16", drop=0.0),
        # a training batch's way back: gradients of the answers, the router weights and the tokens
        dict(name="gradient 16384 x 8", kind="gradient", T=16384, k=8, E=512, C=2048, dtype="bf16", drop=0.0),
        # activations of one training batch in front of a linear layer
        dict(name="quantize rows 8192", kind="quantize", how="row", B=1, R=8192, C=4096, dtype="bf16", f8="e4m3"),
        # the expert bucket after a Muon step: forward and transposed operand in one pass
        dict(name="quantize bucket 512", kind="quantize", how="tile", B=512, R=2048, C=512, dtype="bf16", f8="e4m3"),
        # output gradients laid out for the weight gradients of 64 experts
        dict(name="quantize columns 32771", kind="columns", P=32771, E=64, C=2048, dtype="bf16", f8="e5m2"),
        # four sequences decoding through an MLP matrix of the 11008 x 4096 bucket
        dict(name="product 4 x 11008 x 4096", kind="product", B=1, M=4, N=11008, K=4096, out="bf16", a="e4m3", b="e4m3",
             b_scale="tile"),
        # the same matrix's input gradient for a training batch (e5m2 gradients)
        dict(name="product 8192 x 4096 x 11008", kind="product", B=1, M=8192, N=4096, K=11008, out="bf16", a="e5m2",
             b="e4m3", b_scale="tile"),
        # 32 sequences decoding: 256 rows over 512 experts, most of them empty or with one row
        dict(name="experts 32 x 8", kind="experts", T=32, k=8, E=512, N=512, K=2048, out="bf16", a="e4m3", b="e4m3"),
        # a training batch through the expert bucket
        dict(name="experts 16384 x 8", kind="experts", T=16384, k=8, E=512, N=512, K=2048, out="bf16", a="e4m3",
             b="e4m3"),
        # weight gradients of a few wide experts from a short batch, in fp32
        dict(name="weights 1003 over 8", kind="weights", P=1003, E=8, N=300, K=1000, out="f32", a="e5m2", b="e4m3"),
        # weight gradients of the expert bucket from a training batch
        dict(name="weights 131072 over 512", kind="weights", P=131072, E=512, N=2048, K=512, out="bf16", a="e5m2",
             b="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A side of a weight: mostly a multiple of 64, sometimes any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(lo, n // 64 * 64)


def draw(rng):
    kind = rng.choice(["gather", "return", "gradient", "quantize", "columns", "product", "product", "experts", "experts",
                       "weights"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    f8 = lambda: rng.choice(["e4m3", "e4m3", "e5m2"])  # noqa: E731
    if kind in ("gather", "return", "gradient"):
        return dict(kind=kind, T=_log(rng, 1, 12000), k=rng.choice([1, 2, 4, 6, 8]), E=rng.choice([8, 60, 64, 128, 256, 512]),
                    C=_width(rng, 128, 4096), dtype=dt, drop=rng.choice([0.0, 0.0, 0.02]))
    if kind == "quantize":
        how = rng.choice(["row", "tile"])
        B = _log(rng, 1, 64)
        return dict(kind=kind, how=how, B=B, R=_log(rng, 1, max(16, 16384 // B)), C=_width(rng, 64, 8192), dtype=dt, f8=f8())
    if kind == "columns":
        return dict(kind=kind, P=_log(rng, 1, 40000), E=rng.choice([1, 8, 60, 128]), C=_width(rng, 64, 4096), dtype=dt, f8=f8())
    if kind == "product":
        return dict(kind=kind, B=rng.choice([1, 1, 1, 2, 5]), M=_log(rng, 1, 4096), N=_width(rng, 64, 11008),
                    K=_width(rng, 64, 8192), out=rng.choice(["bf16", "f16", "f32"]), a=f8(), b=f8(),
                    b_scale=rng.choice(["row", "tile", "tile"]))
    N, K = _width(rng, 64, 2048), _width(rng, 64, 2048)
    if kind == "experts":
        return dict(kind=kind, T=_log(rng, 1, 8192), k=rng.choice([1, 2, 4, 8]), E=rng.choice([8, 60, 64, 128, 256]),
                    N=N, K=K, out=rng.choice(["bf16", "f16", "f32"]), a=f8(), b=f8())
    return dict(kind=kind, P=_log(rng, 1, 40000), E=rng.choice([1, 8, 60, 128]), N=N, K=K,
                out=rng.choice(["bf16", "f32"]), a=f8(), b=f8())


def _up(n):
    return -(-n // BLOCK) * BLOCK


def _size(dt):
    return torch.empty((), dtype=DT[dt]).element_size()


def work(case):
    c = case
    kind = c["kind"]
    if kind in ("gather", "return", "gradient"):
        P, s = c["T"] * c["k"], _size(c["dtype"])
        row, ids = c["C"] * s, 4 * P
        if kind == "gather":  # ids; plan written; tokens read once, rows written
            return {"bytes": 8 * P + 2 * ids + 4 * (c["E"] + 1) + (c["T"] + P) * row, "flops": 0}
        if kind == "return":
            return {"bytes": ids + 4 * P + (c["T"] + P) * row, "flops": 2 * P * c["C"]}
        # the answers' gradients and the weights': T + P rows read, P written; the tokens': P read, T written
        return {"bytes": 2 * ids + 2 * 4 * P + (2 * c["T"] + 3 * P) * row, "flops": 4 * P * c["C"]}
    if kind == "quantize":
        n, p = c["B"] * c["R"] * c["C"], c["B"] * c["R"] * _up(c["C"])
        if c["how"] == "row":
            return {"bytes": n * _size(c["dtype"]) + p + p // 32, "flops": 3 * n}
        return {"bytes": n * _size(c["dtype"]) + p + c["B"] * c["C"] * _up(c["R"]), "flops": 3 * n}
    if kind == "columns":
        n = c["P"] * c["C"]
        return {"bytes": n * _size(c["dtype"]) + n + n // 32, "flops": 3 * n}
    if kind == "product":
        Kp = _up(c["K"])
        sb = c["N"] if c["b_scale"] == "row" else -(-c["N"] // BLOCK)
        return {"bytes": c["B"] * ((c["M"] + c["N"]) * Kp + (c["M"] + sb) * (Kp // 32) + c["M"] * c["N"] * _size(c["out"])),
                "flops": 2 * c["B"] * c["M"] * c["N"] * c["K"]}
    if kind == "experts":
        P, Kp = c["T"] * c["k"], _up(c["K"])
        used = c["E"] * (1 - (1 - 1 / c["E"]) ** P)  # experts that some token chose
        return {"bytes": c["T"] * (Kp + Kp // 32) + used * c["N"] * Kp + P * (4 + c["N"] * _size(c["out"])),
                "flops": 2 * P * c["N"] * c["K"]}
    return {"bytes": c["P"] * (c["N"] + c["K"]) * (1 + 1 / 32) + c["E"] * c["N"] * c["K"] * _size(c["out"]),
            "flops": 2 * c["P"] * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, shape, dt):
    """Normal values with a spread of channel sizes, a few channels far larger."""
    x = torch.randn(shape, generator=g, device=DEV)
    c = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEV))
    c = torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.004, 20 * c, c)
    return (x * c).to(DT[dt])


def _weights(g, shape, dt="bf16"):
    return (0.02 * torch.randn(shape, generator=g, device=DEV)).to(DT[dt])


def _choices(g, T, k, E, drop):
    """Each token's k experts (distinct where E allows), some more popular than others."""
    bias = 0.5 * torch.randn(E, generator=g, device=DEV)
    ids = torch.empty((T, k), dtype=torch.int64, device=DEV)
    for a in range(0, T, 4096):
        n = min(4096, T - a)
        u = torch.rand((n, E), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
        ids[a:a + n] = (bias - torch.log(-torch.log(u))).topk(min(k, E), dim=1).indices
    if drop:
        ids = torch.where(torch.rand((T, k), generator=g, device=DEV) < drop, -1, ids)
    return ids


def _lengths(g, P, E):
    """Row counts of E experts that add up to P; with several experts one is empty."""
    share = torch.exp(0.6 * torch.randn(E, generator=g, device=DEV))
    if E > 2:
        share[E // 3] = 0
    cut = (share.cumsum(0) / share.sum() * P).round().to(torch.int64)
    cut[-1] = P
    return torch.cat([cut.new_zeros(1), cut]).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind = c["kind"]
    if kind in ("gather", "return", "gradient"):
        T, k, E, C = c["T"], c["k"], c["E"], c["C"]
        ids = _choices(g, T, k, E, c["drop"])
        s = dict(case=c, ids=ids)
        if kind == "gather":
            s["x"] = _activations(g, (T, C), c["dtype"])
            return s
        s["plan"] = _sort(ids, E)
        s["w"] = torch.softmax(torch.randn((T, k), generator=g, device=DEV), dim=1)
        s["y"] = _activations(g, (T * k, C), c["dtype"])
        if kind == "gradient":
            s["dout"] = (0.1 * torch.randn((T, C), generator=g, device=DEV)).to(DT[c["dtype"]])
            s["dx"] = (0.1 * torch.randn((T * k, C), generator=g, device=DEV)).to(DT[c["dtype"]])
        return s
    if kind == "quantize":
        shape = (c["B"], c["R"], c["C"])
        x = _activations(g, shape, c["dtype"]) if c["how"] == "row" else _weights(g, shape, c["dtype"])
        return dict(case=c, x=x)
    if kind == "columns":
        return dict(case=c, x=_activations(g, (c["P"], c["C"]), c["dtype"]), offsets=_lengths(g, c["P"], c["E"]))
    if kind == "product":
        a = _quantize_rows(_activations(g, (c["B"], c["M"], c["K"]), "bf16"), c["a"])
        w = _weights(g, (c["B"], c["N"], c["K"]))
        b = _quantize_rows(w, c["b"]) if c["b_scale"] == "row" else _quantize_tiles(w, c["b"])
        return dict(case=c, a=a, b=b)
    if kind == "experts":
        ids = _choices(g, c["T"], c["k"], c["E"], 0.0)
        plan = _sort(ids, c["E"])
        a = _quantize_rows(_activations(g, (c["T"], c["K"]), "bf16"), c["a"])
        b = _quantize_tiles(_weights(g, (c["E"], c["N"], c["K"])), c["b"])
        return dict(case=c, a=a, b=b, plan=plan, longest=max(1, int(plan[0].diff().max())))
    offsets = _lengths(g, c["P"], c["E"])
    dy = (0.1 * torch.randn((c["P"], c["N"]), generator=g, device=DEV)).to(torch.bfloat16)
    x = _activations(g, (c["P"], c["K"]), "bf16")
    return dict(case=c, offsets=offsets, a=_quantize_columns(dy, offsets, c["a"]), b=_quantize_columns(x, offsets, c["b"]),
                longest=max(1, int(offsets.diff().max())))


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _sort(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    P = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = counts[:E].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(P, device=ids.device)
    rows = torch.where(key < E, place, -1).to(torch.int32).reshape(T, k)
    tokens = torch.where(key[order] < E, order // k, -1).to(torch.int32)
    return offsets, rows, tokens


def _gather(x, tokens):
    return torch.where((tokens >= 0)[:, None], x[tokens.clamp(min=0).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def _combine(y, rows, w):
    picked = torch.where((rows >= 0)[..., None], y[rows.clamp(min=0).long()].float(), 0.0)
    return (picked if w is None else picked * w[..., None]).sum(1).to(y.dtype)


def _combine_gradient(dout, y, rows, w):
    T, k = rows.shape
    there = rows >= 0
    at = rows.clamp(min=0).long()
    d = dout.float()
    dw = torch.where(there, (y[at].float() * d[:, None]).sum(-1), 0.0)
    # the rows behind the last expert's stay zero; a dropped choice writes to a row that is cut off
    dy = torch.zeros((y.shape[0] + 1, y.shape[1]), dtype=y.dtype, device=y.device)
    dy[torch.where(there, at, y.shape[0]).reshape(-1)] = (w[..., None] * d[:, None]).to(y.dtype).reshape(-1, y.shape[1])
    return dy[:-1], dw


def _pad(x, rows=0, cols=0):
    return torch.nn.functional.pad(x, (0, cols, 0, rows))


def _to8(x, scale, f8):
    return (x * (1.0 / scale)).to(F8[f8])


def _scale_of(size, f8):
    return (size / TOP[f8]).clamp(min=TINY)


def _quantize_rows(x, f8):
    C = x.shape[-1]
    v = _pad(x.float(), 0, _up(C) - C)
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    s = _scale_of(v.abs().amax(-1), f8)
    return _to8(v, s[..., None], f8).flatten(-2), s.transpose(-1, -2).contiguous()


def _quantize_tiles(x, f8):
    """x [B, R, C]: q [B, R, Cp] and scale [B, Cp/128, ceil(R/128)]."""
    B, R, C = x.shape
    v = _pad(x.float(), _up(R) - R, _up(C) - C).reshape(B, _up(R) // BLOCK, BLOCK, _up(C) // BLOCK, BLOCK)
    s = _scale_of(v.abs().amax((2, 4)), f8)
    q = _to8(v, s[:, :, None, :, None], f8).reshape(B, _up(R), _up(C))[:, :R]
    return q.contiguous(), s.transpose(1, 2).contiguous()


def _turned(q, s, R, C):
    """The transposed operand of _quantize_tiles's: [B, C, Rp] and [B, Rp/128, ceil(C/128)]."""
    t = _pad(q[:, :, :C].view(torch.uint8).transpose(1, 2), 0, _up(R) - R)
    return t.contiguous().view(q.dtype), s.transpose(1, 2).contiguous()


def _places(offsets, P):
    """Each sorted row's expert, its place there, and its column in the columns layout."""
    n = offsets.diff().long()
    e = torch.searchsorted(offsets[1:].contiguous(), torch.arange(P, dtype=torch.int32, device=offsets.device), right=True)
    start = torch.zeros_like(offsets, dtype=torch.int64)
    start[1:] = ((n + BLOCK - 1) // BLOCK * BLOCK).cumsum(0)
    at = torch.arange(P, device=offsets.device) - offsets.long()[e]
    return e, at, start[e] + at


def _quantize_columns(x, offsets, f8):
    P, C = x.shape
    cap = BLOCK * (P // BLOCK + offsets.numel() - 1)
    col = _places(offsets, P)[2]
    v = torch.zeros((cap, C), dtype=torch.float32, device=x.device)
    v[col] = x.float()
    v = v.reshape(-1, BLOCK, C)
    s = _scale_of(v.abs().amax(1), f8)
    q = _to8(v, s[:, None], f8).reshape(cap, C).view(torch.uint8)
    return q.t().contiguous().view(F8[f8]), s


def _values(q, s):
    """An operand's values [B, R, Kp] in fp32."""
    v = q.float()
    R = q.shape[-2]
    t = s.transpose(-1, -2)
    if t.shape[-2] != R:
        t = t.repeat_interleave(BLOCK, dim=-2)[..., :R, :]
    v.view(*v.shape[:-1], -1, BLOCK).mul_(t[..., None])
    return v


def _experts(state):
    c, (offsets, _, tokens), L = state["case"], state["plan"], state["longest"]
    x, w = _values(*state["a"]), _values(*state["b"])
    P = tokens.numel()
    e, at, _ = _places(offsets, P)
    padded = torch.zeros((c["E"], L, x.shape[1]), dtype=torch.float32, device=x.device)
    padded[e, at] = x[tokens.long()]
    return torch.bmm(padded, w.transpose(1, 2))[e, at].to(DT[c["out"]])


def _weight_gradients(state):
    c, offsets, L = state["case"], state["offsets"], state["longest"]
    e, at, col = _places(offsets, c["P"])

    def padded(q, s):  # an expert's rows again, behind each other
        v = torch.zeros((c["E"], L, q.shape[0]), dtype=torch.float32, device=q.device)
        v[e, at] = _values(q, s).t()[col]
        return v

    return torch.bmm(padded(*state["a"]).transpose(1, 2).contiguous(), padded(*state["b"])).to(DT[c["out"]])


def run(state):
    c = state["case"]
    kind = c["kind"]
    if own:
        return _run_own(state)
    if kind == "gather":
        plan = _sort(state["ids"], c["E"])
        return (*plan, _gather(state["x"], plan[2]))
    if kind == "return":
        return _combine(state["y"], state["plan"][1], state["w"])
    if kind == "gradient":
        dy, dw = _combine_gradient(state["dout"], state["y"], state["plan"][1], state["w"])
        return dy, dw, _combine(state["dx"], state["plan"][1], None)
    if kind == "quantize":
        if c["how"] == "row":
            return _quantize_rows(state["x"], c["f8"])
        q, s = _quantize_tiles(state["x"], c["f8"])
        return (q, s, *_turned(q, s, c["R"], c["C"]))
    if kind == "columns":
        return _quantize_columns(state["x"], state["offsets"], c["f8"])
    if kind == "product":
        a, b = _values(*state["a"]), _values(*state["b"])
        return torch.bmm(a, b.transpose(1, 2)).to(DT[c["out"]])
    if kind == "experts":
        return _experts(state)
    return _weight_gradients(state)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _run_own(state):
    import newton_schulz_gram_amd as nsg

    c = state["case"]
    kind = c["kind"]
    if kind == "gather":
        plan = nsg.expert_sort(state["ids"], c["E"])
        return (*plan, nsg.expert_dispatch(state["x"], plan))
    if kind == "return":
        return nsg.expert_combine(state["y"], nsg.ExpertPlan(*state["plan"]), state["w"])
    if kind == "gradient":
        plan = nsg.ExpertPlan(*state["plan"])
        dy, dw = nsg.expert_combine_backward(state["dout"], state["y"], plan, state["w"])
        return dy, dw, nsg.expert_combine(state["dx"], plan)
    if kind == "quantize":
        return nsg.quantize_fp8(state["x"], block=c["how"], dtype=F8[c["f8"]], transposed=c["how"] == "tile")
    if kind == "columns":
        return nsg.quantize_fp8_columns(state["x"], state["offsets"], dtype=F8[c["f8"]])
    if kind == "product":
        return nsg.gemm_fp8_nt(*state["a"], *state["b"], out_dtype=DT[c["out"]])
    if kind == "experts":
        return nsg.expert_gemm_fp8(*state["a"], *state["b"], state["plan"][0], rows=state["plan"][2], out_dtype=DT[c["out"]])
    return nsg.expert_wgrad_fp8(*state["a"], *state["b"], state["offsets"], out_dtype=DT[c["out"]])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _round8(v, f8):
    """Nearest value of the 8 bit type, ties to the even one; v in fp64, no larger than the type's largest by more than rounding."""
    bits, low = (3, -6) if f8 == "e4m3" else (2, -14)
    e = torch.frexp(v)[1].to(torch.float64) - 1
    step = torch.exp2(e.clamp(min=low) - bits)
    return torch.where(v == 0, v, torch.round(v / step) * step)


def _exact_block(v, f8):
    """v [..., 128 values of one block]: (rounded values, scale [..., 1])."""
    s = (v.abs().amax(-1, keepdim=True) / TOP[f8]).clamp(min=TINY)
    return _round8(v / s, f8), s


def _exact_bounds(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def _exact_operand(q, s):
    """fp64 values of a 2-d operand."""
    R, Kp = q.shape
    per_row = s.shape[1] == R
    full = s.t().double()[torch.arange(R, device=q.device) if per_row else torch.arange(R, device=q.device) // BLOCK]
    return q.double() * full[:, torch.arange(Kp, device=q.device) // BLOCK]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "gather":
        x, E = s["x"].double(), c["E"]
        ids = s["ids"].reshape(-1).cpu()
        out = torch.zeros((ids.numel(), c["C"]), dtype=torch.float64, device=DEV)
        lists = torch.cat([torch.nonzero(ids == e)[:, 0] for e in range(E)])
        out[:lists.numel()] = x[(lists // c["k"]).to(DEV)]
        return None, None, None, out
    if kind == "return":
        rows, w, y = s["plan"][1], s["w"].double(), s["y"]
        out = torch.zeros((c["T"], c["C"]), dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            r = rows[:, j].long()
            out[r >= 0] += w[r >= 0, j, None] * y[r[r >= 0]].double()
        return out
    if kind == "gradient":
        rows, w = s["plan"][1], s["w"].double()
        d = s["dout"].double()
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(w.shape, dtype=torch.float64, device=DEV)
        dx = torch.zeros(d.shape, dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            t = torch.nonzero(rows[:, j] >= 0)[:, 0]
            r = rows[t, j].long()
            dy[r] = w[t, j, None] * d[t]
            dw[t, j] = (s["y"][r].double() * d[t]).sum(1)
            dx[t] += s["dx"][r].double()
        return dy, dw, dx
    if kind == "quantize":
        B, R, C = s["x"].shape
        Rp, Cp = _up(R), _up(C)
        v = torch.zeros((B, Rp, Cp), dtype=torch.float64, device=DEV)
        v[:, :R, :C] = s["x"].double()
        if c["how"] == "row":
            q, sc = _exact_block(v[:, :R].unflatten(2, (-1, BLOCK)), c["f8"])
            return q.flatten(2), sc[..., 0].transpose(1, 2)
        tiles = v.reshape(B, Rp // BLOCK, BLOCK, Cp // BLOCK, BLOCK).permute(0, 1, 3, 2, 4).flatten(3)
        q, sc = _exact_block(tiles, c["f8"])
        q = q.unflatten(3, (BLOCK, BLOCK)).permute(0, 1, 3, 2, 4).reshape(B, Rp, Cp)
        return q[:, :R], sc[..., 0].transpose(1, 2), q.transpose(1, 2)[:, :C], sc[..., 0]
    if kind == "columns":
        C, nb = c["C"], c["P"] // BLOCK + c["E"]
        v = torch.zeros((C, nb * BLOCK), dtype=torch.float64, device=DEV)
        at = 0
        for _, a, b in _exact_bounds(s["offsets"]):
            v[:, at:at + b - a] = s["x"][a:b].double().t()
            at += _up(b - a)
        q, sc = _exact_block(v.reshape(C, nb, BLOCK), c["f8"])
        return q.flatten(1), sc[..., 0].t()
    if kind == "product":
        (qa, sa), (qb, sb) = s["a"], s["b"]
        return torch.stack([_exact_operand(qa[i], sa[i]) @ _exact_operand(qb[i], sb[i]).t() for i in range(c["B"])])
    if kind == "experts":
        x, (qw, sw) = _exact_operand(*s["a"]), s["b"]
        offsets, _, tokens = s["plan"]
        out = torch.zeros((tokens.numel(), c["N"]), dtype=torch.float64, device=DEV)
        for e, a, b in _exact_bounds(offsets):
            if b > a:
                out[a:b] = x[tokens[a:b].long()] @ _exact_operand(qw[e], sw[e]).t()
        return out
    dy, x = _exact_operand(*s["a"]), _exact_operand(*s["b"])
    out = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device=DEV)
    at = 0
    for e, a, b in _exact_bounds(s["offsets"]):
        out[e] = dy[:, at:at + b - a] @ x[:, at:at + b - a].t()
        at += _up(b - a)
    return out
