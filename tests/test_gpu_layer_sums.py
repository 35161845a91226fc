"""GPU tests of the sums over many tokens and rows that layer norm's gradient and the router
take, past 32-bit offsets: inputs whose results fp32 holds exactly, whatever the order of
the additions, so that every output of every row is compared for equality and a row, a
workgroup's sum or a turn that is lost or read twice shows.

Layer norm: rows of +1 and -1, as many of each, without eps: mean 0 and rstd 1, so xh is the
row itself.  dy is whole numbers up to 4, weights are 1/2, 1 or 2: g = dy weight is a
multiple of 1/2 up to 8, its sums over a row's C = 2^n columns stay below 2^20 and their
means are multiples of 2^-(n + 1); dx needs at most 5 + n + 1 <= 22 bits.  Sums over the
rows stay below 4 * 2^20 < 2^24.

Router: a token has four experts with logit 0, all others -inf: e^0 = 1, the scores' sum is 4,
each p is 1/4, and of the two lowest experts each weighs 1/2.  Sums of p are multiples of
1/4 below 2^21, their quotient by N (below 2^24) is rounded once."""
import pytest
import torch

import newton_schulz_gram_amd as nsg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def integers(lo, hi, shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def pieces(n, width):
    """Ranges of rows of at most 2^26 elements."""
    step = max(1, (1 << 26) // width)
    return [(a, min(n, a + step)) for a in range(0, n, step)]


# past 2^31 elements: each kernel (256 and 1024 lanes a row, weights in registers and in LDS, rows
# that do not fit in registers); then one of every width
@pytest.mark.parametrize("R,C,dt", [(540_000, 4096, "bf16"), (135_000, 16384, "f32"), (70_000, 32768, "bf16"),
                                    (33_333, 64, "f16"), (20_001, 128, "bf16"), (10_007, 256, "f32"), (7001, 512, "bf16"),
                                    (4099, 1024, "f16"), (3001, 2048, "f32"), (1003, 8192, "bf16"), (517, 16384, "f16"),
                                    (300, 65536, "bf16"), (1001, 4, "bf16"), (1001, 2, "f32")])
def test_layer_norm_of_rows_of_ones(R, C, dt):
    t = DT[dt]
    x, dy = torch.empty(R, C, dtype=t, device="cuda"), torch.empty(R, C, dtype=t, device="cuda")
    for i, (a, b) in enumerate(pieces(R, C)):
        half = 2 * integers(0, 1, (b - a, C // 2), 2 * i) - 1
        x[a:b, :C // 2], x[a:b, C // 2:] = half, -half
        dy[a:b] = integers(-4, 4, (b - a, C), 2 * i + 1)
    w = 2.0 ** integers(-1, 1, (C,), 98).float()
    bias = integers(-8, 8, (C,), 99).float()
    y, stats = nsg.layer_norm(x, w, bias, eps=0.0)
    assert stats[0].eq(0).all() and stats[1].eq(1).all()
    dx, dw, db = nsg.layer_norm_backward(dy, x, stats, w)
    want_w, want_b = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    for a, b in pieces(R, C):
        f, d = x[a:b].float(), dy[a:b].float()
        assert torch.equal(y[a:b], (f * w + bias).to(t)), a
        # (means in 64 bits: exact in any order; the rest is exact in fp32)
        g = d * w
        mean, dot = (v.sum(1, keepdim=True, dtype=torch.float64).div(C).float() for v in (g, g * f))
        assert torch.equal(dx[a:b], (g - mean - f * dot).to(t)), a
        want_w += (d * f).sum(0, dtype=torch.float64)
        want_b += d.sum(0, dtype=torch.float64)
    assert torch.equal(dw.double(), want_w) and torch.equal(db.double(), want_b)


# past 2^31 logits (groups of 32 lanes, a wave each), then one of every width
@pytest.mark.parametrize("T,E,dt", [((1 << 31) // 256 + 4000, 256, "bf16"), ((1 << 31) // 1024 + 4000, 1024, "bf16"),
                                    ((1 << 31) // 512 + 3999, 512, "f16"), ((1 << 24) - 5, 16, "f16"), (1_000_003, 60, "f32"),
                                    (300_001, 128, "bf16"), (2047, 300, "f32"), (2049, 37, "bf16")])
@pytest.mark.parametrize("bias", [False, True])
def test_router_of_four_equal_experts(T, E, dt, bias):
    k, t = 2, DT[dt]
    l = torch.empty(T, E, dtype=t, device="cuda")
    at = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 1, E // 3 + 1, E // 2 + 1], device="cuda")
    for i, (a, b) in enumerate(pieces(T, E)):
        g = torch.Generator(device="cuda").manual_seed(i)
        e = (torch.randint(0, E, (b - a, 1), generator=g, device="cuda") + offsets) % E
        l[a:b] = -float("inf")
        l[a:b].scatter_(1, e, 0.0)
        at[a:b] = e.sort(1).values
    # a bias that is the same for all changes no choice (1/4 + 1/8 is exact)
    b = torch.full((E,), 0.125, device="cuda") if bias else None
    r = nsg.expert_route(l, k, bias=b, balance=True)
    assert torch.equal(r.ids, at[:, :k]) and r.weights.eq(0.5).all()
    chosen, met = (torch.bincount(v.reshape(-1), minlength=E) for v in (at[:, :k], at))
    assert torch.equal(r.counts[:E].long(), chosen) and r.counts[E] == T
    # (rounded once: 53 bits are more than twice fp32's 24 and 2)
    assert torch.equal(r.probs, (met.double() * 0.25 / T).float())
    # products and probs are off by u each, E / (k N) by 2 u, sums by one for each addition: one in
    # a thread, 6 steps of lanes, 16 waves; the last product
    loss = E / (k * T) * (chosen.double() * r.probs.double()).sum()
    assert abs(r.loss.double() - loss) <= (1 + 2 + 1 + 6 + 16 + 1) * U * loss
    # the weights' gradient: v_j (g_j - sum g v) with v = 1/2, whole g
    dw = integers(-4, 4, (T, k), 5).float()
    dl = nsg.expert_route_backward(l, r.ids, dw)
    d = 0.25 * (dw[:, 0] - dw[:, 1])
    for a, b in pieces(T, E):
        want = torch.zeros(b - a, E, device="cuda").scatter_(1, at[a:b, :k].long(), torch.stack([d[a:b], -d[a:b]], 1))
        assert torch.equal(dl[a:b], want.to(t)), a
