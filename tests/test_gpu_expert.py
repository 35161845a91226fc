"""GPU tests of the expert-layer operators against the fp64 oracle: tokens sorted
by expert and back with their gradients, 8-bit operands with block scales, their
products (plain, batched, by expert, weight gradients).

Tolerances count roundings, u = 2^-24 for fp32 and half(t) = eps / 2 for the
output's type, and are absolute against the sum of the sizes of the terms:
  combine   k products and k sums in fp32: (2 k) u sum |w y|, then half(t) |v|
  dw        C products and sums in fp32, in any order: (2 C) u sum |d y|
  products  the 128 products of a block are exact in fp32 (8-bit mantissas);
            their sum inside the matrix instruction is taken as truncating:
            128 * 2 u; one rounding of the scales' product, one per block's
            multiply-add: (K / 128 + 2) u; all of sum |a b|; then half(t) |v|.
            For 16-bit outputs the 8-bit instructions also cut the products of 8
            consecutive k off at 2^-13 of the largest one's power of two, which
            loses less than 7 * 2^-13 of the largest product of each 8 (cut_off).
"""
import numpy as np
import pytest
import torch

import newton_schulz_gram_amd as nsg
from oracle import expert_oracle as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().float().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def normal(shape, dt, seed, scale=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy((scale * g.standard_normal(shape)).astype(np.float32)).to(DT[dt])


def choices(T, k, E, seed, drop=0.1):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, size=(T, k))
    ids[g.random((T, k)) < drop] = -1
    if T * k > 3:
        ids.reshape(-1)[1] = E  # past the last expert: dropped too
        ids.reshape(-1)[2] = -7
    return ids


def plan_of(ids, E):
    o, r, t = ref.expert_sort(ids, E)
    return nsg.ExpertPlan(*(torch.from_numpy(v.astype(np.int32)).cuda() for v in (o, r, t)))


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 512), (7, 3, 5), (64, 1, 64), (513, 8, 60), (1000, 2, 1024),
                                   (4096, 1, 3), (4097, 1, 512), (3001, 7, 100), (70000, 8, 512)])
@pytest.mark.parametrize("wide", [True, False])
def test_sort(T, k, E, wide):
    ids = choices(T, k, E, seed=T + k)
    p = nsg.expert_sort(torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda(), E)
    exp = ref.expert_sort(ids, E)
    for got, e, name in zip(p, exp, ("offsets", "rows", "tokens")):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), e), name


@pytest.mark.parametrize("fill", [-1, 0, 5, 6])
def test_sort_all_alike(fill):
    """All choices dropped, or all on the first or last expert (empty ones around)."""
    ids = np.full((777, 5), fill)
    p = nsg.expert_sort(torch.from_numpy(ids).cuda(), 6)
    for got, e in zip(p, ref.expert_sort(ids, 6)):
        assert np.array_equal(got.cpu().numpy(), e)


def test_sort_huge_ids_are_dropped():
    ids = torch.tensor([[1 << 32, -(1 << 40)], [2, (1 << 62) + 1]]).cuda()
    p = nsg.expert_sort(ids, 3)
    assert p.offsets.tolist() == [0, 0, 0, 1] and p.rows.tolist() == [[-1, -1], [0, -1]] and p.tokens.tolist() == [1, -1, -1, -1]


# ---------------------------------------------------------------------------
# dispatch, combine, gradients
# ---------------------------------------------------------------------------
def pitched(t, pad):
    """The same matrix with `pad` more elements between its rows, on the GPU."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t.cuda()
    return big[:, :t.shape[1]]


SHAPES = [(1, 8, 512, 2048), (5, 2, 3, 64), (33, 4, 8, 1), (17, 3, 5, 129), (40, 8, 64, 1000), (257, 1, 4, 520), (3, 12, 4, 4104)]


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_dispatch(T, k, E, C, dt, pad):
    ids = choices(T, k, E, seed=1)
    x = normal((T, C), dt, 2)
    if T > 2:
        x[2, 0] = float("inf")
        x[1, -1] = float("nan")
    out = nsg.expert_dispatch(pitched(x, pad) if pad else x.cuda(), plan_of(ids, E))
    assert out.dtype == DT[dt]
    assert np.array_equal(f64(out), ref.dispatch(f64(x), ref.expert_sort(ids, E)[2]), equal_nan=True)


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_combine(T, k, E, C, dt, weighted, pad):
    ids = choices(T, k, E, seed=3)
    if T > 4:
        ids[4] = -1  # a token with no expert
    y = normal((T * k, C), dt, 4)
    w = torch.softmax(normal((T, k), "f32", 5), dim=1) if weighted else None
    plan = plan_of(ids, E)
    out = nsg.expert_combine(pitched(y, pad) if pad else y.cuda(), plan, w.cuda() if weighted else None)
    exp, size = ref.combine(f64(y), ref.expert_sort(ids, E)[1], f64(w) if weighted else None)
    tol = 2 * k * U * size + half(DT[dt]) * (np.abs(exp) + 2 * k * U * size)
    assert np.all(np.abs(f64(out) - exp) <= tol)
    if T > 4:
        assert not out[4].any()


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_combine_backward(T, k, E, C, dt, weighted, pad):
    ids = choices(T, k, E, seed=6)
    y, dout = normal((T * k, C), dt, 7), normal((T, C), dt, 8)
    w = torch.softmax(normal((T, k), "f32", 9), dim=1) if weighted else None
    dy, dw = nsg.expert_combine_backward(pitched(dout, pad) if pad else dout.cuda(), pitched(y, pad) if pad else y.cuda(),
                                         plan_of(ids, E), w.cuda() if weighted else None)
    edy, edw, size = ref.combine_backward(f64(dout), f64(y), ref.expert_sort(ids, E)[1], f64(w) if weighted else None)
    assert dy.dtype == DT[dt] and dw.dtype == torch.float32
    assert np.all(np.abs(f64(dw) - edw) <= 2 * C * U * size)
    # one fp32 product, one rounding; f16 values below 2^-14 round to steps of 2^-24
    low = 2.0 ** -25 if dt == "f16" else 0.0
    assert np.all(np.abs(f64(dy) - edy) <= (half(DT[dt]) * (1 + U) + U) * np.abs(edy) + low)


def test_gradients_against_differences():
    """combine is linear in y and in the weights: differences of it are exact up to
    rounding, so <dout, combine(y + h v) - combine(y)> = h <dy, v>, and with dw."""
    T, k, E, C = 23, 3, 6, 200
    plan = plan_of(choices(T, k, E, 10), E)
    y, v, dout = (normal(s, "f32", 11 + i).cuda() for i, s in enumerate([(T * k, C), (T * k, C), (T, C)]))
    w, u = (normal((T, k), "f32", 14 + i).cuda() for i in range(2))
    dy, dw = nsg.expert_combine_backward(dout, y, plan, w)
    h = 0.5
    base = f64(nsg.expert_combine(y, plan, w))
    used = np.zeros((T * k, 1))
    used[:int(plan.offsets[-1])] = 1  # rows that no choice leads to have no gradient
    dd = f64(dout)
    size = np.sum(np.abs(dd) * ref.combine(np.abs(f64(y)) + np.abs(f64(v)), plan.rows.cpu().numpy(),
                                           np.abs(f64(w)) + np.abs(f64(u)))[0])
    # every combine rounds (2 k + 1) times; dw sums 2 C terms, dy rounds twice
    tol = (2 * (2 * k + 1) + 2 * C + 2) * U * size
    assert abs(np.sum(dd * (f64(nsg.expert_combine(y + h * v, plan, w)) - base)) - h * np.sum(f64(dy) * used * f64(v))) <= 2 * tol
    assert abs(np.sum(dd * (f64(nsg.expert_combine(y, plan, w + h * u)) - base)) - h * np.sum(f64(dw) * f64(u))) <= 2 * tol
    # dispatch's gradient is combine without weights: <dispatch(x), v> = <x, combine(v)>
    x = normal((T, C), "f32", 20).cuda()
    lhs, rhs = f64(nsg.expert_dispatch(x, plan)) * f64(v), f64(x) * f64(nsg.expert_combine(v, plan))
    assert abs(lhs.sum() - rhs.sum()) <= (k + 1) * U * 2 * np.abs(lhs).sum() + 1e-12


# ---------------------------------------------------------------------------
# 8-bit operands: the same fp32 arithmetic gives the same bytes
# ---------------------------------------------------------------------------
def spiky(shape, dt, seed):
    """Values over many sizes, an all-zero block, one of tiny values."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * 10.0 ** g.uniform(-3, 2, size=shape)
    x[..., : min(128, shape[-1])][..., 0, :] = 0.0
    if shape[-2] > 3:
        x[..., 3, :] *= 1e-6
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt])


QSHAPES = [(1, 1), (1, 128), (3, 129), (16, 1000), (130, 300), (257, 64), (64, 4096), (40, 8)]


@pytest.mark.parametrize("R,C", QSHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("f8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("B", [0, 3])
def test_quantize_rows(R, C, dt, f8, B):
    x = spiky((max(B, 1), R, C), dt, R + C)
    q, s = nsg.quantize_fp8((x if B else x[0]).cuda(), dtype=F8[f8])
    Cp = ref.up128(C)
    assert q.shape == ((B, R, Cp) if B else (R, Cp)) and s.shape == ((B, Cp // 128, R) if B else (Cp // 128, R))
    q, s = f64(q).reshape(-1, R, Cp), s.cpu().numpy().reshape(-1, Cp // 128, R)
    for b in range(len(q)):
        eq, es = ref.quantize_rows(x[b].float().numpy(), f8)
        assert np.array_equal(s[b], es) and np.array_equal(q[b], eq)


@pytest.mark.parametrize("R,C", QSHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("f8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("B", [0, 3])
def test_quantize_tiles(R, C, dt, f8, B):
    x = spiky((max(B, 1), R, C), dt, R + C)
    xs = (x if B else x[0]).cuda()
    q, s, qt, st = nsg.quantize_fp8(xs, block="tile", dtype=F8[f8], transposed=True)
    q1, s1 = nsg.quantize_fp8(xs, block="tile", dtype=F8[f8])
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, s)
    Rp, Cp = ref.up128(R), ref.up128(C)
    q, qt = f64(q).reshape(-1, R, Cp), f64(qt).reshape(-1, C, Rp)
    s, st = s.cpu().numpy().reshape(-1, Cp // 128, Rp // 128), st.cpu().numpy().reshape(-1, Rp // 128, Cp // 128)
    for b in range(len(q)):
        eq, es = ref.quantize_tiles(x[b].float().numpy(), f8)
        assert np.array_equal(s[b], es) and np.array_equal(q[b], eq) and np.array_equal(st[b], es.T)
        assert np.array_equal(qt[b][:, :R], eq[:, :C].T) and not qt[b][:, R:].any()


@pytest.mark.parametrize("P,E,C", [(0, 3, 40), (1, 1, 1), (5, 4, 130), (128, 1, 128), (300, 3, 64), (1000, 7, 257), (2000, 40, 136)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("f8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("gather", [False, True])
def test_quantize_columns(P, E, C, dt, f8, gather):
    g = np.random.default_rng(P + E)
    cut = np.sort(g.integers(0, P + 1, size=E - 1))
    offsets = np.concatenate([[0], cut, [P]]).astype(np.int32)
    if E > 3:
        offsets[2] = offsets[1]   # an expert without rows
        offsets[-1] -= min(2, P - offsets[-2])  # rows behind the last expert's
    x = spiky((max(P, 4), C), dt, 3)
    rows = g.integers(0, len(x), size=P).astype(np.int32)
    if P > 4:
        rows[3] = -1
        rows[4] = len(x)
    sorted_x = ref.dispatch(f64(x), rows) if gather else f64(x)[:P]
    if gather:
        qt, s = nsg.quantize_fp8_columns(x.cuda(), torch.from_numpy(offsets).cuda(), torch.from_numpy(rows).cuda(), dtype=F8[f8])
    else:
        qt, s = nsg.quantize_fp8_columns(x[:P].contiguous().cuda(), torch.from_numpy(offsets).cuda(), dtype=F8[f8])
    eq, es = ref.quantize_columns(sorted_x.astype(np.float32), offsets, f8)
    assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(f64(qt), eq)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["row", "tile", "columns"])
@pytest.mark.parametrize("f8", ["e4m3", "e5m2"])
def test_quantize_infinities_and_nan(dt, how, f8):
    """They do not change their block's scale and stay where they are."""
    x = normal((130, 200), dt, 30)
    x[5, 7], x[6, 130], x[129, 0], x[64, 64] = float("inf"), float("-inf"), float("nan"), float("nan")
    x[70, :] = float("nan")
    v = x.float().numpy()
    if how == "columns":
        o = np.array([0, 100, 130], dtype=np.int32)
        q, s = nsg.quantize_fp8_columns(x.cuda(), torch.from_numpy(o).cuda(), dtype=F8[f8])
        eq, es = ref.quantize_columns(v, o, f8)
    else:
        q, s = nsg.quantize_fp8(x.cuda(), block=how, dtype=F8[f8])
        eq, es = (ref.quantize_rows if how == "row" else ref.quantize_tiles)(v, f8)
    assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(f64(q), eq, equal_nan=True)
    assert np.isnan(f64(q)).any()


@pytest.mark.parametrize("dt,ends", [("bf16", (1e-38, 3e38)), ("f32", (1e-44, 3.4e38)), ("f16", (6e-8, 65504.0))])
def test_quantize_ends_of_the_range(dt, ends):
    x = torch.zeros((4, 256), dtype=DT[dt])
    x[0, :128], x[1, 5], x[2, 200], x[3, 0] = ends[0], ends[1], -ends[1], ends[0]
    x[1, 6] = ends[0]
    q, s = nsg.quantize_fp8(x.cuda())
    eq, es = ref.quantize_rows(x.float().numpy(), "e4m3")
    assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(f64(q), eq)


@pytest.mark.parametrize("pad", [8, 3])
def test_quantize_pitched_rows(pad):
    x = normal((70, 264), "bf16", 31)
    p = pitched(x, pad)
    for how in ("row", "tile"):
        a, b = nsg.quantize_fp8(p, block=how), nsg.quantize_fp8(x.cuda(), block=how)
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    o = torch.tensor([0, 30, 70], dtype=torch.int32).cuda()
    a, b = nsg.quantize_fp8_columns(p, o), nsg.quantize_fp8_columns(x.cuda(), o)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def operand(shape, f8, seed, how="row"):
    """(q, scale) on the GPU and its fp64 values."""
    x = normal(shape, "f32", seed) * torch.from_numpy(10.0 ** np.random.default_rng(seed + 1).uniform(-2, 2, size=(shape[0], 1)).astype(np.float32))
    q, s = (ref.quantize_rows if how == "row" else ref.quantize_tiles)(x.numpy(), f8)
    return (torch.from_numpy(q).float().to(F8[f8]).cuda(), torch.from_numpy(s.copy()).cuda()), ref.values(q, s)


def product(av, bv):
    return (*ref.product(av, bv), ref.cut_off(av, bv))


def check_product(out, exp, size, cut, K, what=""):
    t = out.dtype
    fuzz = (128 * 2 + K // 128 + 2) * U * size + (0 if t == torch.float32 else cut)
    low = 2.0 ** -25 if t == torch.float16 else 0.0
    tol = fuzz + half(t) * (np.abs(exp) + fuzz) + low
    got = f64(out)
    # the largest number is (2 - eps) 2^e; from half a step past it, (2 - eps / 2) 2^e,
    # numbers round to infinity (f16: 65504, and infinity from 65520 on)
    edge = torch.finfo(t).max / (2 - torch.finfo(t).eps) * (2 - half(t))
    over, under = np.abs(exp) - fuzz >= edge, np.abs(exp) + fuzz < edge
    assert np.all(np.isinf(got[over]))
    assert np.all(np.abs(got - exp)[under] <= tol[under]), (what, np.max((np.abs(got - exp) / tol)[under]))


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 128), (3, 130, 300), (16, 100, 1000), (17, 257, 128), (40, 512, 640),
                                   (64, 48, 2048), (65, 300, 200), (128, 128, 256), (200, 1000, 384), (257, 129, 1100)])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kinds", [("row", "tile"), ("row", "row"), ("tile", "tile"), ("tile", "row")])
def test_gemm(M, N, K, out, kinds):
    (a, av), (b, bv) = operand((M, K), "e4m3", 40, kinds[0]), operand((N, K), "e4m3", 50, kinds[1])
    check_product(nsg.gemm_fp8_nt(*a, *b, out_dtype=DT[out]), *product(av, bv), K=a[0].shape[1])


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M", [2, 33, 150, 300])
@pytest.mark.parametrize("how", ["row", "tile"])
def test_gemm_types(fa, fb, M, how):
    (a, av), (b, bv) = operand((M, 700), fa, 41), operand((320, 700), fb, 51, how)
    check_product(nsg.gemm_fp8_nt(*a, *b, out_dtype=torch.float32), *product(av, bv), K=768)


@pytest.mark.parametrize("M", [1, 20, 130])
def test_gemm_batched(M):
    ops = [[operand((r, 500), "e4m3", 60 + 7 * i + r, h) for i in range(3)] for r, h in ((M, "row"), (200, "tile"))]
    (qa, sa), (qb, sb) = ((torch.stack([o[0][0] for o in side]), torch.stack([o[0][1] for o in side])) for side in ops)
    out = nsg.gemm_fp8_nt(qa, sa, qb, sb, out_dtype=torch.float32)
    for i in range(3):
        check_product(out[i], *product(ops[0][i][1], ops[1][i][1]), K=512)
        # a batch's product is the single one's, bit for bit
        assert torch.equal(out[i], nsg.gemm_fp8_nt(qa[i], sa[i], qb[i], sb[i], out_dtype=torch.float32))


@pytest.mark.parametrize("how", ["row", "tile"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_tile_sizes_agree(how, out):
    """One product alone, among 20 and among 200 runs on tiles of 64, 128 and (16-bit
    outputs) 256: the same sums in the same order, bit for bit."""
    (a, av), (b, bv) = operand((300, 640), "e5m2", 75), operand((290, 640), "e4m3", 76, how)
    one = nsg.gemm_fp8_nt(*a, *b, out_dtype=DT[out])
    check_product(one, *product(av, bv), K=640)
    for n in (20, 200):
        many = nsg.gemm_fp8_nt(*(t.expand(n, *t.shape).contiguous() for t in (*a, *b)), out_dtype=DT[out])
        assert torch.equal(many, one.expand_as(many))


def test_gemm_exact_integers():
    """Small whole numbers with power-of-two scales: every sum is exact, so the
    lane layout of both operands, the block order and the stores are pinned."""
    g = np.random.default_rng(70)
    for M, N, K in [(5, 70, 256), (48, 200, 640), (300, 300, 384)]:
        a, b = g.integers(-8, 9, size=(M, K)), g.integers(-8, 9, size=(N, K))
        sa, sb = 2.0 ** g.integers(-3, 4, size=(K // 128, M)), 2.0 ** g.integers(-3, 4, size=(K // 128, N))
        to = lambda v, s: (torch.from_numpy(v).float().to(F8["e4m3"]).cuda(), torch.from_numpy(s).float().cuda())  # noqa: E731
        out = nsg.gemm_fp8_nt(*to(a, sa), *to(b, sb), out_dtype=torch.float32)
        assert np.array_equal(f64(out), ref.values(a, sa) @ ref.values(b, sb).T)


@pytest.mark.parametrize("M", [3, 200])
def test_gemm_nan_stays_in_its_row_and_column(M):
    (a, av), (b, bv) = operand((M, 256), "e4m3", 71), operand((150, 256), "e5m2", 72)
    a[0][2, 100] = float("nan")
    b[0][7, 3] = float("inf")
    out = f64(nsg.gemm_fp8_nt(*a, *b, out_dtype=torch.float32))
    assert np.isnan(out[2]).all() and not np.isfinite(out[:, 7]).any()
    rest = np.delete(np.delete(out, 2, 0), 7, 1)
    assert np.isfinite(rest).all()


def lengths(P, E, seed, tail=0):
    g = np.random.default_rng(seed)
    o = np.concatenate([[0], np.sort(g.integers(0, P - tail + 1, size=E - 1)), [P - tail]]).astype(np.int32)
    if E > 2:
        o[1] = 0
    return o


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 64, 128), (1, 8, 64, 256, 512), (6, 2, 4, 100, 300), (50, 4, 16, 130, 256),
                                       (300, 2, 3, 260, 640), (700, 1, 5, 64, 128), (40, 8, 512, 70, 128)])
@pytest.mark.parametrize("how", ["row", "tile"])
@pytest.mark.parametrize("types", [("e4m3", "e4m3", "bf16"), ("e5m2", "e4m3", "f32"), ("e4m3", "e5m2", "f16")])
def test_expert_gemm(T, k, E, N, K, how, types):
    ids = choices(T, k, E, 80)
    plan, (offsets, _, tokens) = plan_of(ids, E), ref.expert_sort(ids, E)
    (a, av) = operand((T, K), types[0], 81)
    w = [operand((N, K), types[1], 82 + e % 7, how) for e in range(E)]
    qb, sb = torch.stack([o[0][0] for o in w]), torch.stack([o[0][1] for o in w])
    out = nsg.expert_gemm_fp8(*a, qb, sb, plan.offsets, rows=plan.tokens, out_dtype=DT[types[2]])
    exp = np.zeros((3, T * k, N))
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        exp[:, s] = product(av[tokens[s]], w[e][1])
    check_product(out, *exp, K=a[0].shape[1])
    assert not out[offsets[-1]:].any()


@pytest.mark.parametrize("P,E", [(1, 1), (37, 4), (500, 6), (1500, 3)])
def test_expert_gemm_rows_in_order(P, E):
    o = lengths(P, E, 5, tail=min(3, P - 1))
    (a, av) = operand((P, 384), "e4m3", 90)
    w = [operand((200, 384), "e4m3", 91 + e, "tile") for e in range(E)]
    out = nsg.expert_gemm_fp8(*a, torch.stack([x[0][0] for x in w]), torch.stack([x[0][1] for x in w]),
                              torch.from_numpy(o).cuda(), out_dtype=torch.float32)
    exp = np.zeros((3, P, 200))
    for e in range(E):
        exp[:, o[e]:o[e + 1]] = product(av[o[e]:o[e + 1]], w[e][1])
    check_product(out, *exp, K=384)
    assert not out[o[-1]:].any()


def test_expert_gemm_rows_out_of_range_are_zero():
    (a, av) = operand((5, 128), "e4m3", 95)
    (b, bv) = operand((64, 128), "e4m3", 96, "tile")
    rows = torch.tensor([4, -1, 5, 0, 1 << 30], dtype=torch.int32).cuda()
    a[0][0, 0] = float("nan")  # row 0 is read in their place
    out = nsg.expert_gemm_fp8(*a, b[0][None], b[1][None], torch.tensor([0, 5], dtype=torch.int32).cuda(), rows=rows,
                              out_dtype=torch.float32)
    assert not out[[1, 2, 4]].any() and torch.isnan(out[3]).all() and out[0].isfinite().all()


@pytest.mark.parametrize("P,E,N,K", [(0, 2, 30, 40), (1, 1, 64, 64), (200, 1, 130, 70), (333, 5, 64, 300), (1003, 8, 300, 200),
                                     (600, 3, 257, 129)])
@pytest.mark.parametrize("types", [("e5m2", "e4m3", "f32"), ("e4m3", "e4m3", "bf16"), ("e5m2", "e5m2", "f16")])
def test_expert_wgrad(P, E, N, K, types):
    o = lengths(P, E, 6) if P else np.zeros(E + 1, dtype=np.int32)
    sides = []
    for C, f8, seed in ((N, types[0], 100), (K, types[1], 101)):
        q, s = ref.quantize_columns(normal((P, C), "f32", seed).numpy(), o, f8)
        sides.append(((torch.from_numpy(np.ascontiguousarray(q)).float().to(F8[f8]).cuda(), torch.from_numpy(s.copy()).cuda()),
                      ref.values(q, s)))
    (a, av), (b, bv) = sides
    out = nsg.expert_wgrad_fp8(*a, *b, torch.from_numpy(o).cuda(), out_dtype=DT[types[2]])
    at = 0
    for e in range(E):
        n = o[e + 1] - o[e]
        check_product(out[e], *product(av[:, at:at + n], bv[:, at:at + n]), K=ref.up128(int(n)))
        if n == 0:
            assert not out[e].any()
        at += ref.up128(int(n))


# ---------------------------------------------------------------------------
# wrong device data, far offsets, streams, graphs, the layer as a whole
# ---------------------------------------------------------------------------
def test_wrong_plans_stay_in_bounds():
    """Offsets that run backwards or past the end, rows past the end: clamped."""
    P, E = 300, 4
    x = normal((P, 128), "bf16", 110).cuda()
    (a, _) = operand((P, 128), "e4m3", 111)
    (b, _) = operand((64, 128), "e4m3", 112, "tile")
    qb, sb = b[0][None].expand(E, -1, -1).contiguous(), b[1][None].expand(E, -1, -1).contiguous()
    for o in ([0, 400, 100, -5, 300], [-9, 300, 300, 1 << 30, 7], [250, 0, 300, 0, 300]):
        off = torch.tensor(o, dtype=torch.int32).cuda()
        out = nsg.expert_gemm_fp8(*a, qb, sb, off)
        qt, s = nsg.quantize_fp8_columns(x, off)
        g = nsg.expert_wgrad_fp8(qt, s, qt, s, off)
        plan = nsg.ExpertPlan(off, torch.full((P, 1), 1 << 29, dtype=torch.int32).cuda(), torch.full((P,), P, dtype=torch.int32).cuda())
        assert nsg.expert_dispatch(x, plan).shape == x.shape and not nsg.expert_combine(x, plan).any()
        dy, dw = nsg.expert_combine_backward(x, x, plan)
        assert not dw.any()
        torch.cuda.synchronize()
        assert out.shape == (P, 64) and g.shape == (E, 128, 128) and dy.shape == x.shape


def test_offsets_past_32_bits():
    """Rows beyond 2^32 bytes and 2^31 elements of every large array."""
    T, C = 1_100_000, 4096  # 4.5 GB in 8 bits, 9 GB in bf16
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    last = normal((3, C), "bf16", 120)
    x[-3:] = last.cuda()
    q, s = nsg.quantize_fp8(x)
    eq, es = ref.quantize_rows(last.float().numpy(), "e4m3")
    assert np.array_equal(f64(q[-3:]), eq) and np.array_equal(s[:, -3:].cpu().numpy(), es)
    (b, bv) = operand((64, C), "e4m3", 121, "tile")
    rows = torch.tensor([T - 3, 0, T - 1, T - 2], dtype=torch.int32).cuda()
    off = torch.tensor([0, 4], dtype=torch.int32).cuda()
    out = nsg.expert_gemm_fp8(q, s, b[0][None], b[1][None], off, rows=rows, out_dtype=torch.float32)
    exp = product(ref.values(eq, es), bv)
    check_product(out[[0, 3, 2]], *exp, K=C)
    many = rows.repeat(100)  # as many rows as take the tile kernel
    for dt in (torch.float32, torch.bfloat16):
        tiled = nsg.expert_gemm_fp8(q, s, b[0][None], b[1][None], torch.tensor([0, 400], dtype=torch.int32).cuda(), rows=many,
                                    out_dtype=dt)
        check_product(tiled[[396, 399, 398]], *exp, K=C)
        assert torch.equal(tiled[:4], tiled[396:]) and not tiled[1].any()
    full = nsg.gemm_fp8_nt(q, s, *b, out_dtype=torch.float32)
    check_product(full[-3:], *exp, K=C)
    assert not full[:-3].any()
    del full
    rows_all = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).reshape(T, 1).contiguous()
    turned = nsg.ExpertPlan(torch.tensor([0, T], dtype=torch.int32).cuda(), rows_all, rows)
    for back in (nsg.expert_combine(x, turned), nsg.expert_dispatch(x, turned)):
        assert torch.equal(back[:3].cpu(), last.flip(0)) and not back[3:].any()
        del back


def test_wgrad_of_very_many_rows():
    """More than 2^24 rows: the rows of a tile are over 2^32 bytes apart."""
    P = (1 << 24) + 1000
    o = torch.tensor([0, 300, P - 200, P], dtype=torch.int32).cuda()
    x = torch.zeros((P, 300), dtype=torch.bfloat16, device="cuda")
    ends = normal((500, 300), "bf16", 170)
    x[:300], x[-200:] = ends[:300].cuda(), ends[300:].cuda()
    x[5000] = 1.0
    q, s = nsg.quantize_fp8_columns(x, o)
    del x
    for dt in (torch.float32, torch.bfloat16):
        out = nsg.expert_wgrad_fp8(q[:300], s, q[:300], s, o, out_dtype=dt)
        for e, part in ((0, ends[:300]), (2, ends[300:])):
            eq, es = ref.quantize_columns(part.float().numpy(), [0, len(part)], "e4m3")
            v = ref.values(eq[:, :ref.up128(len(part))], es[:ref.up128(len(part)) // 128])
            check_product(out[e], *product(v, v), K=ref.up128(len(part)))
        # 1 is 448 times the scale 1 / 448, which is rounded (1 + u), once in each operand; the
        # scales' product and the multiply-add round once more: (1 + u)^4, which in bf16 is 1
        assert (out[1].float() - 1).abs().max() <= (5 * U if dt == torch.float32 else 0)


def layer(x, ids, w, W, dout, E):
    """One expert linear layer forward and backward, as a training step runs it."""
    plan = nsg.expert_sort(ids, E)
    xq = nsg.quantize_fp8(x)
    wq, ws, wtq, wts = nsg.quantize_fp8(W, block="tile", transposed=True)
    y = nsg.expert_gemm_fp8(*xq, wq, ws, plan.offsets, rows=plan.tokens)
    out = nsg.expert_combine(y, plan, w)
    dy, dw = nsg.expert_combine_backward(dout, y, plan, w)
    dyq = nsg.quantize_fp8(dy, dtype=torch.float8_e5m2)
    dx = nsg.expert_combine(nsg.expert_gemm_fp8(*dyq, wtq, wts, plan.offsets), plan)
    dyc = nsg.quantize_fp8_columns(dy, plan.offsets, dtype=torch.float8_e5m2)
    xc = nsg.quantize_fp8_columns(x, plan.offsets, rows=plan.tokens)
    dW = nsg.expert_wgrad_fp8(*dyc, *xc, plan.offsets)
    return out, dw, dx, dW


def layer_inputs(T, k, E, N, K, seed):
    ids = choices(T, k, E, seed, drop=0.05)
    return (normal((T, K), "bf16", seed).cuda(), torch.from_numpy(ids).cuda(), torch.softmax(normal((T, k), "f32", seed + 1), 1).cuda(),
            normal((E, N, K), "bf16", seed + 2, 0.05).cuda(), normal((T, N), "bf16", seed + 3, 0.1).cuda())


@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 4, 128, 256), (150, 4, 6, 200, 264)])
def test_layer_and_muon_step(T, k, E, N, K):
    """A step as a whole: the layer's outputs and gradients near those of the fp64
    layer without 8-bit rounding, and muon_step takes its weight gradients.  8-bit
    e4m3 operands are off by 2^-4 relative each at most, e5m2 gradients by 2^-3:
    (1 + 2^-4)(1 + 2^-4) - 1 < 0.13 of the terms' sizes forward, and
    (1 + 2^-3)(1 + 2^-4) - 1 < 0.2 backward, more with what the forward's error
    and bf16 rounding (2^-8, three times) bring."""
    x, ids, w, W, dout = layer_inputs(T, k, E, N, K, 130)
    out, dw, dx, dW = layer(x, ids, w, W, dout, E)
    xv, wv, Wv, dv = f64(x), f64(w), f64(W), f64(dout)
    iv = ids.cpu().numpy()
    e_out, s_out = np.zeros((T, N)), np.zeros((T, N))
    e_dw, s_dw = np.zeros((T, k)), np.zeros((T, k))
    e_dx, s_dx = np.zeros((T, K)), np.zeros((T, K))
    e_dW, s_dW = np.zeros((E, N, K)), np.zeros((E, N, K))
    for t in range(T):
        for j in range(k):
            e = iv[t, j]
            if not 0 <= e < E:
                continue
            y, ys = Wv[e] @ xv[t], np.abs(Wv[e]) @ np.abs(xv[t])
            g = wv[t, j] * dv[t]
            e_out[t] += wv[t, j] * y
            s_out[t] += wv[t, j] * ys
            e_dw[t, j], s_dw[t, j] = dv[t] @ y, np.abs(dv[t]) @ ys
            e_dx[t] += g @ Wv[e]
            s_dx[t] += np.abs(g) @ np.abs(Wv[e])
            e_dW[e] += np.outer(g, xv[t])
            s_dW[e] += np.outer(np.abs(g), np.abs(xv[t]))
    # small elements of a block round to its absolute grid: 2^-10 of the block's largest at most,
    # which the blocks' sizes here (normal values) keep below the terms' own sizes
    fwd, bwd = 0.13 + 3 * 2.0 ** -8, 0.2 + 4 * 2.0 ** -8
    tiny = 1e-6
    assert np.all(np.abs(f64(out) - e_out) <= fwd * s_out + tiny)
    assert np.all(np.abs(f64(dw) - e_dw) <= fwd * s_dw + tiny)
    assert np.all(np.abs(f64(dx) - e_dx) <= bwd * s_dx + tiny)
    assert np.all(np.abs(f64(dW) - e_dW) <= bwd * s_dW + np.max(s_dW) * 2.0 ** -9 + tiny)
    M = torch.zeros((E, N, K), dtype=torch.float32, device="cuda")
    status = torch.ones(E, dtype=torch.int32, device="cuda")
    before = W.clone()
    nsg.muon_step(W, M, dW, mu=0.9, lr=0.02, status=status)
    assert status.tolist() == [0] * E and torch.equal(M, dW.float()) and W.isfinite().all() and not torch.equal(W, before)


def test_layer_twice_is_the_same_bit_for_bit():
    a = layer_inputs(700, 4, 16, 256, 256, 140)
    for p, q in zip(layer(*a, 16), layer(*a, 16)):
        assert torch.equal(p, q)


def test_layer_on_another_stream():
    a = layer_inputs(200, 2, 8, 128, 256, 150)
    exp = layer(*a, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(*a, 8)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(got, exp):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,E", [(2, 8), (900, 64)])
def test_layer_graph_replay(T, E):
    """The whole layer captured once: offsets stay on the device, so one graph
    serves any routing.  Every replay against the eager result, with eager work
    between."""
    k, N, K = 8, 128, 256
    fresh = [layer_inputs(T, k, E, N, K, 160 + 10 * i) for i in range(3)]
    bufs = tuple(t.clone() for t in fresh[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(*bufs, E)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer(*bufs, E)
    for i in range(5):
        for b, f in zip(bufs, fresh[i % 3]):
            b.copy_(f)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, layer(*fresh[i % 3], E)):
            assert torch.equal(p, q), i


# ---------------------------------------------------------------------------
# calls that the documentation allows and that a program may make
# ---------------------------------------------------------------------------
def test_two_layers_at_once():
    """Two layers on two streams that run at the same time, each as alone."""
    jobs = [layer_inputs(900, 4, 16, 256, 256, 210), layer_inputs(60, 8, 16, 256, 512, 220)]
    exp = [layer(*a, 16) for a in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*jobs[i], 16))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for p, q in zip(outs, exp[i]):
                assert torch.equal(p, q)


def test_two_graphs_share_a_sort_workspace():
    """The sort's workspace holds nothing between calls: two graphs replayed in turn
    on one stream use one."""
    T, k, E = 5000, 4, 100
    ws = torch.empty(nsg.expert_sort_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    ids = [torch.from_numpy(choices(T, k, E, seed=230 + i)).cuda() for i in range(2)]
    graphs, plans = [], []
    for i in range(2):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            plans.append(nsg.expert_sort(ids[i], E, workspace=ws))
    for n in range(4):
        ws.fill_(0xFF)
        for i in range(2):
            ids[i].copy_(torch.from_numpy(choices(T, k, E, seed=240 + 2 * n + i)))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for got, e in zip(plans[i], ref.expert_sort(ids[i].cpu().numpy(), E)):
                assert np.array_equal(got.cpu().numpy(), e)


def test_one_expert_many_times_in_a_token():
    """The same expert in every choice of a token: each choice has its own row and
    counts on its own, in the sum and in the gradients."""
    T, k, C = 40, 6, 72
    ids = np.repeat(np.arange(T)[:, None] % 3, k, 1)
    p = plan_of(ids, 3)
    x, w = normal((T, C), "f32", 250).cuda(), normal((T, k), "f32", 251).cuda()
    y = nsg.expert_dispatch(x, p)
    got = f64(nsg.expert_combine(y, p, w))
    exp = f64(w).sum(1)[:, None] * f64(x)
    size = np.abs(f64(w)).sum(1)[:, None] * np.abs(f64(x))
    assert np.all(np.abs(got - exp) <= (2 * k + 1) * U * size)
    dy, dw = nsg.expert_combine_backward(x, y, p, w)
    s = (f64(x) ** 2).sum(1)[:, None]
    assert np.all(np.abs(f64(dw) - s) <= 2 * C * U * s)
    for j in range(k):
        assert torch.equal(dy[p.rows[:, j].long()], w[:, j:j + 1] * x)


# 10 x 16 tiles of 256 x 256, of which one kernel needs 160, and 128 x 128 tiles
@pytest.mark.parametrize("M,N", [(2600, 4100), (1000, 4100)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_large_gemm_nan_stays_in_its_row_and_column(M, N, out):
    x, w = normal((M, 200), "bf16", 260).cuda(), normal((N, 200), "bf16", 261).cuda()
    clean = nsg.gemm_fp8_nt(*nsg.quantize_fp8(x), *nsg.quantize_fp8(w), out_dtype=DT[out])
    x[M - 1, 199] = float("nan")
    w[N - 1, 3] = float("inf")
    got = nsg.gemm_fp8_nt(*nsg.quantize_fp8(x), *nsg.quantize_fp8(w), out_dtype=DT[out])
    assert got[M - 1].isnan().all() and not got[:, N - 1].isfinite().any()
    assert clean.isfinite().all() and torch.equal(got[:M - 1, :N - 1], clean[:M - 1, :N - 1])


def test_wgrad_of_the_most_rows():
    """2^25 rows of one column, all 1.  An operand's block is 448 times its scale, which
    is rounded (1 + u); a block's 128 equal products are summed exactly, and its
    multiply-add rounds once: 2^18 blocks in order, (2^18 + 4) u of 2^25 in all."""
    P = 1 << 25
    x = torch.ones((P, 1), dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    q = nsg.quantize_fp8_columns(x, o)
    out = nsg.expert_wgrad_fp8(*q, *q, o, out_dtype=torch.float32)
    assert abs(out.item() - P) <= ((1 << 18) + 4) * U * P


# ---------------------------------------------------------------------------
# refusals of GPU tensors: checked on the host, before any launch
# ---------------------------------------------------------------------------
def test_refusals():
    T, k, E, C = 10, 2, 4, 256
    p = plan_of(choices(T, k, E, seed=270), E)
    x, y = torch.zeros((T, C), device="cuda"), torch.zeros((T * k, C), device="cuda")
    w = torch.zeros((T, k), device="cuda")
    q, s = nsg.quantize_fp8(x)
    W = torch.zeros((E, 64, C), device="cuda")
    wq, ws = nsg.quantize_fp8(W, block="tile")
    c = nsg.quantize_fp8_columns(y, p.offsets)
    wide = torch.zeros((T, k, 2), dtype=torch.int64, device="cuda")
    shifted = torch.zeros(T * C + 16, dtype=torch.uint8, device="cuda")[1:T * C + 1].view(torch.float8_e4m3fn).view(T, C)
    one = torch.zeros((1, C), device="cuda")
    cases = [
        lambda: nsg.expert_sort(wide[..., 0], E),                                  # strided ids
        lambda: nsg.expert_sort(w, E),                                             # ids of floats
        lambda: nsg.expert_sort(wide[..., 0].contiguous(), 0),
        lambda: nsg.expert_sort(wide[..., 0].contiguous(), 1025),
        lambda: nsg.expert_dispatch(one.expand(T, C), p),                          # rows that overlap
        lambda: nsg.expert_dispatch(x.t(), p),
        lambda: nsg.expert_dispatch(y, p),                                         # not the plan's tokens
        lambda: nsg.expert_dispatch(x.double(), p),
        lambda: nsg.expert_dispatch(x, p._replace(offsets=p.offsets.cpu())),
        lambda: nsg.expert_dispatch(x, p._replace(rows=p.rows.long())),
        lambda: nsg.expert_dispatch(x, p._replace(offsets=p.offsets[:0])),
        lambda: nsg.expert_combine(x, p, w),
        lambda: nsg.expert_combine(y, p, w.bfloat16()),
        lambda: nsg.expert_combine(y, p, w.t().contiguous().t()),
        lambda: nsg.expert_combine(y, p, w[:, :1].contiguous()),
        lambda: nsg.expert_combine_backward(x.bfloat16(), y, p, w),                # two dtypes
        lambda: nsg.expert_combine_backward(x[:, :8], y, p, w),
        lambda: nsg.quantize_fp8(x, block="column"),
        lambda: nsg.quantize_fp8(x, transposed=True),
        lambda: nsg.quantize_fp8(x, dtype=torch.bfloat16),
        lambda: nsg.quantize_fp8(W[:, ::2].transpose(0, 1)),                       # batches not behind each other
        lambda: nsg.quantize_fp8_columns(y, p.offsets.long()),
        lambda: nsg.quantize_fp8_columns(y, p.offsets, rows=p.tokens.cpu()),
        lambda: nsg.gemm_fp8_nt(q, s, wq[0], ws),                                  # scales of the batch
        lambda: nsg.gemm_fp8_nt(q, s, wq, ws),
        lambda: nsg.gemm_fp8_nt(q, s.t(), wq[0], ws[0]),
        lambda: nsg.gemm_fp8_nt(q, s.bfloat16(), wq[0], ws[0]),
        lambda: nsg.gemm_fp8_nt(q[:, :128], s[:1], wq[0], ws[0]),                  # a slice of its rows
        lambda: nsg.gemm_fp8_nt(q[:, :128].contiguous(), s[:1], wq[0], ws[0]),     # another K
        lambda: nsg.gemm_fp8_nt(shifted, s, wq[0], ws[0]),                         # not at 16 bytes
        lambda: nsg.gemm_fp8_nt(q, s, wq[0], ws[0], out_dtype=torch.float64),
        lambda: nsg.gemm_fp8_nt(q, s, wq[0], ws[0], out=torch.zeros((64, T), device="cuda")),
        lambda: nsg.expert_gemm_fp8(*nsg.quantize_fp8(torch.zeros((300, C), device="cuda"), block="tile"), wq, ws, p.offsets),
        lambda: nsg.expert_gemm_fp8(q, s, wq, ws, p.offsets[:-1], rows=p.tokens),
        lambda: nsg.expert_gemm_fp8(q, s, wq, ws, p.offsets, rows=p.tokens.long()),
        lambda: nsg.expert_wgrad_fp8(*c, *nsg.quantize_fp8_columns(torch.zeros((300, C), device="cuda"), p.offsets), p.offsets),
        lambda: nsg.expert_wgrad_fp8(q, s, q, s, p.offsets),                       # fewer columns than 128 E
    ]
    for i, call in enumerate(cases):
        with pytest.raises((ValueError, TypeError, nsg.NSGError)):
            call()
            pytest.fail(f"case {i} was not refused")
    torch.cuda.synchronize()


@pytest.mark.parametrize("how", ["row", "tile"])
def test_partly_filled_large_tiles(how):
    """256 x 256 tiles of which an expert's rows, or the last rows and columns of a
    matrix, fill a part: the same bits as each expert's product alone, which takes
    smaller tiles and adds in the same order (above 32 rows; fewer go to the kernel that
    splits K)."""
    E, K, N, P = 40, 264, 1100, 10300
    g = np.random.default_rng(280)
    cuts = np.sort(g.integers(0, P - 77, size=E - 1))
    o = np.concatenate([[0], cuts, [P - 77]])
    x, W = normal((P, K), "bf16", 281).cuda(), normal((E, N, K), "bf16", 282).cuda()
    q, s = nsg.quantize_fp8(x)
    wq, ws = nsg.quantize_fp8(W, block=how)
    out = nsg.expert_gemm_fp8(q, s, wq, ws, torch.from_numpy(o.astype(np.int32)).cuda())
    some = 0
    for e in range(E):
        b, n = o[e], o[e + 1] - o[e]
        if n > 32:
            alone = nsg.gemm_fp8_nt(q[b:b + n].contiguous(), s[:, b:b + n].contiguous(), wq[e], ws[e])
            assert torch.equal(out[b:b + n], alone), e
            some += 1
    assert some > 20 and not out[P - 77:].any()
    whole = nsg.gemm_fp8_nt(q, s, wq[3], ws[3])
    for b in range(0, P, 1000):
        part = nsg.gemm_fp8_nt(q[b:b + 1000].contiguous(), s[:, b:b + 1000].contiguous(), wq[3], ws[3])
        assert torch.equal(whole[b:b + 1000], part)
