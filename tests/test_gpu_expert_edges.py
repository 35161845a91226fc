"""GPU tests of the expert-layer operators at the edges of their ranges."""
import pytest
import torch

import newton_schulz_gram_amd as nsg

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def whole(shape, seed, top=8):
    """Whole numbers -top .. top as e4m3 on the GPU: the products of 8 of them are within
    2^-13 of each other and sums below 2^24, so that every kernel's sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(torch.float32).to(E4M3)


@pytest.mark.parametrize("M,out", [(1, torch.float32), (3, torch.bfloat16)])
def test_the_largest_batch_of_few_rows(M, out):
    """65535 products with matrices of 2048 x 128 (17 GB): more workgroups than a launch of
    the kernel for few rows holds."""
    B, N, some = 65535, 2048, 255
    a, base = whole((B, M, 128), 1), whole((some, N, 128), 2)
    sa = torch.exp2(torch.arange(B, device="cuda") % 5 - 2.0).view(B, 1, 1).expand(B, 1, M).contiguous()
    sb = torch.exp2(torch.arange(N // 128, device="cuda") % 3 - 1.0).expand(B, 1, N // 128).contiguous()
    b = base.view(torch.uint8).repeat(B // some, 1, 1).view(E4M3)
    got = nsg.gemm_fp8_nt(a, sa, b, sb, out_dtype=out)
    assert got.shape == (B, M, N)
    scale = sb[0, 0].repeat_interleave(128).double()
    for r in range(some):
        exp = (a[r::some].double() * sa[r::some].double().transpose(1, 2)).flatten(0, 1) @ base[r].double().t() * scale
        assert torch.equal(got[r::some].flatten(0, 1), exp.to(out)), r


# ---------------------------------------------------------------------------
# empty sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_products_of_rows_without_elements_are_zero(out, block):
    """quantize_fp8 takes rows of no elements; their products are empty sums."""
    x, w = torch.zeros((200, 0), device="cuda"), torch.zeros((3, 140, 0), device="cuda")
    a, b = nsg.quantize_fp8(x), nsg.quantize_fp8(w, block=block)
    assert a[0].shape == (200, 0) and b[0].shape == (3, 140, 0)
    for got, shape in ((nsg.gemm_fp8_nt(*a, b[0][0], b[1][0], out_dtype=out), (200, 140)),
                       (nsg.gemm_fp8_nt(*b, *b, out_dtype=out), (3, 140, 140))):
        assert got.dtype == out and got.shape == shape and not got.any()
    used = torch.full((200, 140), float("nan"), dtype=out, device="cuda")
    assert nsg.gemm_fp8_nt(*a, b[0][0], b[1][0], out=used) is used and not used.any()
    plan = nsg.expert_sort(torch.arange(400, device="cuda").view(200, 2) % 4, 3)
    got = nsg.expert_gemm_fp8(*a, *b, plan.offsets, rows=plan.tokens, out_dtype=out)
    assert got.shape == (400, 140) and not got.any()


def test_expert_product_of_no_tokens_is_zero():
    """Rows that all point past the end of A, which has none."""
    a = nsg.quantize_fp8(torch.zeros((0, 256), device="cuda"))
    b = nsg.quantize_fp8(torch.ones((2, 64, 256), device="cuda"), block="tile")
    offsets = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    got = nsg.expert_gemm_fp8(*a, *b, offsets, rows=torch.tensor([0, 1, -1, 7, 0], dtype=torch.int32, device="cuda"))
    assert got.shape == (5, 64) and not got.any()


# ---------------------------------------------------------------------------
# the order of sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("C", [1, 64, 129, 1000, 2048])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 2), (8, 0), (5, 7)])
def test_gradients_do_not_depend_on_pitch_or_alignment(C, dt, pad, shift):
    """Views whose rows lie apart or start anywhere give the bits of packed rows."""
    T, k, E = 60, 3, 5
    g = torch.Generator(device="cuda").manual_seed(C)
    plan = nsg.expert_sort(torch.randint(-1, E, (T, k), generator=g, device="cuda"), E)
    w = torch.randn((T, k), generator=g, device="cuda")

    def moved(x):
        big = torch.full((x.shape[0] * (C + pad) + shift,), float("nan"), dtype=dt, device="cuda")
        view = big[shift:].view(x.shape[0], C + pad)[:, :C]
        view.copy_(x)
        return view

    dout, y = (torch.randn((n, C), generator=g, device="cuda").to(dt) for n in (T, T * k))
    dy, dw = nsg.expert_combine_backward(dout, y, plan, w)
    for a, b in ((moved(dout), y), (dout, moved(y)), (moved(dout), moved(y))):
        dy2, dw2 = nsg.expert_combine_backward(a, b, plan, w)
        assert torch.equal(dw, dw2) and torch.equal(dy, dy2)
    assert torch.equal(nsg.expert_combine(moved(y), plan, w), nsg.expert_combine(y, plan, w))
    assert torch.equal(nsg.expert_dispatch(moved(dout), plan), nsg.expert_dispatch(dout, plan))


# ---------------------------------------------------------------------------
# whole-line stores: 16-bit outputs whose rows take 16-byte stores, in whole column
# tiles, leave by lanes that swap halves.  Tiles of 256 x 256 are taken from 160 full
# ones on (with experts only from 96 rows per expert on, 192 with row scales), tiles of
# 128 x 128 below that, from 257 of 64 x 64 on.  All sums are exact, so the results are
# the exact ones rounded once, whatever the order.
# ---------------------------------------------------------------------------
def operand(shape, seed, f8, how="row"):
    """An operand [..., R, K] of whole numbers with power-of-two scales, and its values."""
    R, K = shape[-2:]
    q = whole(shape, seed).float().to(f8)
    n = R if how == "row" else -(-R // 128)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = torch.exp2(torch.randint(-1, 2, (*shape[:-2], K // 128, n), generator=g, device="cuda").float())
    each = s if how == "row" else s.repeat_interleave(128, -1)[..., :R]
    return (q, s), q.double() * each.transpose(-1, -2).repeat_interleave(128, -1).double()


# 256 x 256 tiles: 14 matrices with 3 x 4 full ones, and 10 x 16; 128 x 128: the others
@pytest.mark.parametrize("batch,M,N,K", [(1, 901, 1096, 384), (14, 901, 1096, 128), (1, 2601, 4104, 256), (1, 1100, 1024, 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kinds", [("row", "tile"), ("row", "row"), ("tile", "tile")])
def test_whole_line_stores(batch, M, N, K, out, kinds):
    (a, av), (b, bv) = operand((batch, M, K), 10, E4M3, kinds[0]), operand((batch, N, K), 20, E5M2, kinds[1])
    got = nsg.gemm_fp8_nt(*a, *b, out_dtype=out)
    for i in range(batch):
        assert torch.equal(got[i], (av[i] @ bv[i].t()).to(out)), i


def segments(P, E, seed, tail):
    """Offsets of E experts in P rows: odd starts and lengths, an expert without rows,
    `tail` rows behind the last."""
    g = torch.Generator().manual_seed(seed)
    cut = torch.sort(torch.randint(0, P - tail + 1, (E - 1,), generator=g)).values
    cut[1] = cut[0]
    return torch.cat([torch.zeros(1, dtype=torch.long), cut, torch.tensor([P - tail])]).to(torch.int32).cuda()


# 256 x 256 tiles: 40 x 4 full ones; 128 x 128
@pytest.mark.parametrize("P,E", [(10300, 40), (1501, 12)])
@pytest.mark.parametrize("N", [1096, 1024])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("how", ["row", "tile"])
def test_whole_line_stores_of_experts(P, E, N, out, how):
    T, K = 1200, 256
    (a, av), (b, bv) = operand((T, K), 30, E5M2), operand((E, N, K), 40, E4M3, how)
    o = segments(P, E, 50, tail=77)
    g = torch.Generator(device="cuda").manual_seed(60)
    rows = torch.randint(-20, T + 20, (P,), generator=g, device="cuda", dtype=torch.int32)  # some are no rows of A
    got = nsg.expert_gemm_fp8(*a, *b, o, rows=rows, out_dtype=out)
    there = (rows >= 0) & (rows < T)
    x = torch.where(there[:, None], av[rows.clamp(0, T - 1).long()], 0.0)
    for e in range(E):
        s = slice(int(o[e]), int(o[e + 1]))
        assert torch.equal(got[s], (x[s] @ bv[e].t()).to(out)), e
    assert not got[int(o[-1]):].any()


def columns(P, o, C, seed, f8):
    """Columns-layout operand of whole numbers [C, cap] with scales by block, and its values."""
    E = o.numel() - 1
    cap = nsg.fp8_columns(P, E)
    n = o.diff().long().cpu()
    start = torch.cat([torch.zeros(1, dtype=torch.long), ((n + 127) // 128 * 128).cumsum(0)])
    used = torch.zeros(cap, device="cuda")
    for e in range(E):
        used[start[e]:start[e] + n[e]] = 1
    (q, s), _ = operand((C, cap), seed, f8)
    q = (q.float() * used).to(f8)
    return (q, s), q.double() * s.t().repeat_interleave(128, -1).double(), start


# 256 x 256 tiles: 2 x 4 full ones for each of 20 experts; 128 x 128
@pytest.mark.parametrize("P,E", [(3001, 20), (1003, 5)])
@pytest.mark.parametrize("N,K", [(520, 1096), (519, 1024)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_whole_line_stores_of_weight_gradients(P, E, N, K, out):
    o = segments(P, E, 70, tail=0)
    (a, av, start), (b, bv, _) = columns(P, o, N, 80, E5M2), columns(P, o, K, 90, E4M3)
    got = nsg.expert_wgrad_fp8(*a, *b, o, out_dtype=out)
    for e in range(E):
        s = slice(int(start[e]), int(start[e + 1]))
        assert torch.equal(got[e], (av[:, s] @ bv[:, s].t()).to(out)), e


# ---------------------------------------------------------------------------
# operands whose rows lie past 32-bit offsets, in every kernel that takes them
# ---------------------------------------------------------------------------
# T rows of 4096 bytes are 4.5 GB; 256 x 256 tiles: 40 x 4 full ones; 128 x 128
@pytest.mark.parametrize("P,E", [(10300, 40), (1501, 12)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["row", "tile"])
def test_far_rows_of_experts(P, E, out, how):
    T, K, N, some = 1_100_000, 4096, 1096, 500
    (few, fs), fv = operand((2 * some, K), 100, E4M3)
    q = torch.zeros((T, K), dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.ones((K // 128, T), device="cuda")
    at = torch.cat([torch.arange(some), torch.arange(T - some, T)]).cuda()
    q.view(torch.uint8)[at] = few.view(torch.uint8)
    s[:, at] = fs
    (b, bv) = operand((E, N, K), 110, E4M3, how)
    o = segments(P, E, 120, tail=9)
    g = torch.Generator(device="cuda").manual_seed(130)
    pick = torch.randint(0, 2 * some, (P,), generator=g, device="cuda")
    got = nsg.expert_gemm_fp8(q, s, *b, o, rows=at[pick].to(torch.int32), out_dtype=out)
    for e in range(E):
        r = slice(int(o[e]), int(o[e + 1]))
        assert torch.equal(got[r], (fv[pick[r]] @ bv[e].t()).to(out)), e
    assert not got[int(o[-1]):].any()


# rows are P bytes: 256 of them from P = 2^24 on, 128 from 2^25 on are more than 2^32.
# 256 x 256 tiles: 2 x 2 full ones for each of 40 experts; 128 x 128
@pytest.mark.parametrize("P,N,K,out", [((1 << 24) + 1000, 512, 520, torch.bfloat16), (1 << 25, 264, 272, torch.bfloat16),
                                       (1 << 25, 264, 272, torch.float32)])
def test_far_rows_of_weight_gradients(P, N, K, out):
    E, each = 40, 150
    n = torch.full((E,), each)
    n[20] = P - (E - 1) * each  # one expert has nearly all rows, the others lie on both sides
    o = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(torch.int32).cuda()
    cap = nsg.fp8_columns(P, E)
    start = torch.cat([torch.zeros(1, dtype=torch.long), ((n + 127) // 128 * 128).cumsum(0)])
    q = torch.zeros((K, cap), dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.ones((cap // 128, K), device="cuda")
    values = []  # 256 columns of each expert hold numbers: its rows, or its last ones
    for e in range(E):
        (v, vs), _ = operand((K, 256), 140 + e, E4M3)
        v[:, each if e != 20 else 256 - int(-n[e] % 128):] = 0  # columns that are no row
        c = int(start[e]) if e != 20 else int(start[21]) - 256
        q.view(torch.uint8)[:, c:c + 256] = v.view(torch.uint8)
        s[c // 128:c // 128 + 2] = vs
        values.append(v.double() * vs.t().repeat_interleave(128, -1).double())
    qa, sa = q[K - N:], s[:, K - N:].contiguous()
    got = nsg.expert_wgrad_fp8(qa, sa, q, s, o, out_dtype=out)
    for e in range(E):
        assert torch.equal(got[e], (values[e][K - N:] @ values[e].t()).to(out)), e


# ---------------------------------------------------------------------------
# scales whose product is past the largest fp32 number
# ---------------------------------------------------------------------------
def large_block(op, how, exponent, kinds):
    """The operand with the scale 2^exponent in its second block, where row r holds only
    its element 5, kinds[r % len(kinds)]; and its values."""
    q, s = op[0].float(), op[1].clone()
    R = q.shape[-2]
    q[..., 128:256] = 0
    q[..., 133] = torch.tensor(kinds, device="cuda")[torch.arange(R, device="cuda") % len(kinds)]
    s[..., 1, :] = 2.0 ** exponent
    q = q.to(op[0].dtype)
    each = s if how == "row" else s.repeat_interleave(128, -1)[..., :R]
    return (q, s), q.double() * each.transpose(-1, -2).repeat_interleave(128, -1).double()


# 2^-9 is e4m3's smallest number: 2^-18 2^140 is a number, 2^-9 2^140 is infinite
A_KINDS, B_KINDS = (0.0, 2.0 ** -9, 1.0), (0.0, 2.0 ** -9)


# the kernels for few rows, for few tiles, tiles of 128 x 128 and 256 x 256 (16-bit outputs)
@pytest.mark.parametrize("batch,M,N", [(1, 3, 200), (1, 20, 100), (2, 100, 200), (1, 901, 1096), (14, 901, 1096), (14, 901, 1091)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kinds", [("row", "tile"), ("row", "row"), ("tile", "tile")])
def test_scales_with_an_infinite_product(batch, M, N, out, kinds):
    """A block sum of 0 adds nothing and a small one a number, as by the definition,
    although the product of the scales alone is infinite."""
    a, av = large_block(operand((batch, M, 384), 200, E4M3, kinds[0])[0], kinds[0], 70, A_KINDS)
    b, bv = large_block(operand((batch, N, 384), 210, E4M3, kinds[1])[0], kinds[1], 70, B_KINDS)
    got = nsg.gemm_fp8_nt(*a, *b, out_dtype=out)
    for i in range(batch):
        exp = (av[i] @ bv[i].t()).float().to(out)
        assert torch.equal(got[i], exp), i
        assert M < 3 or out == torch.float16 or exp[1, 1] == 2.0 ** 122 and exp[2, 1] == float("inf") and exp[2, 0].isfinite()


@pytest.mark.parametrize("P,E,N", [(9, 3, 100), (300, 4, 200), (1501, 12, 1096), (10300, 40, 1096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["row", "tile"])
def test_scales_of_experts_with_an_infinite_product(P, E, N, out, how):
    T = 1200
    a, av = large_block(operand((T, 384), 220, E4M3)[0], "row", 70, A_KINDS)
    b, bv = large_block(operand((E, N, 384), 230, E4M3, how)[0], how, 70, B_KINDS)
    o = segments(P, E, 240, tail=2)
    g = torch.Generator(device="cuda").manual_seed(250)
    rows = torch.randint(-20, T, (P,), generator=g, device="cuda", dtype=torch.int32)
    got = nsg.expert_gemm_fp8(*a, *b, o, rows=rows, out_dtype=out)
    x = torch.where((rows >= 0)[:, None], av[rows.clamp(min=0).long()], 0.0)
    for e in range(E):
        s = slice(int(o[e]), int(o[e + 1]))
        assert torch.equal(got[s], (x[s] @ bv[e].t()).float().to(out)), e
    assert not got[int(o[-1]):].any()


@pytest.mark.parametrize("E,N,K", [(1, 100, 70), (5, 520, 1096), (20, 520, 1096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_scales_of_weight_gradients_with_an_infinite_product(E, N, K, out):
    P = 384 * E  # three blocks for each expert
    o = (384 * torch.arange(E + 1)).to(torch.int32).cuda()
    (a, _, _), (b, _, _) = columns(P, o, N, 260, E4M3), columns(P, o, K, 270, E4M3)
    got_a, av = zip(*[large_block((a[0][:, c:c + 384], a[1][c // 128:c // 128 + 3]), "row", 70, A_KINDS) for c in range(0, P, 384)])
    got_b, bv = zip(*[large_block((b[0][:, c:c + 384], b[1][c // 128:c // 128 + 3]), "row", 70, B_KINDS) for c in range(0, P, 384)])
    join = lambda whole, parts: (torch.cat([p[0] for p in parts] + [whole[0][:, P:]], 1).contiguous(),  # noqa: E731
                                 torch.cat([p[1] for p in parts] + [whole[1][P // 128:]]))
    got = nsg.expert_wgrad_fp8(*join(a, got_a), *join(b, got_b), o, out_dtype=out)
    for e in range(E):
        assert torch.equal(got[e], (av[e] @ bv[e].t()).float().to(out)), e


@pytest.mark.parametrize("M,N", [(3, 200), (100, 200), (901, 1096)])
def test_infinite_sums_and_nan_are_not_computed_away(M, N):
    """What is infinite or NaN by the definition stays so, also next to such scales."""
    (a, _), (b, _) = operand((M, 384), 280, E4M3), operand((N, 384), 290, E4M3)
    a, av = large_block(a, "row", 70, (1.0, 0.0))
    b, bv = large_block(b, "row", 70, (1.0, -1.0, 0.0))
    a[0][1, 300] = float("nan")
    got = nsg.gemm_fp8_nt(*a, *b, out_dtype=torch.float32)
    exp = (av @ bv.t()).float()
    exp[1] = float("nan")
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), exp.nan_to_num(7.0, 8.0, 9.0))
    assert exp[0, 0] == float("inf") and exp[0, 1] == -float("inf") and exp[0, 2].isfinite()


@pytest.mark.parametrize("M,N", [(3, 200), (100, 200), (901, 1096)])
@pytest.mark.parametrize("f8", [E4M3, E5M2])
def test_scales_with_a_subnormal_product(M, N, f8):
    """sa sb is rounded to a multiple of 2^-149, so that a block of 128 products adds an
    error of 2^-150 times their sum's size; then one rounding a block."""
    (a, av), (b, bv) = operand((M, 384), 300, f8), operand((N, 384), 310, f8)
    a, b = (a[0], a[1] * 1.37 * 2.0 ** -66), (b[0], b[1] * 1.19 * 2.0 ** -66)
    av, bv = (q.double() * s.double().t().repeat_interleave(128, -1) for q, s in (a, b))
    got = nsg.gemm_fp8_nt(*a, *b, out_dtype=torch.float32).double()
    size = sum((a[0][:, k:k + 128].double() @ b[0][:, k:k + 128].double().t()).abs() for k in range(0, 384, 128))
    exp = av @ bv.t()
    assert torch.all((got - exp).abs() <= size * 2.0 ** -150 * (1 + 2.0 ** -20) + 3 * 2.0 ** -149 + 4 * 2.0 ** -24 * exp.abs())
    assert got.abs().max() > 0


@pytest.mark.parametrize("M,N,batch", [(3, 200, 1), (100, 200, 1), (901, 1096, 1), (901, 1096, 14)])
def test_large_products_that_cancel(M, N, batch):
    """448^2 and -448^2 in different groups of 8 and numbers of 1 beside them.  fp32 outputs
    hold the sum exactly; 16-bit outputs are off by 7 * 2^-13 of the largest product of each
    group at most, then by one rounding (the sum of 14 is a number of both types)."""
    a, b = torch.ones((batch, M, 128), device="cuda"), torch.zeros((batch, N, 128), device="cuda")
    a[..., 0], a[..., 64] = 448, 448
    b[..., 0], b[..., 64] = 448, -448
    b[..., 1:8], b[..., 65:72] = 1, 1
    one = torch.ones((batch, 1, M), device="cuda"), torch.ones((batch, 1, N), device="cuda")
    args = a.to(E4M3), one[0], b.to(E4M3), one[1]
    assert torch.all(nsg.gemm_fp8_nt(*args, out_dtype=torch.float32) == 14)
    bound = 2 * 7 * 2.0 ** -13 * 448 ** 2
    for out in (torch.bfloat16, torch.float16):
        off = (nsg.gemm_fp8_nt(*args, out_dtype=out).double() - 14).abs().max()
        assert off <= bound + torch.finfo(out).eps / 2 * (14 + bound)
