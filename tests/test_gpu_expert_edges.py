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
