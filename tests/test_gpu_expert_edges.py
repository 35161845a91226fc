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
