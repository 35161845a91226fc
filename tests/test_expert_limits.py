"""Sizes at the ends of the expert layer's limits that a launch can hold, on the C entry
points.  Without a GPU a call that passes every check ends in a failed launch, with
addresses that nothing follows; with one these calls are not made."""
import pytest
import torch

import newton_schulz_gram_amd as nsg

P16 = 0x10000  # an aligned address that no call may follow
SHAPE, HIP = 3, 5

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch kernels on addresses that are none")


def gemm(batch, M, N, K=128, out=1, block=1):
    return nsg.lib().nsg_gemm_fp8_nt(3, 3, out, batch, M, N, K, P16, P16, 0, P16, P16, block, P16, None)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 128])
@pytest.mark.parametrize("N", [2048, 4096])
@pytest.mark.parametrize("out", [0, 1, 2])
@pytest.mark.parametrize("block", [0, 1])
def test_the_largest_batch_of_few_rows(M, N, out, block):
    """65535 matrices of 2048 or 4096 x 128 are 17 or 34 GB: the kernel for few rows needs
    more threads than a launch has, the tile kernel does not."""
    assert gemm(65535, M, N, out=out, block=block) == HIP


@pytest.mark.parametrize("M,N", [(16, 65536), (1 << 25, 65536)])
def test_more_tiles_than_a_launch_holds(M, N):
    assert gemm(65535, M, N) == SHAPE


def quantize(block, B, R, C=128, ld=None):
    return nsg.lib().nsg_quantize_fp8(P16, 1, B, R, C, C if ld is None else ld, block, 3, P16, P16, None, None, None)


@pytest.mark.parametrize("block,B,R,ld,code", [
    (1, 1, 128 * 65535, None, HIP), (1, 1, 128 * 65535 + 1, None, SHAPE), (0, 1, 1 << 25, None, HIP), (0, 1, (1 << 25) + 1, None, SHAPE),
    (0, 65535, 1048560, None, HIP), (0, 65535, 1048561, None, SHAPE), (0, 32767, 1048561, None, HIP), (1, 65535, 1000, None, HIP),
    (0, 1, 4, 1 << 31, HIP), (0, 1, 4, (1 << 31) + 1, SHAPE),
])
def test_the_documented_limits_of_the_quantisers(block, B, R, ld, code):
    assert quantize(block, B, R, ld=ld) == code
