"""The block-scaled product's two larger tile shapes (128 columns, and pairs of CTAs on 256
x 256) over many K blocks: whole groups of four scales and more, odd counts, a last block of
16, results whose rows bulk stores cannot take, and what the smaller shapes are tested for.
The comment at the shape's choice gives its rule; with 148 SMs the sizes below take
the pairs (300 x 9000: 72 tiles in one wave, 2600 x 3900) and the 128 columns (1500 x 4000,
900 x 5000).  Tolerance as in test_fp8_gpu, whose longest sum is 64 blocks."""
import pytest
import torch

from linear_attention_token_shortconv_b200 import gdn
from test_fp8_gpu import BF16, E4M3, F32, agree, operands

pytestmark = pytest.mark.gpu

PAIRS, WIDE = (300, 9000), (1500, 4000)


@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(300, 9000, 1040), (300, 9000, 2064), (300, 9000, 640), (2600, 3900, 1168),
                                   (1500, 4000, 1040), (1500, 4000, 2064), (900, 5000, 640), (900, 5000, 4112)],
                         ids=lambda v: str(v))
def test_many_blocks(cuda_device, M, N, K, out):
    ops = operands(M, N, K, cuda_device, seed=M + K)
    agree(*ops, gdn.gemm_fp8(*ops, out_dtype=out))
    assert gdn.device_error_status() == (0, 0)


@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N", [PAIRS, WIDE])
def test_strided(cuda_device, M, N, out):
    """Operands and a result inside wider buffers, the result's rows at odd addresses."""
    K = 1168
    a, sa, b, sb = operands(M, N, K, cuda_device, seed=7)
    wa = torch.zeros(M, K + 48, device=cuda_device).to(E4M3)
    wb = torch.full((N, K + 16), 5.0, device=cuda_device).to(E4M3)
    wa[:, 16:K + 16], wb[:, :K] = a, b
    c = torch.full((M, N + 11), 3.0, dtype=out, device=cuda_device)
    gdn.gemm_fp8(wa[:, 16:K + 16], sa, wb[:, :K], sb, out=c[:, 5:N + 5])
    agree(a, sa, b, sb, c[:, 5:N + 5])
    assert bool((c[:, :5] == 3).all()) and bool((c[:, N + 5:] == 3).all())


@pytest.mark.parametrize("M,N", [PAIRS, WIDE])
def test_scales_far_apart(cuda_device, M, N):
    """Blocks whose scales differ by many orders of magnitude, zero scales among them."""
    a, sa, b, sb = operands(M, N, 1168, cuda_device, seed=8)
    one = [1.0, 1e-20, 1e15, 0.0, 3.0, 1e-10, 1e5, 1.0, 0.0, 7.0]
    two = [1.0, 1e18, 1e-15, 1.0, 1e-3, 1e10, 1e-4, 2.0, 1.0, 0.0]
    sa, sb = sa * torch.tensor(one, device=cuda_device), sb * torch.tensor(two, device=cuda_device)
    agree(a, sa, b, sb, gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32))


@pytest.mark.parametrize("M,N", [PAIRS, WIDE])
@pytest.mark.parametrize("k", [3, 600, 1160])
def test_nan_stays_in_its_row_and_column(cuda_device, M, N, k):
    a, sa, b, sb = operands(M, N, 1168, cuda_device, seed=9)
    want = gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32)
    row, col = M - 30, N - 130
    a.view(torch.uint8)[row, k] = 0x7F
    b.view(torch.uint8)[col, k] = 0x7F
    got = gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32)
    bad = torch.zeros(M, N, dtype=torch.bool, device=cuda_device)
    bad[row], bad[:, col] = True, True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("M,N", [PAIRS, WIDE])
def test_same_inputs_same_bits(cuda_device, M, N):
    ops = operands(M, N, 2064, cuda_device, seed=10)
    first = gdn.gemm_fp8(*ops, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(first, gdn.gemm_fp8(*ops, out_dtype=F32))
