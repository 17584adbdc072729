"""Results of the block-scaled product inside wider buffers whose rows are whole 16 bytes
apart while the result's own width is not: what lies beside it and behind it stays as it was,
in every tile shape.  Tolerance as in test_fp8_gpu."""
import pytest
import torch

from linear_attention_token_shortconv_b200 import gdn
from test_fp8_gpu import BF16, F32, agree, operands

pytestmark = pytest.mark.gpu


# at most 64 tokens, 64 columns (also with K split), 128 columns, pairs; widths of less than
# 16 bytes, of a tile and one more, and one less than whole 16 bytes
@pytest.mark.parametrize("M,N,K", [(5, 93, 304), (64, 131, 2064), (65, 1, 128), (71, 221, 16), (188, 5, 288),
                                   (130, 257, 4112), (893, 93, 304), (333, 2047, 1040), (1500, 3999, 272),
                                   (900, 4865, 144), (300, 8999, 272), (2600, 3873, 144)], ids=str)
@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
def test_neighbours_stay(cuda_device, M, N, K, out):
    ops = operands(M, N, K, cuda_device, seed=M + N)
    vec = 16 // out.itemsize
    for pad in (-N % vec, -N % vec + vec):
        c = torch.full((M + 2, N + pad), 7.0, dtype=out, device=cuda_device)
        assert c.stride(0) % vec == 0
        gdn.gemm_fp8(*ops, out=c[1:-1, :N])
        agree(*ops, c[1:-1, :N])
        assert bool((c[1:-1, N:] == 7).all()) and bool((c[0] == 7).all()) and bool((c[-1] == 7).all())
    assert gdn.device_error_status() == (0, 0)
