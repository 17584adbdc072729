"""Element offsets past 32 bits in every tensor that can have them: what lies behind them
is right and what lies before is not written over."""
import pytest
import torch

from linear_attention_token_shortconv_b200 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _weights(H, P, N, dev, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    return dict(conv_w=rnd(H * P + 2 * N, 4) * 0.5, A=torch.zeros(H, device=dev), b_dt=torch.full((H,), -3.0, device=dev))


def test_prefill(cuda_device):
    """600000 and 100 tokens, 32 heads of 128: x and out have 2.46e9 elements.  The second
    sequence gives the bits that it gives by itself."""
    H, P, N, lens = 32, 128, 64, [600000, 100]
    rows, dev = sum(lens), cuda_device
    w = _weights(H, P, N, dev)
    x = torch.empty(rows, H, P, dtype=BF16, device=dev).normal_()
    B, C = (torch.empty(rows, 1, N, dtype=BF16, device=dev).normal_() for _ in range(2))
    dt = torch.zeros(rows, H, dtype=BF16, device=dev)
    cu = torch.tensor([0, lens[0], rows], dtype=torch.int32, device=dev)
    out, S, tail = gdn.ssm_prefill(x, B, C, dt, **w, cu_seqlens=cu)
    k = lens[0]
    out1, S1, tail1 = gdn.ssm_prefill(x[k:], B[k:], C[k:], dt[k:], **w)
    assert torch.equal(out[k:], out1) and torch.equal(S[1], S1[0]) and torch.equal(tail[1], tail1[0])
    head, _, _ = gdn.ssm_prefill(x[:64], B[:64], C[:64], dt[:64], **w)
    assert torch.equal(out[:64], head) and bool(torch.isfinite(S).all())
    del out, x
    torch.cuda.empty_cache()


def test_decode(cuda_device):
    """4200 sequences of 32 heads of 128, N = 128: the states have 2.2e9 elements."""
    H, P, N, n, dev = 32, 128, 128, 4200, cuda_device
    w = _weights(H, P, N, dev)
    S = torch.empty(n, H, N, P, device=dev).normal_()
    hist = torch.empty(n, 3, H * P + 2 * N, dtype=BF16, device=dev).normal_()
    x = torch.empty(n, H, P, dtype=BF16, device=dev).normal_()
    B, C = (torch.empty(n, 1, N, dtype=BF16, device=dev).normal_() for _ in range(2))
    dt = torch.zeros(n, H, dtype=BF16, device=dev)
    pick = [0, n // 2, n - 1]
    S1, hist1 = S[pick].clone(), hist[pick].clone()
    out = gdn.ssm_decode_step(x, B, C, dt, w["conv_w"], hist, w["A"], w["b_dt"], S)
    out1 = gdn.ssm_decode_step(x[pick], B[pick], C[pick], dt[pick], w["conv_w"], hist1, w["A"], w["b_dt"], S1)
    assert torch.equal(out[pick], out1) and torch.equal(S[pick], S1) and torch.equal(hist[pick], hist1)
    del S
    torch.cuda.empty_cache()


@pytest.mark.parametrize("block", [1, 128])
def test_quant(cuda_device, block):
    """40000 x 65536: 2.6e9 elements."""
    x = torch.empty(40000, 65536, dtype=BF16, device=cuda_device).normal_()
    q, scale = gdn.quant_fp8(x, block)
    for lo in (0, 128 * 200, 39936):
        q1, s1 = gdn.quant_fp8(x[lo:lo + 64] if block == 1 else x[lo:lo + 128], block)
        n = q1.shape[0]
        assert torch.equal(q[lo:lo + n].view(torch.uint8), q1.view(torch.uint8))
        assert torch.equal(scale[lo // block:lo // block + s1.shape[0]], s1)
    del x, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N", [(66000, 40000), (16, 140000000)], ids=["tokens", "features"])
def test_gemm(cuda_device, M, N):
    """2.6e9 and 2.2e9 results (K = 64 and 16); rows and columns of them by themselves."""
    K = 64 if M > 16 else 16
    dev = cuda_device
    mat = lambda r: torch.empty(r, K, device=dev, dtype=BF16).normal_().to(torch.float8_e4m3fn)
    a, b = mat(M), mat(N)
    sa = torch.rand(M, 1, device=dev) + 0.5
    sb = torch.rand(-(-N // 128), 1, device=dev) + 0.5
    c = gdn.gemm_fp8(a, sa, b, sb)
    for r, n in ((0, 0), (M - 1, 0), (0, N - 64), (M - 1, N - 64), (M // 2, N // 128 // 2 * 128)):
        ref = (a[r].double() * sa[r].double()) @ (b[n:n + 64].double() * sb[n // 128].double()).t()
        size = (a[r].double().abs() * sa[r]) @ (b[n:n + 64].double().abs() * sb[n // 128]).t()
        got = c[r, n:n + 64].double()
        # one rounding to bf16, and a few fp32 ones of the scale and the sum of 64 exact products
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size).all())
    del a, b, c
    torch.cuda.empty_cache()
