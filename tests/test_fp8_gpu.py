"""The e4m3 quantiser and the block-scaled product (gdn_quant_fp8, gdn_gemm_fp8).

The quantiser's bytes and scales are a function of the values (IEEE fp32 divisions, one
rounding to nearest even) and have to be equal to the plain form's.  The product's terms
are exact; its fp32 sums are off by at most 2^-24 of the sum of absolute values per
addition along the longest path (at most 128 within a block and 64 blocks here, far
fewer in a tree): 2^-17 of the sum of absolute values; a bf16 result by 2^-8 of the value
on top."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def plain_quant(x, block):
    R, C = x.shape
    rb, cb = -(-R // block), -(-C // 128)
    p = torch.zeros(rb * block, cb * 128, device=x.device)
    p[:R, :C] = x.float()
    t = p.view(rb, block, cb, 128)
    amax = torch.clamp(t.abs().amax((1, 3), keepdim=True), min=2.0 ** -64)
    top = torch.full_like(amax, 448.0)
    q = (t * torch.div(top, amax)).to(E4M3).view(rb * block, cb * 128)[:R, :C]
    return q, torch.div(amax, top).view(rb, cb)


def same_bytes(got, want):
    return torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 16), (3, 128), (128, 144), (129, 2064), (257, 112), (1000, 512)])
def test_quant(cuda_device, R, C, dtype, block):
    g = torch.Generator().manual_seed(R + C)
    x = (torch.randn(R, C, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(dtype).to(cuda_device)
    q, scale = gdn.quant_fp8(x, block)
    qr, sr = plain_quant(x, block)
    assert same_bytes(q, qr) and torch.equal(scale, sr)


@pytest.mark.parametrize("block", [1, 128])
def test_quant_edges(cuda_device, block):
    """Zeros, values below the smallest scale, the largest finite values, ties, and a
    strided input and output."""
    wide = torch.zeros(130, 320, device=cuda_device)
    x = wide[:, 16:304]
    x[0] = 0.0
    x[1] = 1e-30
    x[2] = torch.finfo(F32).max
    x[3] = torch.arange(288, device=cuda_device) / 16.0 - 9.0
    x[4, :128] = 448.0 * torch.linspace(-1, 1, 128, device=cuda_device)
    x[129] = -1.5
    q = torch.full((130, 304), 1.0, device=cuda_device).to(E4M3)[:, :288]
    gq, gs = gdn.quant_fp8(x, block, q=q)
    qr, sr = plain_quant(x, block)
    assert gq is q and same_bytes(q, qr) and torch.equal(gs, sr)
    assert bool((q._base.float()[:, 288:] == 1.0).all())


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_quant_not_finite(cuda_device, block, bad):
    """A NaN or an infinity marks its own block only."""
    x = torch.ones(256, 256, device=cuda_device)
    x[5, 7] = bad
    q, s = gdn.quant_fp8(x, block)
    qr, sr = plain_quant(x, block)
    assert torch.equal(torch.isnan(s), torch.isnan(sr)) and torch.equal(torch.isinf(s), torch.isinf(sr))
    ok = torch.isfinite(sr)
    assert int((~ok).sum()) == 1 and torch.equal(s[ok], sr[ok])
    assert torch.isnan(q.float()[5, 7]) and torch.equal(q.float()[128:], qr.float()[128:])


def operands(M, N, K, device, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(device)
    b = (torch.randn(N, K, generator=g) * K ** -0.5).to(device)
    qa, sa = plain_quant(a, 1)
    qb, sb = plain_quant(b, 128)
    return qa.contiguous(), sa, qb.contiguous(), sb


def agree(a, sa, b, sb, c):
    ref, size = so.product(a, sa, b, sb)
    bound = (2.0 ** -8 if c.dtype == BF16 else 0.0) * ref.abs() + 2.0 ** -17 * size + 1e-30
    assert bool(((c.double() - ref).abs() <= bound).all()), float(((c.double() - ref).abs() / bound).max())


SIZES = [(1, 128, 128), (4, 1000, 272), (17, 129, 2064), (33, 640, 1024), (64, 96, 4112), (65, 300, 512),
         (128, 256, 128), (129, 257, 400), (333, 2048, 4112), (700, 1031, 640), (1500, 4000, 256), (2600, 3900, 144),
         (1, 1, 16), (3, 5, 32), (130, 7, 8192)]


@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_gemm(cuda_device, M, N, K, out):
    ops = operands(M, N, K, cuda_device, seed=M + N)
    agree(*ops, gdn.gemm_fp8(*ops, out_dtype=out))
    assert gdn.device_error_status() == (0, 0)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
def test_gemm_strided(cuda_device, M, out):
    """Operands and result inside wider buffers; what lies beside the result stays."""
    a, sa, b, sb = operands(M, 200, 304, cuda_device)
    wa = torch.zeros(M, 384, device=cuda_device).to(E4M3)
    wb = torch.full((200, 320), 5.0, device=cuda_device).to(E4M3)
    wa[:, 16:320], wb[:, :304] = a, b
    c = torch.full((M, 211), 3.0, dtype=out, device=cuda_device)
    gdn.gemm_fp8(wa[:, 16:320], sa, wb[:, :304], sb, out=c[:, 5:205])
    agree(a, sa, b, sb, c[:, 5:205])
    assert bool((c[:, :5] == 3).all()) and bool((c[:, 205:] == 3).all())


def test_gemm_scales_far_apart(cuda_device):
    """Blocks whose scales differ by many orders of magnitude, zero scales among them."""
    for M in (8, 200):
        a, sa, b, sb = operands(M, 260, 640, cuda_device)
        sa = sa * torch.tensor([1.0, 1e-20, 1e15, 0.0, 3.0], device=cuda_device)
        sb = sb * torch.tensor([1.0, 1e18, 1e-15, 1.0, 1e-3], device=cuda_device)
        agree(a, sa, b, sb, gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32))


def test_gemm_nan_stays_in_its_row_and_column(cuda_device):
    for M in (40, 200):
        a, sa, b, sb = operands(M, 300, 256, cuda_device)
        want = gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32)
        a.view(torch.uint8)[7, 3] = 0x7F
        b.view(torch.uint8)[11, 200] = 0x7F
        got = gdn.gemm_fp8(a, sa, b, sb, out_dtype=F32)
        bad = torch.zeros(M, 300, dtype=torch.bool, device=cuda_device)
        bad[7], bad[:, 11] = True, True
        assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])


def test_gemm_empty(cuda_device):
    a, sa, b, sb = operands(3, 40, 64, cuda_device)
    assert gdn.gemm_fp8(a[:0], sa[:0], b, sb).shape == (0, 40)
    assert gdn.gemm_fp8(a, sa, b[:0], sb[:0]).shape == (3, 0)


def test_same_inputs_same_bits(cuda_device):
    for M in (16, 333):
        ops = operands(M, 512, 4096, cuda_device)
        first = gdn.gemm_fp8(*ops, out_dtype=F32)
        for _ in range(3):
            assert torch.equal(first, gdn.gemm_fp8(*ops, out_dtype=F32))


def test_layer_of_both(cuda_device):
    """The operators as a layer uses them: 8-bit in-projection, the mixer on its column
    blocks, 8-bit out-projection; a prompt, then single tokens, captured into a graph on
    another stream.  Each step is checked on the inputs that it was given."""
    import test_ssm_gpu as ts
    H, G, P, N, d = 4, 1, 64, 128, 256
    hp, gn = H * P, G * N
    width = 2 * hp + 2 * gn + 8
    g = torch.Generator().manual_seed(3)
    lens = [90, 39]
    params = so.make_inputs(lens, H, G, P, N, BF16, cuda_device, state=False)
    hidden = torch.randn(sum(lens), d, generator=g).to(BF16).to(cuda_device)
    step_in = torch.randn(2, d, generator=g).to(BF16).to(cuda_device)
    w_in = gdn.quant_fp8((torch.randn(width, d, generator=g) * d ** -0.5).to(cuda_device), 128)
    w_out = gdn.quant_fp8((torch.randn(d, hp, generator=g) * hp ** -0.5).to(cuda_device), 128)
    cu = torch.tensor([0, 90, 129], dtype=torch.int32, device=cuda_device)

    def columns(p):
        return {"z": p[:, :hp].unflatten(1, (H, P)), "x": p[:, hp:2 * hp].unflatten(1, (H, P)),
                "B": p[:, 2 * hp:2 * hp + gn].unflatten(1, (G, N)),
                "C": p[:, 2 * hp + gn:2 * hp + 2 * gn].unflatten(1, (G, N)),
                "dt": p[:, 2 * hp + 2 * gn:2 * hp + 2 * gn + H]}

    def layer(x, state):
        qx = gdn.quant_fp8(x)
        proj = gdn.gemm_fp8(*qx, *w_in)
        c = columns(proj)
        if state is None:
            y, S, tail = gdn.ssm_prefill(c["x"], c["B"], c["C"], c["dt"], params["conv_w"], params["A"],
                                         params["b_dt"], conv_b=params["conv_b"], D=params["D"], z=c["z"],
                                         cu_seqlens=cu)
        else:
            S, tail = state
            y = gdn.ssm_decode_step(c["x"], c["B"], c["C"], c["dt"], params["conv_w"], tail, params["A"],
                                    params["b_dt"], S, conv_b=params["conv_b"], D=params["D"], z=c["z"])
        qy = gdn.quant_fp8(y.flatten(1))
        return qx, proj, y, S, tail, qy, gdn.gemm_fp8(*qy, *w_out)

    def run():
        first = layer(hidden, None)
        kept = first[3].clone(), first[4].clone()
        return first, kept, layer(step_in, kept)

    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        first, kept, second = run()
    graph.replay()
    torch.cuda.synchronize()
    for (qx, proj, y, S, tail, qy, out), lengths, S0, hist in ((first, lens, None, None),
                                                               (second, [1, 1], first[3], first[4])):
        agree(*qx, *w_in, proj)
        ref, Sr, tr, ya, Sa = so.batch({**params, **columns(proj), "S0": S0, "hist": hist}, lengths)
        ts.check(y, ref, ya, ts.EBF, ts.EOP)
        ts.check(S, Sr, Sa, name="state")
        assert torch.equal(tail, tr)
        assert same_bytes(qy[0], plain_quant(y.flatten(1), 1)[0])
        agree(*qy, *w_out, out)
    assert gdn.device_error_status() == (0, 0)
