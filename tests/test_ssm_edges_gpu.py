"""The selective state-space mixer at its edges: values that are not finite inside a
sequence, several streams at once, buffers of the caller's own layout, long segmented
prompts in place, and the wait self-test of its pipelines."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn
from test_ssm_gpu import BF16, F32, agree, bounds, check, prefill

pytestmark = pytest.mark.gpu

T, HIT, H, G, P, N = 150, 75, 4, 2, 64, 128
HP, GN = H * P, G * N


def _hit(inp, place, value):
    """One value of token HIT, which lies inside the second chunk of 64."""
    col = {"x": HP + 5, "B": 2 * HP + 7, "C": 2 * HP + GN + 7, "z": 5, "dt": 2 * HP + 2 * GN}[place]
    inp["proj"][HIT, col] = value


def _touched(place):
    """out [T, H, P] and S [H, N, P] elements that the value may reach: by the formulas it
    goes forward in time only, and x, z, dt and B, C each along their own axes."""
    out, S = torch.zeros(T, H, P, dtype=torch.bool), torch.zeros(H, N, P, dtype=torch.bool)
    if place == "x":
        out[HIT:, 0, 5], S[0, :, 5] = True, True
    elif place == "z":
        out[HIT, 0, 5] = True
    elif place == "dt":
        out[HIT:, 0], S[0] = True, True
    elif place == "B":
        out[HIT:, :H // G], S[:H // G, 7] = True, True
    else:
        out[HIT:HIT + 4, :H // G] = True
    return out, S


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("place", ["x", "B", "C", "z", "dt"])
def test_not_finite_goes_where_the_formulas_take_it(cuda_device, dtype, place, value):
    """What the value cannot reach is as accurate as without it; at its own token, where
    the formulas give NaN or an infinity, the result is not finite either."""
    inp = so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=11)
    y, Sr, _, ya, Sa = so.batch(inp, [T])
    _hit(inp, place, value)
    out, S, _ = prefill(inp, [T])
    rel, operands = bounds(dtype, dtype)
    may, may_S = (m.to(cuda_device) for m in _touched(place))
    check(out[~may], y[~may], ya[:, ~may], rel, operands)
    check(S[0][~may_S], Sr[0][~may_S], Sa[:, 0][:, ~may_S], name="state")
    if place == "x" and value != value:
        assert torch.isnan(out[HIT:, 0, 5]).all() and torch.isnan(S[0, 0, :, 5]).all()
    if place == "B" and value != value:
        assert torch.isnan(out[HIT, :H // G]).all() and torch.isnan(S[0, :H // G, 7]).all()
    if place == "dt" and value != value:
        assert torch.isnan(out[HIT:, 0]).all() and torch.isnan(S[0, 0]).all()


@pytest.mark.parametrize("lens,heads", [([2000], 4), ([700, 0, 1500, 64], 2), ([575, 576, 577, 129, 768], 6), ([127, 128, 3000], 40)],
                         ids=["one", "ragged", "multiples", "many_heads"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_long_prompts_in_place(cuda_device, dtype, lens, heads):
    """Few heads, so that the sequence itself is split: state and history in place."""
    inp = so.make_inputs(lens, heads, 1, P, N, dtype, cuda_device, seed=3)
    S0, hist = inp["S0"].clone(), inp["hist"].clone()
    out, S, tail = agree(inp, lens)
    inp["S0"], inp["hist"] = S0, hist
    again, S_in, tail_in = prefill(inp, lens, S_final=S0, conv_tail=hist)
    assert S_in.data_ptr() == S0.data_ptr() and tail_in.data_ptr() == hist.data_ptr()
    assert torch.equal(again, out) and torch.equal(S_in, S) and torch.equal(tail_in, tail)


def test_two_streams_at_once(cuda_device):
    """Calls on two streams do not share their scratch memory."""
    cases = [([900, 300], 4, 21), ([500, 1, 64], 8, 22)]
    made = [(so.make_inputs(lens, h, 1, P, N, BF16, cuda_device, seed=s), lens) for lens, h, s in cases]
    alone = [prefill(i, l) for i, l in made]
    cus = [torch.tensor([0] + list(torch.tensor(l).cumsum(0)), dtype=torch.int32, device=cuda_device) for _, l in made]
    xs = [torch.randn(700, 512, generator=torch.Generator().manual_seed(s)).to(BF16).to(cuda_device) for s in (1, 2)]
    ws = [torch.randn(300, 512, generator=torch.Generator().manual_seed(s)).to(BF16).to(cuda_device) for s in (3, 4)]
    mul = lambda k, s=None: gdn.gemm_fp8(*gdn.quant_fp8(xs[k], stream=s), *gdn.quant_fp8(ws[k], 128, stream=s), stream=s)
    products = [mul(0), mul(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got, got_products = [[], []], [[], []]
    for _ in range(5):
        for k, (i, _) in enumerate(made):
            with torch.cuda.stream(streams[k]):
                got[k].append(gdn.ssm_prefill(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], i["A"], i["b_dt"],
                                              conv_b=i["conv_b"], D=i["D"], z=i["z"], S0=i["S0"],
                                              conv_hist=i["hist"], cu_seqlens=cus[k]))
                got_products[k].append(mul(k))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert all(torch.equal(u, v) for u, v in zip(r, alone[k]))
        assert all(torch.equal(r, products[k]) for r in got_products[k])


@pytest.mark.parametrize("family", [gdn.ERRF_SSM, gdn.ERRF_FP8])
def test_expired_wait_is_reported(cuda_device, family):
    """The pipelines' bounded waits report in their own family; the next call works."""
    gdn.device_error_status(clear=True)
    gdn.selftest_wait_timeout(family, max_polls=1024)
    assert gdn.device_error_status(clear=True) == (5, family)
    lens = [70]
    agree(so.make_inputs(lens, 2, 1, P, N, BF16, cuda_device), lens)
    assert gdn.device_error_status() == (0, 0)
