"""The selective state-space mixer at its edges: values that are not finite inside a
sequence, several streams at once, buffers of the caller's own layout, long segmented
prompts in place, and the wait self-test of its pipelines."""
import os
import subprocess
import sys

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


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("hit", [5, 700, 1990])
def test_not_finite_in_a_long_prompt(cuda_device, dtype, hit):
    """The same where the sequence is cut: NaN in one column of x goes through the segments."""
    T = 2000
    inp = so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=12)
    clean, Sc, _ = prefill(inp, [T])
    inp["proj"][hit, HP + 5] = float("nan")
    out, S, _ = prefill(inp, [T])
    reach = torch.zeros(T, H, P, dtype=torch.bool, device=cuda_device)
    reach[hit:, 0, 5] = True
    assert torch.isnan(out[reach]).all() and torch.isnan(S[0, 0, :, 5]).all()
    near = reach.clone()
    near[:, 0] = True                       # one power of two scales a head's values in a chunk
    assert torch.equal(out[~near], clean[~near])
    # two results of one value: twice its rounding (2^-8), or twice 2^-18 and some
    rel = 2.0 ** -7 if dtype == BF16 else 2.0 ** -16
    size = clean[~reach].float().abs().max()
    assert (out[~reach].float() - clean[~reach].float()).abs().max() <= rel * size
    keep = [c for c in range(P) if c != 5]
    assert torch.equal(S[0, 1:], Sc[0, 1:]) and torch.isfinite(S[0, 0, :, keep]).all()


@pytest.mark.parametrize("lens,heads", [([2000], 4), ([700, 0, 1500, 64], 2), ([575, 576, 577, 129, 768], 6), ([127, 128, 3000], 40),
                                        ([1000, 70, 3000, 1, 500], 40), ([1500, 64, 1400, 5], 72)],
                         ids=["one", "ragged", "multiples", "many_heads", "one_cut_of_five", "two_cut_of_four"])
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


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_long_memory(cuda_device, dtype):
    """Decays within 1e-3 of 1 and the same at every token: rounded to fp32 each would be
    off by up to 2^-25 in the same direction, 5000 of them by 1e-4 of the state."""
    lens = [5000]
    inp = so.make_inputs(lens, H, G, P, N, dtype, cuda_device, seed=13)
    inp["proj"][:, 2 * HP + 2 * GN:] = 0.0
    inp["A"] = torch.tensor([-3.0, -4.3, -5.1, -6.7], device=cuda_device)
    agree(inp, lens)


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


def test_results_belong_to_their_stream(cuda_device):
    """A result that is dropped while its stream may still write it is not handed to work
    of another stream."""
    i = so.make_inputs([300], 4, 1, P, N, BF16, cuda_device)
    x = torch.randn(700, 512, device=cuda_device)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    calls = [lambda: gdn.quant_fp8(x, stream=s),
             lambda: (gdn.gemm_fp8(*gdn.quant_fp8(x, stream=s), *gdn.quant_fp8(x, 128, stream=s), stream=s),),
             lambda: gdn.ssm_prefill(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], i["A"], i["b_dt"], stream=s),
             lambda: (gdn.ssm_decode_step(i["x"], i["B"], i["C"], i["dt"], i["conv_w"],
                                          i["x"].new_zeros(300, 3, i["conv_w"].shape[0]), i["A"], i["b_dt"],
                                          torch.zeros(300, 4, N, P, device=cuda_device), stream=s),)]
    for call in calls:
        torch.cuda.synchronize()
        results = call()
        kinds = [(r.data_ptr(), r.shape, r.dtype) for r in results]
        del results
        taken = [torch.empty(shape, dtype=dtype, device=cuda_device) for _, shape, dtype in kinds]
        assert not {t.data_ptr() for t in taken} & {p for p, _, _ in kinds}
    torch.cuda.synchronize()


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, "tests")
import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn
dev = torch.device("cuda:0")
ins = [so.make_inputs([700, 300], 4, 1, 64, 128, d, dev) for d in (torch.bfloat16, torch.float32)]
cu = torch.tensor([0, 700, 1000], dtype=torch.int32, device=dev)
one = so.make_inputs([1, 1], 4, 1, 64, 128, torch.bfloat16, dev)
a, b = torch.randn(2048, 512, device=dev), torch.randn(2048, 512, device=dev)
def calls():
    outs = []
    for i in ins:
        outs += gdn.ssm_prefill(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], i["A"], i["b_dt"], conv_b=i["conv_b"],
                                D=i["D"], z=i["z"], S0=i["S0"], conv_hist=i["hist"], cu_seqlens=cu)
    S, hist = one["S0"].clone(), one["hist"].clone()
    outs += [gdn.ssm_decode_step(one["x"], one["B"], one["C"], one["dt"], one["conv_w"], hist, one["A"], one["b_dt"], S), S]
    for rows in (2048, 100, 3):
        outs.append(gdn.gemm_fp8(*gdn.quant_fp8(a[:rows]), *gdn.quant_fp8(b, 128)))
    return outs
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    got = calls()
g.replay()
g.replay()
torch.cuda.synchronize()
for u, v in zip(got, calls()):
    assert torch.equal(u, v)
print("same")
"""


def test_first_calls_of_a_process_captured(cuda_device):
    """What a first call sets up (attributes, the pool, the pairs that fit) needs no call
    outside a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_offsets_out_of_range(cuda_device):
    """Offsets past the tokens, negative or falling are clamped: the sequences that are
    well formed come out right and nothing outside out and the states is written."""
    lens, H = [60, 90, 50], 4
    for dtype in (F32, BF16):
        inp = so.make_inputs(lens, H, 1, P, N, dtype, cuda_device, seed=8)
        clean, Sc, _ = prefill(inp, lens)
        guard = torch.full((3, H, P), 5.0, dtype=dtype, device=cuda_device)
        for cu, whole in (([-7, 60, 150, 4000], [0, 1, 2]), ([0, 60, 40, 200], [0])):
            buf = torch.cat([guard, torch.zeros_like(clean), guard])
            out, S, _ = gdn.ssm_prefill(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], inp["A"], inp["b_dt"],
                                        conv_b=inp["conv_b"], D=inp["D"], z=inp["z"], S0=inp["S0"],
                                        conv_hist=inp["hist"], out=buf[3:-3],
                                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
            assert torch.equal(buf[:3], guard) and torch.equal(buf[-3:], guard)
            for n in whole:
                b, e = sum(lens[:n]), sum(lens[:n + 1])
                assert torch.equal(S[n], Sc[n])
                if len(whole) == 3:
                    assert torch.equal(out[b:e], clean[b:e])
