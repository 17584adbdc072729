"""A state that holds infinities keeps them: a decay above zero times an infinity is that
infinity, and no other element learns of it."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn
from test_ssm_gpu import BF16, F32, bounds, check, prefill

pytestmark = pytest.mark.gpu

H, G, P, N = 4, 2, 64, 128
INF = float("inf")
SPOTS = [(0, 3, 5, INF), (1, 127, 63, -INF), (3, 64, 0, INF)]


def _slow(inp):
    """Decays of 1e-3 and less a token: none underflows over the prompt."""
    inp["A"] = torch.full((H,), -5.0, device=inp["x"].device)
    for h, n, p, v in SPOTS:
        inp["S0"][0, h, n, p] = v
    return inp


def _columns(device):
    hit = torch.zeros(H, P, dtype=torch.bool, device=device)
    for h, _, p, _ in SPOTS:
        hit[h, p] = True
    return hit


def _same_state(S, Sr, Sa):
    ok = torch.isfinite(Sr)
    assert torch.equal(S[~ok].double(), Sr[~ok]) and int((~ok).sum()) == len(SPOTS)
    check(S[ok], Sr[ok], Sa[:, ok], name="state")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 16, 70, 1500])
def test_prefill(cuda_device, dtype, T):
    inp = _slow(so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=51))
    y, Sr, _, ya, Sa = so.batch(inp, [T])
    out, S, _ = prefill(inp, [T])
    _same_state(S, Sr, Sa)
    hit = _columns(cuda_device)
    rel, operands = bounds(dtype, dtype)
    check(out[:, ~hit], y[:, ~hit], ya[:, :, ~hit], rel, operands)
    assert torch.equal(out[:, hit].double(), y[:, hit])          # infinities, by their sign


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_step(cuda_device, dtype):
    steps = 5
    inp = _slow(so.make_inputs([steps], H, G, P, N, dtype, cuda_device, seed=52))
    y, Sr, tail, ya, Sa = so.batch(inp, [steps])
    S, hist = inp["S0"].clone(), inp["hist"].clone()
    outs = []
    for t in range(steps):
        sl = slice(t, t + 1)
        outs.append(gdn.ssm_decode_step(inp["x"][sl], inp["B"][sl], inp["C"][sl], inp["dt"][sl], inp["conv_w"], hist,
                                        inp["A"], inp["b_dt"], S, conv_b=inp["conv_b"], D=inp["D"], z=inp["z"][sl]))
    _same_state(S, Sr, Sa)
    hit = _columns(cuda_device)
    out = torch.cat(outs)
    check(out[:, ~hit], y[:, ~hit], ya[:, :, ~hit], bounds(dtype, dtype)[0])
    assert torch.equal(out[:, hit].double(), y[:, hit]) and torch.equal(hist, tail)
