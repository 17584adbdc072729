"""The state-space mixer on values far down the negative side, where SiLU is zero to any
precision: x, B, C and the gate from -1e4 to the lowest bf16, on every path, against the
recurrence in 64 bits and against the step.

Tolerances as in test_ssm_gpu, with one size made smaller.  The oracle's second bound takes
an activation by the sum inside its convolution, for SiLU passes that sum's rounding on
with a slope of at most 1.1.  Where SiLU is 0 in 64 bits (below -709) the slope is below
1e-300 and the rounding, a few 2^-24 of the sum, leaves the sum below -700: nothing is
passed on, and the size is 0 there."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn
from test_ssm_gpu import BF16, EBF, F32, agree, bounds, check, prefill

pytestmark = pytest.mark.gpu

T, HIT, H, G, P, N = 100, 70, 4, 2, 64, 128
HP, GN = H * P, G * N
COLS = {"z": slice(0, HP), "x": slice(HP, 2 * HP), "B": slice(2 * HP, 2 * HP + GN),
        "C": slice(2 * HP + GN, 2 * HP + 2 * GN)}
LOWEST = float(torch.finfo(BF16).min)


@pytest.fixture
def flat(monkeypatch):
    plain = so.conv

    def conv(raw, w, b):
        v, size = plain(raw, w, b)
        return v, torch.where(v == 0, 0.0, size)

    monkeypatch.setattr(so, "conv", conv)


def _inputs(dtype, device, places, value, rows=(HIT,)):
    """All taps between 0.1 and 0.25, so that one such value brings the four tokens it
    reaches down without overflow; every third column of the places."""
    inp = so.make_inputs([T], H, G, P, N, dtype, device, seed=31)
    g = torch.Generator().manual_seed(32)
    inp["conv_w"] = (0.1 + 0.15 * torch.rand(HP + 2 * GN, 4, generator=g)).to(device)
    for place in places:
        for r in rows:
            inp["proj"][r, COLS[place]][::3] = value
    return inp


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("value", [-1e4, -1e20, LOWEST])
@pytest.mark.parametrize("places", ["z", "x", "B", "C", "zxBC"])
def test_prefill(cuda_device, flat, dtype, out_dtype, places, value):
    agree(_inputs(dtype, cuda_device, places, value), [T], out_dtype=out_dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [-1e4, -1e20, LOWEST])
@pytest.mark.parametrize("places", ["z", "x", "B", "C", "zxBC"])
def test_step_continues_the_prompt(cuda_device, flat, dtype, places, value):
    """The value in the token that a step takes: the same result as in one prompt."""
    inp = _inputs(dtype, cuda_device, places, value, rows=(T - 1,))
    y, S_ref, tail, ya, Sa = so.batch(inp, [T])
    part = {k: (v[:T - 1] if k in ("x", "B", "C", "dt", "z") else v) for k, v in inp.items()}
    _, S, hist = prefill(part, [T - 1])
    one = slice(T - 1, T)
    out = gdn.ssm_decode_step(inp["x"][one], inp["B"][one], inp["C"][one], inp["dt"][one], inp["conv_w"], hist,
                              inp["A"], inp["b_dt"], S, conv_b=inp["conv_b"], D=inp["D"], z=inp["z"][one])
    whole, S_whole, _ = agree(inp, [T])
    check(out, y[one], ya[:, one], EBF if dtype == BF16 else 0.0)
    check(S, S_ref, Sa, name="state")
    assert torch.equal(hist, tail)
    # where the formula gives zero, both give zero
    gone = y[T - 1] == 0
    assert torch.equal(gone, _gone(places, cuda_device))
    assert bool((whole[T - 1][gone] == 0).all()) and bool((out[0][gone] == 0).all())


def _gone(places, device):
    col = torch.arange(HP, device=device).view(H, P)
    return (col % 3 == 0) if "z" in places else torch.zeros(H, P, dtype=torch.bool, device=device)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_gate_over_its_range(cuda_device, dtype):
    """The gate from -200 to 200, a value a column, and at infinities and NaN."""
    inp = so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=33)
    inp["proj"][:, COLS["z"]] = torch.linspace(-200.0, 200.0, HP, device=cuda_device).to(dtype)
    agree(inp, [T])
    for i, value in enumerate((float("inf"), float("-inf"), float("nan"))):
        inp["proj"][HIT, i] = value
    want = so.batch(inp, [T])[0][HIT, 0, :3]
    for out in (prefill(inp, [T])[0], prefill(inp, [T], out_dtype=F32)[0]):
        assert torch.isinf(out[HIT, 0, 0]) and float(out[HIT, 0, 0]) == float(want[0])
        assert torch.isnan(want[1:]).all() and torch.isnan(out[HIT, 0, 1:3]).all()
