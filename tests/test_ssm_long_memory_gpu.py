"""A state that remembers 32768 tokens.  Equal steps give every token (and every chunk of
64) the same decay, whose rounding to fp32 then adds up instead of cancelling, up to
2^-25 of the state each.  The rates are picked, in 64 bits, where a chunk's decay rounds
worst.

Tolerance.  Two errors add up over a long memory.  (1) The fp32 state is rounded once at
every update, one a token in fp32 and one a chunk on the chunked path.  With random inputs
these are independent: uniform within half a unit, at most 2^-24 of the value, so of a
standard deviation of 2^-24.8; n of them 2^-24.8 sqrt(n) of the values that they are made
on, which are at most 2.2 times the last one (e^0.5 to e^2 of decay, 7.4 at the fastest:
the bound takes 8), and 6 deviations for 32768 elements: 6 * 8 * 2^-24.8 sqrt(n) at most.
The mean over a head's 8192 elements, each by its own sign, has 1 / 90 of that.  (2) The
log-decay as a whole, L <= 2: exp(A) and the step are each off by at most 2^-22 (2 units
of expf, 3 of log1pf and expf), the sum of a chunk's by 2^-22, so 2 * 3 * 2^-22 < 2^-19 of
the state, the same in all elements.  The mean, where (1) is nothing, is held to 2^-19 and
what 6 deviations leave; roundings that add up reach 1.5e-5 = 2^-16 there."""
import math

import pytest
import torch

import ssm_oracle as so
from test_ssm_gpu import BF16, E32, F32, bounds, check, prefill

pytestmark = pytest.mark.gpu

T, H, G, P, N = 32768, 4, 2, 64, 128


def _worst_rates(b_dt):
    """Per head the A, of 400 near the wanted memory, whose decay over 64 equal steps lies
    farthest from fp32."""
    rates = []
    for h, b in enumerate(b_dt.double().tolist()):
        step = math.log1p(math.exp(b))
        near = torch.log(torch.tensor((h + 1) / 2 / 32768 / step, dtype=torch.float64))
        A = (near + torch.arange(400) * 1e-4).float()
        decay = torch.exp(-64 * torch.exp(A.double()) * step)
        off = (decay.float().double() - decay).abs()
        assert off.max() > 0.45 * 2.0 ** -24          # half a unit in the last place is 2^-25
        rates.append(float(A[off.argmax()]))
    return torch.tensor(rates)


def _same_state(S, Sr, Sa, updates, name):
    walk = 6 * 8 * 2.0 ** -24.8 * math.sqrt(updates)
    bad = (S.double() - Sr).abs() > walk * Sr.abs() + E32 * Sa[1]
    assert not bad.any(), (name, int(bad.sum()))
    drift = ((S.double() - Sr) * Sr.sign()).sum((1, 2)) / Sr.abs().sum((1, 2))
    assert bool((drift.abs() <= 2.0 ** -19 + walk / math.sqrt(N * P)).all()), (name, drift.tolist())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_equal_steps(cuda_device, dtype):
    """The state before the prompt is far larger than what the prompt adds, and is still
    there at its end.  Alone the prompt is cut into segments; beside 600 empty sequences
    it is not."""
    inp = so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=41)
    inp["proj"][:, 2 * H * P + 2 * G * N:] = 0.0
    inp["A"] = _worst_rates(inp["b_dt"]).to(cuda_device)
    inp["S0"] *= 5000.0
    y, Sr, tail, ya, Sa = so.batch(inp, [T])
    rel, operands = bounds(dtype, dtype)
    updates = T if dtype == F32 else T // 64
    # y passes the state's error on, relative to the sum of its terms' sizes
    rel_y = operands + 6 * 8 * 2.0 ** -24.8 * math.sqrt(updates)
    empty = 600
    many = dict(inp, S0=torch.cat([inp["S0"], inp["S0"].new_zeros(empty, H, N, P)]),
                hist=torch.cat([inp["hist"], inp["hist"].new_zeros(empty, *inp["hist"].shape[1:])]))
    for name, i, lens in (("cut", inp, [T]), ("whole", many, [T] + [0] * empty)):
        out, S, _ = prefill(i, lens)
        _same_state(S[0], Sr[0], Sa[:, 0], updates, name)
        check(out, y, ya, rel, rel_y, name="out, " + name)
