"""Tokens of one chunk whose steps and whose B differ by many orders of magnitude: a small
token's own share of y and of the state is as accurate as a large one's wherever the large
one does not reach it, before it comes or after a decay has taken it away.  No skip, no
gate and no state before, so nothing hides that share.  Tolerances as in test_ssm_gpu."""
import pytest
import torch

import ssm_oracle as so
from test_ssm_gpu import BF16, E32, F32, agree, bounds, check, prefill

pytestmark = pytest.mark.gpu


def _inputs(T, dtype, device, P, N, seed):
    return so.make_inputs([T], 4, 2, P, N, dtype, device, seed=seed, gate=False, state=False, bias=False)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("first", [10, 31, 33, 50, 64, 90])
def test_small_steps_before_large_ones(cuda_device, dtype, P, N, first):
    """Steps near 1e-10 in the first tokens, near 1 behind them."""
    inp = _inputs(100, dtype, cuda_device, P, N, seed=61)
    inp["dt"][:first] -= 18.0
    inp["dt"][first:] += 3.0
    agree(inp, [100])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("cut", [10, 30, 40])
def test_small_tokens_behind_a_decay(cuda_device, dtype, P, N, cut):
    """B of 2^-30 from one token on, and then a step so large that all before it is gone:
    what is left of y and of the state is the small tokens'."""
    inp = _inputs(100, dtype, cuda_device, P, N, seed=62)
    hp, gn = 4 * P, 2 * N
    inp["proj"][cut:, 2 * hp:2 * hp + gn] *= 2.0 ** -30
    inp["dt"][cut + 4] = 400.0
    agree(inp, [100])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_of_unlike_size(cuda_device, dtype):
    """B's rows spread over 2^-40 .. 2^40, growing and falling, the steps likewise."""
    T, P, N = 150, 64, 128
    inp = _inputs(T, dtype, cuda_device, P, N, seed=63)
    hp, gn = 4 * P, 2 * N
    e = 40.0 * torch.sin(torch.arange(T, device=cuda_device) / 12.0)
    inp["proj"][:, 2 * hp:2 * hp + gn] *= torch.exp2(e.round())[:, None].to(dtype)
    inp["dt"][:] += (e / 8).to(dtype)[:, None]
    agree(inp, [T])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("at", [3, 40, 70])
def test_large_x_forgotten(cuda_device, dtype, P, N, at):
    """A token whose x is 2^12 times its neighbours', near the documented 2^15, which fast
    decays take away inside the chunk."""
    inp = _inputs(100, dtype, cuda_device, P, N, seed=64)
    hp = 4 * P
    inp["proj"][at, hp:2 * hp] *= 2.0 ** 12
    inp["A"] = torch.full((4,), 5.0, device=cuda_device)
    agree(inp, [100])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 3, 100])
def test_small_elements_of_B(cuda_device, dtype, P, N, T):
    """Every other column of B 2^12 times smaller than its neighbours: their rows of the state
    are as accurate as the others', as far as pairs of fp16 reach.  A row of B has its largest
    in 2^13 .. 2^14 and the pair's second part a least step of 2^-24, so an element is off by
    2^-22 of itself, which test_ssm_gpu's bound holds, or by 2^-25 <= 2^-38 of the row's
    largest.  The largest is at most the row's sum, so the state is off by 2^-38 of its
    sizes' sum over n on top; with B's largest in 8 .. 16 it was 2^-28 of the largest."""
    inp = _inputs(T, dtype, cuda_device, P, N, seed=65)
    hp, gn = 4 * P, 2 * N
    inp["proj"][:, 2 * hp + 1:2 * hp + gn:2] *= 2.0 ** -12
    out, S, _ = prefill(inp, [T])
    y, Sr, _, ya, Sa = so.batch(inp, [T])
    check(out, y, ya, *bounds(dtype, dtype))
    floor = 0.0 if dtype == F32 else 2.0 ** -38 * Sa[0].sum(2, keepdim=True)
    assert bool(((S.double() - Sr).abs() <= E32 * Sa[1] + floor + 1e-30).all())
