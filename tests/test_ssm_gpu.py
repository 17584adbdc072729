"""The selective state-space mixer (gdn_ssm_prefill, gdn_ssm_decode_step) against the
recurrence in 64 bits.

Tolerances, per element.  fp32: a result of sums of n fp32 products is off by a few
units of 2^-24 per term of the sum of absolute values; exp, log1p and the divisions by
at most a few more (the decays multiply, each off by about 2^-23).  2^-18 of the sum of
absolute values covers 64 such units; the sum is the oracle's second bound, which counts
what cancels inside the convolution.  A bf16 result is rounded once more: 2^-8 of the
value.  The chunked path of bf16 tensors rounds the operands of the products that make
y to fp16 (2^-11 each): C, the chunk scores and x, or C and the state; with the state's
own error at most 4 of them, so 2^-9 of the oracle's first bound on top.  States are fp32
on every path."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
E32, EBF, EOP = 2.0 ** -18, 2.0 ** -8, 2.0 ** -9


def check(got, ref, sizes, rel=0.0, operands=0.0, name="out"):
    bound = rel * ref.abs() + operands * sizes[0] + E32 * sizes[1] + 1e-30
    bad = (got.to(torch.float64) - ref).abs() > bound
    bad |= ~torch.isfinite(got)
    assert not bad.any(), (name, int(bad.sum()), float(((got.double() - ref).abs() / bound).max()))


def bounds(in_dtype, out_dtype):
    return (EBF if out_dtype == BF16 else 0.0), (EOP if in_dtype == BF16 and out_dtype == BF16 else 0.0)


def prefill(inp, lens=None, **kw):
    cu = None
    if lens is not None:
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=inp["x"].device)
    return gdn.ssm_prefill(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], inp["A"], inp["b_dt"],
                           conv_b=inp["conv_b"], D=inp["D"], z=inp["z"], S0=inp["S0"], conv_hist=inp["hist"],
                           cu_seqlens=cu, **kw)


def agree(inp, lens, out_dtype=None, **kw):
    out_dtype = out_dtype or inp["x"].dtype
    out, S, tail = prefill(inp, lens, out_dtype=out_dtype, **kw)
    y, Sr, tr, ya, Sa = so.batch(inp, lens)
    rel, operands = bounds(inp["x"].dtype, out_dtype)
    check(out[:y.shape[0]], y, ya, rel, operands)
    check(S, Sr, Sa, name="state")
    assert torch.equal(tail, tr)
    return out, S, tail


SHAPES = [  # H, G, P, N
    (2, 1, 64, 128), (4, 2, 64, 64), (3, 3, 128, 128), (5, 1, 64, 128), (2, 2, 128, 64), (6, 2, 64, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("H,G,P,N", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_prefill_shapes(cuda_device, H, G, P, N, dtype):
    """Every head and state size, shared and own groups, an odd number of heads."""
    lens = [70, 129]
    agree(so.make_inputs(lens, H, G, P, N, dtype, cuda_device, seed=H + P), lens)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2], [3], [63], [64], [65], [0, 5, 0, 0, 1, 200, 0], [17, 0, 64, 128, 3, 1, 130]],
                         ids=lambda v: "-".join(map(str, v)))
def test_prefill_lengths(cuda_device, lens, dtype):
    """Lengths around the chunk and the convolution's reach, empty sequences among them."""
    agree(so.make_inputs(lens, 2, 1, 64, 128, dtype, cuda_device, seed=len(lens)), lens)


@pytest.mark.parametrize("gate,state,bias", [(False, False, False), (True, False, False), (False, True, True)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prefill_optional_inputs(cuda_device, dtype, gate, state, bias):
    lens = [100, 41]
    agree(so.make_inputs(lens, 4, 2, 64, 128, dtype, cuda_device, gate=gate, state=state, bias=bias), lens)


def test_prefill_mixed_types(cuda_device):
    lens = [90]
    agree(so.make_inputs(lens, 2, 1, 64, 128, BF16, cuda_device), lens, out_dtype=F32)
    agree(so.make_inputs(lens, 2, 1, 64, 128, F32, cuda_device), lens, out_dtype=BF16)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prefill_long(cuda_device, dtype):
    """One sequence that is split over its length (and its neighbours that are not)."""
    lens = [1500, 10, 700]
    agree(so.make_inputs(lens, 2, 1, 64, 128, dtype, cuda_device, seed=3), lens)


def test_prefill_equal_lengths_need_no_offsets(cuda_device):
    inp = so.make_inputs([70, 70, 70], 2, 1, 64, 64, BF16, cuda_device)
    a = prefill(inp, [70, 70, 70])
    b = prefill(inp, None, num_seqs=3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_behind_the_last_sequence_stay(cuda_device, dtype):
    """Padding rows behind cu[-1] hold NaN: they are not read, and out keeps its values there."""
    lens = [33, 70]
    inp = so.make_inputs(lens, 2, 1, 64, 128, dtype, cuda_device, extra=80)
    inp["proj"][103:] = float("nan")
    out = torch.full((183, 2, 64), 7.0, dtype=dtype, device=cuda_device)
    agree(inp, lens, out=out)
    assert bool((out[103:] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_nan_stays_in_its_sequence(cuda_device, dtype):
    """A sequence of NaN and infinities between two others does not reach them."""
    lens = [37, 20, 90]
    inp = so.make_inputs(lens, 2, 1, 64, 128, dtype, cuda_device, seed=9)
    clean, Sc, _ = prefill(inp, lens)
    inp["proj"][37:57] = float("nan")
    inp["proj"][40:44] = float("inf")
    out, S, _ = prefill(inp, lens)
    keep = [i for i in range(147) if not 37 <= i < 57]
    assert torch.equal(out[keep], clean[keep]) and torch.equal(S[[0, 2]], Sc[[0, 2]])
    assert bool(torch.isnan(S[1]).any())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 30])
def test_prefill_far_from_one(cuda_device, dtype, scale):
    """Values far outside fp16's range: the operands of the chunked path are scaled."""
    lens = [150]
    inp = so.make_inputs(lens, 2, 1, 64, 128, dtype, cuda_device, state=False)
    hp, gn = 128, 128
    inp["conv_b"] = None
    inp["proj"][:, hp:2 * hp] *= scale                       # x
    inp["proj"][:, 2 * hp:2 * hp + gn] *= 1.0 / scale        # B
    agree(inp, lens)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prefill_extreme_steps(cuda_device, dtype):
    """Steps of zero (logit -inf side), of hundreds (the state is forgotten at once), and
    decay rates from none to immediate."""
    lens = [140]
    inp = so.make_inputs(lens, 4, 1, 64, 128, dtype, cuda_device)
    inp["dt"][10:20] = -300.0
    inp["dt"][50:53] = 400.0
    inp["dt"][90] = -30000.0
    inp["A"][0], inp["A"][1] = -40.0, 6.0
    agree(inp, lens)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_pieces_join(cuda_device, dtype):
    """A prompt in two pieces with state and history fed back in place, then single
    tokens, against one run of the whole."""
    T, cut, H, G, P, N = 200, 131, 4, 2, 64, 128
    inp = so.make_inputs([T], H, G, P, N, dtype, cuda_device, seed=5)
    y, S_ref, tail_ref, ya, Sa = so.batch(inp, [T])
    rel, operands = bounds(dtype, dtype)
    S, hist = inp["S0"].clone(), inp["hist"].clone()
    outs = []
    for lo, hi in ((0, cut), (cut, 190)):
        part = {k: (v[lo:hi] if k in ("x", "B", "C", "dt", "z") else v) for k, v in inp.items()}
        part["S0"], part["hist"] = S, hist
        out, S2, h2 = prefill(part, [hi - lo], S_final=S, conv_tail=hist)
        assert S2 is S and h2 is hist
        outs.append(out)
    for t in range(190, T):
        sl = slice(t, t + 1)
        outs.append(gdn.ssm_decode_step(inp["x"][sl], inp["B"][sl], inp["C"][sl], inp["dt"][sl], inp["conv_w"], hist,
                                        inp["A"], inp["b_dt"], S, conv_b=inp["conv_b"], D=inp["D"], z=inp["z"][sl]))
    check(torch.cat(outs), y, ya, rel, operands)
    check(S, S_ref, Sa, name="state")
    assert torch.equal(hist, tail_ref)


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("H,G,P,N", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_decode_step(cuda_device, H, G, P, N, dtype, out_dtype):
    for B in (1, 3, 9):
        inp = so.make_inputs([1] * B, H, G, P, N, dtype, cuda_device, seed=B)
        y, S_ref, tail, ya, Sa = so.batch(inp, [1] * B)
        S, hist = inp["S0"].clone(), inp["hist"].clone()
        out = gdn.ssm_decode_step(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], hist, inp["A"],
                                  inp["b_dt"], S, conv_b=inp["conv_b"], D=inp["D"], z=inp["z"], out_dtype=out_dtype)
        check(out, y, ya, EBF if out_dtype == BF16 else 0.0)
        check(S, S_ref, Sa, name="state")
        assert torch.equal(hist, tail)


def test_decode_optional_inputs(cuda_device):
    inp = so.make_inputs([1, 1], 2, 1, 64, 128, BF16, cuda_device, gate=False, bias=False)
    y, S_ref, tail, ya, Sa = so.batch(inp, [1, 1])
    S, hist = inp["S0"].clone(), inp["hist"].clone()
    out = gdn.ssm_decode_step(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], hist, inp["A"], inp["b_dt"], S)
    check(out, y, ya, EBF)
    check(S, S_ref, Sa, name="state")


def test_streams_and_graphs(cuda_device):
    """Prefill and step on a side stream, and captured into one graph that is replayed on
    new inputs."""
    lens = [80, 50]
    inp = so.make_inputs(lens, 2, 1, 64, 128, BF16, cuda_device, seed=1)
    other = so.make_inputs(lens, 2, 1, 64, 128, BF16, cuda_device, seed=2)
    want = prefill(inp, lens), prefill(other, lens)
    step = lambda i, S, h: gdn.ssm_decode_step(i["x"][:2], i["B"][:2], i["C"][:2], i["dt"][:2], i["conv_w"], h, i["A"],
                                               i["b_dt"], S, conv_b=i["conv_b"], D=i["D"], z=i["z"][:2])
    want_step = []
    for i, w in ((inp, want[0]), (other, want[1])):
        S, h = w[1].clone(), w[2].clone()
        want_step.append((step(i, S, h), S, h))
    live = {k: (v.clone() if v is not None and k != "proj" else v) for k, v in inp.items()}
    live["proj"] = inp["proj"].clone()
    hp, gn = 128, 128
    live.update(z=live["proj"][:, :hp].unflatten(1, (2, 64)), x=live["proj"][:, hp:2 * hp].unflatten(1, (2, 64)),
                B=live["proj"][:, 2 * hp:2 * hp + gn].unflatten(1, (1, 128)),
                C=live["proj"][:, 2 * hp + gn:2 * hp + 2 * gn].unflatten(1, (1, 128)),
                dt=live["proj"][:, 2 * hp + 2 * gn:2 * hp + 2 * gn + 2])
    cu = torch.tensor([0, 80, 130], dtype=torch.int32, device=cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both():
        out, S, tail = gdn.ssm_prefill(live["x"], live["B"], live["C"], live["dt"], live["conv_w"], live["A"],
                                       live["b_dt"], conv_b=live["conv_b"], D=live["D"], z=live["z"], S0=live["S0"],
                                       conv_hist=live["hist"], cu_seqlens=cu)
        return out, step(live, S, tail), S, tail

    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want_step[0][0])
    assert torch.equal(got[2], want_step[0][1]) and torch.equal(got[3], want_step[0][2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = both()
    for k in ("proj", "conv_w", "conv_b", "A", "b_dt", "D", "S0", "hist"):
        live[k].copy_(other[k])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want_step[1][0])
    assert torch.equal(got[2], want_step[1][1]) and torch.equal(got[3], want_step[1][2])
    assert gdn.device_error_status() == (0, 0)


def test_same_inputs_same_bits(cuda_device):
    lens = [300, 64]
    inp = so.make_inputs(lens, 6, 2, 64, 128, BF16, cuda_device)
    first = prefill(inp, lens)
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(first, prefill(inp, lens)))


def test_no_tokens(cuda_device):
    inp = so.make_inputs([0, 0], 2, 1, 64, 128, BF16, cuda_device)
    out, S, tail = prefill(inp, [0, 0])
    assert out.shape == (0, 2, 64) and torch.equal(S, inp["S0"]) and torch.equal(tail, inp["hist"])
