"""The state-space mixer at the largest numbers of sequences and of heads that it takes, and
two captured graphs of it replayed at once.  Tolerances as in test_ssm_gpu."""
import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn
from test_ssm_gpu import BF16, EBF, F32, agree, bounds, check, prefill

pytestmark = pytest.mark.gpu


def _pick(inp, keep, device):
    """The one-token sequences `keep` of a batch of one-token sequences."""
    keep = torch.tensor(keep, device=device)
    return {k: (v[keep] if k in ("x", "B", "C", "dt", "z", "S0", "hist") else v) for k, v in inp.items()}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_most_sequences(cuda_device, dtype):
    """65535 sequences of a token each, prompt and step."""
    n, H, G, P, N = 65535, 2, 1, 64, 64
    inp = so.make_inputs([1] * n, H, G, P, N, dtype, cuda_device, seed=71)
    keep = [0, 1, 511, 512, 513, 32768, n - 2, n - 1]
    some = _pick(inp, keep, cuda_device)
    y, Sr, tail, ya, Sa = so.batch(some, [1] * len(keep))
    rel, operands = bounds(dtype, dtype)
    for cu in (torch.arange(n + 1, dtype=torch.int32, device=cuda_device), None):
        out, S, hist = gdn.ssm_prefill(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], inp["A"], inp["b_dt"],
                                       conv_b=inp["conv_b"], D=inp["D"], z=inp["z"], S0=inp["S0"],
                                       conv_hist=inp["hist"], cu_seqlens=cu, num_seqs=n)
        check(out[keep], y, ya, rel, operands)
        check(S[keep], Sr, Sa, name="state")
        assert torch.equal(hist[keep], tail)
        del out, S, hist
    S, hist = inp["S0"].clone(), inp["hist"].clone()
    out = gdn.ssm_decode_step(inp["x"], inp["B"], inp["C"], inp["dt"], inp["conv_w"], hist, inp["A"], inp["b_dt"], S,
                              conv_b=inp["conv_b"], D=inp["D"], z=inp["z"])
    check(out[keep], y, ya, EBF if dtype == BF16 else 0.0)
    check(S[keep], Sr, Sa, name="state, step")
    assert torch.equal(hist[keep], tail)
    del inp, S, hist, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 65535 // 5])
def test_most_heads(cuda_device, dtype, G):
    """65535 heads of 64, one group and groups of five (an odd number of 64 columns)."""
    H, P, N, lens = 65535, 64, 64, [3, 67]
    inp = so.make_inputs(lens, H, G, P, N, dtype, cuda_device, seed=72, state=False)
    out, S, tail = prefill(inp, lens)
    per = H // G
    cut = lambda t, a, b: t[:, a:b]
    rel, operands = bounds(dtype, dtype)
    hp, gn = H * P, G * N
    for h in (0, 5 * 4321, H - 5):                 # five heads from here, all of one group
        g = h // per
        chan = torch.cat([torch.arange(h * P, (h + 5) * P), hp + torch.arange(g * N, (g + 1) * N),
                          hp + gn + torch.arange(g * N, (g + 1) * N)]).to(cuda_device)
        part = dict(x=cut(inp["x"], h, h + 5), z=cut(inp["z"], h, h + 5), dt=cut(inp["dt"], h, h + 5),
                    B=cut(inp["B"], g, g + 1), C=cut(inp["C"], g, g + 1), conv_w=inp["conv_w"][chan],
                    conv_b=inp["conv_b"][chan], S0=None, hist=None,
                    **{k: inp[k][h:h + 5] for k in ("A", "b_dt", "D")})
        y, Sr, tr, ya, Sa = so.batch(part, lens)
        check(out[:, h:h + 5], y, ya, rel, operands)
        check(S[:, h:h + 5], Sr, Sa, name="state")
        assert torch.equal(tail[:, :, chan], tr)
    del inp, out, S, tail
    torch.cuda.empty_cache()


def test_two_graphs_at_once(cuda_device):
    """Two captured graphs, replayed on two streams at once and again after the first is
    gone: their scratch memory is their own."""
    cases = [([2000], 4, F32, 73), ([1500, 64, 700], 8, BF16, 74), ([900, 300], 4, BF16, 75)]
    made = [(so.make_inputs(lens, h, 1, 64, 128, d, cuda_device, seed=s), lens) for lens, h, d, s in cases]
    want = [prefill(i, lens) for i, lens in made]
    cus = [torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=cuda_device)
           for _, lens in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    graphs, got = [], []
    for (i, _), cu, s in zip(made, cus, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(gdn.ssm_prefill(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], i["A"], i["b_dt"],
                                       conv_b=i["conv_b"], D=i["D"], z=i["z"], S0=i["S0"], conv_hist=i["hist"],
                                       cu_seqlens=cu))
        graphs.append(g)
    for live in ([0, 1, 2], [1, 2]):
        for k in live:
            for t in got[k]:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for k in live:
                with torch.cuda.stream(streams[k]):
                    graphs[k].replay()
        torch.cuda.synchronize()
        for k in live:
            assert all(torch.equal(u, v) for u, v in zip(got[k], want[k]))
        if live[0] == 0:
            graphs[0].reset()
    assert gdn.device_error_status() == (0, 0)
