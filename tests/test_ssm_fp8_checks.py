"""Host-side refusals of the state-space mixer and of the block-scaled product, on the
CPU: the binding refuses tensors the library would misread, and the library refuses bad
arguments before it touches CUDA."""
import ctypes

import pytest
import torch

import ssm_oracle as so
from linear_attention_token_shortconv_b200 import gdn

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
H, G, P, N = 4, 2, 64, 128
CHANS = H * P + 2 * G * N


# ---------------------------------------------------------------- the binding

def _inputs():
    return so.make_inputs([9, 5], H, G, P, N, BF16, "cpu")


def _prefill(i, **kw):
    kw = {**dict(conv_b=i["conv_b"], D=i["D"], z=i["z"], S0=i["S0"], conv_hist=i["hist"],
                 cu_seqlens=torch.tensor([0, 9, 14], dtype=torch.int32)), **kw}
    return gdn.ssm_prefill(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], i["A"], i["b_dt"], **kw)


def _step(i, **kw):
    kw = {**dict(conv_b=i["conv_b"], D=i["D"], z=i["z"]), **kw}
    n = i["x"].shape[0]
    hist = kw.pop("hist", torch.zeros(n, 3, CHANS, dtype=BF16))
    S = kw.pop("S", torch.zeros(n, H, N, P))
    return gdn.ssm_decode_step(i["x"], i["B"], i["C"], i["dt"], i["conv_w"], hist, i["A"], i["b_dt"], S, **kw)


def test_valid_host_tensors_reach_the_device_check():
    """Column blocks of one projection are taken as they are; the device is refused last."""
    for call in (_prefill, _step):
        with pytest.raises(ValueError, match="CUDA device"):
            call(_inputs())
    x = torch.zeros(6, 256, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.quant_fp8(x[:, :128])
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gemm_fp8(x.to(E4M3), torch.ones(6, 2), x.to(E4M3), torch.ones(1, 2))


@pytest.mark.parametrize("key,bad,err,word", [
    ("x", lambda t: t.half(), TypeError, "x"),
    ("x", lambda t: t.flatten(1), ValueError, "x"),
    ("x", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), ValueError, "x"),    # not packed in a token
    ("x", lambda t: t[:1].expand(14, H, P), ValueError, "x"),                            # tokens overlap
    ("B", lambda t: t.float(), TypeError, "B"),
    ("B", lambda t: t[:-1], ValueError, "B"),
    ("C", lambda t: t[:, :1], ValueError, "C"),
    ("C", lambda t: t[:, :, :64], ValueError, "C"),
    ("dt", lambda t: t[:, :2], ValueError, "dt_logit"),
    ("dt", lambda t: t.float(), TypeError, "dt_logit"),
    ("z", lambda t: t[:, :2], ValueError, "z"),
    ("conv_w", lambda t: t[:-1], ValueError, "conv_w"),
    ("conv_w", lambda t: t.to(BF16), TypeError, "conv_w"),
    ("conv_w", lambda t: t.t().contiguous().t(), ValueError, "conv_w"),
    ("conv_b", lambda t: t[:-1], ValueError, "conv_b"),
    ("A", lambda t: t.double(), TypeError, "A"),
    ("b_dt", lambda t: t[:2], ValueError, "b_dt"),
    ("D", lambda t: t.to(BF16), TypeError, "D"),
])
def test_mixer_refuses_bad_tensors(key, bad, err, word):
    i = _inputs()
    i[key] = bad(i[key])
    for call in (_prefill, _step):
        with pytest.raises(err, match=word):
            call(i)


@pytest.mark.parametrize("kw,err,word", [
    (dict(S0=torch.zeros(1, H, N, P)), ValueError, "S0"),
    (dict(S0=torch.zeros(2, H, P, N)), ValueError, "S0"),
    (dict(S_final=torch.zeros(2, H, N, P, dtype=BF16)), TypeError, "S_final"),
    (dict(conv_hist=torch.zeros(2, 3, CHANS)), TypeError, "conv_hist"),
    (dict(conv_tail=torch.zeros(2, 4, CHANS, dtype=BF16)), ValueError, "conv_tail"),
    (dict(cu_seqlens=torch.tensor([0, 9, 14])), TypeError, "cu_seqlens"),
    (dict(out=torch.zeros(14, H, P, dtype=torch.float16)), TypeError, "out"),
    (dict(out=torch.zeros(13, H, P, dtype=BF16)), ValueError, "out"),
    (dict(out=torch.zeros(14, H, 2 * P, dtype=BF16)[:, :, :P]), ValueError, "out"),
])
def test_prefill_refuses_bad_states_and_results(kw, err, word):
    with pytest.raises(err, match=word):
        _prefill(_inputs(), **kw)


def test_step_refuses_bad_states():
    i = _inputs()
    for kw, err, word in ((dict(S=None), ValueError, "S"), (dict(hist=None), ValueError, "conv_hist"),
                          (dict(S=torch.zeros(13, H, N, P)), ValueError, "S"),
                          (dict(S=torch.zeros(14, H, N, P, dtype=BF16)), TypeError, "S"),
                          (dict(S=torch.zeros(14, H, P, N).transpose(2, 3)), ValueError, "S"),
                          (dict(hist=torch.zeros(14, 3, CHANS)), TypeError, "conv_hist")):
        with pytest.raises(err, match=word):
            _step(i, **kw)


def test_quant_refuses_bad_tensors():
    x = torch.zeros(6, 256)
    for args, kw, err, word in (
            ((x.half(),), {}, TypeError, "x"),
            ((x[0],), {}, ValueError, "x"),
            ((x, 64), {}, ValueError, "block_rows"),
            ((x.t(),), {}, ValueError, "x"),
            ((x[:1].expand(6, 256),), {}, ValueError, "x"),
            ((x,), dict(q=torch.zeros(6, 256, dtype=torch.uint8)), TypeError, "q"),
            ((x,), dict(q=torch.zeros(5, 256, dtype=torch.uint8).view(E4M3)), ValueError, "q"),
            ((x,), dict(scale=torch.zeros(6, 3)), ValueError, "scale"),
            ((x,), dict(scale=torch.zeros(2, 6).t()), ValueError, "scale")):
        with pytest.raises(err, match=word):
            gdn.quant_fp8(*args, **kw)


def test_gemm_refuses_bad_tensors():
    a, b = torch.zeros(6, 256, dtype=torch.uint8).view(E4M3), torch.zeros(130, 256, dtype=torch.uint8).view(E4M3)
    sa, sb = torch.ones(6, 2), torch.ones(2, 2)
    for args, kw, err, word in (
            ((a.float(), sa, b, sb), {}, TypeError, "a"),
            ((a, sa, b.float(), sb), {}, TypeError, "b"),
            ((a, sa, b[:, :128], sb), {}, ValueError, "b"),
            ((a[0], sa, b, sb), {}, ValueError, "a"),
            ((a, sa[:, :1], b, sb), {}, ValueError, "a_scale"),
            ((a, sa, b, sb[:1]), {}, ValueError, "b_scale"),
            ((a, sa.double(), b, sb), {}, TypeError, "a_scale"),
            ((a, sa, b, sb), dict(out_dtype=torch.float16), TypeError, "out"),
            ((a, sa, b, sb), dict(out=torch.zeros(6, 129)), ValueError, "out"),
            ((a, sa, b, sb), dict(out=torch.zeros(130, 6).t()), ValueError, "out")):
        with pytest.raises(err, match=word):
            gdn.gemm_fp8(*args, **kw)


# ---------------------------------------------------------------- the library

FAKE = [ctypes.c_void_p(4096 * (i + 1)) for i in range(20)]


@pytest.fixture(scope="module")
def lib():
    from linear_attention_token_shortconv_b200 import build
    build.build()
    return gdn.load()


def _dims(**kw):
    base = dict(num_seqs=2, total_tokens=14, H=H, G=G, P=P, N=N, conv_k=4, in_dtype=1, out_dtype=1)
    return gdn.SsmDims(**{**base, **kw})


DIMS = [
    (dict(num_seqs=0), INVALID), (dict(total_tokens=-1), INVALID), (dict(H=0), INVALID), (dict(G=0), INVALID),
    (dict(G=3), INVALID), (dict(in_dtype=2), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(ld_x=H * P - 8), INVALID), (dict(ld_dt=H - 1), INVALID), (dict(ld_B=-8), INVALID),
    (dict(P=32), UNSUPPORTED), (dict(N=256), UNSUPPORTED), (dict(conv_k=3), UNSUPPORTED),
    (dict(ld_z=(1 << 30) + 8), UNSUPPORTED), (dict(H=65536, G=1), UNSUPPORTED),
    (dict(H=65535, G=65535, P=128), UNSUPPORTED),                        # channels
    (dict(ld_x=H * P + 4), ALIGNMENT), (dict(ld_C=G * N + 1), ALIGNMENT),
    (dict(in_dtype=0, ld_x=H * P + 2), ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", DIMS, ids=[",".join(f"{k}={v}" for k, v in kw.items()) for kw, _ in DIMS])
def test_mixer_dims(lib, kw, status):
    d, n = _dims(**kw), ctypes.c_size_t()
    assert lib.gdn_ssm_prefill_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status
    assert lib.gdn_ssm_prefill(ctypes.byref(d), *FAKE[:16], None) == status
    kw = dict(kw)
    if "num_seqs" not in kw and "total_tokens" not in kw:
        kw.update(num_seqs=2, total_tokens=2)
        assert lib.gdn_ssm_decode_step(ctypes.byref(_dims(**kw)), *FAKE[:13], None) == status


def test_mixer_lengths(lib):
    """Equal lengths have to divide the tokens; a step has one token a sequence."""
    equal = FAKE[:13] + [None] + FAKE[14:16]
    assert lib.gdn_ssm_prefill(ctypes.byref(_dims(total_tokens=15)), *equal, None) == INVALID
    assert lib.gdn_ssm_decode_step(ctypes.byref(_dims()), *FAKE[:13], None) == INVALID
    assert lib.gdn_ssm_decode_step(ctypes.byref(_dims(num_seqs=65536, total_tokens=65536)), *FAKE[:13], None) == UNSUPPORTED
    assert lib.gdn_ssm_prefill(None, *FAKE[:16], None) == INVALID
    assert lib.gdn_ssm_prefill_workspace_size(ctypes.byref(_dims()), None) == INVALID


# x B C dt conv_w conv_b A b_dt D z S0 hist cu out S_final tail
@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 6, 7, 13])
def test_prefill_needs_its_pointers(lib, i):
    args = list(FAKE[:16])
    args[i] = None
    assert lib.gdn_ssm_prefill(ctypes.byref(_dims()), *args, None) == INVALID


@pytest.mark.parametrize("i", range(16))
def test_prefill_alignment(lib, i):
    args = list(FAKE[:16])
    args[i] = ctypes.c_void_p(args[i].value + {3: 1, 6: 2, 7: 2, 8: 2, 12: 2}.get(i, 8))
    assert lib.gdn_ssm_prefill(ctypes.byref(_dims()), *args, None) == ALIGNMENT


# x B C dt conv_w conv_b hist A b_dt D z S out
@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 6, 7, 8, 11, 12])
def test_step_needs_its_pointers(lib, i):
    args = list(FAKE[:13])
    args[i] = None
    assert lib.gdn_ssm_decode_step(ctypes.byref(_dims(total_tokens=2)), *args, None) == INVALID


@pytest.mark.parametrize("i", range(13))
def test_step_alignment(lib, i):
    args = list(FAKE[:13])
    args[i] = ctypes.c_void_p(args[i].value + {3: 1, 7: 2, 8: 2, 9: 2}.get(i, 8))
    assert lib.gdn_ssm_decode_step(ctypes.byref(_dims(total_tokens=2)), *args, None) == ALIGNMENT


def test_workspace_grows_with_the_tokens(lib):
    sizes = [gdn.ssm_prefill_workspace_size(1, t, 32, 1, 64, 128) for t in (0, 64, 4096, 65536)]
    assert sizes == sorted(sizes) and sizes[-1] > sizes[1] > 0
    assert gdn.ssm_prefill_workspace_size(2, 100, 4, 2, 64, 64, F32) >= 100 * (4 * 64 + 2 * 2 * 64) * 4


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), OK), (dict(cols=0), OK), (dict(rows=-1), INVALID), (dict(block=64), INVALID),
    (dict(cols=24), INVALID), (dict(ld_x=240), INVALID), (dict(ld_q=240), INVALID), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(x=ctypes.c_void_p(4104)), ALIGNMENT), (dict(q=ctypes.c_void_p(4104)), ALIGNMENT),
    (dict(scale=ctypes.c_void_p(4098)), ALIGNMENT), (dict(ld_x=258), ALIGNMENT), (dict(ld_q=264), ALIGNMENT),
    (dict(rows=(1 << 31) - 1, cols=256), UNSUPPORTED), (dict(rows=65535 * 128 + 1, block=128), UNSUPPORTED),
], ids=str)
def test_quant_arguments(lib, kw, status):
    a = {**dict(rows=6, cols=256, x=FAKE[0], ld_x=256, dtype=0, block=1, q=FAKE[1], ld_q=256, scale=FAKE[2]), **kw}
    assert lib.gdn_quant_fp8(a["rows"], a["cols"], a["x"], a["ld_x"], a["dtype"], a["block"], a["q"], a["ld_q"],
                             a["scale"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=24), INVALID),
    (dict(lda=240), INVALID), (dict(ldb=240), INVALID), (dict(ldc=129), INVALID), (dict(dtype=3), INVALID),
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID),
    (dict(c=None), INVALID),
    (dict(a=ctypes.c_void_p(4104)), ALIGNMENT), (dict(b=ctypes.c_void_p(4104)), ALIGNMENT),
    (dict(sa=ctypes.c_void_p(4098)), ALIGNMENT), (dict(sb=ctypes.c_void_p(4098)), ALIGNMENT),
    (dict(c=ctypes.c_void_p(4097)), ALIGNMENT), (dict(c=ctypes.c_void_p(4098), dtype=0), ALIGNMENT),
    (dict(lda=264), ALIGNMENT), (dict(ldb=264), ALIGNMENT),
    (dict(M=0x7fffff01), UNSUPPORTED),
], ids=str)
def test_gemm_arguments(lib, kw, status):
    a = {**dict(M=6, N=130, K=256, a=FAKE[0], lda=256, sa=FAKE[1], b=FAKE[2], ldb=256, sb=FAKE[3], c=FAKE[4], ldc=130,
                dtype=1), **kw}
    assert lib.gdn_gemm_fp8(a["M"], a["N"], a["K"], a["a"], a["lda"], a["sa"], a["b"], a["ldb"], a["sb"], a["c"],
                            a["ldc"], a["dtype"], None) == status
