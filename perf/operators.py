"""Cases of the selective state-space mixer and the 8-bit projections around it.

Four operators: `prefill` (short causal convolution, selective scan and gate over
packed prompts), `decode` (the same for one token per sequence, state and
convolution history updated in place), `quant` (values to e4m3 with one scale per
block of 128) and `gemm` (the product of two such matrices).  `run` computes each
from elementary torch operations, or with `own` through the package.

The mixer's token tensors are column blocks [z | x | B | C | dt] of one projection
result, as an in-projection leaves them, so they are strided views.
"""
import math

import torch

own = False

CHUNK = 64      # tokens per chunk of the plain chunked scan
FMAX = 448.0    # largest e4m3 value
TINY = 2.0 ** -64


def listed():
    return [
        # the next 37 tokens of a prompt that is already in the state (a chunked prompt, a tool's answer)
        dict(name="prefill continued 37", op="prefill", lens="37", H=32, G=1, P=64, N=128, dtype="bf16", gate=True,
             state=True),
        # a serving batch of ragged prompts, an empty one and a single token among them; B and C shared by 8 heads
        dict(name="prefill ragged batch", op="prefill", lens="2050,1,0,777,64,4095,333,1290", H=64, G=8, P=64, N=128,
             dtype="bf16", gate=True, state=True),
        # the pretraining shape of this repository's layer (d_model 2048): 4 sequences of 4096
        dict(name="prefill 4x4096", op="prefill", lens="4096,4096,4096,4096", H=64, G=1, P=64, N=128, dtype="bf16",
             gate=True, state=False),
        # one long prompt: few heads, so the sequence itself has to be split
        dict(name="prefill 1x32768", op="prefill", lens="32768", H=32, G=1, P=128, N=128, dtype="bf16", gate=True,
             state=False),
        # fp32 end to end, no gate, small state
        dict(name="prefill fp32", op="prefill", lens="1000,999", H=16, G=2, P=64, N=64, dtype="fp32", gate=False,
             state=True),
        # one chat: latency
        dict(name="decode B=1", op="decode", B=1, H=64, G=1, P=64, N=128, dtype="bf16", gate=True),
        # a full serving batch: the states are streamed
        dict(name="decode B=256", op="decode", B=256, H=32, G=1, P=128, N=128, dtype="bf16", gate=True),
        # the layer's activations before a projection
        dict(name="quant rows 16384x2048", op="quant", R=16384, C=2048, block=1, dtype="bf16"),
        # a weight matrix of odd height, once at load
        dict(name="quant tiles 8513x2064", op="quant", R=8513, C=2064, block=128, dtype="fp32"),
        # in-projection for a handful of single tokens: the weights are streamed
        dict(name="gemm M=4", op="gemm", M=4, N=8512, K=2048, out="bf16"),
        # out-projection of a ragged prompt, fp32 result
        dict(name="gemm M=333", op="gemm", M=333, N=2048, K=4112, out="fp32"),
        # in-projection of the pretraining shape
        dict(name="gemm M=16384", op="gemm", M=16384, N=8512, K=2048, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "quant", "gemm", "gemm"])
    if op == "prefill":
        H = rng.choice([8, 12, 16, 24, 32, 64])
        f32 = rng.random() < 0.2
        total = _log(rng, 1, 2048 if f32 else 16384)
        n = min(rng.choice([1, 1, 2, 4, 7]), total)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return dict(op=op, lens=",".join(map(str, lens)), H=H, G=rng.choice([g for g in (1, 2, 4, 8) if H % g == 0]),
                    P=rng.choice([64, 128]), N=rng.choice([64, 128]), dtype="fp32" if f32 else "bf16",
                    gate=rng.random() < 0.7, state=rng.random() < 0.5)
    if op == "decode":
        H = rng.choice([8, 12, 16, 32, 64])
        return dict(op=op, B=_log(rng, 1, 128), H=H, G=rng.choice([g for g in (1, 2, 4, 8) if H % g == 0]),
                    P=rng.choice([64, 128]), N=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    gate=rng.random() < 0.7)
    if op == "quant":
        return dict(op=op, R=_log(rng, 1, 8192), C=16 * _log(rng, 1, 256), block=rng.choice([1, 128]),
                    dtype=rng.choice(["bf16", "fp32"]))
    return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 8192), K=16 * _log(rng, 4, 256),
                out=rng.choice(["bf16", "bf16", "fp32"]))


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _lens(case):
    return [int(s) for s in case["lens"].split(",")]


# --------------------------------------------------------------------- inputs

def _mixer_params(s, gen):
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    chans = H * P + 2 * G * N
    dev = "cuda"
    s["conv_w"] = torch.randn(chans, 4, generator=gen, device=dev) * 0.5
    s["conv_b"] = torch.randn(chans, generator=gen, device=dev) * 0.1
    s["A"] = torch.log(torch.rand(H, generator=gen, device=dev) * 15 + 1)             # decay rates 1 .. 16
    step = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))   # 0.001 .. 0.1
    s["b_dt"] = step + torch.log(-torch.expm1(-step))                                  # softplus(b_dt) = step
    s["D"] = 1 + 0.1 * torch.randn(H, generator=gen, device=dev)
    return chans


def _projection(s, rows, gen, dtype):
    """[z | x | B | C | dt] as the column blocks of one product, rows padded to whole 16 bytes."""
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    width = (2 * H * P + 2 * G * N + H + 7) // 8 * 8
    s["proj"] = torch.randn(rows, width, generator=gen, device="cuda").to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dev = "cuda"
    if case["op"] == "prefill":
        lens = _lens(case)
        dtype = _dtype(case["dtype"])
        chans = _mixer_params(s, gen)
        _projection(s, sum(lens), gen, dtype)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["longest"] = max(lens)
        shape = (len(lens), s["H"], s["N"], s["P"])
        s["S0"] = torch.randn(shape, generator=gen, device=dev) * 0.15 if case["state"] else None
        s["hist"] = torch.randn(len(lens), 3, chans, generator=gen, device=dev).to(dtype) if case["state"] else None
    elif case["op"] == "decode":
        dtype = _dtype(case["dtype"])
        chans = _mixer_params(s, gen)
        _projection(s, s["B"], gen, dtype)
        s["S"] = torch.randn(s["B"], s["H"], s["N"], s["P"], generator=gen, device=dev) * 0.15
        s["hist"] = torch.randn(s["B"], 3, chans, generator=gen, device=dev).to(dtype)
    elif case["op"] == "quant":
        x = torch.randn(s["R"], s["C"], generator=gen, device=dev)
        # rows of unlike size, as activations have them
        x *= torch.exp(torch.randn(s["R"], 1, generator=gen, device=dev))
        s["x"] = x.to(_dtype(case["dtype"]))
    else:
        a = torch.randn(s["M"], s["K"], generator=gen, device=dev)
        a *= torch.exp(torch.randn(s["M"], 1, generator=gen, device=dev))
        b = torch.randn(s["N"], s["K"], generator=gen, device=dev) * s["K"] ** -0.5
        s["a"], s["a_scale"] = _quant(a, 1)
        s["b"], s["b_scale"] = _quant(b, 128)
    return s


# ---------------------------------------------------------------- plain forms

def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _columns(s):
    """z, x, B, C [rows, heads or groups, width] and dt [rows, H] as views of the projection."""
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    p, hp, gn = s["proj"], H * P, G * N
    z = p[:, :hp].unflatten(1, (H, P))
    x = p[:, hp:2 * hp].unflatten(1, (H, P))
    B = p[:, 2 * hp:2 * hp + gn].unflatten(1, (G, N))
    C = p[:, 2 * hp + gn:2 * hp + 2 * gn].unflatten(1, (G, N))
    dt = p[:, 2 * hp + 2 * gn:2 * hp + 2 * gn + H]
    return z if s["gate"] else None, x, B, C, dt


def _conv(s, raw, T):
    """The short convolution of raw [n, 3 + T, channels] with bias, then SiLU."""
    w = s["conv_w"]
    c = raw[:, 0:T] * w[:, 0] + raw[:, 1:T + 1] * w[:, 1] + raw[:, 2:T + 2] * w[:, 2] + raw[:, 3:T + 3] * w[:, 3]
    return _silu(c + s["conv_b"])


def _plain_prefill(s):
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    proj = s["proj"]
    hp, gn, R, Q = H * P, G * N, H // G, CHUNK
    dev = proj.device
    cu = s["cu_seqlens"].long()
    n, T = cu.numel() - 1, s["longest"]
    nc = max(1, -(-T // Q))
    Tp = nc * Q
    # the packed tokens laid out as [sequence, position], zeros behind each end
    pos = torch.arange(Tp, device=dev)
    valid = pos[None] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(valid, cu[:-1, None] + pos[None], 0)
    xbc = proj[:, hp:2 * hp + 2 * gn]
    rows = torch.where(valid[..., None], xbc[at].float(), 0.0)
    hist = s["hist"].float() if s["hist"] is not None else rows.new_zeros(n, 3, hp + 2 * gn)
    raw = torch.cat([hist, rows], 1)
    act = torch.where(valid[..., None], _conv(s, raw, Tp), 0.0)
    x = act[..., :hp].unflatten(2, (H, P))
    B = act[..., hp:hp + gn].unflatten(2, (G, N))
    C = act[..., hp + gn:].unflatten(2, (G, N))
    dt = _softplus(proj[:, 2 * hp + 2 * gn:2 * hp + 2 * gn + H][at].float() + s["b_dt"])
    dt = torch.where(valid[..., None], dt, 0.0)
    # log-decays and their running sums in 64 bits: differences of long sums are exponentiated
    la = (-torch.exp(s["A"].double()) * dt.double()).view(n, nc, Q, H)
    L = torch.cumsum(la, 2)
    total = L[:, :, -1]                                                       # [n, nc, H]
    xc = (x * dt[..., None]).view(n, nc, Q, G, R, P).permute(0, 1, 3, 4, 2, 5)   # [n, nc, G, R, Q, P]
    Bc = B.view(n, nc, Q, G, N).permute(0, 1, 3, 2, 4)                         # [n, nc, G, Q, N]
    Cc = C.view(n, nc, Q, G, N).permute(0, 1, 3, 2, 4)
    Lh = L.permute(0, 1, 3, 2)                                                # [n, nc, H, Q]
    causal = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    seg = torch.where(causal, Lh[..., :, None] - Lh[..., None, :], -math.inf)
    decay = torch.exp(seg.float()).view(n, nc, G, R, Q, Q)
    del seg
    scores = torch.matmul(Cc, Bc.transpose(-1, -2))                            # [n, nc, G, Q, Q]
    y = torch.matmul(scores[:, :, :, None] * decay, xc)                        # within the chunk
    del decay
    # each chunk's own addition to the state, and the state before each chunk
    to_end = torch.exp((total[:, :, None] - L).float()).permute(0, 1, 3, 2).view(n, nc, G, R, Q, 1)
    U = torch.matmul(Bc.transpose(-1, -2)[:, :, :, None], xc * to_end)         # [n, nc, G, R, N, P]
    E = torch.cat([total.new_zeros(n, 1, H), torch.cumsum(total, 1)], 1).permute(0, 2, 1)   # [n, H, nc + 1]
    i = torch.arange(nc + 1, device=dev)
    carry = torch.where(i[:, None] > i[None, :nc], E[:, :, :, None] - E[:, :, None, 1:], -math.inf)
    carry = torch.exp(carry.float())                                           # [n, H, nc + 1, nc]
    Uh = U.reshape(n, nc, H, N * P).permute(0, 2, 1, 3)
    S = torch.matmul(carry, Uh)                                                # [n, H, nc + 1, N P]
    if s["S0"] is not None:
        S = S + torch.exp(E.float())[..., None] * s["S0"].reshape(n, H, 1, N * P)
    S_final = S[:, :, nc].reshape(n, H, N, P)
    Sc = S[:, :, :nc].permute(0, 2, 1, 3).reshape(n, nc, G, R, N, P)
    y = y + torch.exp(Lh.float()).view(n, nc, G, R, Q, 1) * torch.matmul(Cc[:, :, :, None], Sc)
    y = y.permute(0, 1, 4, 2, 3, 5).reshape(n, Tp, H, P) + s["D"][:, None] * x
    if s["gate"]:
        y = y * _silu(proj[:, :hp][at].float().unflatten(2, (H, P)))
    out = torch.empty(proj.shape[0], H, P, dtype=proj.dtype, device=dev)
    out[at[valid]] = y[valid].to(proj.dtype)
    # the last three raw rows of each sequence, older history where it is shorter
    last = (cu[1:] - cu[:-1])[:, None] + torch.arange(3, device=dev)[None]      # rows of `raw`
    tail = torch.gather(raw, 1, last[..., None].expand(n, 3, raw.shape[2])).to(proj.dtype)
    return {"out": out, "state": S_final, "tail": tail}


def _plain_decode(s):
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    proj, S, hist = s["proj"], s["S"], s["hist"]
    hp, gn, R = H * P, G * N, H // G
    raw = torch.cat([hist, proj[:, None, hp:2 * hp + 2 * gn]], 1)
    act = _conv(s, raw.float(), 1)[:, 0]
    x = act[:, :hp].unflatten(1, (H, P))
    B = act[:, hp:hp + gn].unflatten(1, (G, N)).repeat_interleave(R, 1)
    C = act[:, hp + gn:].unflatten(1, (G, N)).repeat_interleave(R, 1)
    dt = _softplus(proj[:, 2 * hp + 2 * gn:2 * hp + 2 * gn + H].float() + s["b_dt"])
    a = torch.exp(-torch.exp(s["A"]) * dt)
    S.mul_(a[..., None, None]).add_((B * dt[..., None])[..., None] * x[..., None, :])
    y = (S * C[..., None]).sum(2) + s["D"][:, None] * x
    if s["gate"]:
        y = y * _silu(proj[:, :hp].float().unflatten(1, (H, P)))
    hist.copy_(raw[:, 1:])
    return {"out": y.to(proj.dtype), "state": S, "hist": hist}


def _quant(x, block):
    """e4m3 values [R, C] and the scale of each 1 x 128 (block 1) or 128 x 128 block."""
    R, C = x.shape
    rb, cb = -(-R // block), -(-C // 128)
    xp = torch.zeros(rb * block, cb * 128, device=x.device)
    xp[:R, :C] = x
    t = xp.view(rb, block, cb, 128)
    amax = torch.clamp(t.abs().amax((1, 3), keepdim=True), min=TINY)
    top = torch.full_like(amax, FMAX)
    q = (t * torch.div(top, amax)).to(torch.float8_e4m3fn).view(rb * block, cb * 128)
    return q[:R, :C].contiguous(), torch.div(amax, top).view(rb, cb)


def _expand(q, scale, block):
    """The values that q and its scales stand for."""
    w = q.float()
    R, C = w.shape
    return w * scale.repeat_interleave(block, 0)[:R].repeat_interleave(128, 1)[:, :C]


def _plain_gemm(s):
    c = torch.matmul(_expand(s["a"], s["a_scale"], 1), _expand(s["b"], s["b_scale"], 128).t())
    return c.to(_dtype(s["out"]))


def run(s):
    op = s["op"]
    if own:
        from linear_attention_token_shortconv_b200 import gdn
        if op == "prefill":
            z, x, B, C, dt = _columns(s)
            out, state, tail = gdn.ssm_prefill(x, B, C, dt, s["conv_w"], s["A"], s["b_dt"], conv_b=s["conv_b"],
                                               D=s["D"], z=z, S0=s["S0"], conv_hist=s["hist"],
                                               cu_seqlens=s["cu_seqlens"])
            return {"out": out, "state": state, "tail": tail}
        if op == "decode":
            z, x, B, C, dt = _columns(s)
            out = gdn.ssm_decode_step(x, B, C, dt, s["conv_w"], s["hist"], s["A"], s["b_dt"], s["S"],
                                      conv_b=s["conv_b"], D=s["D"], z=z)
            return {"out": out, "state": s["S"], "hist": s["hist"]}
        if op == "quant":
            q, scale = gdn.quant_fp8(s["x"], block_rows=s["block"])
            return {"q": q, "scale": scale}
        return gdn.gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=_dtype(s["out"]))
    if op == "prefill":
        return _plain_prefill(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "quant":
        q, scale = _quant(s["x"].float(), s["block"])
        return {"q": q, "scale": scale}
    return _plain_gemm(s)


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "quant":
        el = case["R"] * case["C"]
        scales = -(-case["R"] // case["block"]) * -(-case["C"] // 128)
        return {"bytes": el * (1 + (2 if case["dtype"] == "bf16" else 4)) + 4 * scales, "flops": 3 * el}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        scales = 4 * kb * (M + -(-N // 128))
        return {"bytes": M * K + N * K + scales + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    chans, esz = H * P + 2 * G * N, 2 if case["dtype"] == "bf16" else 4
    params = chans * 20 + 12 * H
    if op == "decode":
        tokens, seqs = case["B"], case["B"]
        states, hist = 2, 2
    else:
        tokens, seqs = sum(_lens(case)), len(_lens(case))
        states, hist = (2, 2) if case["state"] else (1, 1)
    per_token = esz * (chans + H + H * P * (2 if case["gate"] else 1))
    flops = tokens * (9 * chans + H * (5 * N * P + 8 * P))   # the recurrence; the convolution and activations
    return {"bytes": tokens * per_token + seqs * (4 * H * N * P * states + 3 * chans * esz * hist) + params,
            "flops": flops}


# ---------------------------------------------------------------------- exact

def _exact_mixer(s, raw, dt, z, S, lens):
    """The recurrence token by token in 64 bits: raw [n, 3 + T, channels], dt [n, T, H]; S [n, H, N, P]."""
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    T = dt.shape[1]
    w, b = s["conv_w"].double(), s["conv_b"].double()
    c = sum(raw[:, j:j + T] * w[:, j] for j in range(4)) + b
    act = c * torch.sigmoid(c)
    x = act[..., :H * P].reshape(-1, T, H, P)
    head = torch.arange(H, device=dt.device) // (H // G)
    B = act[..., H * P:H * P + G * N].reshape(-1, T, G, N)
    C = act[..., H * P + G * N:].reshape(-1, T, G, N)
    step = torch.nn.functional.softplus(dt + s["b_dt"].double(), threshold=1e6)
    a = torch.exp(-torch.exp(s["A"].double()) * step)
    y = torch.zeros_like(x)
    for t in range(T):
        live = (t < lens)[:, None, None, None]
        new = S * a[:, t, :, None, None] + (B[:, t][:, head] * step[:, t, :, None])[..., None] * x[:, t, :, None, :]
        S = torch.where(live, new, S)
        y[:, t] = torch.einsum("bhnp,bhn->bhp", S, C[:, t][:, head])
    y = y + s["D"].double()[:, None] * x
    return (y if z is None else y * z * torch.sigmoid(z)), S


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x, block = s["x"].double(), case["block"]
        R, C = x.shape
        rows = torch.arange(R, device=x.device) // block
        cols = torch.arange(C, device=x.device) // 128
        cell = (rows[:, None] * (-(-C // 128)) + cols[None]).reshape(-1)
        top = torch.zeros(int(cell[-1]) + 1, dtype=torch.float64, device=x.device)
        top.scatter_reduce_(0, cell, x.abs().reshape(-1), "amax")
        top.clamp_(min=TINY)
        q = (x.reshape(-1) * FMAX / top[cell]).float().view(R, C).to(torch.float8_e4m3fn)
        return {"q": q, "scale": (top / FMAX).view(-(-R // block), -(-C // 128))}
    if op == "gemm":
        a, b, M, N = s["a"].double(), s["b"].double(), case["M"], case["N"]
        c = torch.zeros(M, N, dtype=torch.float64, device=a.device)
        for k in range(s["a_scale"].shape[1]):
            block = slice(128 * k, 128 * (k + 1))
            cols = s["b_scale"][:, k].double()[torch.arange(N, device=a.device) // 128]
            c += (a[:, block] * s["a_scale"][:, k:k + 1].double()) @ (b[:, block] * cols[:, None]).t()
        return c
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    proj = s["proj"].double()
    lo, hi = H * P, 2 * H * P + 2 * G * N
    if op == "decode":
        raw = torch.cat([s["hist"].double(), proj[:, None, lo:hi]], 1)
        z = proj[:, None, :lo].reshape(-1, 1, H, P) if case["gate"] else None
        y, S = _exact_mixer(s, raw, proj[:, None, hi:hi + H], z, s["S"].double(), torch.ones(s["B"], device="cuda"))
        return {"out": y[:, 0], "state": S, "hist": None}
    lens = _lens(case)
    n, T = len(lens), max(lens)
    raw = torch.zeros(n, 3 + T, hi - lo, dtype=torch.float64, device="cuda")
    dt = torch.zeros(n, T, H, dtype=torch.float64, device="cuda")
    z = torch.zeros(n, T, H, P, dtype=torch.float64, device="cuda") if case["gate"] else None
    at = 0
    for i, m in enumerate(lens):
        if s["hist"] is not None:
            raw[i, :3] = s["hist"][i].double()
        raw[i, 3:3 + m] = proj[at:at + m, lo:hi]
        dt[i, :m] = proj[at:at + m, hi:hi + H]
        if z is not None:
            z[i, :m] = proj[at:at + m, :lo].reshape(m, H, P)
        at += m
    S = torch.zeros(n, H, N, P, dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    y, S = _exact_mixer(s, raw, dt, z, S, torch.tensor(lens, device="cuda"))
    return {"out": torch.cat([y[i, :m] for i, m in enumerate(lens)]), "state": S, "tail": None}
