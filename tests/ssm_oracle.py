"""The selective state-space mixer and the block-scaled product in 64 bits, token by
token and without any of the library's code, shared by their tests.

Beside each result the mixer returns two bounds of the sizes that were added to make it,
the same recurrence on absolute values.  The first takes the activated channels by their
value: a rounding of an operand of the products by a relative e moves the result by at
most e times it.  The second takes them by 1.1 times the sum of absolute values inside
the convolution, c = b + sum_j w_j r_j: fp32 arithmetic gets c to a few 2^-24 of that sum
and not of |c| (the taps may cancel), and SiLU, whose slope is below 1.1, passes the error
on; |SiLU(c)| <= |c| <= the sum, so the second bound covers the first."""
import torch

F64 = torch.float64


def conv(raw, w, b):
    """raw [3 + T, C] -> SiLU of the width-4 causal convolution [T, C], and 1.1 times the
    sum of absolute values inside it."""
    T = raw.shape[0] - 3
    c = sum(raw[j:j + T] * w[:, j] for j in range(4))
    size = sum(raw[j:j + T].abs() * w[:, j].abs() for j in range(4))
    if b is not None:
        c, size = c + b, size + b.abs()
    return c / (1 + torch.exp(-c)), 1.1 * size


def sequence(x, B, C, dt, conv_w, A, b_dt, conv_b, D, z, S0, hist):
    """One sequence: x [T, H, P], B, C [T, G, N], dt [T, H].  Returns out, S, tail and
    the two bounds of sizes for out and S, all float64 (tail in its own dtype)."""
    T, H, P = x.shape
    G, N = B.shape[1:]
    raw_in = torch.cat([x.reshape(T, H * P), B.reshape(T, G * N), C.reshape(T, G * N)], 1)
    if hist is None:
        hist = raw_in.new_zeros(3, raw_in.shape[1])
    rows = torch.cat([hist, raw_in])
    act, act_size = conv(rows.to(F64), conv_w.to(F64), None if conv_b is None else conv_b.to(F64))
    head = torch.arange(H, device=x.device) // (H // G)
    split = lambda t: (t[:, :H * P].reshape(T, H, P), t[:, H * P:H * P + G * N].reshape(T, G, N)[:, head],
                       t[:, H * P + G * N:].reshape(T, G, N)[:, head])
    xh, Bh, Ch = split(act)
    xs, Bs, Cs = split(act_size)
    s = dt.to(F64) + b_dt.to(F64)
    step = torch.clamp(s, min=0) + torch.log1p(torch.exp(-s.abs()))
    a = torch.exp(-torch.exp(A.to(F64)) * step)
    S = torch.zeros(H, N, P, dtype=F64, device=x.device) if S0 is None else S0.to(F64).clone()
    # S and y with their two bounds: value, sizes by value, sizes by the convolution's sum
    S = torch.stack([S, S.abs(), S.abs()])
    X, Bx, Cx = torch.stack([xh, xh.abs(), xs]), torch.stack([Bh, Bh.abs(), Bs]), torch.stack([Ch, Ch.abs(), Cs])
    y = torch.zeros_like(X)
    for t in range(T):
        S = a[t][:, None, None] * S + (step[t][:, None] * Bx[:, t])[..., None] * X[:, t][:, :, None, :]
        y[:, t] = torch.einsum("ihnp,ihn->ihp", S, Cx[:, t])
    if D is not None:
        d = D.to(F64)[:, None]
        y = y + torch.stack([d, d.abs(), d.abs()])[:, None] * X
    if z is not None:
        g = z.to(F64) / (1 + torch.exp(-z.to(F64)))
        y = y * torch.stack([g, g.abs(), g.abs()])
    return y[0], S[0], rows[rows.shape[0] - 3:], y[1:], S[1:]


def batch(inp, lens):
    """Packed sequences of the given lengths; the keys of make_inputs."""
    outs, at = [], 0
    for i, n in enumerate(lens):
        sl = slice(at, at + n)
        pick = lambda k: None if inp[k] is None else inp[k][sl]
        outs.append(sequence(inp["x"][sl], inp["B"][sl], inp["C"][sl], inp["dt"][sl], inp["conv_w"], inp["A"],
                             inp["b_dt"], inp["conv_b"], inp["D"], pick("z"),
                             None if inp["S0"] is None else inp["S0"][i],
                             None if inp["hist"] is None else inp["hist"][i]))
        at += n
    y, S, tail, ya, Sa = zip(*outs)
    return torch.cat(y), torch.stack(S), torch.stack(tail), torch.cat(ya, 1), torch.stack(Sa, 1)


def make_inputs(lens, H, G, P, N, dtype, device, seed=0, gate=True, state=True, bias=True, extra=0):
    """Inputs as column blocks [z | x | B | C | dt] of one projection (strided views);
    `extra` tokens behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(lens) + extra
    hp, gn = H * P, G * N
    width = (2 * hp + 2 * gn + H + 7) // 8 * 8
    proj = torch.randn(rows, width, generator=g).to(dtype).to(device)
    chans = hp + 2 * gn
    rnd = lambda *s: torch.randn(*s, generator=g).to(device)
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)   # 0.001 .. 0.1
    return {"proj": proj, "z": proj[:, :hp].unflatten(1, (H, P)) if gate else None,
            "x": proj[:, hp:2 * hp].unflatten(1, (H, P)),
            "B": proj[:, 2 * hp:2 * hp + gn].unflatten(1, (G, N)),
            "C": proj[:, 2 * hp + gn:2 * hp + 2 * gn].unflatten(1, (G, N)),
            "dt": proj[:, 2 * hp + 2 * gn:2 * hp + 2 * gn + H],
            "conv_w": rnd(chans, 4) * 0.5, "conv_b": rnd(chans) * 0.1 if bias else None,
            "A": torch.log(torch.rand(H, generator=g) * 15 + 1).to(device),
            "b_dt": (step + torch.log(-torch.expm1(-step))).to(device),
            "D": 1 + 0.1 * rnd(H) if bias else None,
            "S0": 0.2 * rnd(len(lens), H, N, P) if state else None,
            "hist": rnd(len(lens), 3, chans).to(dtype) if state else None}


def product(a, a_scale, b, b_scale):
    """sum over 128-blocks of a_scale b_scale (a b^T) in float64, and the same on
    absolute values."""
    M, K = a.shape
    N = b.shape[0]
    cols = torch.arange(N, device=a.device) // 128
    c = torch.zeros(M, N, dtype=F64, device=a.device)
    ca = torch.zeros_like(c)
    for k in range(a_scale.shape[1]):
        u = a[:, 128 * k:128 * (k + 1)].to(F64) * a_scale[:, k:k + 1].to(F64)
        v = b[:, 128 * k:128 * (k + 1)].to(F64) * b_scale[:, k].to(F64)[cols][:, None]
        c += u @ v.t()
        ca += u.abs() @ v.abs().t()
    return c, ca
