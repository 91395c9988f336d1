"""Plain fp64 forms of the latent attention operators, and their inputs, for the tests.

Everything here is written from the operators' definitions with numpy-like torch operations in 64
bits on the CPU; nothing of the package's arithmetic is used.
"""
import math

import torch

DC, DR, ROW = 512, 64, {0: 1152, 1: 656}
BF16_HALF = 2.0 ** -8          # relative error of a rounding to bf16, at most
F32_STEP = 2.0 ** -23          # a sum's step in fp32, rounded in any direction


def gen(seed):
    return torch.Generator().manual_seed(seed)


def latents(g, T, loud=1.0):
    c = torch.randn(T, DC, generator=g) * loud
    return c.to(torch.bfloat16), torch.randn(T, DR, generator=g).to(torch.bfloat16)


def e4m3_values():
    """The type's 256 values by its definition (1 sign, 4 exponent bits of bias 7, 3 fraction bits)."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if (b & 127) == 127 else (-x if b >= 128 else x))
    return torch.tensor(v, dtype=torch.float64)


def quantise(c):
    """(codes uint8, scale fp64) of latents [T, DC] by trying every code."""
    x = c.double()
    fin = torch.isfinite(x)
    amax = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(dim=1)
    pw = torch.tensor([2.0 ** e for e in range(-117, 120)], dtype=torch.float64)
    s = torch.where(amax > 0, pw[torch.searchsorted(448.0 * pw, amax).clamp_max(len(pw) - 1)], torch.ones_like(amax))
    val = e4m3_values()[:127]                                  # codes 0 .. 126, ascending
    y = (x / s[:, None]).abs().clamp_max(448.0)
    y = torch.where(fin, y, torch.zeros_like(y))
    hi = torch.searchsorted(val, y.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    up, down = val[hi] - y, y - val[lo]
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = code + 128 * torch.signbit(x)
    code = torch.where(fin, code, torch.full_like(code, 127))
    return code.to(torch.uint8), s


def pack(c, r, dtype):
    """Cache rows [T, row bytes] of tokens."""
    if dtype == 0:
        return torch.cat([c, r], dim=1).contiguous().view(torch.uint8)
    code, s = quantise(c)
    rows = torch.zeros(c.shape[0], ROW[1], dtype=torch.uint8)
    rows[:, :DC] = code
    rows[:, DC:DC + 128] = r.contiguous().view(torch.uint8)
    rows[:, DC + 128:DC + 132] = s.float()[:, None].contiguous().view(torch.uint8)
    return rows


def unpack(rows, dtype):
    """fp64 (latents, position keys) of cache rows."""
    if dtype == 0:
        x = rows.contiguous().view(torch.bfloat16).double()
        return x[:, :DC], x[:, DC:]
    s = rows[:, DC + 128:DC + 132].contiguous().view(torch.float32).double()
    return e4m3_values()[rows[:, :DC].long()] * s, rows[:, DC:DC + 128].contiguous().view(torch.bfloat16).double()


def paged(lens, page, dtype, seed, loud=1.0, junk=None):
    """A cache over shuffled pages whose rows past each sequence's end hold `junk` bytes; returns
    (cache [P, page, row], table [N, M], per sequence fp64 (c, r))."""
    g = gen(seed)
    need = [-(-x // page) for x in lens]
    P = sum(need) + 2
    perm = torch.randperm(P, generator=g).to(torch.int32)
    cache = torch.zeros(P, page, ROW[dtype], dtype=torch.uint8)
    if junk is not None:
        cache[:] = junk
    table = torch.full((len(lens), max(max(need), 1) + 1), P + 5, dtype=torch.int32)   # entries past the end: invalid
    at, held = 0, []
    for n, x in enumerate(lens):
        table[n, :need[n]] = perm[at:at + need[n]]
        c, r = latents(g, x, loud)
        rows = pack(c, r, dtype) if x else torch.zeros(0, ROW[dtype], dtype=torch.uint8)
        held.append(unpack(rows, dtype) if x else (torch.zeros(0, DC, dtype=torch.float64), torch.zeros(0, DR, dtype=torch.float64)))
        for i in range(need[n]):
            part = rows[i * page:(i + 1) * page]
            cache[perm[at + i], :part.shape[0]] = part
        at += need[n]
    return cache, table, held


def attend(q, key, val, scale, see):
    """One query row over its first `see` keys: (out, lse, bound) in fp64.  `bound` is the largest
    error that the operator's roundings can make in each output: the result's and the
    probabilities' rounding to bf16, and the fp32 sums of the scores (one step a term, of the sum
    of magnitudes) and of the weighted values (one step a term)."""
    if see <= 0:
        z = torch.zeros(val.shape[1], dtype=torch.float64)
        return z, -math.inf, z, 0.0
    k, v = key[:see], val[:see]
    x = (k @ q) * scale
    lse = torch.logsumexp(x, 0)
    p = torch.exp(x - lse)
    o = p @ v
    dx = float(((k.abs() @ q.abs()) * abs(scale)).max()) * (k.shape[1] + 2) * F32_STEP + 2.0 ** -21   # exp2's and its argument's
    mass = p @ v.abs()
    bound = BF16_HALF * o.abs() + (BF16_HALF + 2 * dx + see * F32_STEP) * mass * (1 + BF16_HALF) + 1e-30
    return o, float(lse), bound, dx + (see + 2) * F32_STEP + abs(float(lse)) * F32_STEP


def check_rows(got, got_lse, rows):
    """got [R, D], got_lse [R] or None against a list of attend() results."""
    g = got.double().cpu()
    for i, (o, lse, bound, dl) in enumerate(rows):
        err = (g[i] - o).abs()
        assert torch.isfinite(g[i]).all(), f"row {i}: non-finite output"
        worst = float((err / bound.clamp_min(1e-30)).max())
        assert worst <= 1.0, f"row {i}: error {float(err.max()):.3e}, {worst:.2f} x the bound"
        if got_lse is not None:
            l = float(got_lse[i])
            assert (l == lse) if math.isinf(lse) else abs(l - lse) <= dl, f"row {i}: lse {l} vs {lse} (bound {dl:.2e})"
