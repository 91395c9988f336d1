"""Absorbed attention in 64 bits with a tolerance for each output of its own, narrow enough for rows over thousands of tokens,
whose outputs are small beside the values that they are sums of."""
import torch

from tests import _latent as L


def rows(q, c, r, scale, see):
    """q [R, 576] over tokens c [T, 512], r [T, 64] where see [R, T]: (out, lse, tolerance of out, of lse), fp64.

    The weights p are rounded to bf16 before the product (over e4m3 to at least as many bits), each by at most 2^-8 of itself
    and independently: a rounding's standard deviation is at most 2^-8 / sqrt(3) of p, that of an output
    2^-8 / sqrt(3) sqrt(sum p^2 v^2), and six of those hold over some millions of outputs.  Beside them: the output's own
    rounding, 2^-8 of it; scores, off by a step of fp32 a term of their sums and by exp2's 2^-21, over e4m3 by 2^-17 of the
    queries' largest in the few of 512 terms that their second code does not reach (together below 2^-15 here), which move all
    weights of a row alike or less; and the sums over the tokens, a step of fp32 each eight."""
    key = torch.cat([c, r], dim=1)
    x = (q.double() @ key.T) * scale
    dx = (q.double().abs() @ key.abs().T * scale).amax(dim=1, keepdim=True) * 578 * L.F32_STEP + 2.0 ** -21 + 2.0 ** -15
    x = torch.where(see, x, torch.full_like(x, -torch.inf))
    lse = torch.logsumexp(x, dim=1, keepdim=True)
    p = torch.where(torch.isfinite(lse), torch.exp(x - lse), torch.zeros_like(x))
    o, mass = p @ c, p @ c.abs()
    sigma = torch.sqrt(p.square() @ c.square()) * 2.0 ** -8 / 3 ** 0.5
    steps = c.shape[0] / 8 * L.F32_STEP
    tol = 2.0 ** -8 * o.abs() + 6 * sigma + (2 * dx + steps) * mass + 1e-30
    return o, lse[:, 0], tol, dx[:, 0] + c.shape[0] * L.F32_STEP + lse[:, 0].abs() * L.F32_STEP


def check(got, got_lse, want, what):
    o, lse, tol, dl = want
    err = (got.double().cpu() - o).abs()
    assert torch.isfinite(err).all(), what
    assert (err <= tol).all(), f"{what}: {float((err / tol).max()):.2f} x the tolerance"
    l = got_lse.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(none, torch.isinf(l)), what
    assert ((l - lse).abs()[~none] <= dl[~none]).all(), what
