"""kda_token_logprobs against its definition in 64 bits."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
H24 = 2.0 ** -24                                                # half a step of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def order(row):
    """Indices by value, largest first, equal ones by index."""
    return torch.sort(row.double(), descending=True, stable=True).indices


def expected(row, t, scale, top):
    """(log prob, rank, entropy, top log probs, top tokens) in fp64, and bounds of the first, third and fourth.

    A term 2^y, y = (x - m) c: two roundings of y (and one of c), 3 half steps of |y| ln 2 relative, ex2's 2^-22; the sum
    adds at most a half step a term of a thread's own (V / 512 and 32 more) and a dozen of the joins.  So the log of the
    sum is off by `ds`; the entropy by that and by the same relative errors in the weighted mean of y."""
    x = row.double() * scale
    V = x.numel()
    m = x.max()
    ls = torch.logsumexp(x - m, 0) if m > -math.inf else torch.tensor(0.0, dtype=torch.float64)
    p = torch.exp(x - m - ls) if m > -math.inf else torch.zeros_like(x)
    y = torch.where(p > 0, (x - m).abs(), torch.zeros_like(x))
    ey, eyy = float((p * y).sum()), float((p * y * y).sum())
    n = V / 512 + 60
    ds = 3 * H24 * ey + 2.0 ** -22 + n * H24 + float(ls) * 4 * H24 + 1e-30
    dent = ds + 3 * H24 * eyy + ey * (2.0 ** -22 + (2 * n + 8) * H24) + (float(ls) + ey) * 4 * H24
    lp = torch.where(x > -math.inf, x - m - ls, torch.full_like(x, -math.inf))
    ent = float(ls) + ey if m > -math.inf else 0.0
    lp = torch.where(lp < -torch.finfo(F32).max, torch.full_like(lp, -math.inf), lp)   # beyond fp32: -inf
    o = order(row)
    rank = None if t is None else int((o == t).nonzero()[0]) + 1
    near = lambda v: ds + 4 * H24 * ((v + ls).abs() + abs(float(ls)))    # the difference, the product, the sum
    return lp, rank, ent, o[:top], near, dent


def check(x, tok, top, scale, got):
    lp, rank, ent, tlp, ttok = [None if g is None else g.cpu() for g in got]
    for r in range(x.shape[0]):
        t = None if tok is None else int(tok[r])
        e_lp, e_rank, e_ent, e_top, near, dent = expected(x[r], t, scale, top)
        if t is not None:
            assert int(rank[r]) == e_rank, (r, int(rank[r]), e_rank)
            if e_lp[t] == -math.inf:
                assert lp[r] == -math.inf
            else:
                assert abs(float(lp[r]) - float(e_lp[t])) <= float(near(e_lp[t])), (r, float(lp[r]), float(e_lp[t]))
        assert abs(float(ent[r]) - e_ent) <= dent, (r, float(ent[r]), e_ent, dent)
        if top:
            k = e_top.numel()
            assert torch.equal(ttok[r, :k].long(), e_top), (r, ttok[r, :k].tolist(), e_top.tolist())
            w = e_lp[e_top]
            fin = w > -math.inf
            assert (tlp[r, :k][~fin] == -math.inf).all()
            assert ((tlp[r, :k].double() - w).abs()[fin] <= near(w)[fin]).all()
            assert (ttok[r, k:] == -1).all() and (tlp[r, k:] == -math.inf).all()


def run(x, tok, top=0, scale=1.0, pad=0, lead=0):
    """x [R, V] as a view of wider rows: `pad` elements after each, the first row `lead` elements into the memory."""
    R, V = x.shape
    buf = torch.full((lead + R * (V + pad),), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[lead:].view(R, V + pad)[:, :V]
    v.copy_(x)
    return kda.token_logprobs(v, None if tok is None else torch.tensor(tok, dtype=torch.int32, device=DEV), top=top, scale=scale)


def rows(R, V, dtype, seed, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * sharp).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,V,top,pad,lead,scale", [
    (1, 1, 1, 0, 0, 1.0), (3, 2, 5, 3, 1, 0.5), (2, 31, 32, 0, 3, 1.0), (5, 1000, 20, 1, 0, 1.0), (2, 4095, 8, 0, 5, 2.0),
    (2, 4097, 32, 7, 7, 0.3), (3, 32001, 5, 0, 1, 1.0), (4, 100003, 20, 29, 0, 0.7), (1, 131072, 32, 0, 0, 1.0),
    (2, 160001, 1, 0, 3, 1.0), (700, 513, 3, 0, 0, 1.0), (2, 20000, 0, 0, 0, 1.0)])
def test_rows(dtype, R, V, top, pad, lead, scale):
    x = rows(R, V, dtype, seed=R + V)
    g = torch.Generator().manual_seed(V)
    tok = torch.randint(0, V, (R,), generator=g).tolist()
    tok[0], tok[-1] = (0, V - 1) if R > 1 else (V // 2, V // 2)
    got = run(x, tok, top, scale, pad, lead)
    _ok()
    check(x, tok, top, scale, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [3000, 70001])
def test_ties_and_orders(dtype, V):
    """Constant rows, few values, ascending and descending rows, zeros of both signs, one value far above."""
    x = torch.zeros(8, V)
    x[1] = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).float()
    x[2] = torch.arange(V) * (30.0 / V)
    x[3] = -torch.arange(V) * (30.0 / V)
    x[4, ::2] = -0.0
    x[5, V // 3] = 80.0
    x[6, 5:V - 5:7] = 1.0
    x[7] = -3.0e38
    x = x.to(dtype)
    tok = [V - 1, V // 2, 0, V - 1, 1, V // 3, 12, 5]
    for top in (1, 20, 32):
        got = run(x, tok, top, 1.0, pad=1, lead=1)
        _ok()
        check(x, tok, top, 1.0, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_masked_vocabularies(dtype):
    """-inf and the type's lowest value in all but a few places, or everywhere."""
    V = 50001
    lowest = torch.finfo(dtype).min
    for mask in (-math.inf, lowest):
        x = torch.full((5, V), mask)
        x[0, [3, 40000, 50000]] = torch.tensor([1.0, -2.0, 0.5])
        x[1, 17] = -4.0
        x[3, 20000:20007] = 2.0
        x[4] = rows(1, V, F32, 3)[0]
        x[4, 100:] = mask
        x = x.to(dtype)
        tok = [40000, 18, 7, 20006, 60]
        got = run(x, tok, 20)
        _ok()
        check(x, tok, 20, 1.0, got)
        if mask == -math.inf:
            assert got[0][2] == -math.inf and got[2][2] == 0 and got[4][2].tolist() == list(range(20))
        else:
            assert abs(float(got[0][2]) + math.log(V)) < 1e-4 and abs(float(got[2][2]) - math.log(V)) < 1e-4


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_nan_and_infinity(dtype):
    x = rows(4, 20011, dtype, 5)
    x[0, 20010] = float("nan")
    x[1, 4444] = float("inf")
    x[2, 0] = float("-inf")
    got = run(x, [1, 4444, 0, 9], 5)
    _ok()
    for r in (0, 1):
        assert torch.isnan(got[0][r]) and got[1][r] == 0 and torch.isnan(got[2][r])
        assert torch.isnan(got[3][r]).all() and (got[4][r] == -1).all()
    check(x[2:], [0, 9], 5, 1.0, [g[2:] for g in got])
    assert got[0][2] == -math.inf and got[1][2] == 20011


def test_largest_values_side_by_side():
    """Most of the largest values fall to the same few threads: more than are put in order at once."""
    V = 131072
    x = rows(2, V, F32, 6, sharp=1.0)
    i = torch.arange(V)
    x[0, (i // 4) % 512 < 8] += 100.0                           # every chunk of 16 bytes that 8 of 512 threads take
    x[1] = 0.0
    x[1, (i // 4) % 512 < 4] = 1.0 + (i[(i // 4) % 512 < 4] % 977) * 2.0 ** -10
    got = run(x, [0, 5], 32)
    _ok()
    check(x, [0, 5], 32, 1.0, got)


def test_padding_rows_and_bad_tokens():
    x = rows(5, 9001, BF, 8)
    tok = [4, -1, 9000, -7, 0]
    got = run(x, tok, 4)
    _ok()
    on = [0, 2, 4]
    check(x[on], [tok[i] for i in on], 4, 1.0, [g[on] for g in got])
    for r in (1, 3):
        assert got[0][r] == 0 and got[1][r] == 0 and got[2][r] == 0 and (got[3][r] == -math.inf).all() and (got[4][r] == -1).all()
    got = run(x, [4, 9001, 9000, 1, 0], 4)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert got[1][1] == 0 and (got[4][1] == -1).all()
    _ok()


def test_without_tokens_and_without_alternatives():
    x = rows(3, 5003, F32, 9)
    a = run(x, None, 6)
    b = run(x, [1, 2, 3], 0)
    _ok()
    assert a[0] is None and a[1] is None and b[3] is None and b[4] is None
    check(x, None, 6, 1.0, a)
    check(x, [1, 2, 3], 0, 1.0, b)


def test_row_offsets_past_32_bits_and_repeats():
    V = 131072
    R = (1 << 31) // V + 3
    x = torch.empty(R, V, dtype=BF, device=DEV).normal_(0, 2.0, generator=torch.Generator(device=DEV).manual_seed(4))
    tok = torch.randint(0, V, (R,), device=DEV).to(torch.int32)
    a = kda.token_logprobs(x, tok, top=3)
    b = kda.token_logprobs(x, tok, top=3)
    _ok()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    some = [0, R // 2, R - 2, R - 1]
    check(x[some].cpu(), [int(tok[i]) for i in some], 3, 1.0, [g[some] for g in a])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-6, 0.02, 1.0, 1e6])
def test_large_logits_and_scales(dtype, scale):
    """Logits far from 0, where neighbours of the type are far apart; lowest values and -inf side by side; scales that
    leave a row flat, or one token alone."""
    V = 30011
    x = rows(6, V, F32, 11)
    x[1] = x[1] * 100 + 1e6
    x[2] = x[2] * 1e28 + 9e29
    x[3] = torch.finfo(dtype).min
    x[3, ::2] = -math.inf
    x[4] = torch.finfo(dtype).min / 3
    x[4, 5:9000:3] = torch.finfo(dtype).min
    x[5, :] = -math.inf
    x[5, 17], x[5, 29000] = -3.0e38, -1.0e38
    x = x.to(dtype)
    tok = [7, 9, 11, 1, 6, 17]
    for R in (6, 1):
        got = run(x[:R] if R > 1 else x[3:4], tok if R > 1 else tok[3:4], 7, scale, pad=2)
        _ok()
        check(x[:R] if R > 1 else x[3:4], tok if R > 1 else tok[3:4], 7, scale, got)


def test_rows_alone_and_together():
    """Few rows are spread over several CTAs each, many are not: the same tokens and ranks, and sums to within rounding."""
    x = rows(700, 65000, BF, 12)
    tok = torch.randint(0, 65000, (700,), generator=torch.Generator().manual_seed(1)).tolist()
    many = run(x, tok, 32)
    for r0, r1 in ((0, 1), (5, 8), (100, 140), (0, 300)):
        few = run(x[r0:r1], tok[r0:r1], 32)
        _ok()
        assert torch.equal(few[1], many[1][r0:r1]) and torch.equal(few[4], many[4][r0:r1])
        for i in (0, 2, 3):
            assert torch.allclose(few[i], many[i][r0:r1], rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [30000, 105187])
def test_entropy_of_sharp_rows(dtype, V):
    """The entropy is the difference of the log of a sum and a mean exponent.  Terms are at most 2^6 of their
    reference, so both are below 8 where a few tokens hold the row, a rounding of either is at most 8 half steps, and a
    dozen of those at random (the sums' last additions, the quotient, the logarithm) are 28: in nats, 28 ln 2 2^-24."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(150, V, generator=g) * 3.2).to(dtype)
    _, _, ent, _, _ = kda.token_logprobs(x.to(DEV), None, scale=1.9)
    _ok()
    lp = torch.log_softmax(x.double() * 1.9, -1)
    ref = -(lp.exp() * lp).sum(-1)
    err = float((ent.double().cpu() - ref).pow(2).mean().sqrt())
    assert err <= 28 * math.log(2) * H24, f"{err:.2g}"
