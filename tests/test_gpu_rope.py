"""kda_latent_append_rope: the rotation against whole-number arithmetic, everything else as kda_latent_append."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L

mpmath = pytest.importorskip("mpmath")
pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")]
BITS = 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def angles(pos, freq):
    """fp64 angles in (-pi, pi] of pos * freq, the product and its remainder in whole numbers."""
    mpmath.mp.prec = 2 * BITS
    inv = int(mpmath.floor(mpmath.mpf(2) ** BITS / (2 * mpmath.pi)))     # turns a radian
    out = torch.zeros(len(pos), len(freq), dtype=torch.float64)
    for j, f in enumerate(freq.double().tolist()):
        m, e = int(f * 2.0 ** 149), 149                                  # a float is a whole number of 2^-149
        for i, p in enumerate(pos):
            turns = (p * m * inv >> e) % (1 << BITS)
            turns = turns - (1 << BITS) if turns >> (BITS - 1) else turns
            out[i, j] = float(2 * mpmath.pi * mpmath.mpf(turns) / mpmath.mpf(2) ** BITS)
    return out


def rotate(x, ang, inter):
    """fp64 rotation of x [T, ..., 64] by ang [T, 32], and a bound of the operator's error: the angle to within 2^-23,
    sine and cosine to a step, two products and a sum in fp32 (together below 2^-21 of the pair's magnitudes), and the
    rounding to bf16."""
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    while ang.dim() < a.dim():
        ang = ang[:, None]
    c, s = torch.cos(ang), torch.sin(ang)
    y, z, mag = a * c - b * s, a * s + b * c, a.abs() + b.abs()
    glue = (lambda u, v: torch.stack([u, v], -1).flatten(-2)) if inter else (lambda u, v: torch.cat([u, v], -1))
    y, mag = glue(y, z), glue(mag, mag)
    err = 2.0 ** -21 * mag
    return y, err + 2.0 ** -8 * (y.abs() + err) + 1e-38


def freqs():
    return (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float()


def near(got, ref):
    y, bound = ref
    err = (got.double().cpu() - y).abs()
    assert (err <= bound).all(), f"{float((err / bound).max()):.2f} x the bound"


def run(dtype, pos, H=3, inter=False, page=16, slots=None, freq=None, layout="alone", seed=0, in_place=False):
    T = len(pos)
    g = L.gen(seed)
    c, r = L.latents(g, T)
    wide = {"alone": 64, "expanded": 192, "absorbed": 576}[layout]
    both = torch.cat([c, r, c[:, :64]], dim=1).to(DEV)
    q = torch.randn(T, H, wide, generator=g).to(torch.bfloat16)
    qd = q.to(DEV)
    P = -(-T // page) + 1
    if slots is None:
        slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32)
    freq = freqs() if freq is None else freq
    cache = kda.latent_cache(P, page, dtype)
    out = qd[..., -64:] if in_place else torch.full((T, H, wide), 7.0, dtype=torch.bfloat16, device=DEV)[..., -64:]
    got = kda.latent_append_rope(both[:, :512], both[:, 512:576], cache, dtype, slots.to(DEV),
                                 torch.tensor(pos, dtype=torch.int32, device=DEV), freq.to(DEV), q=qd[..., -64:], q_out=out,
                                 interleaved=inter)
    assert got is out
    if in_place and wide > 64:                                  # only the position parts have changed
        assert torch.equal(qd[..., :-64].cpu(), q[..., :-64])
    plain = kda.latent_cache(P, page, dtype)
    kda.latent_append(both[:, :512], both[:, 512:576], plain, dtype, slots.to(DEV))
    return c, r, q[..., -64:], got.cpu(), cache.cpu().view(-1, L.ROW[dtype]), plain.cpu().view(-1, L.ROW[dtype]), slots, freq


def check(dtype, pos, inter, res):
    c, r, q, got, cache, plain, slots, freq = res
    ang = angles(pos, freq)
    at = slots.long()
    lo = L.DC if dtype else 2 * L.DC
    near(cache[at][:, lo:lo + 128].contiguous().view(torch.bfloat16), rotate(r, ang, inter))
    near(got, rotate(q, ang, inter))
    cache, plain = cache.clone(), plain.clone()
    cache[at, lo:lo + 128] = 0
    plain[at, lo:lo + 128] = 0
    assert torch.equal(cache, plain)                            # latents, scales and other rows: the plain append's bytes


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("pos,H,layout", [
    ([0], 1, "alone"), ([1, 0, 5], 3, "expanded"), ([2 ** 31 - 1, -5, -2 ** 31, 1000003, 142000], 5, "absorbed"),
    (list(range(130990, 131073)), 4, "alone"), (list(range(17)), 64, "expanded"), ([7] * 40, 33, "absorbed")])
def test_rotation(dtype, inter, pos, H, layout):
    res = run(dtype, pos, H, inter, layout=layout, page=48, seed=len(pos) + H)
    _ok()
    check(dtype, pos, inter, res)


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
def test_frequencies(inter):
    """Larger than a turn a position, denormal, negative, zero; and what is too large is NaN in its pair alone."""
    f = freqs()
    f[:8] = torch.tensor([1.5, 6.2831855, 1000.25, 4.0e9, -0.3, 0.0, 1e-39, 2.0 ** -100])
    pos = [0, 1, 77, 100000, 2 ** 31 - 1, -9]
    res = run(1, pos, 4, inter, freq=f, seed=3)
    _ok()
    check(1, pos, inter, res)
    f[3], f[4] = 2.0 ** 32, float("inf")
    c, r, q, got, cache, plain, slots, freq = run(1, pos, 4, inter, freq=f, seed=3)
    pairs = got.unflatten(-1, (32, 2)) if inter else got.unflatten(-1, (2, 32)).transpose(-1, -2)
    assert torch.isnan(pairs[..., 3:5, :].float()).all() and torch.isfinite(pairs[..., 5:, :].float()).all()


@pytest.mark.parametrize("layout", ["alone", "expanded"])
def test_in_place(layout):
    pos = [5, 900, 33, 4]
    res = run(0, pos, 6, True, layout=layout, in_place=True, seed=8)
    _ok()
    check(0, pos, True, res)


@pytest.mark.parametrize("dtype", CACHES)
def test_padding_and_bad_slots(dtype):
    """Tokens of a negative slot leave the cache and their rows of q_out as they were; slots past the cache are reported."""
    pos = list(range(6))
    slots = torch.tensor([3, -1, 7, -9, 0, 12], dtype=torch.int32)
    c, r, q, got, cache, plain, _, freq = run(dtype, pos, 5, slots=slots, seed=4)
    _ok()
    on = [0, 2, 4, 5]
    near(got[on], rotate(q[on], angles([pos[i] for i in on], freq), False))
    assert (got[[1, 3]] == 7).all()
    assert not cache[[i for i in range(cache.shape[0]) if i not in (3, 7, 0, 12)]].any()
    slots[2] = cache.shape[0]
    c, r, q, got, *_ = run(dtype, pos, 5, slots=slots, seed=4)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert (got[2] == 7).all()
    _ok()


def test_without_queries_and_with_outputs_of_its_own():
    g = L.gen(1)
    c, r = (t.to(DEV) for t in L.latents(g, 9))
    pos, slots = torch.arange(9, dtype=torch.int32, device=DEV) + 50, torch.arange(9, dtype=torch.int32, device=DEV)
    a, b = kda.latent_cache(1, 16, 1), kda.latent_cache(1, 16, 1)
    assert kda.latent_append_rope(c, r, a, 1, slots, pos, freqs().to(DEV)) is None
    q = torch.randn(9, 2, 64, generator=g).to(torch.bfloat16)
    out = kda.latent_append_rope(c, r, b, 1, slots, pos, freqs().to(DEV), q=q.to(DEV))
    _ok()
    assert torch.equal(a, b) and out.shape == (9, 2, 64)
    near(out, rotate(q, angles(pos.tolist(), freqs()), False))


def test_many_tokens_repeat():
    pos = [(i * 7919) % 200000 for i in range(5000)]
    x = run(1, pos, 8, seed=5)
    y = run(1, pos, 8, seed=5)
    _ok()
    assert torch.equal(x[3], y[3]) and torch.equal(x[4], y[4])
    some = list(range(0, 5000, 617))
    near(x[3][some], rotate(x[2][some], angles([pos[i] for i in some], x[7]), False))
