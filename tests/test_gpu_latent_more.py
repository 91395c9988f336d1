"""More shapes of the latent attention: many sequences, row counts around the tiles, empty caches, and
values at the ends of their ranges, against plain fp64 forms."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _check(lens, K, H, page, dtype, seed, pick=None, scale=192 ** -0.5, q=None, paged=None):
    cache, table, held = paged or L.paged(lens, page, dtype, seed)
    if q is None:
        q = torch.randn(len(lens), K, H, 576, generator=L.gen(seed + 1)).to(torch.bfloat16)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), dtype, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), scale, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    rows, at = [], []
    for n, length in enumerate(lens):
        key = torch.cat(held[n], dim=1)
        for j in range(K):
            for h in range(H):
                i = (n * K + j) * H + h
                if pick is None or i % pick == 0 or length < K:
                    rows.append(L.attend(q[n, j, h].double(), key, held[n][0], scale, length - (K - 1 - j)))
                    at.append(i)
    L.check_rows(out.view(-1, L.DC)[at], lse.view(-1)[at], rows)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("N,K,H", [(70, 1, 3), (200, 2, 16), (33, 1, 64)])
def test_many_sequences_of_mixed_lengths(dtype, N, K, H):
    """More sequences than lanes of a warp, empty ones among them, and more than CTAs."""
    g = L.gen(N)
    lens = [int(x) for x in torch.randint(0, 400, (N,), generator=g)]
    for i in (0, 3, 31, 32, N - 1):
        lens[i] = 0
    lens[5], lens[6] = 3000, 64
    _check(lens, K, H, 16, dtype, seed=N, pick=7)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("K,H", [(1, 15), (1, 16), (1, 17), (1, 33), (5, 13), (1, 65), (3, 43), (1, 129)])
def test_row_counts_around_the_tiles(dtype, K, H):
    _check([70, 330, 2], K, H, 32, dtype, seed=K * H)


@pytest.mark.parametrize("dtype", CACHES)
def test_nothing_cached(dtype):
    q = torch.randn(3, 2, 8, 576, generator=L.gen(1)).to(torch.bfloat16).to(DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for pages, cols in ((0, 0), (4, 0), (4, 2)):
        out, lse = kda.latent_decode(q, kda.latent_cache(pages, 16, dtype), dtype,
                                     torch.zeros(3, cols, dtype=torch.int32, device=DEV), lens, 0.07, want_lse=True)
        assert kda.kda_device_status() == kda.KDA_OK
        assert not out.any() and (lse == -math.inf).all()
    # and a length that the empty pool cannot hold
    lens[1] = 5
    out, lse = kda.latent_decode(q, kda.latent_cache(0, 16, dtype), dtype, torch.zeros(3, 2, dtype=torch.int32, device=DEV),
                                 lens, 0.07, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert not out.any() and (lse == -math.inf).all()


def test_e4m3_scales_far_apart():
    """Tokens whose scales differ by tens of powers of two, and queries of very small and large rows:
    the scale of each token moves between the two products."""
    lens = [300]
    g = L.gen(40)
    c, r = L.latents(g, 300)
    c = (c.float() * torch.exp2(torch.randint(-30, 4, (300, 1), generator=g).float())).to(torch.bfloat16)
    page, table = 64, torch.tensor([[2, 0, 3, 4, 1]], dtype=torch.int32)
    cache = torch.zeros(6, page, 656, dtype=torch.uint8)
    rows = L.pack(c, r, 1)
    for i in range(5):
        part = rows[i * 64:(i + 1) * 64]
        cache[table[0, i], :part.shape[0]] = part
    held = [L.unpack(rows, 1)]
    q = torch.randn(1, 1, 20, 576, generator=g)
    q[0, 0, :10] *= torch.exp2(torch.arange(-20, 0, 2).float())[:, None]
    q[0, 0, 10:, :512:5] *= 2.0 ** -12                          # rows of far apart magnitudes
    _check(lens, 1, 20, page, 1, seed=0, q=q.to(torch.bfloat16), paged=(cache, table, held))


@pytest.mark.parametrize("power", [-100, -60, 60, 110])
def test_e4m3_latents_at_the_ends_of_the_range(power):
    """All latents near 2^power: scores of position keys alone (the latents' part over- or underflows
    into them evenly), sums that must not overflow.  Below 2^-80 the weighted latents may vanish (the
    8-bit terms end at 2^-16 of fp16's one), so only their size is checked there."""
    g = L.gen(45)
    lens = [150]
    c, r = L.latents(g, 150)
    c = (c.float().clamp(-4, 4) * 2.0 ** power).to(torch.bfloat16)
    rows = L.pack(c, r, 1)
    cache = torch.zeros(4, 64, 656, dtype=torch.uint8)
    table = torch.tensor([[1, 3, 0]], dtype=torch.int32)
    for i in range(3):
        part = rows[i * 64:(i + 1) * 64]
        cache[table[0, i], :part.shape[0]] = part
    q = torch.zeros(1, 1, 16, 576)
    q[..., 512:] = torch.randn(1, 1, 16, 64, generator=g)
    q = q.to(torch.bfloat16)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), 1, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 0.3, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    held = L.unpack(rows, 1)
    rows64 = [L.attend(q[0, 0, h].double(), torch.cat(held, 1), held[0], 0.3, 150) for h in range(16)]
    if power >= -80:
        L.check_rows(out[0, 0], lse[0, 0], rows64)
    else:
        for h in range(16):
            assert abs(float(lse[0, 0, h]) - rows64[h][1]) <= rows64[h][3]
        assert float(out.double().abs().max()) <= 8 * 2.0 ** power


def test_e4m3_one_loud_token_among_many():
    """One token takes nearly all the weight and thousands share the rest: their small weights must not
    be lost to the 8-bit terms."""
    T = 20000
    cache, table, held = L.paged([T], 64, 1, seed=50)
    r = torch.zeros(T, 64, dtype=torch.float64)
    r[777, 0] = 16.0                                            # its score: 16 powers of two above the others' level
    for t in (777,):
        cache[table[0, t // 64], t % 64, 512:640] = r[t].to(torch.bfloat16).view(torch.uint8)
    for t in range(T):
        if t != 777:
            cache[table[0, t // 64], t % 64, 512:640] = 0
    held = [(held[0][0], r)]
    q = torch.zeros(1, 1, 16, 576)
    q[..., 512] = math.log(2.0)
    q[..., :512] = torch.randn(1, 1, 16, 512, generator=L.gen(51)) * 0.02
    _check([T], 1, 16, 64, 1, seed=0, scale=1.0, q=q.to(torch.bfloat16), paged=(cache, table, held))


def test_expanded_without_keys():
    q = torch.randn(7, 2, 192, generator=L.gen(1)).to(torch.bfloat16).to(DEV)
    k = torch.zeros(0, 2, 128, device=DEV, dtype=torch.bfloat16)
    r = torch.zeros(0, 64, device=DEV, dtype=torch.bfloat16)
    cq, ck = torch.tensor([0, 3, 7], dtype=torch.int32), torch.tensor([0, 0, 0], dtype=torch.int32)
    out, lse = kda.latent_prefill(q, k, k, r, cq, ck, 0.07, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    assert not out.any() and (lse == -math.inf).all()


def test_expanded_many_short_sequences():
    g = L.gen(60)
    lens = [int(x) for x in torch.randint(0, 90, (75,), generator=g)]
    tq = sum(lens)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    q, k, v, r = mk(tq, 2, 192), mk(tq, 2, 128), mk(tq, 2, 128), mk(tq, 64)
    cu = torch.nn.functional.pad(torch.tensor(lens).cumsum(0), (1, 0)).to(torch.int32)
    out, lse = kda.latent_prefill(*(x.to(DEV) for x in (q, k, v, r)), cu, cu, 192 ** -0.5, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    for n in range(0, 75, 4):
        a, b = int(cu[n]), int(cu[n + 1])
        for h in range(2):
            key = torch.cat([k[a:b, h], r[a:b]], dim=1).double()
            L.check_rows(out[a:b, h], lse[a:b, h], [L.attend(q[a + i, h].double(), key, v[a:b, h].double(), 192 ** -0.5, i + 1)
                                                    for i in range(b - a)])
