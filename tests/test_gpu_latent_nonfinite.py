"""NaN and infinities in the latent cache: they reach the rows that see them and no others, and cost no time."""
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


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def _best(call):
    """Shortest of several passes, in microseconds."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(3):
        call()
    best = math.inf
    for _ in range(8):
        ev[0].record()
        call()
        ev[1].record()
        torch.cuda.synchronize()
        best = min(best, ev[0].elapsed_time(ev[1]) * 1e3)
    return best


# (a call from Python takes 20 us or so of its own: a few microseconds more of that are not the kernel's)
def _near(got, clean):
    assert got <= 2 * clean + 20, f"{got:.0f} us against {clean:.0f} us without a NaN"


# ---- absorbed ------------------------------------------------------------------------------------

def _absorbed(N, T, K, H, dtype, seed):
    """q, cache, table, lens of N sequences of T tokens, written through the package's own append."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    per = -(-T // 64)
    table = torch.randperm(N * per, generator=g, device=DEV).to(torch.int32).view(N, per)
    cache = kda.latent_cache(N * per, 64, dtype)
    t = torch.arange(T, device=DEV)
    for n in range(N):
        kda.latent_append(rn(T, 512), rn(T, 64), cache, dtype, (table[n].long()[t // 64] * 64 + t % 64).to(torch.int32))
    return rn(N, K, H, 576), cache, table, torch.full((N,), T, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("N,T", [(3, 6000), (160, 1500)])       # sequences of many CTAs, CTAs of a sequence or more
def test_absorbed_with_a_nan_in_an_early_token(dtype, N, T):
    K, H = 4, 32
    q, cache, table, lens = _absorbed(N, T, K, H, dtype, seed=N)
    call = lambda: kda.latent_decode(q, cache, dtype, table, lens, 0.07, want_lse=True)
    out, lse = call()
    clean = _best(call)
    cache[table[1, 0].long(), 0, :512] = 0xFF                   # token 0 of sequence 1
    got, got_lse = call()
    _ok()
    assert torch.isnan(got[1].float()).all() and torch.isnan(got_lse[1]).all()
    for n in (0, 2, N - 1):
        assert torch.equal(got[n], out[n]) and torch.equal(got_lse[n], lse[n])
    _near(_best(call), clean)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("lens", [[70, 5, 129, 3], [20000]])
def test_absorbed_last_tokens_that_earlier_queries_do_not_see(dtype, lens):
    """The last three tokens hold NaN latents; query j of four sees j of them."""
    K, H, page = 4, 8, 16
    cache, table, held = L.paged(lens, page, dtype, seed=sum(lens))
    q = torch.randn(len(lens), K, H, 576, generator=L.gen(3)).to(torch.bfloat16)
    for n, length in enumerate(lens):
        for t in range(max(0, length - 3), length):
            cache[table[n, t // page], t % page, 3:500] = 0x7F if dtype else 0xFF
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), dtype, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), 0.07, want_lse=True)
    _ok()
    for n, length in enumerate(lens):
        key = torch.cat(held[n], dim=1)
        rows = [L.attend(q[n, 0, h].double(), key, held[n][0], 0.07, length - 3) for h in range(H)]
        L.check_rows(out[n, 0], lse[n, 0], rows)
        for j in range(1, K):
            if length - 3 + j > max(0, length - 3):
                assert torch.isnan(out[n, j].float()).all() and torch.isnan(lse[n, j]).all()


@pytest.mark.parametrize("lens", [[70, 9], [20000]])
@pytest.mark.parametrize("back", [2, 8])                        # seen by the last two queries of four, by all of them
def test_absorbed_infinite_latent_without_weight(lens, back):
    """A latent of -inf that every query multiplies by a positive number scores -inf: its weight is 0, and
    0 * inf spoils its channel alone."""
    K, H, page, ch = 4, 5, 32, 137
    cache, table, held = L.paged(lens, page, 0, seed=4)
    q = torch.randn(len(lens), K, H, 576, generator=L.gen(5)).to(torch.bfloat16)
    q[..., ch] = 0.5
    for n, length in enumerate(lens):
        t = length - back
        cache[table[n, t // page], t % page, 2 * ch:2 * ch + 2] = torch.tensor([-math.inf]).to(torch.bfloat16).view(torch.uint8)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), 0, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), 0.07, want_lse=True)
    _ok()
    rest = [c for c in range(512) if c != ch]
    for n, length in enumerate(lens):
        t = length - back
        key, val = torch.cat(held[n], dim=1), held[n][0]
        for j in range(K):
            see = length - (K - 1 - j)
            if see > t:                                         # the same without that token
                k, v, s = torch.cat([key[:t], key[t + 1:]]), torch.cat([val[:t], val[t + 1:]])[:, rest], see - 1
                assert torch.isnan(out[n, j, :, ch].float()).all()
            else:
                k, v, s = key, val[:, rest], see
            L.check_rows(out[n, j][:, rest], lse[n, j], [L.attend(q[n, j, h].double(), k, v, 0.07, s) for h in range(H)])
