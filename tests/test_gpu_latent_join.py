"""Absorbed attention of many sequences, chains and trees, whose longest ones several CTAs work on: every joined row against
64 bits, with a tolerance of its own outputs' size."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _join as J
from tests import _latent as L
from tests import _tree as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("N,K,H", [
    (20, 2, 8), (20, 8, 32),        # few sequences: every warp of the joining kernel counts them
    (33, 8, 32), (32, 12, 24),      # rows or sequences enough: the cut ones alone
    (128, 2, 8), (129, 2, 8), (129, 4, 64), (300, 1, 16), (300, 5, 32)])
def test_joined_rows(N, K, H, dtype, tree):
    lens = [0 if n % 11 == 5 else K + (n * 37) % 400 + (3000 if n % 50 == 7 else 0) for n in range(N)]
    cache, table, held = L.paged(lens, 32, dtype, seed=N + K)
    q = torch.randn(N, K, H, 576, generator=L.gen(N + 1)).to(torch.bfloat16)
    rows = [T.tree(K, n, 3, nodes=1 + n % K) for n in range(N)] if tree else [list(range(-1, K - 1))] * N
    args = (q.to(DEV), cache.to(DEV), dtype, table.to(DEV), _i32(lens))
    out, lse = (kda.latent_decode_tree(*args, _i32(rows), 0.07, want_lse=True) if tree else
                kda.latent_decode(*args, 0.07, want_lse=True))
    assert kda.kda_device_status() == kda.KDA_OK
    out, lse = out.cpu(), lse.cpu()
    some = [n for n in range(N) if lens[n] > 3000 or n % 7 == 0 or lens[n] == 0]
    for n in some:
        if lens[n] == 0:
            assert not out[n].any() and (lse[n] == -torch.inf).all()
            continue
        see = torch.zeros(K, lens[n], dtype=torch.bool)
        for j in range(K):
            p = T.path(rows[n], j)
            if p:
                see[j, :lens[n] - K] = True
                see[j, [lens[n] - K + i for i in p]] = True
        pick = sorted({0, H // 2, H - 1})
        want = J.rows(q[n][:, pick].reshape(-1, 576), *held[n], 0.07, see.repeat_interleave(len(pick), dim=0))
        J.check(out[n][:, pick].reshape(-1, 512), lse[n][:, pick].reshape(-1), want, f"sequence {n} of {lens[n]} tokens")
