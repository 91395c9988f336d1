"""kda_latent_decode_tree against a plain attention in 64 bits over each node's own tokens."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L
from tests import _tree as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def expected(q, held, rows, scale, n, pick=None):
    """attend() of each of sequence n's rows (j, h) over the context and the node's path."""
    K, H = q.shape[1:3]
    c, r = held[n]
    key = torch.cat([c, r], dim=1)
    ctx = key.shape[0] - K
    out = []
    for j in range(K):
        p = T.path(rows[n], j) if ctx >= 0 else []
        idx = torch.tensor(list(range(ctx)) + [ctx + i for i in p], dtype=torch.long) if p else torch.zeros(0, dtype=torch.long)
        for h in range(H):
            if pick is None or (j, h) in pick:
                out.append(L.attend(q[n, j, h].double(), key[idx], c[idx], scale, len(idx)))
    return out


def run(q, cache, table, lens, rows, scale, dtype, **o):
    return kda.latent_decode_tree(q.to(DEV), cache.to(DEV), dtype, table.to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV),
                                  torch.tensor(rows, dtype=torch.int32, device=DEV), scale, want_lse=True, **o)


def case(ctx, K, H, page, dtype, seed, reach=4, scale=192 ** -0.5, q_std=1.0, junk=None, full=False):
    lens = [0 if x is None else x + K for x in ctx]
    cache, table, held = L.paged(lens, page, dtype, seed, junk=junk)
    g = L.gen(seed + 1)
    q = (torch.randn(len(lens), K, H, 576, generator=g) * q_std).to(torch.bfloat16)
    rows = [T.tree(K, seed + n, reach, nodes=K if full or n % 2 == 0 else max(1, K - 1 - n)) for n in range(len(lens))]
    out, lse = run(q, cache, table, lens, rows, scale, dtype)
    _ok()
    for n, x in enumerate(lens):
        if x == 0:
            assert not out[n].any() and (lse[n] == -math.inf).all()
            continue
        exp = expected(q, held, rows, scale, n)
        L.check_rows(out[n].reshape(-1, L.DC), lse[n].reshape(-1), exp)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("ctx,K,H,page,reach", [
    ([0], 1, 1, 16, 1),
    ([0, 5, None, 63, 64], 1, 3, 16, 1),        # one node; a sequence that is not there
    ([0, 1, 60, 130], 8, 4, 32, 3),             # no context; trees that end in the next tile
    ([700, 33, 257], 5, 8, 48, 5),              # pages that no tile divides
    ([300, 64, 1], 4, 32, 64, 4),               # 128 rows
    ([500], 8, 64, 16, 8),                      # 512 rows
    ([100, 31], 64, 2, 16, 64),                 # trees of 64, over two tiles
    ([40, 3], 64, 8, 48, 1),                    # chains of 64
    ([6000, 5], 6, 4, 64, 2),                   # one long, one short: several CTAs a sequence
    ([3000], 33, 1, 1024, 7),
])
def test_trees(dtype, ctx, K, H, page, reach):
    case(ctx, K, H, page, dtype, seed=sum(x or 0 for x in ctx) + K + H, reach=reach)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("scale,q_std", [(192 ** -0.5, 30.0), (0.0, 1.0), (-0.07, 4.0)])
def test_scales(dtype, scale, q_std):
    case([333, 1500], 6, 8, 64, dtype, seed=5, scale=scale, q_std=q_std)


@pytest.mark.parametrize("dtype", CACHES)
def test_a_chain_is_what_latent_decode_gives(dtype):
    lens, K, H = [70, 900, 64], 4, 8
    cache, table, held = L.paged(lens, 16, dtype, seed=3)
    q = torch.randn(3, K, H, 576, generator=L.gen(4)).to(torch.bfloat16)
    out, lse = run(q, cache, table, lens, [list(range(-1, K - 1))] * 3, 0.07, dtype)
    _ok()
    for n, x in enumerate(lens):
        rows = [L.attend(q[n, j, h].double(), torch.cat(held[n], 1), held[n][0], 0.07, x - (K - 1 - j))
                for j in range(K) for h in range(H)]
        L.check_rows(out[n].reshape(-1, L.DC), lse[n].reshape(-1), rows)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("ctx", [10, 61, 2000], ids=["one_tile", "two_tiles", "several_ctas"])
def test_nan_in_a_branch(dtype, ctx):
    """NaN in the cache past the end, in one node's row and in a place without a node (its query too) reaches the node's
    descendants only."""
    K, H, page = 8, 4, 16
    lens = [ctx + K]
    row = [-1, 0, 0, 1, 2, 2, 3, -2]                            # node 1: its descendants are 3 and 6
    cache, table, held = L.paged(lens, page, dtype, seed=ctx, junk=0xFF)
    q = torch.randn(1, K, H, 576, generator=L.gen(ctx + 1)).to(torch.bfloat16)
    q[0, 7] = float("nan")
    for j in (1, 7):
        at = ctx + j
        cache[table[0, at // page], at % page, :(L.DC if dtype else 2 * L.DC)] = 0xFF
    out, lse = run(q, cache, table, lens, [row], 0.07, dtype)
    _ok()
    exp = expected(q, held, [row], 0.07, 0)
    for j in (0, 2, 4, 5, 7):
        L.check_rows(out[0, j], lse[0, j], exp[j * H:(j + 1) * H])
    for j in (1, 3, 6):
        assert torch.isnan(out[0, j].float()).all() and torch.isnan(lse[0, j]).all()


def test_infinite_latent_of_a_node_bf16():
    """A latent of -inf that scores -inf leaves the sums alone, and its channel is NaN for those that see it."""
    K, H, page, ctx = 4, 2, 16, 100
    row = [-1, 0, 0, 1]
    cache, table, held = L.paged([ctx + K], page, 0, seed=5)
    q = torch.randn(1, K, H, 576, generator=L.gen(6)).to(torch.bfloat16)
    q[..., 7] = 1.0
    at = ctx + 1
    cache[table[0, at // page], at % page].view(torch.bfloat16)[7] = float("-inf")
    out, lse = run(q, cache, table, [ctx + K], [row], 0.07, 0)
    _ok()
    exp = expected(q, held, [row], 0.07, 0)
    for j in (0, 2):
        L.check_rows(out[0, j], lse[0, j], exp[j * H:(j + 1) * H])
    for j in (1, 3):
        assert torch.isnan(out[0, j, :, 7].float()).all() and torch.isfinite(out[0, j, :, 8:].float()).all()


def test_bad_parents_lengths_and_pages_are_reported():
    K, H, page = 4, 4, 16
    lens = [50, 40, 30]
    cache, table, held = L.paged(lens, page, 0, seed=2)
    q = torch.randn(3, K, H, 576, generator=L.gen(1)).to(torch.bfloat16)
    rows = [[-1, 0, 2, 2], [-1, -2, 1, 0], [-1, 0, 0, 1]]       # itself, and its child; a child of no node
    out, lse = run(q, cache, table, lens, rows, 0.07, 0)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    for n in range(3):
        L.check_rows(out[n].reshape(-1, L.DC), lse[n].reshape(-1), expected(q, held, rows, 0.07, n))
    assert not out[0, 2].any() and not out[0, 3].any() and not out[1, 2].any()
    rows = [[-1, 0, 0, 1]] * 3
    for bad in (-1, 3, 10000):                                 # shorter than the tree; past the table
        out, lse = run(q, cache, table, [50, bad, 30], rows, 0.07, 0)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        assert not out[1].any() and (lse[1] == -math.inf).all()
        for n in (0, 2):
            L.check_rows(out[n].reshape(-1, L.DC), lse[n].reshape(-1), expected(q, held, rows, 0.07, n))
    _ok()


@pytest.mark.parametrize("dtype", CACHES)
def test_repeats_bit_for_bit_and_in_a_graph(dtype):
    """A captured call follows new lengths, parents and queries."""
    ctx, K, H = [5000, 1, 900, 64, 2222], 6, 16
    lens = [x + K for x in ctx]
    cache, table, held = L.paged(lens, 64, dtype, seed=20)
    q = torch.randn(5, K, H, 576, generator=L.gen(21)).to(torch.bfloat16).to(DEV)
    cache, table = cache.to(DEV), table.to(DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rows = [T.tree(K, n, 3) for n in range(5)]
    par = torch.tensor(rows, dtype=torch.int32, device=DEV)
    call = lambda: kda.latent_decode_tree(q, cache, dtype, table, ld, par, 0.07, want_lse=True)
    a = call()
    assert all(torch.equal(x, y) for _ in range(3) for x, y in zip(call(), a))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, a))
    par.copy_(torch.tensor([T.tree(K, n + 50, 6, nodes=3) for n in range(5)], dtype=torch.int32))
    q.copy_(torch.randn(5, K, H, 576, generator=L.gen(22)))
    ld.copy_(torch.tensor([K, K + 1, 700, 40, 2000], dtype=torch.int32))
    graph.replay()
    want = call()
    torch.cuda.synchronize()
    _ok()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
