"""kda_decode_tree where decays leave 2^-100 .. 2^100 on some paths: nodes below such a decay are right, and all others, of
other branches, heads and sequences, have the bits that they have without it."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _tree as T
from tests.test_gpu_tree_state import CH, HD, DEV, check, inputs, run

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _same_but_below(got, clean, rows, n, h, node):
    """Sequence n's head h has changed below `node` alone."""
    for m in range(got.shape[0]):
        for j in range(got.shape[1]):
            for g in range(got.shape[2]):
                if not (m == n and g == h and node in T.path(rows[m], j)):
                    assert torch.equal(got[m, j, g], clean[m, j, g]), (m, j, g)


@pytest.mark.parametrize("decay", [-INF, -200.0, -75.0], ids=["gone", "underflows", "small"])
@pytest.mark.parametrize("D,K", [(64, 6), (128, 8), (64, 13), (128, 16), (64, 20), (128, 32), (64, 33), (64, 48), (128, 40), (128, 64)])
def test_a_far_decay_stays_in_its_branch(D, K, decay):
    """All channels, or one, of one node of one of three heads of two sequences."""
    x, pool = inputs(2, K, 3, D, CH, seed=D + K)
    rows = [T.tree(K, 2, 4), T.tree(K, 3, 3, nodes=K - 1)]
    clean = run(x, pool, rows, [0, 1])
    kda.kda_device_status()
    for n, h, node in ((0, 0, 2), (0, 1, 1), (1, 2, 3)):
        for channel in (slice(0, D), slice(D - 3, D - 2)):
            y = [t.clone() for t in x]
            y[3][n, node, h, channel] = decay
            got = run(y, pool, rows, [0, 1])
            assert kda.kda_device_status() == kda.KDA_OK
            check(got, y, pool, rows, [0, 1])
            _same_but_below(got, clean, rows, n, h, node)


@pytest.mark.parametrize("D,K", [(64, 5), (64, 14), (64, 27), (64, 50), (128, 14)])
def test_a_sequence_does_not_see_what_it_is_batched_with(D, K):
    """Sequences of one head, whose decays are far in every other one: each as in a call of its own."""
    N = 9
    x, pool = inputs(N, K, 1, D, HD, seed=K)
    x[3][1::2] -= 40.0
    rows = [T.tree(K, n, 1 + n % 5) for n in range(N)]
    got = run(x, pool, rows, decay=HD)
    for n in range(N):
        alone = run([t[n:n + 1] for t in x], pool, rows[n:n + 1], [n], decay=HD)
        assert torch.equal(got[n], alone[0]), n
    assert kda.kda_device_status() == kda.KDA_OK
    check(got, x, pool, rows, list(range(N)))


@pytest.mark.parametrize("D,K", [(64, 12), (128, 12), (64, 40), (128, 25)])
def test_near_nodes_of_a_head_whose_other_nodes_are_far(D, K):
    """A chain whose decays add up to a far one half way: its first nodes as in the chain without the rest."""
    x, pool = inputs(1, K, 2, D, CH, seed=3, shift=-2.0)
    x[3][0, K // 2, 0] = -80.0
    chain = list(range(-1, K - 1))
    got = run(x, pool, [chain])
    cut = run(x, pool, [[p if j < K // 2 else -2 for j, p in enumerate(chain)]])
    assert kda.kda_device_status() == kda.KDA_OK
    assert torch.equal(got[0, :K // 2], cut[0, :K // 2])
    check(got, x, pool, [chain], [0])
