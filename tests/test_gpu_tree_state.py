"""kda_decode_tree against the recurrence in 64 bits along every path, and against kda_decode_multi on chains."""
import pytest
import torch
import torch.nn.functional as F

from kimi_delta_attention_06_gb300 import kda
from tests import _tree as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
CH, HD, NO = kda.KDA_DECAY_CHANNEL, kda.KDA_DECAY_HEAD, kda.KDA_DECAY_NONE


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def inputs(N, K, H, D, decay, seed, shift=-2.0, s0=0.2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    la = None if decay == NO else -F.softplus(rn(*((N, K, H, D) if decay == CH else (N, K, H))) + shift)
    return [unit(rn(N, K, H, D)), unit(rn(N, K, H, D)), rn(N, K, H, D).to(torch.bfloat16), la,
            torch.sigmoid(rn(N, K, H)).to(torch.bfloat16)], rn(N + 2, H, D, D) * s0


def run(x, pool, rows, slots=None, out=torch.float32, decay=CH, **o):
    d = [None if t is None else t.to(DEV) for t in x]
    par = torch.tensor(rows, dtype=torch.int32, device=DEV)
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV)
    return kda.decode_tree(*d, pool.to(DEV), par, state_slots=sl, out_dtype=out, decay=decay, **o)


def check(got, x, pool, rows, slots, out=torch.float32):
    q, k, v, la, beta = x
    got = got.double().cpu()
    for n, row in enumerate(rows):
        ref, bound = T.state_outputs(q[n], k[n], v[n], None if la is None else la[n], beta[n], pool[slots[n]], row)
        if out == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        err = (got[n] - ref).abs()
        assert torch.isfinite(got[n]).all()
        assert (err <= bound + 1e-30).all(), f"sequence {n}: {float((err / (bound + 1e-30)).max()):.2f} x the bound"
        for j in range(len(row)):
            if not T.path(row, j):
                assert not got[n, j].any()


@pytest.mark.parametrize("decay", [CH, HD, NO], ids=["channel", "head", "none"])
@pytest.mark.parametrize("N,K,H,D,reach", [
    (1, 1, 1, 64, 1), (1, 1, 1, 128, 1), (2, 2, 3, 128, 1), (3, 7, 2, 64, 3), (3, 8, 2, 128, 4), (2, 9, 1, 128, 9),
    (2, 16, 2, 128, 1), (2, 17, 1, 64, 5), (1, 31, 1, 128, 31), (2, 33, 1, 128, 6), (1, 48, 2, 64, 12), (1, 64, 1, 128, 1),
    (1, 64, 1, 64, 64)])
def test_trees(N, K, H, D, reach, decay):
    x, pool = inputs(N, K, H, D, decay, seed=N + K + D)
    rows = [T.tree(K, n + K, reach, nodes=K if n == 0 else max(1, K - n - 1)) for n in range(N)]
    slots = [(2 * n + 1) % (N + 2) for n in range(N)]
    got = run(x, pool, rows, slots, decay=decay)
    _ok()
    check(got, x, pool, rows, slots)
    got = run(x, pool, rows, slots, out=torch.bfloat16, decay=decay)
    _ok()
    check(got, x, pool, rows, slots, torch.bfloat16)


def test_without_slots_and_with_shared_ones():
    x, pool = inputs(3, 6, 2, 128, CH, seed=4)
    rows = [T.tree(6, n, 3) for n in range(3)]
    check(run(x, pool, rows), x, pool, rows, [0, 1, 2])
    check(run(x, pool, rows, [4, 4, 0]), x, pool, rows, [4, 4, 0])
    _ok()


@pytest.mark.parametrize("shift,s0", [(6.0, 1.0), (40.0, 1.0), (-9.0, 30.0)], ids=["fast", "gone_at_once", "slow_large"])
def test_decays(shift, s0):
    """alpha from 1e-20 a node (products vanish) to nearly 1; large states."""
    x, pool = inputs(2, 12, 2, 128, CH, seed=9, shift=shift, s0=s0)
    rows = [T.tree(12, 5, 2), T.tree(12, 6, 12)]
    got = run(x, pool, rows, [0, 1])
    _ok()
    check(got, x, pool, rows, [0, 1])


def test_chain_equals_the_multi_token_verify():
    N, K, H, D = 4, 8, 4, 128
    x, pool = inputs(N, K, H, D, CH, seed=2)
    d = [t.to(DEV) for t in x]
    ref = torch.empty(N, K, H, D, device=DEV)
    kda.kda_decode_multi(*d, pool.to(DEV), N + 2, None, None, 0, ref, kda.KDA_OUT_F32, N, K, H, D, D)
    got = run(x, pool, [list(range(-1, K - 1))] * N)
    _ok()
    assert float((got - ref).abs().max()) <= 1e-5 * float(ref.abs().max())


def test_nothing_reaches_a_node_that_is_no_descendant():
    """NaN and infinities in one branch, and in places that hold no node, leave the others as they are."""
    x, pool = inputs(1, 8, 2, 128, CH, seed=7)
    row = [-1, 0, 0, 1, 2, 2, 3, -5]
    clean = run(x, pool, [row])
    for bad in (float("nan"), float("inf")):
        y = [t.clone() for t in x]
        for i in (0, 1, 2, 4):
            y[i][0, 1] = bad                                    # node 1: its descendants are 3 and 6
            y[i][0, 7] = bad                                    # no node
        y[3][0, 7] = bad
        got = run(y, pool, [row])
        _ok()
        for j in (0, 2, 4, 5, 7):
            assert torch.equal(got[0, j], clean[0, j]), j
        for j in (1, 3, 6):
            assert not torch.isfinite(got[0, j]).all()


def test_bad_parents_and_slots_are_reported():
    x, pool = inputs(3, 5, 2, 64, CH, seed=3)
    rows = [[-1, 0, 5, 1, 2], [-1, 0, 2, -3, 3], [-1, 0, 1, 2, 3]]     # after its child; itself; a child of no node
    got = run(x, pool, rows, [0, 1, 2])
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    check(got, x, pool, rows, [0, 1, 2])
    assert not got[0, 2].any() and not got[0, 4].any() and not got[1, 2].any() and not got[1, 4].any()
    good = [[-1, 0, 1, 2, 3]] * 3
    for s in (-1, 5):
        out = torch.full((3, 5, 2, 64), 7.0, device=DEV)
        d = [t.to(DEV) for t in x]
        kda.kda_decode_tree(*d, pool.to(DEV), 5, torch.tensor([0, s, 2], dtype=torch.int32, device=DEV),
                            torch.tensor(good, dtype=torch.int32, device=DEV), out, kda.KDA_OUT_F32, 3, 5, 2, 64, 64)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        assert (out[1] == 7).all()
        check(out[[0, 2]], [t[[0, 2]] for t in x], pool, good[:2], [0, 2])
    _ok()


def test_repeats_bit_for_bit_and_reads_only():
    x, pool = inputs(40, 16, 8, 128, CH, seed=5)
    rows = [T.tree(16, n, 4, nodes=1 + n % 16) for n in range(40)]
    d = [t.to(DEV) for t in x]
    p = pool.to(DEV)
    keep = p.clone()
    par = torch.tensor(rows, dtype=torch.int32, device=DEV)
    a = kda.decode_tree(*d, p, par)
    for _ in range(3):
        assert torch.equal(kda.decode_tree(*d, p, par), a)
    _ok()
    assert torch.equal(p, keep)


def test_state_offsets_past_32_bits():
    """A pool of 2^31 elements and more: the last slot."""
    H, D = 64, 128
    slots = (1 << 31) // (H * D * D) + 2
    pool = torch.zeros(slots, H, D, D, device=DEV)
    x, small = inputs(1, 3, H, D, CH, seed=6)
    pool[-1] = small[0].to(DEV)
    d = [t.to(DEV) for t in x]
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device=DEV)
    at = torch.tensor([slots - 1], dtype=torch.int32, device=DEV)
    got = kda.decode_tree(*d, pool, par, state_slots=at, out_dtype=torch.float32)
    _ok()
    assert torch.equal(got, kda.decode_tree(*d, pool[-1:].clone(), par, out_dtype=torch.float32))


@pytest.mark.parametrize("decay", [CH, HD], ids=["channel", "head"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("K", [3, 8, 13, 16, 29, 32, 50, 64])
def test_many_heads_one_after_another(K, D, decay):
    """More heads than the device works on at once, an odd number of them: each as in a call of its own sequence."""
    N, H = 91, 11
    x, pool = inputs(N, K, H, D, decay, seed=K + D)
    rows = [T.tree(K, n, 1 + n % 7, nodes=max(1, K - n % 5)) for n in range(N)]
    got = run(x, pool, rows, decay=decay)
    _ok()
    for n in (0, 1, 40, 77, 89, 90):
        one = [None if t is None else t[n:n + 1] for t in x]
        alone = run(one, pool, rows[n:n + 1], [n], decay=decay)
        _ok()
        assert torch.equal(got[n], alone[0]), n
    n = 90
    check(got[n:], [None if t is None else t[n:] for t in x], pool[n:], rows[n:], [0])


@pytest.mark.parametrize("D,K,decay", [(64, 6, CH), (64, 48, HD), (128, 16, CH), (128, 30, NO), (128, 64, CH)])
def test_sums_do_not_lean(D, K, decay):
    """The tensor cores take 8 terms a step and round the sum towards zero, by up to 2^-23 of it: D / 8 steps of the state's
    product, K / 8 of the path's, half of that on average and on one side.  With 4 half steps for the rest, that bounds the
    errors' root mean square by (D / 8 + K / 8 + 4) 2^-24 of the outputs'."""
    x, pool = inputs(4, K, 4, D, decay, seed=K + D)
    rows = [T.tree(K, n, 6) for n in range(4)]
    got = run(x, pool, rows, decay=decay).double().cpu()
    _ok()
    q, k, v, la, beta = x
    ref = torch.stack([T.state_outputs(q[n], k[n], v[n], None if la is None else la[n], beta[n], pool[n], rows[n])[0] for n in range(4)])
    rel = float((got - ref).norm() / ref.norm())
    assert rel <= (D / 8 + K / 8 + 4) * 2.0 ** -24, f"{rel:.2g}"


@pytest.mark.parametrize("N,H,D,K", [(256, 32, 128, 16), (300, 32, 128, 7), (512, 32, 64, 13), (100, 32, 128, 25), (256, 16, 64, 40)])
def test_every_channel_of_many_states(N, H, D, K):
    """Queries that pick a channel of the state each, where nothing is written: outputs are its rows, to the 22 bits that the
    products keep.  (CTAs that serve dozens of states one after another: a piece of the next one in a piece's place shows.)"""
    g = torch.Generator(device=DEV).manual_seed(K)
    pool = torch.randn(N, H, D, D, device=DEV, generator=g)
    par = torch.tensor([T.tree(K, n, 6) for n in range(N)], dtype=torch.int32, device=DEV)
    zero = torch.zeros(N, K, H, D, dtype=torch.bfloat16, device=DEV)
    beta = torch.zeros(N, K, H, dtype=torch.bfloat16, device=DEV)
    for it in range(-(-D // K)):
        at = (torch.arange(K, device=DEV) * -(-D // K) + it).clamp_max(D - 1)
        q = zero.clone()
        q.scatter_(3, at.view(1, K, 1, 1).expand(N, K, H, 1), 1.0)
        for _ in range(3):
            o = kda.decode_tree(q, zero, zero, None, beta, pool, par, out_dtype=torch.float32, decay=NO)
            want = pool[:, :, at].permute(0, 2, 1, 3)
            assert ((o - want).abs() <= 2.0 ** -21 * want.abs()).all()
    _ok()


@pytest.mark.parametrize("D,K", [(128, 8), (64, 15), (128, 16), (128, 25), (64, 32), (64, 40), (128, 64)])
@pytest.mark.parametrize("what", ["q", "k", "v", "log_alpha", "beta"])
@pytest.mark.parametrize("shift", [-2.0, 25.0], ids=["near", "far"])
def test_one_bad_input_of_one_node(D, K, what, shift):
    """One input of one node and head holds NaN or an infinity: its descendants in that head (of a query: itself) have no
    finite row, everything else has the bits that it has without."""
    x, pool = inputs(1, K, 3, D, CH, seed=K, shift=shift)          # (far: decays of a path below 2^-100)
    row = T.tree(K, 2, 4)
    node = 3
    clean = run(x, pool, [row])
    at = ["q", "k", "v", "log_alpha", "beta"].index(what)
    for bad in (float("nan"), float("inf")) if what != "log_alpha" else (float("nan"),):
        y = [t.clone() for t in x]
        y[at][0, node, 1] = bad
        got = run(y, pool, [row])
        _ok()
        for j in range(K):
            hit = j == node if what == "q" else node in T.path(row, j)
            for h in range(3):
                if h == 1 and hit:
                    assert not torch.isfinite(got[0, j, h]).any(), (j, h)
                else:
                    assert torch.equal(got[0, j, h], clean[0, j, h]), (j, h)


def test_places_without_any_node():
    """Trees of no node at all beside others: zeros."""
    for K, D in ((3, 128), (20, 64), (50, 128)):
        x, pool = inputs(3, K, 2, D, HD, seed=D)
        rows = [[-2] * K, T.tree(K, 1, 3), [-7] * K]
        got = run(x, pool, rows, decay=HD)
        _ok()
        assert not got[0].any() and not got[2].any()
        check(got, x, pool, rows, [0, 1, 2])
