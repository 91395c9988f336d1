"""The operators over trees, the append with rotation and the log probabilities as a server runs them: on another stream than
the current one, two calls at once, captured and replayed with other inputs, in the sizes where their work is split anew."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L
from tests import _tree as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
LONG = 300_000_000                                              # clocks: about 150 ms
BF, E4 = kda.KDA_CACHE_BF16, kda.KDA_CACHE_E4M3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _rn(g, *s):
    return torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parents(N, K, seed):
    return _i32([T.tree(K, seed + n, 4, nodes=K - n % 3 * (K // 4)) for n in range(N)])


# each: the inputs that a replay may change, and the call on them, which returns outputs of its own

def _append_rope(seed):
    g = L.gen(seed)
    n = 300
    c, r = (t.to(DEV) for t in L.latents(g, n))
    q, pos = _rn(g, n, 5, 64), torch.randint(0, 100000, (n,), generator=g).to(torch.int32).to(DEV)
    slots = torch.randperm(640, generator=g)[:n].to(torch.int32).to(DEV)
    freq = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).to(DEV)
    cache = kda.latent_cache(10, 64, E4)
    x = [c, r, q, pos, slots]
    return x, lambda **o: (kda.latent_append_rope(x[0], x[1], cache, E4, x[4], x[3], freq, q=x[2], **o), cache)


def _attend(seed, N=3, K=9, H=16, dtype=E4):
    lens = [K + 40 * n + 700 * (n == 0) for n in range(N)]
    cache, table, _ = L.paged(lens, 16, dtype, seed=seed)
    g = L.gen(seed)
    cache, table = cache.to(DEV), table.to(DEV)
    x = [_rn(g, N, K, H, 576), _parents(N, K, seed), _i32(lens)]
    return x, lambda **o: kda.latent_decode_tree(x[0], cache, dtype, table, x[2], x[1], 0.07, want_lse=True, **o)


def _attend_few(seed):
    return _attend(seed, N=1, K=4, H=4, dtype=BF)


def _state(seed, K=12):
    g = L.gen(seed)
    N, H, D = 5, 6, 128
    unit = lambda t: (t.float() / t.float().norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    x = [unit(_rn(g, N, K, H, D)), unit(_rn(g, N, K, H, D)), _rn(g, N, K, H, D),
         -torch.rand(N, K, H, D, generator=g).to(DEV), torch.rand(N, K, H, generator=g).to(torch.bfloat16).to(DEV),
         torch.randn(N, H, D, D, generator=g).to(DEV), _parents(N, K, seed)]
    return x, lambda **o: (kda.decode_tree(*x[:6], x[6], **o),)


def _state_large(seed):
    return _state(seed, K=40)


def _scores(seed, R=40, V=30011):
    g = L.gen(seed)
    x = [_rn(g, R, V), torch.randint(0, V, (R,), generator=g).to(torch.int32).to(DEV)]
    return x, lambda **o: kda.token_logprobs(x[0], x[1], 5, 1.3, **o)


def _scores_few(seed):
    return _scores(seed, R=2, V=100003)


MAKES = [_append_rope, _attend, _attend_few, _state, _state_large, _scores, _scores_few]
each = pytest.mark.parametrize("make", MAKES, ids=[f.__name__[1:] for f in MAKES])


def _garbage(like):
    keep = [torch.full((64 * (i % 8 + 1),), 1 << 30, dtype=torch.int32, device=DEV) for i in range(64)]
    return keep + [torch.full_like(t, 77) for t in like for _ in range(2)]


def _same(got, want):
    assert kda.kda_device_status() == kda.KDA_OK
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@each
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_call_on_a_busy_stream(make, raw):
    _, call = make(3)
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    got = call(stream=s.cuda_stream if raw else s)
    busy = not s.query()
    keep = _garbage(want)
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    assert busy, "the call returned after its stream was idle: nothing was tested"
    _same(got, want)
    del keep


@each
def test_outputs_against_work_pending_on_the_current_stream(make):
    _, call = make(4)
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(LONG)
    for t in old:
        t.fill_(77)
    del old, t
    got = call(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    _same(got, want)


@each
def test_two_calls_at_once(make):
    """Calls on two streams that both wait for the same event run side by side: their scratch is their own."""
    calls = [make(5)[1], make(6)[1]]
    want = [[t.clone() for t in call()] for call in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        torch.cuda._sleep(LONG // 50)
        event = torch.cuda.Event()
        event.record()
        for s in streams:
            s.wait_event(event)
        got = [[call(stream=s) for _ in range(4)] for call, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for outs, w in zip(got, want):
            for o in outs:
                _same(o, w)


@each
def test_captured_and_replayed_on_other_inputs(make):
    """Two graphs of the operator, replayed in turn and at once on inputs that change between the replays."""
    made = [make(7), make(8)]
    graphs, outs = [], []
    for x, call in made:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in made]
    for i in range(3):
        for j, (x, _) in enumerate(made):
            for a, b in zip(x, make(20 + 2 * i + j)[0]):
                a.copy_(b)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        for g, (_, call) in zip(got, made):
            _same(g, call())


@pytest.mark.parametrize("dtype", [BF, E4], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N", [512, 513, 700])
def test_many_trees_of_several_row_tiles(N, dtype):
    """Row tiles without nodes are left out where the sequences are few enough to be looked at, and are worked through where
    they are not: the same outputs as calls on a part of the sequences."""
    K, H = 5, 32
    lens = [0 if n % 7 == 3 else K + n % 60 for n in range(N)]
    cache, table, _ = L.paged(lens, 16, dtype, seed=1)
    cache, table, lens = cache.to(DEV), table.to(DEV), _i32(lens)
    q = _rn(L.gen(2), N, K, H, 576)
    rows = [T.tree(K, n, 3, nodes=n % (K + 1)) for n in range(N)]                # some without any node
    rows[9] = [-2, -1, -2, 1, -2]                                                # places between nodes without one
    par = _i32(rows)
    out, lse = kda.latent_decode_tree(q, cache, dtype, table, lens, par, 0.07, want_lse=True)
    for at in (0, 9, N - 20):
        part = slice(at, at + 20)
        o, l = kda.latent_decode_tree(q[part].contiguous(), cache, dtype, table[part].contiguous(), lens[part].contiguous(),
                                      par[part].contiguous(), 0.07, want_lse=True)
        # (fewer sequences are cut into other parts: the sums' order differs)
        assert float((out[part].float() - o.float()).abs().max()) <= 2.0 ** -7 * float(o.float().abs().max())
        both = torch.isfinite(l)
        assert torch.equal(both, torch.isfinite(lse[part])) and float((lse[part] - l)[both].abs().max()) < 1e-4
    for n in range(N):
        for j in range(K):
            if not T.path(rows[n], j) or int(lens[n]) == 0:
                assert not out[n, j].any() and (lse[n, j] == float("-inf")).all()
            else:
                assert torch.isfinite(lse[n, j]).all()
    assert kda.kda_device_status() == kda.KDA_OK


@pytest.mark.parametrize("dtype", [BF, E4], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N,K,H", [(128, 2, 8), (129, 2, 8), (129, 4, 64), (300, 1, 16), (33, 8, 32), (32, 8, 32)])
def test_many_sequences_are_joined_alike(N, K, H, dtype):
    """Sequences enough to be counted by the attention itself, cut anywhere: what calls on a part of them give, chains and trees,
    empty ones and long ones among them."""
    lens = [0 if n % 11 == 5 else K + (n * 37) % 400 + (3000 if n % 50 == 7 else 0) for n in range(N)]
    cache, table, _ = L.paged(lens, 32, dtype, seed=N)
    cache, table, ld = cache.to(DEV), table.to(DEV), _i32(lens)
    q = _rn(L.gen(N + 1), N, K, H, 576)
    par = _i32([T.tree(K, n, 3, nodes=1 + n % K) for n in range(N)])
    calls = [lambda s: kda.latent_decode(q[s].contiguous(), cache, dtype, table[s].contiguous(), ld[s].contiguous(), 0.07, want_lse=True),
             lambda s: kda.latent_decode_tree(q[s].contiguous(), cache, dtype, table[s].contiguous(), ld[s].contiguous(),
                                              par[s].contiguous(), 0.07, want_lse=True)]
    for call in calls:
        out, lse = call(slice(0, N))
        for at in range(0, N, 25):
            part = slice(at, at + 25)
            o, l = call(part)
            # (cut into other parts: the sums' order differs; outputs are rounded to bf16, half a step of 2^-8 a side)
            assert float((out[part].float() - o.float()).abs().max()) <= 2.0 ** -7 * float(o.float().abs().max())
            fin = torch.isfinite(l)
            assert torch.equal(fin, torch.isfinite(lse[part]))
            assert not fin.any() or float((lse[part] - l)[fin].abs().max()) < 1e-4
    assert kda.kda_device_status() == kda.KDA_OK


@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
def test_bad_lengths_among_many_sequences(tree):
    """Lengths that are none count as 0 and are reported, where the attention itself writes what is empty."""
    N, K, H = 200, 3, 32
    lens = [K + n % 90 for n in range(N)]
    cache, table, _ = L.paged(lens, 16, BF, seed=3)
    cache, table = cache.to(DEV), table.to(DEV)
    q, par = _rn(L.gen(4), N, K, H, 576), _i32([T.tree(K, n, 2) for n in range(N)])
    call = lambda ld: (kda.latent_decode_tree(q, cache, BF, table, ld, par, 0.07, want_lse=True) if tree else
                       kda.latent_decode(q, cache, BF, table, ld, 0.07, want_lse=True))
    zero = list(lens)
    for n in (0, 7, 131, N - 1):
        zero[n] = 0
    want = call(_i32(zero))
    assert kda.kda_device_status() == kda.KDA_OK
    bad = list(zero)
    bad[0], bad[7], bad[N - 1] = -5, table.shape[1] * 16 + 1, 2 ** 31 - 1
    got = call(_i32(bad))
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for n in (0, 7, 131, N - 1):
        assert not want[0][n].any() and (want[1][n] == float("-inf")).all()
