"""Trees of drafts through the hybrid server: the append with rotation, both tree passes, the drawn tokens, the commit of the
path and the log probabilities together, against prompts of the same tokens."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from kimi_delta_attention_06_gb300.hybrid_step import HybridModel, HybridServer, main

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _prompts(m, lens, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randint(0, m.V, (n,), device=DEV, generator=g) for n in lens]


def _same(a, b, hist):
    """Two servers hold the same history: the tolerances of the linear steps (bf16 steps of hidden rows of size ~1 and 256
    terms, logits x 0.25: a few hundredths)."""
    assert a.lens.tolist() == b.lens.tolist() == [len(h) for h in hist]
    assert float((a.state - b.state).norm() / a.state.norm()) < 1e-2
    nxt = torch.randint(0, a.m.V, (a.N,), generator=torch.Generator().manual_seed(3)).to(DEV)
    p = [s.prompt([t[None] for t in nxt]) for s in (a, b)]
    assert float((p[0].log() - p[1].log()).abs().max()) < 0.1


@pytest.mark.parametrize("cache", [kda.KDA_CACHE_BF16, kda.KDA_CACHE_E4M3])
@pytest.mark.parametrize("rotary", [0.0, 10000.0])
def test_every_node_sees_its_path(cache, rotary):
    """The distribution after each node of a tree is the one after a prompt that ends with the node's path: read off the
    log probabilities of a path that draws follow on purpose (u_sample and drafts chosen from a first run)."""
    m = HybridModel(seed=2, vocab=64, rotary=rotary)
    lens = [130, 1, 64, 300]
    tok = _prompts(m, lens, 1)
    g = torch.Generator(device=DEV).manual_seed(6)
    last = torch.randint(0, m.V, (4,), device=DEV, generator=g).to(torch.int32)
    # drafts of place 1..: two children of the last token, two of place 2, one of place 4; a place without a draft
    parents = torch.tensor([0, 0, 2, 2, -1, 4], device=DEV).expand(4, -1).contiguous()
    drafts = torch.randint(0, m.V, (4, 6), device=DEV, generator=g).to(torch.int32)
    u = torch.rand(4, 7, device=DEV, generator=g)
    # the tokens that draws give along 0 -> 2 -> 4 -> 6, one place found a run
    for place, above in ((2, 0), (4, 2), (6, 4)):
        srv = HybridServer(m, 4, 400, page=16, cache_dtype=cache)
        srv.prompt(tok)
        tokens, num, _ = srv.step_tree(last, drafts, parents, u)
        depth = {0: 0, 2: 1, 4: 2}[above]
        drafts[:, place - 1] = tokens[:, depth]
        other = {2: 1, 4: 3}.get(place)
        if other:                                              # its sibling holds another token
            drafts[:, other - 1] = (tokens[:, depth] + 1) % m.V
    srv = HybridServer(m, 4, 400, page=16, cache_dtype=cache)
    srv.prompt(tok)
    tokens, num, (lp, rank, entropy, top_lp, top_tok) = srv.step_tree(last, drafts, parents, u, top=3)
    assert num.tolist() == [4] * 4 and (tokens[:, 4:] == -1).all()
    assert torch.equal(tokens[:, :3], drafts[:, [1, 3, 5]])
    hist = [t.tolist() + [int(l)] + d for t, l, d in zip(tok, last, drafts[:, [1, 3, 5]].tolist())]
    ref = HybridServer(m, 4, 400, cache_dtype=cache)
    for i in range(4):                                          # the target's distribution after each node of the path
        ids = [h[:len(t) + 1] if i == 0 else h[len(t) + i:len(t) + i + 1] for h, t in zip(hist, tok)]
        p = ref.prompt([torch.tensor(h, device=DEV) for h in ids]).double()
        want = p.gather(1, tokens[:, i:i + 1].long())[:, 0].log()
        assert float((lp[:, i] - want).abs().max()) < 0.1
        assert float((entropy[:, i] + (p * p.log()).sum(1)).abs().max()) < 0.1
        assert float((top_lp[:, i] - p.topk(3, dim=1).values.log()).abs().max()) < 0.1
    assert (lp[:, 4:] == 0).all() and (rank[:, 4:] == 0).all() and (top_tok[:, 4:] == -1).all()
    assert (rank[:, :4] >= 1).all()
    assert kda.kda_device_status() == kda.KDA_OK
    _same(ref, srv, hist)


def test_tree_loop_keeps_the_history():
    """After several steps with paths of different lengths, the server holds what a prompt of the accepted tokens gives."""
    m = HybridModel(seed=4, vocab=24, rotary=10000.0)
    N, K = 5, 21
    lens = [40, 1, 64, 63, 20]
    tok = _prompts(m, lens, 7)
    srv = HybridServer(m, N, 400, page=16)
    srv.prompt(tok)
    g = torch.Generator(device=DEV).manual_seed(9)
    last = torch.randint(0, m.V, (N,), device=DEV, generator=g).to(torch.int32)
    hist = [list(t.tolist()) for t in tok]
    counts = set()
    for _ in range(8):
        # 18 distinct children of the last token and three of some of them; sequence 1 has fewer
        drafts = torch.stack([torch.randperm(m.V, device=DEV, generator=g)[:K] for _ in range(N)]).to(torch.int32)
        parents = torch.cat([torch.zeros(N, 18, dtype=torch.long, device=DEV),
                             torch.randint(1, 19, (N, 3), device=DEV, generator=g)], dim=1)
        parents[1, 5:] = -1
        tokens, num, _ = srv.step_tree(last, drafts, parents, torch.rand(N, K + 1, generator=g, device=DEV))
        for n in range(N):
            k = int(num[n])
            counts.add(k)
            hist[n] += [int(last[n])] + tokens[n, :k - 1].tolist()
        last = tokens.gather(1, (num - 1).long()[:, None])[:, 0].contiguous()
    assert len(counts) > 1
    ref = HybridServer(m, N, 400, page=64)
    ref.prompt([torch.tensor(h, device=DEV) for h in hist])
    assert kda.kda_device_status() == kda.KDA_OK
    _same(ref, srv, hist)


def test_rotation_leaves_a_model_without_positions_alone():
    """Frequencies of 0 turn nothing: the rotating append in place of the plain one gives the same bits."""
    a = HybridModel(seed=5, vocab=64)
    b = HybridModel(seed=5, vocab=64)
    b.rotary = True
    tok = _prompts(a, [70, 3], 2)
    sa, sb = HybridServer(a, 2, 200), HybridServer(b, 2, 200)
    assert torch.equal(sa.prompt(tok), sb.prompt(tok)) and torch.equal(sa.cache, sb.cache)
    g = torch.Generator(device=DEV).manual_seed(1)
    last, drafts = (torch.randint(0, 64, s, device=DEV, generator=g).to(torch.int32) for s in ((2,), (2, 3)))
    q, ua, us = (torch.rand(*s, device=DEV, generator=g) for s in ((2, 3, 64), (2, 3), (2,)))
    for x, y in zip(sa.step(last, drafts, q, ua, us), sb.step(last, drafts, q, ua, us)):
        assert torch.equal(x, y)
    assert torch.equal(sa.state, sb.state) and torch.equal(sa.cache, sb.cache)


def test_command(capsys):
    main(["--seqs", "3", "--prompt", "50", "--draft", "2", "--branches", "3", "--steps", "3", "--rotary", "10000"])
    assert "3 steps of 6 drafted tokens" in capsys.readouterr().out


def test_without_drafts_and_with_parents_that_are_none():
    """A tree of the last token alone is a step without drafts; a place whose parent is not before it holds no node, is never
    part of a path, and is reported."""
    m = HybridModel(seed=6, vocab=32, rotary=10000.0)
    tok = _prompts(m, [30, 7], 3)
    last = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    a, b = HybridServer(m, 2, 100), HybridServer(m, 2, 100)
    a.prompt(tok), b.prompt(tok)
    u = torch.rand(2, 1, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    empty = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    tokens, num, scores = a.step_tree(last, empty, empty.long(), u)
    b.step(last, empty, torch.empty(2, 0, m.V, device=DEV), torch.empty(2, 0, device=DEV), u[:, 0].contiguous())
    assert num.tolist() == [1, 1] and tokens.shape == (2, 1) and scores[3] is None
    assert kda.kda_device_status() == kda.KDA_OK
    _same(a, b, [t.tolist() + [int(l)] for t, l in zip(tok, last)])
    # every token is drafted below place 1, which is below itself
    c = HybridServer(m, 2, 200)
    c.prompt(tok)
    drafts = torch.arange(33, device=DEV).clamp_max(31).to(torch.int32).expand(2, -1).contiguous()
    parents = torch.ones(2, 33, dtype=torch.long, device=DEV)
    _, num, _ = c.step_tree(last, drafts, parents, torch.rand(2, 34, device=DEV))
    assert num.tolist() == [1, 1]
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
