"""The latent cache, both forms of the latent attention and the verification, together with the KDA
layer, as a serving loop uses them."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from kimi_delta_attention_06_gb300.hybrid_step import HybridModel, HybridServer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _prompts(m, lens, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randint(0, m.V, (n,), device=DEV, generator=g) for n in lens]


@pytest.mark.parametrize("cache", [kda.KDA_CACHE_BF16, kda.KDA_CACHE_E4M3])
def test_expanded_and_absorbed_forms_agree(cache):
    """The same tokens entered as one prompt, as two chunks (the second reads the first back from the
    cache), and as a prompt and a decode step give the same distributions.  The forms round at
    different places (per-head keys and values to bf16, or the absorbed query): bf16 steps of hidden
    rows of size ~1 and 256 terms, so the logits (x 0.25) agree to a few hundredths."""
    m = HybridModel(seed=2)
    lens = [130, 5, 64, 300]
    tok = _prompts(m, lens, 1)
    a = HybridServer(m, 4, 400, cache_dtype=cache)
    pa = a.prompt(tok)
    b = HybridServer(m, 4, 400, page=16, cache_dtype=cache)
    b.prompt([t[:n // 2 + 1] for t, n in zip(tok, lens)])
    pb = b.prompt([t[n // 2 + 1:] for t, n in zip(tok, lens)])
    c = HybridServer(m, 4, 400, page=48, cache_dtype=cache)
    c.prompt([t[:-2] for t in tok])
    K = 1
    g = torch.Generator(device=DEV).manual_seed(5)
    drafts = torch.stack([t[-1] for t in tok]).to(torch.int32)[:, None]
    # a draft that is always accepted (u = 0), then a token drawn: the state is that of all tokens
    q = torch.full((4, K, m.V), 1.0 / m.V, device=DEV)
    tokens, num = c.step(torch.stack([t[-2] for t in tok]).to(torch.int32), drafts, q,
                         torch.zeros(4, K, device=DEV), torch.rand(4, device=DEV, generator=g))
    torch.cuda.synchronize()
    assert kda.kda_device_status() == kda.KDA_OK
    assert num.tolist() == [2] * 4 and torch.equal(tokens[:, 0], drafts[:, 0])
    for s in (b, c):
        assert torch.equal(s.lens, a.lens)
        assert float((s.state - a.state).norm() / a.state.norm()) < 1e-2
    assert float((pa.log() - pb.log()).abs().max()) < 0.1
    # the next token's distribution from both histories
    nxt = tokens[:, 1].contiguous()
    pn = [s.prompt([t[None] for t in nxt]) for s in (a, c)]
    assert float((pn[0].log() - pn[1].log()).abs().max()) < 0.1


def test_speculative_loop_keeps_the_history():
    """After several steps with rejections, the server holds what a prompt of the accepted tokens gives."""
    m = HybridModel(seed=4, vocab=64)
    N, K = 5, 3
    lens = [40, 1, 64, 63, 20]
    tok = _prompts(m, lens, 7)
    srv = HybridServer(m, N, 200, page=16)
    p = srv.prompt(tok)
    g = torch.Generator(device=DEV).manual_seed(9)
    last = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
    hist = [list(t.tolist()) for t in tok]
    counts = set()
    q = (0.5 * p + 0.5 / m.V)[:, None].expand(-1, K, -1).contiguous()
    for _ in range(8):
        drafts = torch.multinomial(q.view(-1, m.V), 1, generator=g).view(N, K).to(torch.int32)
        tokens, num = srv.step(last, drafts, q, torch.rand(N, K, generator=g, device=DEV),
                               torch.rand(N, generator=g, device=DEV))
        for n in range(N):
            k = int(num[n])
            counts.add(k)
            hist[n] += [int(last[n])] + tokens[n, :k - 1].tolist()
        last = tokens.gather(1, (num - 1).long()[:, None])[:, 0].contiguous()
    assert len(counts) > 1                                     # accepted and rejected drafts both occur
    ref = HybridServer(m, N, 200, page=64)
    pr = ref.prompt([torch.tensor(h, device=DEV) for h in hist])
    torch.cuda.synchronize()
    assert kda.kda_device_status() == kda.KDA_OK
    assert torch.equal(ref.lens, srv.lens) and [len(h) for h in hist] == srv.lens.tolist()
    assert float((ref.state - srv.state).norm() / ref.state.norm()) < 1e-2
    pa = [s.prompt([t[None] for t in last]) for s in (ref, srv)]
    assert float((pa[0].log() - pa[1].log()).abs().max()) < 0.1
