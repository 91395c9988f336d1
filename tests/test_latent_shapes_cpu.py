"""Shapes that do not fit together are refused by the binding of the latent attention and verification calls: the
library sees addresses only and would read past the smaller tensor.  (On the CPU: a call that passed every check
would say that its tensors are not on the GPU.)"""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def bf(*s):
    return torch.zeros(*s, dtype=BF)


def i32(*s):
    return torch.zeros(*s, dtype=I32)


def _refused(fn, good, bad):
    """`good` passes all checks but the last; each of `bad` replaces arguments and is refused for its shape."""
    with pytest.raises(ValueError, match="on the GPU"):
        fn(**good)
    for b in bad:
        with pytest.raises(ValueError) as e:
            fn(**{**good, **b})
        assert "on the GPU" not in str(e.value), {k: tuple(v.shape) for k, v in b.items()}


def _cache(dt=kda.KDA_CACHE_E4M3, pages=4, page=16):
    return torch.zeros(pages, page, {0: 1152, 1: 656}[dt], dtype=torch.uint8)


def test_append():
    good = dict(c=bf(5, 512), k_rope=bf(5, 64), cache=_cache(), cache_dtype=1, slots=i32(5), stream=0)
    _refused(kda.latent_append, good, [
        dict(k_rope=bf(4, 64)), dict(slots=i32(4)), dict(c=bf(5, 448)), dict(c=bf(2, 3, 512)),
        dict(k_rope=bf(5, 32)), dict(c=bf(1, 100), k_rope=bf(1, 64), slots=i32(1)),
        dict(c=bf(1, 512), k_rope=bf(1, 8), slots=i32(1)), dict(c=bf(5 * 512)), dict(cache=_cache(0))])
    low = dict(good, total_tokens=5)
    _refused(kda.kda_latent_append, low, [dict(total_tokens=6), dict(slots=i32(3)), dict(k_rope=bf(4, 64))])


@pytest.mark.parametrize("dt", [0, 1])
def test_gather(dt):
    good = dict(cache=_cache(dt), cache_dtype=dt, block_table=i32(2, 3), cu_seqlens_host=torch.tensor([0, 5, 9], dtype=I32),
                cu_seqlens=i32(3), start_pos=i32(2), stream=0)
    bad = [dict(block_table=i32(1, 3)), dict(block_table=i32(6)), dict(cu_seqlens=i32(2)), dict(start_pos=i32(1)),
           dict(cache=_cache(1 - dt))]
    low = dict(good, num_seqs=2, total_tokens=9, c=bf(9, 512), k_rope=bf(9, 64))
    _refused(kda.kda_latent_gather, low, bad + [dict(c=bf(8, 512)), dict(k_rope=bf(8, 64)), dict(c=bf(9, 500)),
                                                dict(k_rope=bf(9, 56)), dict(cu_seqlens_host=i32(2))])
    _refused(kda.latent_gather, good, bad)


@pytest.mark.parametrize("dt", [0, 1])
def test_decode(dt):
    good = dict(q=bf(3, 2, 8, 576), cache=_cache(dt), cache_dtype=dt, block_table=i32(3, 2), seq_lens=i32(3), sm_scale=0.07,
                stream=0)
    bad = [dict(q=bf(3, 2, 8, 192)),                           # not absorbed
           dict(q=bf(3, 2, 8, 512)), dict(seq_lens=i32(2)), dict(block_table=i32(2, 2)), dict(block_table=i32(6))]
    _refused(kda.latent_decode, good, bad)
    low = dict(good, N=3, K=2, H=8, out=bf(3, 2, 8, 512), lse=None)
    _refused(kda.kda_latent_decode, low, bad + [dict(N=4), dict(K=3), dict(H=9)])


def test_prefill():
    cu = torch.tensor([0, 4, 9], dtype=I32)
    good = dict(q=bf(9, 4, 192), k=bf(9, 4, 128), v=bf(9, 4, 128), k_rope=bf(9, 64), cu_q_host=cu, cu_k_host=cu, sm_scale=0.07,
                cu_q=i32(3), cu_k=i32(3), stream=0)
    bad = [dict(q=bf(9, 4, 128)), dict(q=bf(9, 4, 576)), dict(v=bf(8, 4, 128)), dict(v=bf(9, 3, 128)), dict(k=bf(9, 3, 128)),
           dict(k=bf(9, 4, 120)), dict(v=bf(9, 4, 64)), dict(k_rope=bf(8, 64)), dict(k_rope=bf(9, 32)), dict(cu_q=i32(2)),
           dict(cu_k=i32(2)), dict(cu_k_host=cu[:2].contiguous()), dict(k=bf(9, 1, 128), v=bf(9, 1, 128))]
    _refused(kda.latent_prefill, good, bad)
    low = dict(good, num_seqs=2, total_q=9, total_k=9, H=4, causal=1, out=bf(9, 4, 128), lse=None)
    _refused(kda.kda_latent_prefill, low, bad + [dict(total_q=10), dict(total_k=10), dict(H=5), dict(num_seqs=3)])


def test_verify():
    f = lambda *s: torch.zeros(*s)
    good = dict(target_probs=f(3, 5, 7), draft_probs=f(3, 4, 7), draft_tokens=i32(3, 4), u_accept=f(3, 4), u_sample=f(3),
                num_draft=i32(3), stream=0)
    bad = [dict(draft_probs=f(3, 3, 7)), dict(draft_probs=f(3, 4, 6)), dict(draft_probs=f(2, 4, 7)), dict(draft_tokens=i32(3, 3)),
           dict(u_accept=f(3, 3)), dict(u_sample=f(2)), dict(num_draft=i32(2)), dict(draft_tokens=i32(2, 4))]
    _refused(kda.verify_draft, good, bad + [dict(u_accept=f(4, 3)), dict(draft_tokens=i32(4, 3))])
    low = dict(good, N=3, K=4, V=7, tokens=i32(3, 5), num_tokens=i32(3))
    _refused(kda.kda_verify_draft, low, bad + [dict(K=5), dict(V=8), dict(N=4), dict(target_probs=f(3, 4, 7))])


def test_outputs(monkeypatch):
    """Outputs that the caller brings are looked at after the inputs (taken to be on the GPU here)."""
    seen = []
    monkeypatch.setattr(kda, "_on_gpu", lambda *t: seen.append(t))
    q = dict(q=bf(3, 2, 8, 576), cache=_cache(), cache_dtype=1, block_table=i32(3, 2), seq_lens=i32(3), N=3, K=2, H=8,
             sm_scale=0.07, stream=0)
    for out, lse in ((bf(3, 2, 7, 512), None), (bf(3, 2, 8, 512), torch.zeros(3, 2, 7))):
        with pytest.raises(ValueError, match="elements are needed"):
            kda.kda_latent_decode(out=out, lse=lse, **q)
    f = lambda *s: torch.zeros(*s)
    for tokens, num in ((i32(3, 4), i32(3)), (i32(3, 5), i32(2))):
        with pytest.raises(ValueError, match="elements are needed"):
            kda.kda_verify_draft(f(3, 5, 7), None, i32(3, 4), None, f(3, 4), f(3), 3, 4, 7, tokens, num, stream=0)
    cu = torch.tensor([0, 4, 9], dtype=I32)
    with pytest.raises(ValueError, match="elements are needed"):
        kda.kda_latent_prefill(bf(9, 4, 192), bf(9, 4, 128), bf(9, 4, 128), bf(9, 64), i32(3), cu, i32(3), cu, 2, 9, 9, 4, 1, 0.07,
                               bf(9, 3, 128), None, stream=0)
    assert seen


def test_larger_tensors_pass():
    """Buffers that a server keeps may be longer than the call, rows wider than what is read of them."""
    with pytest.raises(ValueError, match="on the GPU"):
        kda.kda_verify_draft(torch.zeros(3, 5, 16), torch.zeros(3, 4, 16), i32(3, 4), None, torch.zeros(3, 4), torch.zeros(3), 3, 4, 13,
                             i32(3, 5), i32(3), stream=0)
    with pytest.raises(ValueError, match="on the GPU"):
        kda.latent_append(bf(3, 576), bf(3, 72), _cache(), 1, i32(3), stream=0)
    with pytest.raises(ValueError, match="on the GPU"):
        kda.latent_decode(bf(3, 2, 8, 576), _cache(), 1, i32(9, 4), i32(9), 0.07, stream=0)
    with pytest.raises(ValueError, match="on the GPU"):
        kda.latent_append(bf(3, 512), bf(3, 64), _cache(), 1, i32(9), stream=0)
