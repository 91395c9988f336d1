"""Host-side refusals of the rotated append, the tree operators and the log probabilities: by the C ABI (the pointers
here are never followed) and by the binding, for tensors that do not fit together (on the CPU, where a call that
passed every check would say that its tensors are not on the GPU)."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda

BAD, UNSUP, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load()


def _call(lib, name, order, base, **over):
    a = dict(base)
    a.update(over)
    return getattr(lib, name)(*(a[k] for k in order))


def test_append_rope_refusals(lib):
    order = ["c", "ldc", "r", "ldr", "cache", "dt", "pages", "page", "slots", "pos", "freq", "inter", "q", "ldq", "hdq", "qo",
             "ldo", "hdo", "T", "H", "st"]
    base = dict(c=0x1000, ldc=576, r=0x2000, ldr=576, cache=0x3000, dt=1, pages=4, page=64, slots=0x4000, pos=0x5000,
                freq=0x6000, inter=0, q=0x7000, ldq=768, hdq=192, qo=0x8000, ldo=256, hdo=64, T=3, H=4, st=None)
    f = lambda **o: _call(lib, "kda_latent_append_rope", order, base, **o)
    for o in (dict(dt=2), dict(pages=-1), dict(page=0), dict(T=-1), dict(ldc=504), dict(ldc=577), dict(ldr=56), dict(c=None),
              dict(r=None), dict(slots=None), dict(pos=None), dict(freq=None), dict(cache=None), dict(c=0x1008),
              dict(r=0x2004), dict(slots=0x4002), dict(pos=0x5001), dict(freq=0x6002), dict(inter=2), dict(inter=-1),
              dict(q=None), dict(qo=None), dict(H=0), dict(H=-1), dict(q=0x7008), dict(qo=0x8004), dict(ldq=60), dict(hdq=56),
              dict(hdq=100), dict(ldo=63), dict(hdo=0), dict(H=1 << 30, T=4)):
        assert f(**o) == BAD, o
    assert f(page=24) == UNSUP and f(page=2048) == UNSUP
    assert f(T=0, c=None, r=None, slots=None) == OK


def test_decode_tree_refusals(lib):
    order = ["q", "k", "v", "la", "beta", "pool", "slots_n", "slots", "parents", "out", "odt", "N", "K", "H", "Dk", "Dv",
             "decay", "st"]
    base = dict(q=0x1000, k=0x2000, v=0x3000, la=0x4000, beta=0x5000, pool=0x6000, slots_n=3, slots=0x7000, parents=0x8000,
                out=0x9000, odt=0, N=2, K=5, H=4, Dk=128, Dv=128, decay=0, st=None)
    f = lambda **o: _call(lib, "kda_decode_tree", order, base, **o)
    for o in (dict(N=-1), dict(K=-1), dict(H=0), dict(slots_n=-1), dict(slots_n=0), dict(decay=3), dict(decay=2), dict(la=None),
              dict(odt=2), dict(q=None), dict(k=None), dict(v=None), dict(beta=None), dict(pool=None), dict(parents=None),
              dict(out=None), dict(q=0x1008), dict(pool=0x6004), dict(out=0x9002), dict(slots=0x7001), dict(parents=0x8002),
              dict(slots=None, slots_n=1), dict(N=1 << 24, K=64, H=4)):
        assert f(**o) == BAD, o
    assert f(Dk=96) == UNSUP and f(Dv=64) == UNSUP and f(K=kda.KDA_TREE_MAX_NODES + 1) == UNSUP
    assert f(N=0) == OK and f(K=0) == OK


def test_latent_decode_tree_refusals(lib):
    order = ["q", "cache", "dt", "pages", "page", "table", "mp", "lens", "parents", "N", "K", "H", "scale", "out", "lse", "st"]
    base = dict(q=0x1000, cache=0x2000, dt=0, pages=4, page=16, table=0x3000, mp=2, lens=0x4000, parents=0x7000, N=2, K=3, H=32,
                scale=0.07, out=0x5000, lse=None, st=None)
    f = lambda **o: _call(lib, "kda_latent_decode_tree", order, base, **o)
    for o in (dict(dt=3), dict(N=-1), dict(K=-1), dict(H=0), dict(mp=-1), dict(scale=float("nan")), dict(q=None),
              dict(lens=None), dict(out=None), dict(table=None), dict(parents=None), dict(parents=0x7002), dict(q=0x1008),
              dict(out=0x5008), dict(lens=0x4001), dict(lse=0x6002), dict(cache=0x2004), dict(mp=1 << 28)):
        assert f(**o) == BAD, o
    assert f(K=17) == UNSUP and f(K=65, H=1) == UNSUP and f(page=40) == UNSUP
    assert f(N=0, parents=None) == OK and f(K=0, parents=None) == OK


def test_token_logprobs_refusals(lib):
    order = ["x", "dt", "ld", "tok", "R", "V", "top", "scale", "lp", "rank", "ent", "tl", "tt", "st"]
    base = dict(x=0x1000, dt=0, ld=100, tok=0x2000, R=3, V=100, top=5, scale=1.0, lp=0x3000, rank=0x4000, ent=0x5000, tl=0x6000,
                tt=0x7000, st=None)
    f = lambda **o: _call(lib, "kda_token_logprobs", order, base, **o)
    for o in (dict(R=-1), dict(V=0), dict(top=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(scale=9e-7), dict(scale=1.1e6), dict(dt=2), dict(ld=99), dict(x=None), dict(x=0x1001), dict(dt=1, x=0x1002),
              dict(tok=None), dict(lp=None), dict(tok=None, lp=None), dict(tl=None), dict(tt=None), dict(tok=0x2002),
              dict(rank=0x4001), dict(ent=0x5002), dict(tl=0x6002), dict(tt=0x7001), dict(R=1 << 27)):
        assert f(**o) == BAD, o
    assert f(top=kda.KDA_LOGPROBS_MAX_TOP + 1) == UNSUP and f(V=(1 << 30) + 1, ld=1 << 31) == UNSUP
    assert f(R=0, x=None) == OK


# ---- the binding -----------------------------------------------------------------------------

def _refused(fn, good, bad, also=ValueError):
    with pytest.raises(ValueError, match="on the GPU"):
        fn(**good)
    for b in bad:
        with pytest.raises(also) as e:
            fn(**{**good, **b})
        assert "on the GPU" not in str(e.value), {k: getattr(v, "shape", v) for k, v in b.items()}


def _z(dt):
    return lambda *s: torch.zeros(*s, dtype=dt)


bf, f32, i32 = _z(BF), _z(F32), _z(I32)


def test_binding_append_rope():
    good = dict(c=bf(5, 512), k_rope=bf(5, 64), cache=torch.zeros(4, 16, 656, dtype=torch.uint8), cache_dtype=1, slots=i32(5),
                positions=i32(5), inv_freq=f32(32), q=bf(5, 4, 192)[..., 128:], q_out=bf(5, 4, 576)[..., 512:], stream=0)
    _refused(kda.latent_append_rope, good, [
        dict(k_rope=bf(4, 64)), dict(slots=i32(4)), dict(positions=i32(4)), dict(inv_freq=f32(31)), dict(c=bf(5, 448)),
        dict(q=bf(4, 4, 64)), dict(q=bf(5, 4, 32)), dict(q=bf(5, 256)), dict(q_out=bf(5, 3, 64)), dict(q_out=bf(4, 4, 64)),
        dict(q=None), dict(q=bf(5, 4, 128)[..., ::2]), dict(cache=torch.zeros(4, 16, 1152, dtype=torch.uint8))])
    _refused(kda.latent_append_rope, good, [dict(positions=torch.zeros(5)), dict(inv_freq=torch.zeros(32).double()),
                                            dict(q=f32(5, 4, 64)), dict(q_out=f32(5, 4, 64))], TypeError)
    low = dict(good, total_tokens=5, H=4, interleaved=0)
    _refused(kda.kda_latent_append_rope, low, [dict(total_tokens=6), dict(H=5)])


def test_binding_decode_tree():
    good = dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 4, 64), v=bf(2, 3, 4, 64), log_alpha=f32(2, 3, 4, 64), beta=bf(2, 3, 4),
                state_pool=f32(3, 4, 64, 64), parents=i32(2, 3), state_slots=i32(2), stream=0)
    _refused(kda.decode_tree, good, [
        dict(k=bf(2, 3, 4, 32)), dict(v=bf(2, 2, 4, 64)), dict(log_alpha=f32(2, 3, 4)), dict(beta=bf(2, 3, 3)),
        dict(state_pool=f32(3, 4, 64, 32)), dict(parents=i32(2, 2)), dict(state_slots=i32(1)), dict(q=bf(2, 3, 64, 4).transpose(2, 3))])
    _refused(kda.decode_tree, good, [dict(parents=f32(2, 3)), dict(q=f32(2, 3, 4, 64)), dict(state_pool=bf(3, 4, 64, 64))], TypeError)


def test_binding_latent_decode_tree():
    good = dict(q=bf(3, 2, 8, 576), cache=torch.zeros(4, 16, 1152, dtype=torch.uint8), cache_dtype=0, block_table=i32(3, 2),
                seq_lens=i32(3), parents=i32(3, 2), sm_scale=0.07, stream=0)
    _refused(kda.latent_decode_tree, good, [dict(q=bf(3, 2, 8, 512)), dict(seq_lens=i32(2)), dict(block_table=i32(2, 2)),
                                            dict(parents=i32(3, 1))])
    _refused(kda.latent_decode_tree, good, [dict(parents=f32(3, 2)), dict(parents=i32(3, 2).long())], TypeError)


def test_binding_token_logprobs():
    good = dict(logits=bf(4, 100), tokens=i32(4), top=3, stream=0)
    _refused(kda.token_logprobs, good, [dict(tokens=i32(3)), dict(logits=bf(100)), dict(logits=bf(100, 4).t(), tokens=i32(4))])
    _refused(kda.token_logprobs, good, [dict(logits=torch.zeros(4, 100, dtype=torch.float16)), dict(tokens=f32(4))], TypeError)
    low = dict(good, R=4, V=100, scale=1.0, logprob=f32(4), rank=i32(4), entropy=f32(4), top_logprob=f32(4, 3), top_token=i32(4, 3))
    _refused(kda.kda_token_logprobs, low, [dict(R=5), dict(V=101)])
