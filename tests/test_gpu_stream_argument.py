"""The functions that allocate outputs, called with stream= another stream than the current one: neither their
copies of host offsets nor their outputs may share memory with work that is pending on either stream."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda, workloads
from tests import _latent as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
LONG = 300_000_000                                              # clocks: about 150 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _rn(g, *s):
    return torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)


def _latent_prefill(seed):
    g = L.gen(seed)
    x = [_rn(g, 500, 4, 192), _rn(g, 700, 4, 128), _rn(g, 700, 4, 128), _rn(g, 700, 64)]
    cq, ck = torch.tensor([0, 200, 500], dtype=torch.int32), torch.tensor([0, 250, 700], dtype=torch.int32)
    return lambda **o: kda.latent_prefill(*x, cq, ck, 0.07, want_lse=True, **o)


def _latent_gather(seed):
    cache, table, _ = L.paged([70, 33, 500], 16, kda.KDA_CACHE_E4M3, seed=seed)
    cache, table = cache.to(DEV), table.to(DEV)
    cu = torch.tensor([0, 70, 103, 603], dtype=torch.int32)
    return lambda **o: kda.latent_gather(cache, kda.KDA_CACHE_E4M3, table, cu, **o)


def _latent_decode(seed):
    cache, table, _ = L.paged([70, 33, 500], 16, kda.KDA_CACHE_BF16, seed=seed)
    cache, table, lens = cache.to(DEV), table.to(DEV), torch.tensor([70, 33, 500], dtype=torch.int32, device=DEV)
    q = _rn(L.gen(seed), 3, 2, 8, 576)
    return lambda **o: kda.latent_decode(q, cache, kda.KDA_CACHE_BF16, table, lens, 0.07, want_lse=True, **o)


def _verify_draft(seed):
    g = L.gen(seed)
    p = torch.softmax(torch.randn(64, 4, 3001, generator=g), -1)
    x = torch.randint(0, 3001, (64, 3), generator=g).to(torch.int32).to(DEV)
    u, us = torch.rand(64, 3, generator=g).to(DEV), torch.rand(64, generator=g).to(DEV)
    p = p.to(DEV)
    return lambda **o: kda.verify_draft(p, None, x, u, us, **o)


def _prefill(seed, start=False):
    c = workloads.prefill_case([200, 56, 300], H=2, D=64, seed=seed, la_shift=0.0, s0_std=0.02, ckpt_stride=64)
    x = [t.to(DEV) for t in (c.q, c.k, c.v, c.log_alpha, c.beta)]
    s0 = c.init_state.to(DEV)
    sp = torch.tensor([3, 0, 64], dtype=torch.int32) if start else None
    return lambda **o: kda.prefill(*x, c.cu_seqlens, init_state=s0, ckpt_stride=64, start_pos_host=sp, **o)


def _prefill_start(seed):
    return _prefill(seed, start=True)


def _decode_step(seed):
    d = workloads.decode_case(N=8, H=4, D=128, steps=1, seed=seed)
    x = [d.steps[0][k].to(DEV) for k in ("q", "k", "v", "log_alpha", "beta")]
    state = d.state.to(DEV)
    return lambda **o: (kda.decode_step(*x, state.clone() if not o else state, **o),)


CALLS = [_latent_prefill, _latent_gather, _latent_decode, _verify_draft, _prefill, _prefill_start, _decode_step]


def _garbage(like):
    """Take the small blocks and those of the outputs' sizes, and write over them."""
    keep = [torch.full((64 * (i % 8 + 1),), 1 << 30, dtype=torch.int32, device=DEV) for i in range(64)]
    keep += [torch.full_like(t, 77) for t in like for _ in range(2)]
    return keep


@pytest.mark.parametrize("make", CALLS, ids=[f.__name__[1:] for f in CALLS])
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_call_waits_on_a_busy_stream(make, raw):
    """The stream is busy for long after the call returns; the current stream's memory is written meanwhile."""
    call = make(3)
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
    assert kda.kda_device_status() == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del keep


@pytest.mark.parametrize("make", CALLS, ids=[f.__name__[1:] for f in CALLS])
def test_outputs_against_work_pending_on_the_current_stream(make):
    """Blocks of the outputs' sizes are freed with writes to them still pending on the current stream."""
    call = make(4)
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
    assert kda.kda_device_status() == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("make", CALLS, ids=[f.__name__[1:] for f in CALLS])
def test_outputs_freed_while_the_current_stream_reads_them(make):
    """Outputs are read by work pending on the current stream and dropped; the next call must not get them."""
    call, other = make(5), make(6)
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if make is _decode_step:                                    # (it moves its state: a call on a fresh copy each time)
        call = make(5)
        torch.cuda.synchronize()
    got = call(stream=s)
    s.synchronize()
    torch.cuda._sleep(LONG)
    read = [t.clone() for t in got]
    del got
    again = other(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
    del again
