"""NaN and infinities in the keys and values of the expanded form: they reach the rows that see them and no others,
and cost no time."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


def _best(call):
    """Shortest of several passes, in microseconds."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(3):
        call()
    best = math.inf
    for _ in range(8):
        ev[0].record()
        call()
        ev[1].record()
        torch.cuda.synchronize()
        best = min(best, ev[0].elapsed_time(ev[1]) * 1e3)
    return best


# (a call from Python takes 20 us or so of its own: a few microseconds more of that are not the kernel's)
def _near(got, clean):
    assert got <= 2 * clean + 20, f"{got:.0f} us against {clean:.0f} us without a NaN"


def _expanded(lens_q, lens_k, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    tq, tk = sum(lens_q), sum(lens_k)
    cu = [torch.nn.functional.pad(torch.tensor(x).cumsum(0), (1, 0)).to(torch.int32) for x in (lens_q, lens_k)]
    return [rn(tq, H, 192), rn(tk, H, 128), rn(tk, H, 128), rn(tk, 64)], cu, [c.to(DEV) for c in cu]


def _run(x, cu, cud, causal):
    return kda.latent_prefill(*x, *cu, 192 ** -0.5, causal=causal, cu_q=cud[0], cu_k=cud[1], want_lse=True)


# (one split over keys, one whole; a NaN in an early key, an early value, one channel of it, and a late value)
@pytest.mark.parametrize("lens_q,lens_k,H", [([4096], [4096], 4), ([300], [8000], 4), ([2048, 2100], [2048, 2100], 12)])
@pytest.mark.parametrize("where", ["key", "value", "channel", "late"])
def test_expanded_with_a_nan(lens_q, lens_k, H, where):
    x, cu, cud = _expanded(lens_q, lens_k, H, seed=H)
    call = lambda: _run(x, cu, cud, True)
    out, lse = call()
    clean = _best(call)
    Lq, Lk = lens_q[0], lens_k[0]
    t = Lk - 100 if where == "late" else 0
    if where == "key":
        x[1][t] = math.nan
    elif where == "channel":
        x[2][t, :, 77] = math.nan
    else:
        x[2][t] = math.nan
    got, got_lse = call()
    _ok()
    first = max(0, t - (Lk - Lq))                               # the first query that sees it
    assert torch.equal(got[:first], out[:first]) and torch.equal(got_lse[:first], lse[:first])
    assert torch.equal(got[Lq:], out[Lq:]) and torch.equal(got_lse[Lq:], lse[Lq:])
    if where == "channel":
        assert torch.isnan(got[:Lq, :, 77].float()).all() and torch.equal(got[..., :77], out[..., :77])
        assert torch.equal(got[..., 78:], out[..., 78:])
    else:
        assert torch.isnan(got[first:Lq].float()).all()
    assert torch.isnan(got_lse[:Lq]).all() if where == "key" else torch.equal(got_lse, lse)
    _near(_best(call), clean)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens_q,lens_k,H", [([4000, 200], [4000, 200], 4), ([200, 3], [8100, 50], 2)])
def test_expanded_neighbour_of_nothing_but_nan(causal, lens_q, lens_k, H):
    """The next sequence's keys and values, which share the first one's last tile, are all NaN."""
    x, cu, cud = _expanded(lens_q, lens_k, H, seed=7)
    call = lambda: _run(x, cu, cud, causal)
    out, lse = call()
    clean = _best(call)
    for i in (1, 2, 3):
        x[i][lens_k[0]:] = math.nan
    got, got_lse = call()
    _ok()
    a = lens_q[0]
    assert torch.equal(got[:a], out[:a]) and torch.equal(got_lse[:a], lse[:a])
    assert torch.isnan(got[a:].float()).all() and torch.isnan(got_lse[a:]).all()
    _near(_best(call), clean)


@pytest.mark.parametrize("Lq,Lk,H", [(300, 300, 2), (129, 257, 1), (200, 5000, 2)])
def test_expanded_infinite_values(Lq, Lk, H):
    """Infinities of either sign and NaN in single channels, on the diagonal and before it: the rows that see
    them get them, in those channels alone; both signs make NaN."""
    x, cu, cud = _expanded([Lq], [Lk], H, seed=11)
    out, lse = _run(x, cu, cud, True)
    base = Lk - Lq
    marks = [(base + 20, 3, math.inf), (base + 21, 70, -math.inf), (base + 100, 3, -math.inf), (base + 127, 127, math.nan),
             (base + 128, 0, math.inf), (Lk - 1, 64, -math.inf), (0, 9, math.inf), (base + 50, 9, math.inf)]
    for t, c, v in marks:
        x[2][t, :, c] = v
    got, got_lse = _run(x, cu, cud, True)
    _ok()
    want = out.clone().float()
    for i in range(Lq):
        for c in {m[1] for m in marks}:
            seen = [v for t, ch, v in marks if ch == c and t <= i + base]
            if seen:
                want[i, :, c] = sum(seen)
    assert torch.equal(got_lse, lse)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got.float()[keep], want[keep])
