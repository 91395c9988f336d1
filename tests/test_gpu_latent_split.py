"""Expanded latent attention of few queries over many keys: the keys are split over CTAs and joined."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L
from tests.test_gpu_latent import DEV, _ok, _prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


# (128 keys a tile; a split takes at least 8 tiles out of the longest series)
@pytest.mark.parametrize("lens_q,lens_k,H,causal,layout", [
    ([1], [5000], 4, True, "dense"),
    ([1], [2561], 1, False, "joint"),                          # 21 tiles, the last of one key
    ([130], [4000], 3, True, "heads"),                         # the second tile has two rows
    ([5, 0, 129, 3], [4000, 7, 129, 6000], 2, True, "dense"),  # split and whole sequences side by side
    ([257, 64], [3000, 64], 2, False, "joint"),
    ([3300], [3000], 1, True, "dense"),                        # rows that see nothing
    ([3, 4], [2, 4100], 2, True, "joint"),
])
def test_split_keys(lens_q, lens_k, H, causal, layout):
    some = [0, 1, 63, 64, 127, 128, 129, 255, 256, 299, 300, 301, 427, 428, 2000]
    _prefill(lens_q, lens_k, H, seed=sum(lens_q) + H, causal=causal, layout=layout, rows=some if min(lens_q) > 0 else None)


@pytest.mark.parametrize("scale,q_std", [(192 ** -0.5, 30.0), (0.0, 1.0), (-0.07, 4.0)])
def test_split_scales(scale, q_std):
    """Sharp scores: whole parts have no weight beside the one with the largest score."""
    _prefill([40], [4500], 2, seed=6, scale=scale, q_std=q_std, rows=[0, 20])


def _inputs(Lq, Lk, H, seed):
    g = L.gen(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    return mk(Lq, H, 192), mk(Lk, H, 128), mk(Lk, H, 128), mk(Lk, 64)


def test_split_rows_that_do_not_see_a_nan():
    Lq, Lk, H, scale = 4, 4000, 2, 192 ** -0.5
    q, k, v, r = _inputs(Lq, Lk, H, 9)
    k[-1] = float("nan")                                       # seen by the last query only
    v[-2] = float("inf")                                       # by the last two
    out, lse = kda.latent_prefill(q.to(DEV), k.to(DEV), v.to(DEV), r.to(DEV), torch.tensor([0, Lq], dtype=torch.int32),
                                  torch.tensor([0, Lk], dtype=torch.int32), scale, want_lse=True)
    _ok()
    assert torch.isnan(out[3].float()).all() and torch.isnan(lse[3]).all()
    assert not torch.isfinite(out[2].float()).any() and torch.isfinite(lse[2]).all()
    for h in range(H):
        key = torch.cat([k[:, h], r], dim=1).double()
        L.check_rows(out[:2, h], lse[:2, h], [L.attend(q[i, h].double(), key[:i + 1 + Lk - Lq], v[:i + 1 + Lk - Lq, h].double(),
                                                       scale, i + 1 + Lk - Lq) for i in range(2)])


def test_split_in_a_graph_and_again():
    q, k, v, r = (x.to(DEV) for x in _inputs(70, 5000, 4, 11))
    cq, ck = torch.tensor([0, 70], dtype=torch.int32), torch.tensor([0, 5000], dtype=torch.int32)
    cqd, ckd = cq.to(DEV), ck.to(DEV)
    call = lambda: kda.latent_prefill(q, k, v, r, cq, ck, 0.07, cu_q=cqd, cu_k=ckd, want_lse=True)
    a = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b = call()
    for _ in range(3):
        b[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        _ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
