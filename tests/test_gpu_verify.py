"""GPU parity of the verification of drafted tokens against a plain form in exact rational
comparisons and 64-bit sums."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests._latent import gen

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _clean(x):
    x = x.double()
    return torch.where((x > 0) & torch.isfinite(x), x, torch.zeros_like(x))


def plain(p, q, x, u, us, nd=None):
    """(tokens, counts, allowed): `allowed[n]` are the tokens that sums off by 1e-11 of the total
    could draw (one token but for thresholds that lie on a border)."""
    N, K1, V = p.shape
    toks = torch.full((N, K1), -1, dtype=torch.int64)
    num = torch.zeros(N, dtype=torch.int64)
    allowed = []
    for n in range(N):
        d = K1 - 1 if nd is None else int(nd[n])
        a = 0
        while a < d:
            t = int(x[n, a])
            pv, qv = float(p[n, a, t]), 1.0 if q is None else float(q[n, a, t])
            if not float(u[n, a]) * qv < pv:
                break
            a += 1
        row = _clean(p[n, a])
        w = row
        if a < d:
            if q is None:
                w = row.clone()
                w[int(x[n, a])] = 0
            else:
                w = (row - _clean(q[n, a])).clamp_min(0)
            if not float(w.sum()) > 0:
                w = row
        toks[n, :a] = x[n, :a].long()
        num[n] = a + 1
        c = w.cumsum(0)
        total = float(c[-1])
        if total > 0:
            want = float(us[n]) * total
            near = ((c > want - 1e-11 * total) & (c - w <= want + 1e-11 * total) & (w > 0)).nonzero()[:, 0].tolist()
            toks[n, a] = int((c > want).to(torch.uint8).argmax())
            allowed.append(set(near))
        else:
            allowed.append({-1})
    return toks, num, allowed


def _case(N, K, V, seed, sharp=2.0, close=0.5, draft=True, pad=0):
    g = gen(seed)
    logits = torch.randn(N, K + 1, V + pad, generator=g) * sharp
    p = torch.softmax(logits[..., :V], -1)
    q = torch.softmax(logits[:, :K, :V] + close * torch.randn(N, K, V, generator=g), -1) if draft else None
    pick = q if draft else p[:, :K]
    x = torch.multinomial(pick.reshape(-1, V), 1, generator=g).view(N, K).to(torch.int32) if K else torch.zeros(N, 0, dtype=torch.int32)
    return p, q, x, torch.rand(N, K, generator=g), torch.rand(N, generator=g)


def _dev(t):
    return None if t is None else t.to(DEV)


def _check(p, q, x, u, us, nd=None):
    t, m = kda.verify_draft(_dev(p), _dev(q), _dev(x), _dev(u), _dev(us), num_draft=_dev(nd))
    assert kda.kda_device_status() == kda.KDA_OK
    wt, wm, allowed = plain(p, q, x, u, us, nd)
    t, m = t.cpu().long(), m.cpu().long()
    assert torch.equal(m, wm)
    for n in range(p.shape[0]):
        a = int(wm[n]) - 1
        assert torch.equal(t[n, :a], wt[n, :a]) and (t[n, a + 1:] == -1).all()
        assert int(t[n, a]) in allowed[n], (n, int(t[n, a]), int(wt[n, a]))
    return wm


@pytest.mark.parametrize("N,K,V,draft", [
    (1, 1, 1, True), (3, 2, 2, False), (5, 4, 31, True), (2, 3, 33, False), (7, 5, 1000, True),
    (4, 3, 8193, True), (2, 2, 40001, False), (1, 3, 131072, True), (200, 4, 5003, True), (400, 2, 999, False),
])
def test_verify(N, K, V, draft):
    _check(*_case(N, K, V, seed=N + K + V, draft=draft))


def test_all_counts_occur_and_thresholds_sweep():
    m = _check(*_case(64, 4, 257, seed=2, close=1.0))
    assert set(m.tolist()) == {1, 2, 3, 4, 5}
    # one row, every threshold: the whole inverse distribution
    p, q, x, u, us = _case(1, 1, 300, seed=3)
    n = 128
    us = torch.cat([torch.linspace(0, 1 - 2.0 ** -24, n - 1), torch.tensor([1 - 2.0 ** -24])])
    big = lambda t: t.expand(n, *t.shape[1:]).contiguous()
    _check(big(p), big(q), big(x), torch.full((n, 1), 0.999999), us)


def test_no_draft_tokens_and_ragged_counts():
    _check(*_case(5, 0, 777, seed=4, draft=False))
    p, q, x, u, us = _case(6, 4, 500, seed=5)
    _check(p, q, x, u, us, nd=torch.tensor([0, 1, 2, 3, 4, 2], dtype=torch.int32))


def test_edges_of_acceptance():
    N, V = 6, 8
    p = torch.full((N, 2, V), 1 / V)
    q = torch.full((N, 1, V), 1 / V)
    x = torch.full((N, 1), 3, dtype=torch.int32)
    u = torch.tensor([[0.0], [1 - 2.0 ** -24], [0.5], [0.5], [0.5], [0.0]])
    us = torch.full((N,), 0.5)
    p[2, 0, 3] = 1 / 16                                        # u q == p exactly: rejected
    q[3, 0, 3] = 0.0                                           # drafted against its own odds: accepted
    p[4, 0, 3] = math.nan                                      # no number: rejected
    p[5, 0, 3] = 0.0                                           # impossible for the target: rejected even at u = 0
    m = _check(p, q, x, u, us)
    assert m.tolist() == [2, 2, 1, 2, 1, 1]


def test_weights_that_vanish():
    N, V = 5, 70
    p = torch.full((N, 2, V), 1 / V)
    q = torch.full((N, 1, V), 2 / V)                           # above p everywhere: no residual
    x = torch.zeros(N, 1, dtype=torch.int32)
    u = torch.full((N, 1), 0.9)
    us = torch.tensor([0.0, 0.3, 0.7, 0.999, 0.5])
    p[1, 0] = 0.0                                              # and no target either: -1
    p[2, 0, 10:] = math.nan
    p[3, 0, 5] = math.inf
    p[4, 0] = 0.0
    p[4, 0, V - 1] = 1e-40                                     # a denormal alone
    m = _check(p, q, x, u, us)
    assert (m == 1).all()


def test_strided_rows_and_another_stream():
    N, K, V, pad = 9, 3, 1237, 35
    p, q, x, u, us = _case(N, K, V, seed=8)
    wide_p = torch.full((N, K + 1, V + pad), math.nan, device=DEV)
    wide_q = torch.full((N, K, V + 3), math.nan, device=DEV)
    wide_p[..., :V], wide_q[..., :V] = p.to(DEV), q.to(DEV)
    args = [x.to(DEV), u.to(DEV), us.to(DEV)]
    a = kda.verify_draft(p.to(DEV), q.to(DEV), *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = kda.verify_draft(wide_p[..., :V], wide_q[..., :V], *args)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _check(p, q, x, u, us)


def test_bad_tokens_and_counts_are_reported_and_skipped():
    p, q, x, u, us = _case(5, 3, 100, seed=9)
    want = kda.verify_draft(*(t.to(DEV) for t in (p, q, x, u, us)))
    x2 = x.clone()
    x2[1, 2], x2[3, 0] = 100, -1
    nd = torch.tensor([3, 3, 4, 3, 3], dtype=torch.int32)
    t, m = kda.verify_draft(*(a.to(DEV) for a in (p, q, x2, u, us)), num_draft=nd.to(DEV))
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    for n in (1, 2, 3):
        assert int(m[n]) == 0 and (t[n] == -1).all()
    for n in (0, 4):
        assert torch.equal(t[n], want[0][n]) and int(m[n]) == int(want[1][n])
    assert kda.kda_device_status() == kda.KDA_OK


def test_accepted_tokens_follow_the_target():
    """Drafts from q, verified against p: the first token of the result is distributed as p."""
    V, N = 12, 40000
    g = gen(12)
    p1 = torch.softmax(torch.randn(V, generator=g), -1)
    q1 = torch.softmax(torch.randn(V, generator=g), -1)
    x = torch.multinomial(q1, N, replacement=True, generator=g).view(N, 1).to(torch.int32)
    p = p1.expand(N, 2, V).contiguous()
    q = q1.expand(N, 1, V).contiguous()
    t, _ = kda.verify_draft(p.to(DEV), q.to(DEV), x.to(DEV), torch.rand(N, 1, generator=g).to(DEV),
                            torch.rand(N, generator=g).to(DEV))
    freq = torch.bincount(t[:, 0].cpu().long(), minlength=V).double() / N
    sd = torch.sqrt(p1.double() * (1 - p1.double()) / N)
    assert ((freq - p1.double()).abs() <= 6 * sd).all()
