"""The tolerance that joined rows are compared with sees a part that is lost, or another sequence's in its place."""
import pytest
import torch

from tests import _join as J
from tests import _latent as L


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,part", [(3261, 192), (400, 64)])
def test_a_wrong_part_is_seen(T, part, dtype):
    g = L.gen(T)
    (c, r), (other, _) = (L.unpack(L.pack(*L.latents(g, T), dtype), dtype) for _ in range(2))
    q = torch.randn(32, 576, generator=g).to(torch.bfloat16)
    see = torch.ones(32, T, dtype=torch.bool)
    o, lse, tol, _ = J.rows(q, c, r, 0.07, see)
    # (a correct result: weights and output rounded)
    p = torch.exp((q.double() @ torch.cat([c, r], 1).T) * 0.07 - lse[:, None])
    good = (p.to(torch.bfloat16).double() @ c).to(torch.bfloat16)
    J.check(good, lse, (o, lse, tol, torch.full_like(lse, 1e-6)), "rounded")
    for wrong in (torch.zeros_like(c), other):
        v = c.clone()
        v[T - part:] = wrong[T - part:]
        bad = (p @ v).to(torch.bfloat16).double()
        assert ((bad - o).abs() > tol).any(dim=1).all()        # in every row
