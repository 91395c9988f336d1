"""Scales of e4m3 cache rows that are no numbers."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


@pytest.mark.parametrize("scale", [math.nan, math.inf])
@pytest.mark.parametrize("lens", [[70, 4], [9000]])
def test_absorbed_scale_that_is_no_number(scale, lens):
    """A cache row whose scale is NaN or infinite makes the rows that see it NaN, and no others."""
    K, H, page = 2, 8, 16
    cache, table, held = L.paged(lens, page, 1, seed=6)
    q = torch.randn(len(lens), K, H, 576, generator=L.gen(7)).to(torch.bfloat16)
    for n, length in enumerate(lens):
        t = length - 1
        cache[table[n, t // page], t % page, 640:644] = torch.tensor([scale], dtype=torch.float32).view(torch.uint8)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), 1, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), 0.07, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    for n, length in enumerate(lens):
        assert torch.isnan(out[n, 1].float()).all() and torch.isnan(lse[n, 1]).all()
        key = torch.cat(held[n], dim=1)
        L.check_rows(out[n, 0], lse[n, 0], [L.attend(q[n, 0, h].double(), key, held[n][0], 0.07, length - 1) for h in range(H)])
