"""Absorbed latent attention of queries at the top of bf16's range."""
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


@pytest.mark.parametrize("dtype", [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")])
def test_largest_queries(dtype):
    """Rows of 2^125 to the largest bf16 value, against a scale that brings their scores to a few units.  (A few
    channels of near magnitudes: the two e4m3 terms hold them exactly; latents small enough that the fp32 sums
    of the products stay finite.)"""
    H, lens, page, scale = 12, [200], 64, 2.0 ** -125
    g = L.gen(21)
    c = (torch.randn(200, 512, generator=g) * 0.1).clamp(-0.4, 0.4).to(torch.bfloat16)
    r = torch.randn(200, 64, generator=g).to(torch.bfloat16)
    rows = L.pack(c, r, dtype)
    cache = torch.zeros(5, page, L.ROW[dtype], dtype=torch.uint8)
    table = torch.tensor([[2, 0, 4, 1]], dtype=torch.int32)
    for i in range(4):
        part = rows[i * page:(i + 1) * page]
        cache[table[0, i], :part.shape[0]] = part
    held = L.unpack(rows, dtype)
    q = torch.zeros(1, 1, H, 576)
    q[0, 0, :, 512:] = torch.randn(H, 64, generator=g) * 2.0 ** 118
    top = [2.0 ** 125, 1.75 * 2.0 ** 125, 2.0 ** 126, 1.75 * 2.0 ** 126, 1.875 * 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127,
           1.75 * 2.0 ** 127, 1.8125 * 2.0 ** 127, 1.9921875 * 2.0 ** 127, -1.9921875 * 2.0 ** 127, 2.0 ** 124]
    for h in range(H):
        q[0, 0, h, 5], q[0, 0, h, 100], q[0, 0, h, 300] = top[h], -0.25 * abs(top[h]), 0.1875 * abs(top[h])
    q = q.to(torch.bfloat16)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), dtype, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 scale, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_OK
    key = torch.cat(held, dim=1)
    L.check_rows(out[0, 0], lse[0, 0], [L.attend(q[0, 0, h].double(), key, held[0], scale, 200) for h in range(H)])
