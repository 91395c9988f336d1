"""kda_latent_append_rope's angles in whole numbers alone (no other package): unit vectors turned by every frequency."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = 256
TURNS = 0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7aef158     # 2^256 / (2 pi), rounded down


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def angle(pos, f):
    """pos * f modulo a turn, in radians from -pi: f is a whole number of 2^-149."""
    t = (pos * int(f * 2.0 ** 149) * TURNS >> 149) % (1 << BITS)
    t = t - (1 << BITS) if t >> (BITS - 1) else t
    return t / (1 << BITS) * 2 * math.pi


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [kda.KDA_CACHE_BF16, kda.KDA_CACHE_E4M3], ids=["bf16", "e4m3"])
def test_unit_vectors(dtype, inter):
    """(1, 0) becomes (cos, sin), (0, 1) (-sin, cos): the angle to within 2^-26 + 2^-32 of a turn (4e-7 of both of them, less than
    2^-21), a step of fp32 each, and the rounding to bf16."""
    pos = [0, 1, 2, 77, 4095, 131071, 1000003, 2 ** 31 - 1, -1, -5000, -2 ** 31]
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float()
    f[5:9] = torch.tensor([1.5, 6.2831855, -0.3, 0.0])
    T = len(pos)
    first = torch.zeros(T, 2, 64, dtype=torch.bfloat16)
    if inter:
        first[:, 0, 0::2] = 1
        first[:, 1, 1::2] = 1
    else:
        first[:, 0, :32] = 1
        first[:, 1, 32:] = 1
    cache = kda.latent_cache(1, 16, dtype)
    c = torch.zeros(T, 512, dtype=torch.bfloat16, device=DEV)
    q = first.to(DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    out = kda.latent_append_rope(c, q[:, 0].contiguous(), cache, dtype, slots, torch.tensor(pos, dtype=torch.int32, device=DEV),
                                 f.to(DEV), q=q, interleaved=inter)
    assert kda.kda_device_status() == kda.KDA_OK
    at = 512 if dtype else 1024
    keys = cache.view(16, -1)[:T, at:at + 128].contiguous().view(torch.bfloat16)
    assert torch.equal(keys, out[:, 0])                         # (the keys were the first head's)
    a = torch.tensor([[angle(p, x) for x in f.double().tolist()] for p in pos], dtype=torch.float64)
    got = out.double().cpu()
    x, y = (got[..., 0::2], got[..., 1::2]) if inter else (got[..., :32], got[..., 32:])
    for g, w in ((x[:, 0], a.cos()), (y[:, 0], a.sin()), (x[:, 1], -a.sin()), (y[:, 1], a.cos())):
        assert ((g - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -20).all()
