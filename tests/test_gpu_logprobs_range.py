"""kda_token_logprobs over rows whose values span more than the type's largest value: differences of two logits are beyond
fp32 there, their log probabilities are not."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests.test_gpu_logprobs import BF, F32, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-6, 0.3, 0.5, 1.0])
@pytest.mark.parametrize("R", [1, 4, 200])
def test_both_signs(dtype, scale, R):
    V = 9001
    x = torch.zeros(R, V)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x[:, 1::3] = low
    x[:, 2::3] = low / 2
    x[:, 40] = high
    x[:, 7000] = high / 2
    x = x.to(dtype)
    tok = [[1, 2, 3, 7000, 40][r % 5] for r in range(R)]
    got = run(x, tok, 20, scale, pad=3)
    assert kda.kda_device_status() == kda.KDA_OK
    check(x, tok, 20, scale, got)
