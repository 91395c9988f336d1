"""kda_token_logprobs over the longest rows that it takes."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests.test_gpu_logprobs import BF, F32, check, rows

pytestmark = pytest.mark.gpu
V = kda.KDA_LOGPROBS_MAX_VOCAB


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _run(x, tok, top):
    got = kda.token_logprobs(x.cuda(), torch.tensor(tok, dtype=torch.int32, device="cuda"), top=top)
    assert kda.kda_device_status() == kda.KDA_OK
    return got


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_longest(dtype):
    x = rows(2, V, dtype, 1)
    tok = [V - 1, V // 3]
    check(x, tok, 32, 1.0, _run(x, tok, 32))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_columns_of_one_slice(dtype):
    """The largest values are a few threads' own, all of them in the last eighth of the row: its CTA looks for one after
    another while the others wait."""
    x = rows(1, V, dtype, 2, sharp=0.25)
    i = torch.arange(7 * V // 8, V)
    n = 16 // x.element_size()
    on = i[i // n % 256 < 80]
    x[0, on] = (4.0 + (on % 5) * 0.5).to(dtype)
    check(x, [V - 7], 32, 1.0, _run(x, [V - 7], 32))
