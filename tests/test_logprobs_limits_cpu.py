"""The longest rows that kda_token_logprobs takes: beyond, fp32 sums and the waits of a row's CTAs for each other do not hold."""
import pytest

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


@pytest.mark.parametrize("dtype", [0, 1], ids=["bf16", "f32"])
def test_vocabularies(dtype):
    def call(V):                                                # (no rows: nothing is launched)
        return kda.load().kda_token_logprobs(0x1000, dtype, V, 0x2000, 0, V, 5, 1.0, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, None)
    assert call(kda.KDA_LOGPROBS_MAX_VOCAB) == kda.KDA_OK
    for V in (kda.KDA_LOGPROBS_MAX_VOCAB + 1, 1 << 28, 1 << 30, (1 << 31) - 1):
        assert call(V) == kda.KDA_ERR_UNSUPPORTED
