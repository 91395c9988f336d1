"""kda.latent_append_rope takes the position parts of queries, and no whole heads: it would turn their first 64 values,
which are not the position part.  (On the CPU: a call that passed every check would say that its tensors are not on the
GPU.)"""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _args(**o):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return {**dict(c=bf(5, 512), k_rope=bf(5, 64), cache=torch.zeros(4, 16, 656, dtype=torch.uint8), cache_dtype=1, slots=i(5),
                   positions=i(5), inv_freq=torch.zeros(32), q=bf(5, 4, 64), q_out=bf(5, 4, 64), stream=0), **o}


@pytest.mark.parametrize("wide", [65, 72, 192, 576])
@pytest.mark.parametrize("which", ["q", "q_out"])
def test_whole_heads_are_refused(which, wide):
    low = dict(total_tokens=5, H=4, interleaved=0)
    for fn, o in ((kda.latent_append_rope, {}), (kda.kda_latent_append_rope, low)):
        with pytest.raises(ValueError, match=f"{which}: .*position parts alone"):
            fn(**_args(**{which: bf(5, 4, wide)}, **o))
        with pytest.raises(ValueError, match="on the GPU"):
            fn(**_args(**{which: bf(5, 4, wide)[..., -64:]}, **o))


def test_one_token_of_one_head():
    """Strides of a single entry say nothing of its width."""
    one = dict(c=bf(1, 512), k_rope=bf(1, 64), slots=torch.zeros(1, dtype=torch.int32), positions=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="position parts alone"):
        kda.latent_append_rope(**_args(**one, q=bf(1, 1, 192), q_out=None))
    with pytest.raises(ValueError, match="on the GPU"):
        kda.latent_append_rope(**_args(**one, q=bf(1, 1, 192)[..., 128:], q_out=None))
