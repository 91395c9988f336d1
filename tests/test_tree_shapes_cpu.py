"""The tree operators read parents as rows of K places and the pool as states of the call's heads: tensors of other rows are
refused where the call knows the shapes, as they would be read askew.  (On the CPU: a call that passed every check would say
that its tensors are not on the GPU.)"""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _state(**o):
    return {**dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 4, 64), v=bf(2, 3, 4, 64), log_alpha=torch.zeros(2, 3, 4, 64), beta=bf(2, 3, 4),
                   state_pool=torch.zeros(3, 4, 64, 64), parents=i32(2, 3), stream=0), **o}


def _attend(**o):
    return {**dict(q=bf(2, 3, 8, 576), cache=torch.zeros(4, 16, 1152, dtype=torch.uint8), cache_dtype=0, block_table=i32(2, 2),
                   seq_lens=i32(2), parents=i32(2, 3), sm_scale=0.07, stream=0), **o}


@pytest.mark.parametrize("call", [lambda **o: kda.decode_tree(**_state(**o)), lambda **o: kda.latent_decode_tree(**_attend(**o))],
                         ids=["state", "attend"])
def test_parents_of_other_places(call):
    for wide in (4, 64):
        with pytest.raises(ValueError, match=r"parents: expected a tensor \[2, 3\]"):
            call(parents=i32(2, wide))
    for rows in (2, 9):                                         # (of more sequences than the call's: the first are read)
        with pytest.raises(ValueError, match="on the GPU"):
            call(parents=i32(rows, 3))


def test_pools_of_other_heads():
    for pool in (torch.zeros(3, 8, 64, 64), torch.zeros(3, 4, 128, 128), torch.zeros(3, 4, 64 * 64), torch.zeros(12, 64, 64)):
        with pytest.raises(ValueError, match="state_pool: expected"):
            kda.decode_tree(**_state(state_pool=pool))
    with pytest.raises(ValueError, match="on the GPU"):
        kda.decode_tree(**_state(state_pool=torch.zeros(7, 4, 64, 64)))

def test_outputs_of_other_types():
    for t in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match="out_dtype"):
            kda.decode_tree(**_state(out_dtype=t))
    for t in (torch.bfloat16, torch.float32):
        with pytest.raises(ValueError, match="on the GPU"):
            kda.decode_tree(**_state(out_dtype=t))
