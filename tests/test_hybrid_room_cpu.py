"""The hybrid server refuses tokens that its pages do not hold, before any of them is entered (an index past the block
table would be a fault on the GPU)."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300.hybrid_step import HybridModel, HybridServer


@pytest.fixture(scope="module")
def model():
    kbuild.build()
    return HybridModel(vocab=16, width=32, heads=1, device="cpu")


def _tokens(*lens):
    return [torch.zeros(n, dtype=torch.int64) for n in lens]


def test_prompt_longer_than_the_pages(model):
    with pytest.raises(ValueError, match="does not fit"):
        HybridServer(model, 2, 100, page=64).prompt(_tokens(5, 129))          # two pages of 64
    srv = HybridServer(model, 2, 100, page=64)
    srv.lens = torch.tensor([3, 120], dtype=torch.int32)
    with pytest.raises(ValueError, match="does not fit"):
        srv.prompt(_tokens(9, 9))
    with pytest.raises(ValueError, match="2 sequences"):
        srv.prompt(_tokens(9))


def test_step_past_the_pages(model):
    srv = HybridServer(model, 2, 64, page=16)
    srv.lens, srv.most = torch.tensor([61, 3], dtype=torch.int32), 61
    step = lambda n, k: srv.step(torch.zeros(n, dtype=torch.int32), torch.zeros(n, k, dtype=torch.int32), None, None, None)
    with pytest.raises(ValueError, match="do not fit"):
        step(2, 3)
    with pytest.raises(ValueError, match="2 sequences"):
        step(1, 1)


def test_the_bound_follows_the_lengths(model):
    """Rejected drafts leave the bound above the lengths: they are read back when it runs out of room."""
    srv = HybridServer(model, 2, 64, page=16)
    srv.lens, srv.most = torch.tensor([20, 30], dtype=torch.int32), 62
    srv._take(4)
    assert srv.most == 34
    srv._take(30)
    assert srv.most == 64
    srv.lens = torch.tensor([20, 61], dtype=torch.int32)
    with pytest.raises(ValueError, match="61 of 64"):
        srv._take(4)
    srv._take(3)
