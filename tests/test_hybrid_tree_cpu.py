"""The hybrid server's tree step refuses what its pages or a tree do not hold, before anything is entered."""
import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300.hybrid_step import HybridModel, HybridServer, main


@pytest.fixture(scope="module")
def srv():
    kbuild.build()
    s = HybridServer(HybridModel(vocab=16, width=32, heads=1, device="cpu", rotary=100.0), 2, 128, page=16)
    s.lens, s.most = torch.tensor([120, 3], dtype=torch.int32), 120
    return s


def _step(srv, n, k, parents=None, u=None):
    return srv.step_tree(torch.zeros(n, dtype=torch.int32), torch.zeros(n, k, dtype=torch.int32),
                         torch.zeros(n, k, dtype=torch.long) if parents is None else parents,
                         torch.zeros(n, k + 1) if u is None else u)


def test_refusals(srv):
    with pytest.raises(ValueError, match="2 sequences"):
        _step(srv, 1, 2)
    with pytest.raises(ValueError, match="parents"):
        _step(srv, 2, 3, parents=torch.zeros(2, 2, dtype=torch.long))
    with pytest.raises(ValueError, match="u_sample"):
        _step(srv, 2, 3, u=torch.zeros(2, 3))
    with pytest.raises(ValueError, match="64 nodes"):
        _step(srv, 2, 64)
    with pytest.raises(ValueError, match="do not fit"):
        _step(srv, 2, 8)
    assert srv.lens.tolist() == [120, 3]


def test_command_refuses_trees_that_are_too_large():
    for args in (["--branches", "0"], ["--branches", "32", "--draft", "2"], ["--branches", "2", "--draft", "0"]):
        with pytest.raises(SystemExit):
            main(args)


def test_frequencies():
    m = HybridModel(vocab=16, width=32, heads=1, device="cpu", rotary=10000.0)
    assert m.rotary and m.inv_freq.shape == (32,) and m.inv_freq[0] == 1
    assert abs(float(m.inv_freq[-1]) * 10000 ** (62 / 64) - 1) < 2e-7
    assert not HybridModel(vocab=16, width=32, heads=1, device="cpu").rotary
