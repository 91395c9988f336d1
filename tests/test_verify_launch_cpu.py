"""The number of CTAs that the verification gives a sequence, by the device it finds."""
import pytest

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def test_choices_of_the_device_it_was_measured_on():
    """152 SMs that hold 14 clusters of 16."""
    f = lambda N, V: kda.kda_debug_verify_cluster(N, V, 152, 14)
    assert f(1, 131072) == 16 and f(9, 131072) == 16 and f(10, 131072) == 8 and f(17, 131072) == 8
    assert f(18, 131072) == 4 and f(38, 131072) == 4 and f(39, 131072) == 2 and f(76, 100003) == 2
    assert f(77, 100003) == 1 and f(256, 100003) == 1 and f(1 << 20, 131072) == 1
    assert f(1, 32768) == 8 and f(1, 32769) == 16
    assert f(1, 8192) == 4 and f(1, 4096) == 2 and f(1, 4095) == 1 and f(1, 1) == 1


@pytest.mark.parametrize("held", [0, 1, 3])
def test_clusters_of_16_that_do_not_fit(held):
    """A device (or a part of one) that refuses them, or holds fewer than there are sequences, takes 8."""
    for N in range(1, 10):
        assert kda.kda_debug_verify_cluster(N, 131072, 152, held) == (16 if N <= held else 8)


def test_an_sm_for_each_cta():
    for sms in (20, 76, 132, 148, 152, 160):
        for N in list(range(1, 40)) + [sms // 2, sms, 2 * sms]:
            for V in (1000, 33000, 131072):
                C = kda.kda_debug_verify_cluster(N, V, sms, 64)
                assert C in (1, 2, 4, 8, 16) and (C == 1 or (N * C <= sms and V // C >= 2048))
                if C == 8:
                    assert N * 8 <= 0.9 * sms
