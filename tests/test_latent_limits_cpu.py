"""Limits of the latent calls, refused on the host before a GPU is touched."""
import pytest

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


@pytest.mark.parametrize("page", [16, 64, 1024])
def test_block_table_of_two_to_the_31_tokens(lib, page):
    """A length near 2^31 overflowed the count of its tiles, and its outputs stayed unwritten."""
    call = lambda pages: lib.kda_latent_decode(0x1000, 0x2000, 0, 4, page, 0x3000, pages, 0x4000, 1, 1, 32, 0.07, 0x5000, None,
                                               None)
    most = kda.KDA_LATENT_MAX_TOKENS // page
    assert most * page == 2**31 - 4096
    for pages in (most + 1, (2**31 - 1) // page):
        assert call(pages) == kda.KDA_ERR_INVALID_ARG


def test_the_limit_is_the_headers():
    import os
    import re
    text = open(os.path.join(os.path.dirname(kbuild.HERE), "include", "kda.h")).read()
    assert int(re.search(r"define KDA_LATENT_MAX_TOKENS (\d+)", text).group(1)) == kda.KDA_LATENT_MAX_TOKENS
