"""Sizes of the packed step's calls that 32-bit launch arithmetic could not hold (no GPU needed).

Every refused call fails validation before anything touches the device.
"""

import pytest

from test_packed_host import _append, _rotary, FAKE, L  # noqa: F401

MOST = 1 << 30


@pytest.mark.parametrize("tokens", [MOST + 1, 2 ** 31 - 64, 2 ** 31 - 1])
def test_tokens_past_the_limit(L, tokens):  # noqa: F811
    """The grid was rounded up in 32 bits: tokens near 2^31 gave a negative number of CTAs."""
    apart = dict(q_out=FAKE + 4096, k=FAKE + 8192, k_out=FAKE + 12288)
    assert _rotary(L, tokens=tokens, **apart) == L.UNSUPPORTED
    assert _rotary(L, tokens=tokens, k_heads=0) == L.UNSUPPORTED
    assert _append(L, tokens=tokens) == L.UNSUPPORTED
