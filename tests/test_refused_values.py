"""Values that a narrower C type would wrap are refused by the binding."""
from __future__ import annotations

import pytest


@pytest.mark.parametrize("window", [-2 ** 31 - 1, -2 ** 32, -2 ** 32 + 5, -2 ** 63, 2 ** 31])
def test_a_window_outside_32_bits_is_refused(window):
    from paged_kv_attention_out_gb300 import binding
    with pytest.raises(ValueError, match="window"):
        binding._score_mod(0.0, None, window, None, 1, 1, 0)


@pytest.mark.parametrize("window", [-2 ** 31, -1, 0, 1, 4096, 2 ** 31 - 1])
def test_a_window_within_them_is_passed_on(window):
    """(the C call refuses the negative ones)"""
    from paged_kv_attention_out_gb300 import binding
    assert binding._score_mod(0.0, None, window, None, 1, 1, 0).window == window
