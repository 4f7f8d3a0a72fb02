"""Refusals of the prompt and cache attention at the edges of fp32 (no device needed)."""
import ctypes as C

import pytest

from tests.test_cache_host import _attn, _cache
from tests.test_step_host import FAKE, _prompt, sv  # noqa: F401


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4028234e38])
def test_scales_beyond_fp32_in_log2_units_are_refused(sv, scale):  # noqa: F811
    """Such a scale's product with log2 e is infinite, and a score of 0 would be NaN."""
    L, n = sv.load_library(), 1 << 40
    assert L.spec_prompt_attend(C.byref(_prompt(scale=scale)), FAKE, FAKE, FAKE, n, None) == 1
    c, a = _cache(), _attn(scale=scale)
    assert L.spec_cache_attend(C.byref(c), C.byref(a), FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), FAKE, FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_weights(C.byref(c), C.byref(a), FAKE, FAKE, None) == 1
