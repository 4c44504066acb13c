"""kv4_attention refuses a softmax scale that is no number, before any CUDA call."""
import ctypes as C
import math

import pytest

import paged_kv_prep_gb300 as pkv
from paged_kv_prep_gb300 import build as pbuild
from paged_kv_prep_gb300._lib import Kv4CacheArgs

P = 4096


@pytest.mark.parametrize("scale,unit", [(math.nan, 1.0), (math.inf, 1.0), (-math.inf, 1.0), (3e38, 1.0), (1e30, 2.0 ** 64), (-1e30, 2.0 ** 64)])
def test_scales_that_are_no_numbers(scale, unit):
    """Times log2(e) and the keys' unit, in fp32."""
    pbuild.build()
    cache = Kv4CacheArgs(P, P, P, P, 10, 16, 2, 128, unit, 1.0)
    assert pkv.lib().pkv_kv4_attention(C.byref(cache), P, 2048, 0, 8, P, 4, P, P, 2, 4, scale, 0, P, 2048, P, P, 1 << 40,
                                       None, None) == pkv.ERR_INVALID_ARG
