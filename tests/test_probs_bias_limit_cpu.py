"""The number of biases that decode_attn_token_probs takes, without a GPU."""
import ctypes

import pytest

import paged_kv_cache_60_gb300 as da
from paged_kv_cache_60_gb300 import build as dabuild

G = 0x100000             # a well-aligned address that nothing may read


@pytest.mark.parametrize("n", [(1 << 30) + 1, 2 ** 31 - 1, -1])
def test_more_biases_than_are_counted(n):
    dabuild.build()
    r = da.TokenRules(bias_starts=G, bias_tokens=G, bias_values=G, n_bias=n)
    lib = da.load_library()
    assert lib.decode_attn_token_probs(2, 0, 100, 0, G, 0, 0, 0x900000, 0, ctypes.byref(r), None, None) == -2
