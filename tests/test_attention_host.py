"""What the attention step's classes refuse before they ask for a GPU."""

import ctypes
import re

import pytest

from fp8_w8a8_quantized_token_amd import Fp8KVCache, _lib
from tests.test_abi import ALIGNED, HEADER


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_a_pool_is_on_a_gpu(device):
    with pytest.raises(ValueError, match="on a GPU"):
        Fp8KVCache(2, 2, device=device)


def test_limits_match_the_header():
    text = open(HEADER).read()
    assert re.search(r"#define FP8W8A8_MAX_REQUESTS \(1 << 20\)", text) and _lib.MAX_REQUESTS == 1 << 20


@pytest.mark.parametrize("tokens,q_heads,k_heads", [(1 << 20, 64, 0), (1 << 20, 32, 32), (1 << 21, 24, 8), (1 << 11, 1, 32767)])
def test_rotary_rows_of_a_launch(tokens, q_heads, k_heads):
    """2^26 rows are one too many (refused on the host: the addresses are not looked at)."""
    plan = ctypes.c_void_p()
    lib = _lib.lib()
    assert lib.fp8_rope_create(128, 1, (ctypes.c_int64 * 1)(64), 1e4, 0, ctypes.byref(plan)) == _lib.OK
    q, k = (ctypes.byref(_lib.Rows(ALIGNED, h, 1 << 23, 128)) if h else None for h in (q_heads, k_heads))
    assert lib.fp8_rope_run(plan, tokens, ALIGNED, q, q, k, k, None) == _lib.ERR_BAD_SHAPE
    lib.fp8_rope_destroy(plan)
