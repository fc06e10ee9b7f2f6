"""What the attention step's classes refuse before they ask for a GPU."""

import pytest

from fp8_w8a8_quantized_token_amd import Fp8KVCache


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_a_pool_is_on_a_gpu(device):
    with pytest.raises(ValueError, match="on a GPU"):
        Fp8KVCache(2, 2, device=device)
