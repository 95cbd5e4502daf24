"""Host-side limits of the attention over block scales, beside test_block_scaled_host.py (CPU only)."""
import pytest

from fp8_paged_kv_reshape_gb300 import binding
from tests.test_block_scaled_host import _decode, _multi


@pytest.mark.parametrize("block_size", [16, 32, 64, 128])
def test_tables_whose_tiles_pass_an_int32(block_size):
    """A length rounded up to a tile of 128 keys has to be an int32: 2^31 - 128 tokens at most."""
    most = (2 ** 31 - 128) // block_size
    for call, over in ((_decode, {}), (_multi, {}), (_multi, dict(qmax=64))):
        args = dict(over, block_size=block_size, num_blocks=1024)
        assert call(max_blocks_per_seq=most, query=None, **args) == binding.ERR_NULL
        assert call(max_blocks_per_seq=most + 1, **args) == binding.ERR_SHAPE
