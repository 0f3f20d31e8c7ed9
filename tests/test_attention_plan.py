"""The attention's workspace follows the SMs of the current device (its grid
does): no GPU needed, the library then plans for 148."""
import pytest
import torch

from tests.test_cache_host import _pdesc, lib  # noqa: F401


def sms():
    if torch.cuda.is_available():
        return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return 148


@pytest.mark.parametrize("G, d, dtype, rows, blocks", [(8, 128, 0, 8, 3), (16, 128, 0, 16, 2), (4, 64, 0, 8, 3),
                                                       (4, 64, 1, 8, 2), (4, 128, 1, 8, 1)])
def test_workspace_follows_the_device(lib, G, d, dtype, rows, blocks):  # noqa: F811
    """Many long sequences: two pieces a run and four words, `blocks` runs an SM
    (bf16: the larger of the 4-bit cache's and the pool's)."""
    got = lib.rkv_attention_workspace_size(_pdesc(S=400, H=8, G=G, d=d, dtype=dtype, mb=4096, nb=1 << 20), 1, 60000)
    runs = sms() * blocks
    floats = runs * (2 * rows * (d + 2) + 4)
    assert got == 256 + -(-4 * floats // 256) * 256
