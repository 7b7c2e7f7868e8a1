"""How the binding takes host counts (no GPU)."""
import array

import numpy as np
import pytest
import torch

from block_diffusion_draft_gb300.dflash_attn import _int32_array


@pytest.mark.parametrize("xs", [
    [3, 0, 17], (3, 0, 17), range(3, 6), bytes([3, 0, 17]), bytes([1, 2, 3, 4]), b"",
    bytearray([9, 8, 7, 6, 5]), memoryview(bytes([5, 6])), array.array("b", [1, -2]),
    array.array("d", [1.0, 2.0]), np.array([4, 5], np.int64), np.array([4.0, 5.0]), [2.9, True],
    torch.tensor([1, 2, 3]), [], [2 ** 32 + 5, -2 ** 31 - 1]], ids=repr)
def test_counts_are_taken_one_by_one(xs):
    want = [(int(x) + 2 ** 31) % 2 ** 32 - 2 ** 31 for x in xs]  # modulo 2^32
    assert list(_int32_array(xs)) == want
