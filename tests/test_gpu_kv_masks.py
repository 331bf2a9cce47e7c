"""What a row of the cache's attention does not see leaves no trace in it."""
import pytest
import torch

import kv_reference as R
from test_gpu_kv_attention import ROOM, _trees, check
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def _beyond(new, masks):
    """The masks with bits set that stand for no row of their sequence: all of them, some, the last one."""
    out, row = [], 0
    for n in new:
        rest = (2 ** 64 - 1) >> n << n
        for i in range(n):
            out.append(masks[row] | rest & [2 ** 64 - 1, 0x5555555555555555, 1 << 63][i % 3])
            row += 1
    return out


@pytest.mark.parametrize("window", [0, 1, 5, 16, 50, 64, 130])
def test_bits_beyond_a_sequences_rows_stand_for_nothing(window):
    """They name no new token: a row's position is counted without them, its own and those that it looks back at."""
    new = [3, 12, 1, 5, 0]
    case = R.Case(new, [103, 90, 70, 5, 9], heads=2, hd=64, bits=4, group=32, page=16, seed=41)
    masks = _trees(new, 3)
    check(case, per=2, window=window, masks=_beyond(new, masks))
    check(case, per=2, window=window, masks=_beyond(new, [0] * len(masks)))     # and nothing else


@pytest.mark.parametrize("window", [0, 1, 50, 130])
def test_bits_beyond_a_sequences_rows_in_tiles_of_256(window):
    new = [48, 63, 50]
    case = R.Case(new, [300, 64, 131], heads=1, hd=128, bits=4, group=64, page=16, seed=42, table_extra=ROOM)
    check(case, per=4, window=window, masks=_beyond(new, _trees(new, 6)))


def test_the_same_bits_with_and_without_them():
    new = [7, 2]
    case = R.Case(new, [60, 33], heads=1, hd=64, bits=4, group=64, page=16, seed=43)
    masks = _trees(new, 8)
    for window in (0, 9):
        assert torch.equal(check(case, per=3, window=window, masks=masks), check(case, per=3, window=window, masks=_beyond(new, masks)))
