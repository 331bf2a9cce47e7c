"""The workspace of the cache's attention holds the partial results of every
tile that a call of its sizes may take (CPU)."""
import pytest

from test_weight_quantization_ttq_b200 import ttq

FORMATS = [(hd, b, g) for hd in (64, 128, 256) for b in (2, 4, 8) for g in (32, 64, 128, 256) if hd // 4 <= g <= hd]


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_the_type_of_the_output_does_not_change_what_is_enough(hd, bits, group):
    """17 to 24 rows of a head go in tiles of 24, or of 32 where Q is taken in two parts (D of K or float32 rows, and an
    output other than bf16), which the sizes given here do not say: they are those of 32 rows."""
    size = ttq.ttq_kv_attention_workspace_size
    for rows in range(17, 33):
        assert size(hd, bits, group, rows, 1, 1) == size(hd, bits, group, 32, 1, 1), rows
    # more rows than 32, in several tiles of 24 or of 32
    for rows in (33, 40, 48, 63, 64, 72, 100):
        assert size(hd, bits, group, rows, 1, 1) >= size(hd, bits, group, 32, 1, 1), rows
