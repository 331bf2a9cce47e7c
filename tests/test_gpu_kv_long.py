"""Sequences of more pages than 24 bits count: the last positions of a context
of 2^28 and more, whose table names a few pages over and over."""
import pytest
import torch

from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.mark.parametrize("page", [16, 32])
def test_the_last_positions_of_a_sequence_of_many_pages(page):
    """Written, read and attended to (through a window) as those of a short sequence with the same pages."""
    hd, H, tail = 64, 2, 7
    cols = 2 ** 24 + 4
    cache, small = (ttq.new_kv_cache(8, page, H, hd, 2, 64) for _ in range(2))
    for c in (cache, small):
        c.pages.fill_(0x33)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((1, cols), 1, **i32)          # a wrong quotient finds page 1, or none
    table[0, -tail:] = torch.arange(tail, 0, -1, **i32)
    kv = [(cols - 1) * page + 5, (tail - 1) * page + 5]
    n = (tail - 2) * page + 5                        # every row in the last pages, none of them page 1's other names
    g = torch.Generator(device="cuda").manual_seed(page)
    K, V = (torch.randn((n, H, hd), generator=g, device="cuda").to(bf16) for _ in range(2))
    Q = torch.randn((3, 4, hd), generator=g, device="cuda").to(bf16)
    out = []
    for c, t, k in ((cache, table, kv[0]), (small, table[:, -tail:].contiguous(), kv[1])):
        rows = ttq.KVBatch(t, torch.tensor([k], **i32), torch.tensor([0, n], **i32), n, n)
        last = ttq.KVBatch(t, torch.tensor([k], **i32), torch.tensor([0, 3], **i32), 3, 3)
        ws = ttq.new_kv_workspace(c, last, 4)
        ttq.ttq_kv_write(c, rows, K, V, ws=ws)
        out.append((c.pages, *ttq.ttq_kv_read(c, rows, ws=ws), ttq.ttq_kv_attention(c, last, Q, 0.1, window=2 * page + 3, ws=ws)))
        torch.cuda.synchronize()
        assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    for a, b in zip(*out[:2]):
        assert torch.equal(a, b)
