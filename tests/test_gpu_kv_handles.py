"""Attributes of a batch and of a cache assigned between calls: as fresh handles."""
import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def test_a_decoding_loop_that_assigns():
    """Steps that give the batch another tensor of lengths, more rows, a wider table; and the cache more pages."""
    case = R.Case([1, 1], [30, 41], heads=2, hd=64, bits=4, group=64, page=16, seed=3, table_extra=4, spare=9)
    free = [p for p in range(case.host.shape[0]) if p not in case.table]
    for b in range(2):
        used = -(-case.kv[b] // 16)
        for i in range(used, used + 3):
            case.table[b, i] = free.pop()
    cache, batch = case.on_gpu()
    other, _ = case.on_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ws = None
    for step in range(4):
        n = 1 + step % 2 * 2                       # 1 or 3 rows a sequence
        kv = torch.tensor([30 + 3 * step, 41 + 3 * step], **i32)
        cu = torch.tensor([0, n, 2 * n], **i32)
        batch.kv_len, batch.cu_new, batch.rows, batch.max_new = kv, cu, 2 * n, n
        if step == 2:
            batch.page_table = torch.cat([batch.page_table, torch.full((2, 5), -1, **i32)], 1)
            cache.pages = torch.cat([cache.pages, torch.zeros_like(cache.pages[:3])])
        junk = [torch.full((2,), 10 ** 6, **i32) for _ in range(8)]   # takes over memory that nothing holds
        fresh = ttq.KVBatch(batch.page_table.clone(), kv.clone(), cu.clone(), 2 * n, n)
        K, V = (torch.randn((2 * n, 2, 64), generator=g, device="cuda").to(bf16) for _ in range(2))
        Q = torch.randn((2 * n, 4, 64), generator=g, device="cuda").to(bf16)
        ws = ttq.new_kv_workspace(cache, batch, 4)
        out = []
        for c, b in ((cache, batch), (other, fresh)):
            ttq.ttq_kv_write(c, b, K, V, ws=ws)
            out.append((c.pages[:len(other.pages)], *ttq.ttq_kv_read(c, b, ws=ws), ttq.ttq_kv_attention(c, b, Q, 0.1, ws=ws)))
        # (as bits: the steps leave positions unwritten, whose random bytes stand for NaN here and there)
        same = [torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*out)]
        assert all(same), (step, same)
        torch.cuda.synchronize()
        assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
        del junk
