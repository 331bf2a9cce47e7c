"""The cache's attention writes nothing behind the workspace that its size function names."""
import pytest
import torch

from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


@pytest.mark.parametrize("hd,bits,group", [(64, 4, 64), (128, 4, 128), (128, 8, 32), (256, 2, 256)])
@pytest.mark.parametrize("dtype,y_dtype,stat", [(bf16, bf16, False), (f16, f16, True), (f32, f32, False)], ids=str)
@pytest.mark.parametrize("n,per", [(1, 1), (1, 9), (3, 7), (24, 1), (5, 5), (33, 2), (64, 4)])
def test_nothing_is_written_behind_it(hd, bits, group, dtype, y_dtype, stat, n, per):
    """A context long enough that every thread block of the grid leaves its partial results, in a table wide enough for
    tiles of 256 rows."""
    H, page, ctx = 2, 64, 40000
    P = -(-ctx // page)
    D = torch.ones((H, hd), device="cuda") if stat else None
    cache = ttq.new_kv_cache(P, page, H, hd, bits, group, ttq.TTQ_QSCHEME_FP8_E4M3 if bits == 8 else 0, D_k=D, D_k_rsqrt=D)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 5000), **i32)
    table[0, :P] = torch.randperm(P, device="cuda").int()
    K, V = torch.randn(2, ctx, H, hd, device="cuda").to(bf16)
    ttq.ttq_kv_write(cache, ttq.KVBatch(table, torch.tensor([ctx], **i32), torch.tensor([0, ctx], **i32), ctx, ctx), K, V)
    batch = ttq.KVBatch(table, torch.tensor([ctx], **i32), torch.tensor([0, n], **i32), n, n)
    size = ttq.ttq_kv_attention_workspace_size(hd, bits, group, H * per, H, n)
    room = torch.full((size + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[:size]
    ttq.ttq_workspace_init(ws)
    Q = torch.randn(n, H * per, hd, device="cuda").to(dtype)
    ttq.ttq_kv_attention(cache, batch, Q, hd ** -0.5, ws=ws, y_dtype=y_dtype)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    assert bool((room[size:] == 0xA5).all())
    with pytest.raises(ttq.TTQError) as e:
        ttq.ttq_kv_attention(cache, batch, Q, hd ** -0.5, ws=room[:size - 16], y_dtype=y_dtype)
    assert e.value.status == ttq.TTQ_ERR_WORKSPACE
