"""The key/value cache called by two host threads at once, each with its own
stream, batch and workspace."""
import threading

import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("hd,dtype", [(256, bf16), (128, f32)], ids=str)
def test_two_threads_read_with_batches_of_different_sizes(hd, dtype):
    """Reads of more than 48 KiB of shared memory a block, of a size that goes with the batch: every call of both
    threads is launched, and gives what it gives alone."""
    case = R.Case([3, 2], [20, 33], heads=2, hd=hd, bits=8, group=hd, page=16, seed=1)
    cache, two = case.on_gpu()
    work, errors = [], []
    for n in (2, 1000):    # the same two sequences, and in the larger batch many without rows behind them
        i32 = dict(dtype=torch.int32, device="cuda")
        table = two.page_table.repeat(n // 2, 1)
        kv = two.kv_len.repeat(n // 2)
        cu = torch.tensor([0, 3] + [5] * (n - 1), **i32)
        batch = ttq.KVBatch(table, kv, cu, 5, 3)
        work.append((batch, ttq.new_kv_workspace(cache, batch), torch.cuda.Stream()))
    want = ttq.ttq_kv_read(cache, two, dtype=dtype)
    start = threading.Barrier(2)
    torch.cuda.synchronize()

    def reads(batch, ws, stream):
        try:
            K, V = (torch.empty_like(x) for x in want)
            args = (cache._arg()[0], batch._arg(0), K.data_ptr(), V.data_ptr(), ttq._dtype_code(K), ws.data_ptr(), ws.nbytes,
                    stream.cuda_stream)
            call = ttq.lib().ttq_kv_read         # as close upon one another as calls can be
            start.wait()
            failed = sum(call(*args) != ttq.TTQ_OK for _ in range(20000))
            assert failed == 0, failed
            stream.synchronize()
            assert torch.equal(K, want[0]) and torch.equal(V, want[1])
        except Exception as e:  # noqa: BLE001 (told to the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=reads, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for _, ws, _ in work:
        assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
