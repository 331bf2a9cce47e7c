"""Writing rows into the quantised key/value cache and reading them back:
codes, scales and zeros bit for bit those of the CPU oracle's quantiser, at
the places that the layout names, with every other byte left alone."""
import numpy as np
import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def _status(ws):
    torch.cuda.synchronize()
    return ttq.ttq_get_status(ws)


def _expected(case, rows, D):
    """The host pages after writing rows = (K, V) [rows][heads][hd] float32."""
    f, want = case.cache, case.host.copy()
    for h in range(f.kv_heads):
        for which in range(2):
            q, s, z = R.quantise(f, rows[which][:, h], None if D[which] is None else D[which][h])
            for b, n in enumerate(case.new):
                for i in range(n):
                    r, p = case.cu[b] + i, case.kv[b] - n + i
                    R.write(want, f, case.table[b, p // f.page_size], p % f.page_size, h, which, q[r], s[r], z[r])
    return want


def _rows(case, dtype, seed=1, spread=True):
    g = torch.Generator().manual_seed(seed)
    shape = (case.rows, case.cache.kv_heads, case.cache.head_dim)
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g)
        if spread:   # groups of very different ranges, and of one sign
            x = x * torch.exp(torch.randn(shape[:2], generator=g) * 2)[..., None]
            x[::3] = x[::3].abs()
            x[1::5] = 0
        out.append(x.to(dtype))
    return out


@pytest.mark.parametrize("dtype", [bf16, f16, f32], ids=str)
@pytest.mark.parametrize("hd,bits,group,scheme,page", [
    (128, 4, 128, R.ASYM, 16), (128, 4, 32, R.SYM, 48), (128, 2, 64, R.ASYM, 32), (128, 8, 64, R.FP8, 64),
    (64, 4, 64, R.ASYM, 16), (64, 2, 32, R.SYM, 32), (64, 8, 32, R.FP8, 16),
    (256, 4, 64, R.ASYM, 32), (256, 2, 256, R.ASYM, 16), (256, 8, 128, R.FP8, 80)])
def test_write_is_the_oracle_bit_for_bit(hd, bits, group, scheme, page, dtype):
    # a single token, none, a run over a page's end, a whole sequence, a sequence inside one page
    case = R.Case([1, 0, 21, 35, 3], [17, 9, 50, 35, 8], heads=3, hd=hd, bits=bits, group=group, scheme=scheme, page=page,
                  seed=hd + bits, extra_rows=4, stat=dtype == f32)
    cache, batch = case.on_gpu()
    K, V = _rows(case, dtype)
    want = _expected(case, (K.float().numpy(), V.float().numpy()), case.D)
    ws = ttq.new_kv_workspace(cache, batch)
    ttq.ttq_kv_write(cache, batch, K.cuda(), V.cuda(), ws=ws)
    assert _status(ws) == (ttq.TTQ_OK, 0)
    assert np.array_equal(cache.pages.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [bf16, f16, f32], ids=str)
@pytest.mark.parametrize("hd,bits,group,page", [(128, 4, 128, 32), (64, 2, 32, 16), (256, 8, 64, 48), (64, 8, 64, 16),
                                                (128, 2, 32, 16), (256, 4, 256, 16)])
@pytest.mark.parametrize("stat", [False, True])
def test_read(hd, bits, group, page, dtype, stat):
    case = R.Case([1, 40, 0, 7], [33, 40, 5, 100], heads=2, hd=hd, bits=bits, group=group, page=page, seed=bits, stat=stat,
                  extra_rows=3)
    cache, batch = case.on_gpu()
    ws = ttq.new_kv_workspace(cache, batch)
    old = torch.full((case.rows, 2, hd), 7.5, dtype=dtype, device="cuda")
    got = ttq.ttq_kv_read(cache, batch, K=old.clone(), V=old.clone(), ws=ws)
    assert _status(ws) == (ttq.TTQ_OK, 0)
    for which in range(2):
        want = np.full(old.shape, 7.5)
        for b, n in enumerate(case.new):
            want[case.cu[b]:case.cu[b] + n] = case.sequence(b, Dr=case.Dr)[which][:, case.kv[b] - n:].transpose(1, 0, 2)
        w = torch.from_numpy(want)
        if not stat:
            assert torch.equal(got[which].cpu(), w.to(dtype))     # s (q - z) is exact in float32, rounded once
        else:
            # D^{-1/2} times the exact value is rounded to float32, then to dtype
            err = (got[which].cpu().double() - w).abs()
            assert bool((err <= w.abs() * (R.HALF_STEP[dtype] + 2.0 ** -23) + (2.0 ** -25 if dtype == f16 else 0)).all())
    # one of the two alone, through the C ABI
    L = ttq.lib()
    only = old.clone()
    assert L.ttq_kv_read(cache._arg()[0], batch._arg(0), None, only.data_ptr(), ttq._dtype_code(only), ws.data_ptr(),
                         ws.numel(), torch.cuda.current_stream().cuda_stream) == ttq.TTQ_OK
    assert torch.equal(only, got[1])


def test_write_takes_slices_of_a_fused_projection():
    case = R.Case([5, 9], [20, 9], heads=2, hd=128, seed=5)
    cache, batch = case.on_gpu()
    qkv = torch.randn(14, 8, 128).to(bf16)      # 4 query heads, 2 of K, 2 of V
    want = _expected(case, (qkv[:, 4:6].float().numpy(), qkv[:, 6:].float().numpy()), case.D)
    x = qkv.cuda()
    ttq.ttq_kv_write(cache, batch, x[:, 4:6], x[:, 6:])
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    # heads-major rows
    cache.pages.copy_(torch.from_numpy(case.host))
    k = qkv[:, 4:6].transpose(0, 1).contiguous().cuda()
    v = qkv[:, 6:].transpose(0, 1).contiguous().cuda()
    ttq.ttq_kv_write(cache, batch, k.transpose(0, 1), v.transpose(0, 1))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    # one head: its stride says nothing
    one = R.Case([3], [3], heads=1, hd=64, bits=4, group=64, seed=6)
    c1, b1 = one.on_gpu()
    x = torch.randn(3, 64).to(bf16).cuda()
    ttq.ttq_kv_write(c1, b1, x.as_strided((3, 1, 64), (64, 1, 1)), x.as_strided((3, 1, 64), (64, 3, 1)))
    want = _expected(one, [x.float().cpu().numpy()[:, None]] * 2, one.D)
    assert np.array_equal(c1.pages.cpu().numpy(), want)
    with pytest.raises(ValueError, match="16-byte aligned"):
        odd = torch.zeros(14 * 260, dtype=bf16, device="cuda").as_strided((14, 2, 128), (260, 130, 1))
        ttq.ttq_kv_write(cache, batch, odd, k.transpose(0, 1))


@pytest.mark.parametrize("bits", [2, 4, 8])
def test_a_group_that_nothing_stands_for_reads_as_nan(bits):
    case = R.Case([6], [22], heads=2, hd=128, bits=bits, group=64, seed=7)
    cache, batch = case.on_gpu()
    K, V = _rows(case, f32, spread=False)
    K[0, 0, 3], K[1, 1, 70], V[2, 0, 127], K[3, 0, 0] = float("nan"), float("inf"), float("-inf"), 3e38
    ws = ttq.new_kv_workspace(cache, batch)
    ttq.ttq_kv_write(cache, batch, K.cuda(), V.cuda(), ws=ws)
    k, v = ttq.ttq_kv_read(cache, batch, dtype=f32, ws=ws)
    st, flags = _status(ws)
    assert st == ttq.TTQ_ERR_NONFINITE and flags == ttq.TTQ_FLAG_NONFINITE | ttq.TTQ_FLAG_SCALE_OVERFLOW
    nan_k, nan_v = torch.zeros(K.shape, dtype=torch.bool), torch.zeros(K.shape, dtype=torch.bool)
    nan_k[0, 0, :64] = nan_k[1, 1, 64:] = nan_k[3, 0, :64] = True
    nan_v[2, 0, 64:] = True
    assert torch.equal(k.cpu().isnan(), nan_k) and torch.equal(v.cpu().isnan(), nan_v)
    K[nan_k], V[nan_v] = 0, 0      # every other group is as it would be without them
    ref = R.Case([6], [22], heads=2, hd=128, bits=bits, group=64, seed=7)
    c2, b2 = ref.on_gpu()
    ttq.ttq_kv_write(c2, b2, K.cuda(), V.cuda())
    k2, v2 = ttq.ttq_kv_read(c2, b2, dtype=f32)
    assert torch.equal(torch.where(nan_k.cuda(), 0.0, k), k2) and torch.equal(torch.where(nan_v.cuda(), 0.0, v), v2)


def test_bad_sequences_and_pages_are_skipped_and_flagged():
    """Lengths, rows and pages out of range: nothing of them is written or
    read, their neighbours are, and the status says so."""
    case = R.Case([4, 4, 4, 4], [20, 20, 20, 20], heads=2, hd=64, bits=4, group=64, page=16, seed=8)
    K, V = _rows(case, bf16)

    def run(change, untouched):
        cache, batch = case.on_gpu()
        change(batch)
        ws = ttq.new_kv_workspace(cache, batch)
        ttq.ttq_kv_write(cache, batch, K.cuda(), V.cuda(), ws=ws)
        assert _status(ws) == (ttq.TTQ_ERR_INVALID_ARG, ttq.TTQ_FLAG_BAD_INDEX)
        ttq.ttq_workspace_init(ws)
        old = torch.full((16, 2, 64), 3.0, dtype=bf16, device="cuda")
        k, _ = ttq.ttq_kv_read(cache, batch, K=old, ws=ws)
        assert _status(ws) == (ttq.TTQ_ERR_INVALID_ARG, ttq.TTQ_FLAG_BAD_INDEX)
        keep = [b for b in range(4) if b not in untouched]
        save = list(case.new)
        case.new = [n if b in keep else 0 for b, n in enumerate(save)]
        want = _expected(case, (K.float().numpy(), V.float().numpy()), case.D)
        case.new = save
        assert np.array_equal(cache.pages.cpu().numpy(), want)
        return k

    k = run(lambda b: b.kv_len.__setitem__(1, 3), [1])             # fewer positions than rows
    assert bool((k[4:8] == 3).all())
    run(lambda b: b.kv_len.__setitem__(2, 10 ** 9), [2])           # beyond its table
    run(lambda b: b.kv_len.__setitem__(0, -1), [0])
    k = run(lambda b: b.page_table.__setitem__((3, 1), 10 ** 6), [3])   # its four rows are on that page
    assert bool((k[12:] == 0).all())
    run(lambda b: b.page_table.__setitem__((3, 1), -1), [3])
    # rows that go down: sequence 1 has none that could be meant
    case.cu[2] = 2
    cache, batch = case.on_gpu()
    ws = ttq.new_kv_workspace(cache, batch)
    ttq.ttq_kv_write(cache, batch, K.cuda(), V.cuda(), ws=ws)
    assert _status(ws)[1] == ttq.TTQ_FLAG_BAD_INDEX
    # rows beyond the tensors, and more rows than max_new
    for cu in ([0, 4, 8, 12, 17], [0, 4, 8, 11, 16], [-1, 4, 8, 12, 16]):
        case.cu = np.asarray(cu, np.int32)
        cache, batch = case.on_gpu()
        batch = ttq.KVBatch(batch.page_table, batch.kv_len, batch.cu_new, 16, 4)
        ws = ttq.new_kv_workspace(cache, batch)
        ttq.ttq_kv_write(cache, batch, K.cuda(), V.cuda(), ws=ws)
        assert _status(ws)[1] == ttq.TTQ_FLAG_BAD_INDEX


def test_pages_beyond_4_gib():
    """Offsets in a cache of more than 2^32 bytes."""
    page = 64
    n = ttq.ttq_kv_page_bytes(page, 8, 128, 8, 128)
    P = (5 << 30) // n
    cache = ttq.new_kv_cache(P, page, 8, 128, 8, 128, ttq.TTQ_QSCHEME_FP8_E4M3)
    table = torch.tensor([[P - 1, 0], [P // 2, P - 2]], dtype=torch.int32, device="cuda")
    batch = ttq.KVBatch(table, torch.tensor([70, 65], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 70, 135], dtype=torch.int32, device="cuda"), 135, 70)
    K = torch.randn(135, 8, 128, device="cuda").to(bf16)
    V = torch.randn(135, 8, 128, device="cuda").to(bf16)
    ws = ttq.new_kv_workspace(cache, batch)
    ttq.ttq_kv_write(cache, batch, K, V, ws=ws)
    k, v = ttq.ttq_kv_read(cache, batch, dtype=f32, ws=ws)
    assert _status(ws) == (ttq.TTQ_OK, 0)
    for got, x in ((k, K), (v, V)):
        # E4M3: half a step of 2^-4 of the value, or of the smallest step of a group whose largest is 448 s
        s = x.float().abs().amax(-1, keepdim=True) / 448 * (1 + 2.0 ** -10)
        assert bool(((got - x.float()).abs() <= x.float().abs() * 2.0 ** -4 + s * 2.0 ** -10).all())


def test_captured_write_and_read_follow_the_batch():
    """One captured step replayed while the lengths move on."""
    case = R.Case([1, 1, 1], [16, 30, 5], heads=2, hd=128, page=16, seed=9, table_extra=3, spare=9)
    for b in range(3):    # room to grow
        used = -(-case.kv[b] // 16)
        case.table[b, used:used + 3] = [p for p in range(case.host.shape[0]) if p not in case.table[:, :]][:3]
    cache, batch = case.on_gpu()
    ws = ttq.new_kv_workspace(cache, batch)
    K, V = torch.zeros((3, 2, 128), dtype=bf16, device="cuda"), torch.zeros((3, 2, 128), dtype=bf16, device="cuda")
    out = torch.zeros_like(K), torch.zeros_like(V)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ttq.ttq_kv_write(cache, batch, K, V, ws=ws)
        ttq.ttq_kv_read(cache, batch, *out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    cache.pages.copy_(torch.from_numpy(case.host))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ttq.ttq_kv_write(cache, batch, K, V, ws=ws)
        ttq.ttq_kv_read(cache, batch, *out, ws=ws)
        batch.kv_len.add_(1)
    batch.kv_len.copy_(torch.tensor(case.kv, dtype=torch.int32))
    for step in range(20):
        k, v = torch.randn(3, 2, 128).to(bf16), torch.randn(3, 2, 128).to(bf16)
        K.copy_(k), V.copy_(v)
        graph.replay()
        case.host = _expected(case, (k.float().numpy(), v.float().numpy()), case.D)
        case.kv = [n + 1 for n in case.kv]
    assert np.array_equal(cache.pages.cpu().numpy(), case.host)
    assert _status(ws) == (ttq.TTQ_OK, 0)


def test_another_stream():
    case = R.Case([3, 8], [40, 8], heads=2, hd=128, seed=11)
    cache, batch = case.on_gpu()
    K, V = _rows(case, bf16)
    want = _expected(case, (K.float().numpy(), V.float().numpy()), case.D)
    K, V = K.cuda(), V.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ttq.ttq_kv_write(cache, batch, K, V, stream=side)
    k, _ = ttq.ttq_kv_read(cache, batch, stream=side)
    side.synchronize()
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    k2, _ = ttq.ttq_kv_read(cache, batch)
    assert torch.equal(k, k2)
