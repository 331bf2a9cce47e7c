"""The key/value cache at the edges of what its documentation allows: the
largest batch, the smallest and largest pages, many rows in one call, shared
pages, calls at the same time, empty ones, extreme scales and windows."""
import numpy as np
import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ok(ws):
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)


@pytest.mark.parametrize("hd,bits,group,scheme,dtype,stat", [
    (128, 4, 64, R.ASYM, bf16, True), (128, 4, 128, R.SYM, f32, False), (256, 8, 64, R.FP8, f32, True),
    (64, 2, 32, R.ASYM, f16, False), (256, 2, 256, R.ASYM, bf16, True), (128, 8, 32, R.FP8, f16, False)], ids=str)
def test_many_rows_in_one_call_are_those_of_many_calls(hd, bits, group, scheme, dtype, stat):
    """More parts of blocks than the grid has warps, against calls of few."""
    H, page, B = 8, 48, 3
    g = torch.Generator(device="cuda").manual_seed(hd + bits)
    kv, new = [4100, 2055, 3001], [4100, 2000, 2999]
    need = -(-max(kv) // page)
    D = [None] * 4
    if stat:
        D[:2] = [torch.randn((H, hd), generator=g, device="cuda").exp() for _ in range(2)]
        D[2:] = [d.rsqrt() for d in D[:2]]
    caches = [ttq.new_kv_cache(B * need, page, H, hd, bits, group, scheme, D_k=D[0], D_v=D[1], D_k_rsqrt=D[2], D_v_rsqrt=D[3])
              for _ in range(2)]
    for c in caches:
        c.pages.fill_(0x5A)
    table = torch.randperm(B * need, generator=g, device="cuda").int().view(B, need)
    cu = np.concatenate([[0], np.cumsum(new)])
    K, V = (torch.randn((int(cu[-1]), H, hd), generator=g, device="cuda").to(dtype) for _ in range(2))
    whole = ttq.KVBatch(table, _ints(kv), _ints(cu), int(cu[-1]), max(new))
    ws = ttq.new_kv_workspace(caches[0], whole)
    ttq.ttq_kv_write(caches[0], whole, K, V, ws=ws)
    for b in range(B):
        for i in range(0, new[b], 100):
            n = min(100, new[b] - i)
            r = slice(int(cu[b]) + i, int(cu[b]) + i + n)
            one = ttq.KVBatch(table[b:b + 1], _ints([kv[b] - new[b] + i + n]), _ints([0, n]), n, n)
            ttq.ttq_kv_write(caches[1], one, K[r], V[r], ws=ws)
    assert torch.equal(caches[0].pages, caches[1].pages)
    k, v = ttq.ttq_kv_read(caches[0], whole, dtype=f32, ws=ws)
    for b in range(B):
        for i in range(0, new[b], 700):
            n = min(700, new[b] - i)
            r = slice(int(cu[b]) + i, int(cu[b]) + i + n)
            one = ttq.KVBatch(table[b:b + 1], _ints([kv[b] - new[b] + i + n]), _ints([0, n]), n, n)
            k1, v1 = ttq.ttq_kv_read(caches[0], one, dtype=f32, ws=ws)
            assert torch.equal(k[r], k1) and torch.equal(v[r], v1)
    _ok(ws)


def test_the_largest_batch():
    """1024 sequences that share 16 contexts: some without rows, some without
    positions, every length around a block's end."""
    kv16 = [1, 15, 16, 17, 31, 32, 33, 47, 2, 64, 65, 5, 80, 3, 11, 96]
    case = R.Case([1] * 16, kv16, heads=2, hd=64, bits=4, group=64, page=16, seed=3)
    cache, _ = case.on_gpu()
    rng = np.random.default_rng(4)
    src = rng.integers(0, 16, 1024)
    new = (rng.random(1024) < 0.8).astype(int)
    kv = np.where(rng.random(1024) < 0.05, 0, np.asarray(kv16)[src])
    new[kv == 0] = 0
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1])
    batch = ttq.KVBatch(torch.from_numpy(case.table[src]).cuda(), _ints(kv), _ints(cu), rows, 1)
    Q16 = torch.randn(16, 6, 64, generator=torch.Generator().manual_seed(5)).to(bf16)
    Q = torch.cat([Q16[s:s + 1] for s, n in zip(src, new) if n]).cuda()
    ws = ttq.new_kv_workspace(cache, batch, 6)
    Y = ttq.ttq_kv_attention(cache, batch, Q, 0.2, ws=ws).cpu().double().numpy()
    _ok(ws)
    want = []
    for b in range(16):
        K, V = case.sequence(b)
        want.append(R.attention(K, V, Q16[b:b + 1].double().numpy(), float(np.float32(0.2)), np.ones((1, kv16[b]), bool)))
    for s, row in zip(src[new == 1], range(rows)):
        y, bound = want[s]
        assert (np.abs(Y[row] - y[0]) <= bound[0] + (np.abs(y[0]) + bound[0]) * 2.0 ** -8 + 1e-5).all()
    # the rows of each context's last position, read by all who have it
    k, _ = ttq.ttq_kv_read(cache, batch, dtype=f32, ws=ws)
    first = {s: r for r, s in reversed(list(enumerate(src[new == 1])))}
    assert all(torch.equal(k[r], k[first[s]]) for r, s in enumerate(src[new == 1]))
    one = ttq.KVBatch(torch.zeros((1025, 1), dtype=torch.int32, device="cuda"), _ints([1] * 1025), _ints(range(1026)), 1025, 1)
    with pytest.raises(ttq.TTQError):
        ttq.ttq_kv_read(cache, one, ws=ws)
    # and written: a row each, to pages of their own
    own = ttq.new_kv_cache(1024, 16, 2, 64, 4, 64)
    own.pages.zero_()
    K, V = torch.randn(2, 1024, 2, 64, device="cuda").to(bf16)
    at = torch.randperm(1024, device="cuda").int().view(1024, 1)
    ttq.ttq_kv_write(own, ttq.KVBatch(at, _ints([7] * 1024), _ints(range(1025)), 1024, 1), K, V, ws=ws)
    some = ttq.new_kv_cache(1024, 16, 2, 64, 4, 64)
    some.pages.zero_()
    for i in range(0, 1024, 16):
        ttq.ttq_kv_write(some, ttq.KVBatch(at[i:i + 16], _ints([7] * 16), _ints(range(17)), 16, 1), K[i:i + 16], V[i:i + 16], ws=ws)
    assert torch.equal(own.pages, some.pages)
    _ok(ws)


def test_pages_of_16_and_of_65536_tokens():
    """The same rows in three caches: bits read and attended to are the same."""
    hd, n = 64, 65536 + 40
    K, V = torch.randn(2, n, 1, hd, device="cuda").to(bf16)
    Q = torch.randn(3, 4, hd, device="cuda").to(bf16)
    out = []
    for page in (16, 65536, 48):
        P = -(-n // page)
        cache = ttq.new_kv_cache(P + 1, page, 1, hd, 2, 64)
        table = torch.randperm(P + 1, device="cuda")[:P].int().view(1, P)
        ws = ttq.new_kv_workspace(cache, ttq.KVBatch(table, _ints([n]), _ints([0, 3]), 3, 3), 4)
        ttq.ttq_kv_write(cache, ttq.KVBatch(table, _ints([n]), _ints([0, n]), n, n), K, V, ws=ws)
        last = ttq.KVBatch(table, _ints([n]), _ints([0, 3]), 3, 3)
        out.append((*ttq.ttq_kv_read(cache, ttq.KVBatch(table, _ints([n]), _ints([0, n]), n, n), ws=ws),
                    ttq.ttq_kv_attention(cache, last, Q, 0.1, ws=ws)))
        _ok(ws)
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def test_calls_at_the_same_time():
    """Two streams, a workspace each: both give what they give alone."""
    work = []
    for seed, (kv, hq) in enumerate([([9000, 300, 5000], 16), ([40, 12000], 8)]):
        g = torch.Generator(device="cuda").manual_seed(seed)
        P = sum(-(-k // 64) for k in kv)
        cache = ttq.new_kv_cache(P, 64, 4, 128, 4, 128)
        need = [-(-k // 64) for k in kv]
        table, at = torch.zeros((len(kv), max(need)), dtype=torch.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = torch.arange(at, at + n)
            at += n
        rows, B = sum(kv), len(kv)
        every = ttq.KVBatch(table.cuda(), _ints(kv), _ints(np.concatenate([[0], np.cumsum(kv)])), rows, max(kv))
        K, V = (torch.randn((rows, 4, 128), generator=g, device="cuda").to(bf16) for _ in range(2))
        ttq.ttq_kv_write(cache, every, K, V)
        batch = ttq.KVBatch(table.cuda(), _ints(kv), _ints(range(B + 1)), B, 1)
        Q = torch.randn((B, hq, 128), generator=g, device="cuda").to(bf16)
        work.append((cache, batch, every, Q, ttq.new_kv_workspace(cache, batch, hq)))
    alone = [(ttq.ttq_kv_attention(c, b, Q, 0.1, ws=ws), *ttq.ttq_kv_read(c, e, ws=ws)) for c, b, e, Q, ws in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(10):
        both = [[], []]
        for i, (s, (c, b, e, Q, ws)) in enumerate(zip(streams, work)):
            for _ in range(4):
                both[i].append((ttq.ttq_kv_attention(c, b, Q, 0.1, ws=ws, stream=s), *ttq.ttq_kv_read(c, e, ws=ws, stream=s)))
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert all(torch.equal(a, b) for one in got for a, b in zip(one, want))
    for *_, ws in work:
        _ok(ws)


@pytest.mark.parametrize("grow", [1, 17])
def test_a_captured_attention_follows_the_lengths(grow):
    """One captured step replayed while contexts grow past blocks and pages
    (by 17: over positions that hold random bytes, NaN among them, so that
    bits are compared)."""
    case = R.Case([2, 1, 0], [14, 30, 3], heads=2, hd=128, page=16, seed=21, table_extra=40, spare=90)
    left = [p for p in range(case.host.shape[0]) if p not in case.table]
    for b in range(3):
        used = -(-case.kv[b] // 16)
        for i in range(used, used + 25):
            case.table[b, i] = left.pop()
    cache, batch = case.on_gpu()
    ws = ttq.new_kv_workspace(cache, batch, 8)
    K, V = torch.zeros((3, 2, 128), dtype=bf16, device="cuda"), torch.zeros((3, 2, 128), dtype=bf16, device="cuda")
    Q = torch.zeros((3, 8, 128), dtype=bf16, device="cuda")
    Y = torch.zeros_like(Q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ttq.ttq_kv_write(cache, batch, K, V, ws=ws)
        ttq.ttq_kv_attention(cache, batch, Q, 0.1, ws=ws, Y=Y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ttq.ttq_kv_write(cache, batch, K, V, ws=ws)
        ttq.ttq_kv_attention(cache, batch, Q, 0.1, ws=ws, Y=Y)
        batch.kv_len.add_(grow)
    batch.kv_len.copy_(_ints(case.kv))
    other = ttq.KVCache(cache.pages.clone(), 16, 2, 128, 4, 128)
    kv = list(case.kv)
    for step in range(20):
        for t in (K, V, Q):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(step)).to(bf16))
        graph.replay()
        now = ttq.KVBatch(batch.page_table, _ints(kv), batch.cu_new, 3, 2)
        ttq.ttq_kv_write(other, now, K, V)
        same = ttq.ttq_kv_attention(other, now, Q, 0.1)
        assert torch.equal(same.view(torch.int16), Y.view(torch.int16))
        assert grow > 1 or bool(Y.isfinite().all())
        assert torch.equal(other.pages, cache.pages)
        kv = [k + grow for k in kv]
    _ok(ws)


def test_scales_windows_and_caps_at_their_ends():
    case = R.Case([3, 1], [70, 40], heads=2, hd=128, seed=22)
    cache, batch = case.on_gpu()
    Q = torch.randn(4, 4, 128, generator=torch.Generator().manual_seed(1)).to(bf16).cuda()
    ws = ttq.new_kv_workspace(cache, batch, 4)
    want = ttq.ttq_kv_attention(cache, batch, Q, 0.1, ws=ws)
    # a window that nothing lies behind
    for window in (70, 2 ** 31, 2 ** 40):
        assert torch.equal(ttq.ttq_kv_attention(cache, batch, Q, 0.1, window=window, ws=ws), want)
    for scale, cap in ((0.0, 0.0), (-0.1, 0.0), (0.1, 1e-3), (0.1, 1e4), (3.0, 0.0)):
        Y = ttq.ttq_kv_attention(cache, batch, Q, scale, softcap=cap, y_dtype=f32, ws=ws).cpu().double().numpy()
        for b in range(2):
            K, V = case.sequence(b)
            r = slice(int(case.cu[b]), int(case.cu[b + 1]))
            see = R.visible(case.new[b], case.kv[b])
            raw = case.sequence(b, of=R.magnitudes)
            y, bound = R.attention(K, V, Q[r].cpu().double().numpy(), float(np.float32(scale)), see, float(np.float32(cap)), raw=raw)
            # (a score's own error stays, however small the cap; binary16 p s_V below its normal range: as in smax = 1, codes 15)
            assert (np.abs(Y[r] - y) <= bound + 70 * 2.0 ** -25 * 2 * 15 + 1e-5).all(), (scale, cap)
    # query rows of zeros: every position counts the same
    Y = ttq.ttq_kv_attention(cache, batch, torch.zeros_like(Q), 0.1, y_dtype=f32, ws=ws)
    Z = ttq.ttq_kv_attention(cache, batch, Q, 0.0, y_dtype=f32, ws=ws)
    assert torch.equal(Y, Z)
    _ok(ws)


def test_calls_without_rows():
    case = R.Case([0, 0], [40, 20], heads=2, hd=64, bits=4, group=64, seed=23)
    cache, batch = case.on_gpu()
    ws = ttq.new_kv_workspace(cache, batch, 4)
    before = cache.pages.clone()
    none = torch.zeros((0, 2, 64), dtype=bf16, device="cuda")
    ttq.ttq_kv_write(cache, batch, none, none, ws=ws)
    k, v = ttq.ttq_kv_read(cache, batch, ws=ws)
    assert k.shape == v.shape == (0, 2, 64)
    assert ttq.ttq_kv_attention(cache, batch, torch.zeros((0, 4, 64), dtype=bf16, device="cuda"), 0.1, ws=ws).shape == (0, 4, 64)
    nobody = ttq.KVBatch(batch.page_table[:0], batch.kv_len[:0], batch.cu_new[:1], 0, 0)
    ttq.ttq_kv_write(cache, nobody, none, none, ws=ws)
    # rows that belong to no sequence stay as they are
    padded = ttq.KVBatch(batch.page_table, batch.kv_len, batch.cu_new, 5, 4)
    Y = torch.full((5, 4, 64), 7.0, dtype=bf16, device="cuda")
    ttq.ttq_kv_attention(cache, padded, torch.randn_like(Y), 0.1, ws=ttq.new_kv_workspace(cache, padded, 4), Y=Y)
    ttq.ttq_kv_write(cache, padded, torch.randn_like(Y[:, :2]), torch.randn_like(Y[:, :2]), ws=ws)
    assert bool((Y == 7).all()) and torch.equal(cache.pages, before)
    _ok(ws)


def test_heads_apart_further_than_rows():
    """K, V laid out [heads][rows][head_dim]."""
    case = R.Case([30, 9], [100, 40], heads=3, hd=128, seed=24)
    K, V = torch.randn(2, 3, 39, 128).to(f16).cuda()
    pages = []
    for a, b in ((K.transpose(0, 1), V.transpose(0, 1)), (K.transpose(0, 1).contiguous(), V.transpose(0, 1).contiguous())):
        cache, batch = case.on_gpu()
        ttq.ttq_kv_write(cache, batch, a, b)
        pages.append(cache.pages)
    assert torch.equal(*pages)
