"""The key/value cache's host side (CPU): its format's sizes and layout, and
what the binding and the C ABI refuse before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

bf16, f32, f16, i32 = torch.bfloat16, torch.float32, torch.float16, torch.int32
FORMATS = [(hd, b, g) for hd in (64, 128, 256) for b in (2, 4, 8) for g in (32, 64, 128, 256) if hd // 4 <= g <= hd]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return ttq.lib()


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_every_code_has_its_own_bits(hd, bits, group):
    """The layout is a bijection of the 16 hd codes onto a part's code bytes,
    a code never straddles a byte, and tokens that share a byte are none."""
    c, p = R.parts(hd, bits, group)
    assert ttq.ttq_kv_page_bytes(48, 3, hd, bits, group) == 3 * 3 * 2 * (c + p) and (2 * (c + p)) % 16 == 0
    for at in R.layout(hd, bits, group):
        assert np.array_equal(np.sort(at.reshape(-1)), np.arange(16 * hd) * bits)
        owner = {}
        for t in range(16):
            for byte in np.unique(at[t] // 8):
                assert owner.setdefault(int(byte), t) == t     # rows are written without reading


def test_page_bytes_refuses_what_is_not_built():
    for args in [(8, 2, 128, 4, 64), (24, 2, 128, 4, 64), (16, 0, 128, 4, 64), (16, 2, 96, 4, 32), (16, 2, 128, 3, 64),
                 (16, 2, 128, 4, 48), (16, 2, 256, 4, 32), (16, 2, 64, 4, 128), (65552, 2, 128, 4, 64)]:
        assert ttq.lib().ttq_kv_page_bytes(*args) == 0, args
        with pytest.raises(ttq.TTQError):
            ttq.ttq_kv_page_bytes(*args)


def test_workspace_size():
    size = ttq.ttq_kv_attention_workspace_size
    assert size(128, 4, 128, 32, 8, 1) >= 4096
    assert size(128, 4, 128, 32, 8, 64) > size(128, 4, 128, 32, 8, 1)
    for args in [(96, 4, 32, 8, 8, 1), (128, 3, 128, 8, 8, 1), (128, 4, 128, 9, 8, 1), (128, 4, 128, 0, 8, 1),
                 (128, 4, 128, 8, 0, 1), (128, 4, 128, 8, 8, 65), (128, 4, 128, 8, 8, -1)]:
        assert size(*args) == 0, args


def _cache(pages=4, page=32, heads=2, hd=128, bits=4, group=64, **kw):
    return ttq.new_kv_cache(pages, page, heads, hd, bits, group, device="cpu", **kw)


def _batch(B=3, T=5, max_new=2):
    return ttq.KVBatch(torch.zeros((B, 2), dtype=i32), torch.zeros(B, dtype=i32), torch.zeros(B + 1, dtype=i32), T, max_new)


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_a_workspace_serves_fewer_rows_too(hd, bits, group):
    """Whatever tile a batch of fewer new rows takes."""
    for per in (1, 3, 4, 5, 8, 33):
        sizes = [ttq.ttq_kv_attention_workspace_size(hd, bits, group, 2 * per, 2, n) for n in range(65)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_handles_check_their_tensors():
    n = ttq.ttq_kv_page_bytes(32, 2, 128, 4, 64)
    with pytest.raises(ValueError, match="pages must be"):
        ttq.KVCache(torch.zeros((4, n + 16), dtype=torch.uint8), 32, 2, 128, 4, 64)
    with pytest.raises(ValueError, match="pages must be"):
        ttq.KVCache(torch.zeros((4, n), dtype=torch.int8), 32, 2, 128, 4, 64)
    with pytest.raises(ValueError, match="D_k must hold 256"):
        _cache(D_k=torch.zeros(128), D_k_rsqrt=torch.zeros(256))
    with pytest.raises(ValueError, match="given together"):
        _cache(D_v=torch.zeros(256))
    with pytest.raises(ttq.TTQError):
        _cache(bits=3)
    with pytest.raises(TypeError, match="kv_len has dtype"):
        ttq.KVBatch(torch.zeros((3, 2), dtype=i32), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=i32), 5, 2)
    with pytest.raises(ValueError, match="cu_new has shape"):
        ttq.KVBatch(torch.zeros((3, 2), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32), 5, 2)
    with pytest.raises(ValueError, match="page_table has shape"):
        ttq.KVBatch(torch.zeros((2, 2), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32), 5, 2)
    with pytest.raises(ValueError, match="negative"):
        _batch(max_new=-1)


def test_calls_check_their_rows():
    cache, batch = _cache(), _batch()
    x = torch.zeros((5, 2, 128), dtype=bf16)
    with pytest.raises(ValueError, match="K has shape"):
        ttq.ttq_kv_write(cache, batch, x[:4], x)
    with pytest.raises(ValueError, match="V has shape"):
        ttq.ttq_kv_write(cache, batch, x, torch.zeros((5, 4, 128), dtype=bf16))
    with pytest.raises(TypeError, match="different dtypes"):
        ttq.ttq_kv_write(cache, batch, x, x.float())
    with pytest.raises(TypeError, match="K has dtype"):
        ttq.ttq_kv_write(cache, batch, x.double(), x)
    with pytest.raises(ValueError, match="contiguous"):
        ttq.ttq_kv_write(cache, batch, torch.zeros((5, 2, 256), dtype=bf16)[..., ::2], x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ttq.ttq_kv_write(cache, batch, x, x)
    with pytest.raises(ValueError, match="K has shape"):
        ttq.ttq_kv_read(cache, batch, K=x[:, :1])
    with pytest.raises(TypeError, match="V has dtype"):
        ttq.ttq_kv_read(cache, batch, V=x, dtype=f16)
    with pytest.raises(TypeError, match="unsupported dtype"):
        ttq.ttq_kv_read(cache, batch, dtype=torch.float64)
    q = torch.zeros((5, 8, 128), dtype=f16)
    with pytest.raises(ValueError, match="multiple of the cache's"):
        ttq.ttq_kv_attention(cache, batch, q[:, :5], 1.0)
    with pytest.raises(ValueError, match="Q has shape"):
        ttq.ttq_kv_attention(cache, batch, q[..., :64], 1.0)
    with pytest.raises(TypeError, match="tree has dtype"):
        ttq.ttq_kv_attention(cache, batch, q, 1.0, tree=torch.zeros(5, dtype=i32))
    with pytest.raises(ValueError, match="tree has shape"):
        ttq.ttq_kv_attention(cache, batch, q, 1.0, tree=torch.zeros((5, 1), dtype=torch.int64))
    with pytest.raises(TypeError, match="Y has dtype"):
        ttq.ttq_kv_attention(cache, batch, q, 1.0, Y=q, y_dtype=bf16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ttq.ttq_kv_attention(cache, batch, q, 1.0)


def _c(**kw):
    c = dict(pages=16, num_pages=4, page_size=32, kv_heads=2, head_dim=128, bits=4, group=64, scheme=0, D_k=None, D_v=None,
             D_k_rsqrt=None, D_v_rsqrt=None)
    c.update(kw)
    return ttq._CacheStruct(*c.values())


def _b(**kw):
    b = dict(page_table=16, table_stride=2, kv_len=16, cu_new=16, batch=3, rows=5, max_new=2)
    b.update(kw)
    return ttq._BatchStruct(*b.values())


def test_c_abi_rejections_before_device_work():
    """Every refusal returns before a CUDA call: there is no device here."""
    L = ttq.lib()
    INV, UNS, WS = ttq.TTQ_ERR_INVALID_ARG, ttq.TTQ_ERR_UNSUPPORTED, ttq.TTQ_ERR_WORKSPACE

    def write(c=None, b=None, K=16, kr=256, kh=128, V=16, dt=1, ws=256, n=4096):
        return L.ttq_kv_write(c or _c(), b or _b(), K, kr, kh, V, 256, 128, dt, ws, n, None)

    shared = [(dict(c=_c(scheme=5)), INV), (dict(c=_c(page_size=40)), INV), (dict(c=_c(kv_heads=0)), INV),
              (dict(c=_c(num_pages=-1)), INV), (dict(c=_c(pages=None)), INV), (dict(c=_c(pages=8)), INV),
              (dict(c=_c(head_dim=80)), UNS), (dict(c=_c(bits=3)), UNS), (dict(c=_c(bits=8)), UNS),
              (dict(c=_c(scheme=2)), UNS), (dict(c=_c(group=16)), UNS), (dict(c=_c(D_k=8)), INV),
              (dict(b=_b(batch=-1)), INV), (dict(b=_b(rows=-1)), INV), (dict(b=_b(rows=1 << 31)), INV),
              (dict(b=_b(batch=1025)), UNS), (dict(b=_b(kv_len=None)), INV), (dict(b=_b(cu_new=2)), INV),
              (dict(b=_b(page_table=None)), INV), (dict(ws=None), INV), (dict(ws=128), INV), (dict(n=64), WS),
              (dict(dt=7), INV)]
    for kw, st in shared + [(dict(K=None), INV), (dict(V=8), INV), (dict(kr=-8), INV), (dict(kr=252), INV),
                            (dict(kh=4), INV)]:
        assert write(**kw) == st, kw
    assert L.ttq_kv_write(None, _b(), 16, 256, 128, 16, 256, 128, 1, 256, 4096, None) == INV
    assert L.ttq_kv_write(_c(), None, 16, 256, 128, 16, 256, 128, 1, 256, 4096, None) == INV

    def read(c=None, b=None, K=16, V=16, dt=1, ws=256, n=4096):
        return L.ttq_kv_read(c or _c(), b or _b(), K, V, dt, ws, n, None)

    for kw, st in shared + [(dict(K=8), INV), (dict(V=40), INV)]:
        assert read(**kw) == st, kw
    size = L.ttq_kv_attention_workspace_size(128, 4, 64, 8, 2, 2)

    def attn(c=None, b=None, Q=16, qr=1024, qh=128, dt=1, heads=8, scale=1.0, cap=0.0, win=0, tree=None, Y=16, ydt=1,
             ws=256, n=size):
        return L.ttq_kv_attention(c or _c(), b or _b(), Q, qr, qh, dt, heads, scale, cap, win, tree, Y, ydt, ws, n, None)

    nan, inf = float("nan"), float("inf")
    for kw, st in shared + [(dict(heads=9), INV), (dict(heads=0), INV), (dict(scale=nan), INV), (dict(scale=inf), INV),
                            (dict(cap=-1.0), INV), (dict(cap=nan), INV), (dict(win=-1), INV), (dict(tree=4), INV),
                            (dict(Q=None), INV), (dict(Y=None), INV), (dict(Y=8), INV), (dict(qr=1020), INV),
                            (dict(ydt=5), INV), (dict(b=_b(max_new=65)), UNS), (dict(n=size - 1), WS)]:
        assert attn(**kw) == st, kw
    # nothing to do is not an error, and launches nothing
    for b in (_b(rows=0), _b(batch=0, kv_len=None, cu_new=None, page_table=None)):
        assert write(b=b) == read(b=b) == attn(b=b) == ttq.TTQ_OK
    assert read(K=None, V=None) == ttq.TTQ_OK
    assert attn(b=_b(max_new=0)) == ttq.TTQ_OK


def test_bad_index_flag_is_an_argument_error():
    f = ttq.ttq_status_from_flags
    assert f(ttq.TTQ_FLAG_BAD_INDEX) == ttq.TTQ_ERR_INVALID_ARG
    assert f(ttq.TTQ_FLAG_BAD_INDEX | ttq.TTQ_FLAG_RANK_DEFICIENT) == ttq.TTQ_ERR_INVALID_ARG
    assert f(ttq.TTQ_FLAG_BAD_INDEX | ttq.TTQ_FLAG_NONFINITE) == ttq.TTQ_ERR_NONFINITE
    assert f(ttq.TTQ_FLAG_BAD_INDEX | ttq.TTQ_FLAG_TIMEOUT) == ttq.TTQ_ERR_TIMEOUT


def test_reference_case_round_trips():
    """The test's own writer and reader of the layout agree."""
    case = R.Case([3, 0], [37, 20], heads=2, hd=64, bits=2, group=32, page=16, seed=3)
    rng = np.random.default_rng(1)
    q, s, z = rng.integers(0, 4, 64), rng.integers(0, 1 << 15, 2), rng.integers(0, 1 << 15, 2)
    R.write(case.host, case.cache, 1, 13, 1, 1, q, s, z)
    got = R.unpack(case.host, case.cache)[1]
    assert np.array_equal(got[0][1, 1, 13], q) and np.array_equal(got[1][1, 1, 13], s) and np.array_equal(got[2][1, 1, 13], z)
