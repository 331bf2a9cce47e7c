"""Attention over the quantised key/value cache against its definition in 64
bits, element by element within the bound that the kernel's own roundings
give (kv_reference.attention)."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def _trees(new, seed):
    """Masks of random trees, one per row: ancestors and itself."""
    rng, out = np.random.default_rng(seed), []
    for n in new:
        bits = []
        for i in range(n):
            up = int(rng.integers(-1, i)) if i else -1
            bits.append((bits[up] if up >= 0 else 0) | 1 << i)
        out += bits
    return out


def _signed(masks):
    return torch.tensor([m - 2 ** 64 if m >= 2 ** 63 else m for m in masks], dtype=torch.int64)


def check(case, per=4, dtype=bf16, y_dtype=None, cap=0.0, window=0, masks=None, q_scale=1.0, seed=0, Q=None):
    f, hd = case.cache, case.cache.head_dim
    cache, batch = case.on_gpu()
    g = torch.Generator().manual_seed(seed)
    hq = f.kv_heads * per
    if Q is None:
        Q = (torch.randn((case.rows, hq, hd), generator=g) * q_scale).to(dtype)
    scale = 1 / math.sqrt(hd)
    ws = ttq.new_kv_workspace(cache, batch, hq)
    Y = torch.full(Q.shape, 9.0, dtype=y_dtype or dtype, device="cuda")
    tree = None if masks is None else _signed(masks + [0] * (case.rows - len(masks))).cuda()
    ttq.ttq_kv_attention(cache, batch, Q.cuda(), scale, softcap=cap, window=window, tree=tree, ws=ws, Y=Y)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    got = Y.cpu().double().numpy()
    assert (got[case.cu[-1]:] == 9.0).all()                  # rows behind the last sequence
    for b, n in enumerate(case.new):
        if n == 0:
            continue
        r = slice(case.cu[b], case.cu[b] + n)
        K, V = case.sequence(b, Dr=case.Dr)
        see = R.visible(n, case.kv[b], window, None if masks is None else masks[r])
        s = R.unpack(case.host[case.table[b, :-(-case.kv[b] // f.page_size)]], f)[1][1]
        s = s.transpose(1, 0, 2, 3).reshape(f.kv_heads, -1, s.shape[3])[:, :case.kv[b]].astype(np.uint16)
        smax = float(s.view(np.float16).max())
        if case.Dr[1] is not None:
            smax *= float(case.Dr[1].max())
        y, bound = R.attention(K, V, Q[r].double().numpy(), float(np.float32(scale)), see, cap,
                               q_rounded=dtype == f32 or case.Dr[0] is not None, smax=smax,
                               code_max=448.0 if f.bits == 8 else 2.0 ** f.bits - 1,
                               raw=case.sequence(b, Dr=case.Dr, of=R.magnitudes))
        tol = bound + (np.abs(y) + bound) * R.HALF_STEP[Y.dtype] + 2.0 ** -24
        bad = ~(np.abs(got[r] - y) <= tol)
        assert not bad.any(), (b, int(bad.sum()), float(np.nanmax(np.abs(got[r] - y) / tol)))
        # and the bound says something: it is well below the values.  Where Q is rounded it holds twice the worst case
        # 2^-11 scale sum |k q| of a score, some 27 / 2^10 of p |V| at q_scale 3, and p |V| is several times |y|.
        # (INT2: a score also holds twice 2^-22 (hd / 16 + 2) scale sum |q| s (64 + 3).)
        part = 0.25 if dtype == f32 or case.Dr[0] is not None or f.bits == 2 else 0.1
        assert bound.mean() <= part * np.sqrt(np.mean(y ** 2)) + 1e-4, (bound.mean(), np.sqrt(np.mean(y ** 2)))
    return Y


FORMATS = [(hd, b, g) for hd in (64, 128, 256) for b in (2, 4, 8) for g in (32, 64, 128, 256) if hd // 4 <= g <= hd]


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_single_tokens_of_every_format(hd, bits, group):
    """One new token a sequence: lengths of one, around a block's and a page's end, and none at all."""
    case = R.Case([1, 1, 1, 0, 1, 1], [1, 16, 17, 40, 97, 150], heads=2, hd=hd, bits=bits, group=group, page=32,
                  seed=hd + bits + group)
    check(case, per=4)


@pytest.mark.parametrize("hd,bits,group", FORMATS)
@pytest.mark.parametrize("n,per", [(5, 3), (9, 4)])
def test_trees_of_every_format(hd, bits, group, n, per):
    """16 and 32 rows a tile, the last tile ragged."""
    new = [n, 2, 0, n - 1]
    case = R.Case(new, [n, 61, 33, 120], heads=2, hd=hd, bits=bits, group=group, page=16, seed=hd + bits + group + n)
    check(case, per=per, masks=_trees(new, n))


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_trees_of_every_format_in_wide_tiles(hd, bits, group):
    """32 rows a tile (16 with heads of 256), one tile and its rows full, ragged and absent."""
    new = [8, 3, 0, 7]
    case = R.Case(new, [50, 3, 33, 71], heads=2, hd=hd, bits=bits, group=group, page=48, seed=hd + bits + group + 1)
    check(case, per=4, masks=_trees(new, 2))


@pytest.mark.parametrize("scheme,bits", [(R.SYM, 4), (R.SYM, 2), (R.ASYM, 4)])
@pytest.mark.parametrize("dtype,y_dtype", [(f16, None), (bf16, f32), (f32, None), (f32, bf16)])
def test_schemes_and_types(scheme, bits, dtype, y_dtype):
    case = R.Case([1, 4], [77, 50], heads=2, hd=128, bits=bits, group=64, scheme=scheme, page=48, seed=4, extra_rows=3)
    check(case, per=2, dtype=dtype, y_dtype=y_dtype)


@pytest.mark.parametrize("bits,group", [(4, 128), (8, 64)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_statistic_and_cap(bits, group, cap):
    """K and V scaled by their statistics; sharp scores that the cap bends."""
    case = R.Case([1, 3], [130, 64], heads=2, hd=128, bits=bits, group=group, page=32, seed=5, stat=True)
    check(case, per=4, cap=cap, q_scale=3.0)


@pytest.mark.parametrize("window", [1, 2, 16, 37, 64, 1000])
@pytest.mark.parametrize("tree", [False, True])
def test_windows(window, tree):
    new = [1, 6, 12, 1]
    case = R.Case(new, [100, 90, 12, 5], heads=1, hd=64, bits=4, group=32, page=16, seed=6)
    check(case, per=2, window=window, masks=_trees(new, 1) if tree else None)


def test_rows_that_see_nothing_are_zero():
    """Masks without a bit: with a context the row sees that alone, without one nothing."""
    new = [3, 4]
    case = R.Case(new, [3, 40], heads=2, hd=128, seed=7)
    Y = check(case, masks=[0, 0b010, 0b111, 0, 0, 0b1000, 0b0001])
    assert bool((Y[0] == 0).all())
    # a window that ends before the context does, for rows that do not see themselves
    Y = check(case, masks=[0] * 7, window=1)
    assert bool((Y == 0).all())


def test_masks_of_64_tokens_and_their_last_bits():
    new = [64, 63]
    case = R.Case(new, [64, 100], heads=1, hd=64, bits=4, group=64, page=64, seed=8)
    masks = _trees(new, 3)
    masks[63] = 2 ** 64 - 1
    check(case, per=1, masks=masks)
    check(case, per=3)      # a chain


@pytest.mark.parametrize("per,heads", [(1, 5), (7, 1), (16, 2), (33, 1)])
def test_head_layouts(per, heads):
    """Query rows that fill no tile, one tile, and several."""
    case = R.Case([1, 2], [40, 33], heads=heads, hd=64, bits=4, group=32, page=16, seed=9)
    check(case, per=per)


def test_long_contexts_are_cut_and_joined():
    """Contexts that many blocks of the grid share, beside short ones."""
    case = R.Case([1, 1, 2, 1], [3000, 7, 1500, 2049], heads=2, hd=64, bits=4, group=64, page=128, seed=10)
    check(case, per=4)
    check(case, per=4, window=1000)


@pytest.mark.parametrize("big", [1e-3, 300.0])
def test_scales_of_every_size(big):
    """V of very different magnitudes in the sequences, and within one:
    the probabilities keep binary16's normal range."""
    case = R.Case([1, 2, 1], [60, 70, 80], heads=2, hd=128, bits=4, group=64, page=16, seed=11,
                  scale_of=lambda which, b: 1.0 if which == 0 else [1e-3, 1.0, big][b])
    check(case, per=2)


def test_sharp_and_flat_softmax():
    case = R.Case([1, 1], [400, 300], heads=1, hd=64, bits=4, group=64, page=16, seed=12)
    check(case, per=2, q_scale=30.0)
    check(case, per=2, q_scale=0.0)
    check(case, per=2, dtype=bf16, Q=torch.randn(2, 2, 64).to(bf16) * torch.tensor([1e-30, 30.0])[:, None, None].to(bf16))


def test_nan_reaches_only_those_that_see_it():
    """A NaN scale in one token's K or V: rows that see it are NaN, all others are as without it."""
    new = [4, 1]
    case = R.Case(new, [30, 50], heads=2, hd=128, bits=4, group=64, page=16, seed=13)
    masks = [0b0001, 0b0011, 0b0101, 0b1001, 0b1]
    clean = check(case, per=2, masks=masks)
    for which in range(2):
        save = case.host.copy()
        p = 27       # the second new token of sequence 0, head 1: seen by rows 1 only
        q, s, z = (a[case.table[0, p // 16], 1, p % 16] for a in R.unpack(case.host, case.cache)[which])
        R.write(case.host, case.cache, case.table[0, p // 16], p % 16, 1, which, q, np.asarray([0x7FFF, s[1]]), z)
        cache, batch = case.on_gpu()
        g = torch.Generator().manual_seed(0)
        Q = torch.randn((case.rows, 4, 128), generator=g).to(bf16).cuda()
        Y = ttq.ttq_kv_attention(cache, batch, Q, 1 / math.sqrt(128), tree=_signed(masks).cuda())
        want = clean.clone()
        nan = torch.zeros(Y.shape, dtype=torch.bool, device="cuda")
        nan[1, 2:, :64 if which else 128] = True       # K: the whole row; V: that group's channels
        assert torch.equal(Y.isnan(), nan)
        assert torch.equal(Y[~nan], want[~nan])
        case.host = save


def test_a_nan_query_keeps_to_its_row():
    case = R.Case([2, 1], [30, 40], heads=1, hd=64, bits=4, group=64, page=16, seed=14)
    cache, batch = case.on_gpu()
    Q = torch.randn(3, 4, 64).to(bf16).cuda()
    clean = ttq.ttq_kv_attention(cache, batch, Q, 0.125)
    Q[1, 2, 5] = float("nan")
    Q[2, 0, 0] = float("inf")
    Y = ttq.ttq_kv_attention(cache, batch, Q, 0.125)
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    assert bool(Y[bad].isnan().all()) and torch.equal(Y[~bad], clean[~bad])


def test_bad_sequences_and_pages():
    """What is out of range is skipped and flagged; the others' rows stand."""
    case = R.Case([1, 1, 1], [40, 50, 60], heads=2, hd=128, page=16, seed=15)
    Q = torch.randn(3, 4, 128).to(bf16).cuda()

    def run(change):
        cache, batch = case.on_gpu()
        change(batch)
        ws = ttq.new_kv_workspace(cache, batch, 4)
        Y = torch.full((3, 4, 128), 5.0, dtype=bf16, device="cuda")
        ttq.ttq_kv_attention(cache, batch, Q, 0.1, ws=ws, Y=Y)
        torch.cuda.synchronize()
        return Y, ttq.ttq_get_status(ws)[1]

    good, flags = run(lambda b: None)
    assert flags == 0
    for kv in (0, -5, 10 ** 9):
        Y, flags = run(lambda b: b.kv_len.__setitem__(1, kv))
        assert flags == ttq.TTQ_FLAG_BAD_INDEX and bool((Y[1] == 5).all())
        assert torch.equal(Y[[0, 2]], good[[0, 2]])
    # a page that is not one of the cache's: as if its positions were not there
    for page in (-1, 10 ** 8):
        Y, flags = run(lambda b: b.page_table.__setitem__((1, 1), page))
        assert flags == ttq.TTQ_FLAG_BAD_INDEX and torch.equal(Y[[0, 2]], good[[0, 2]])
        K, V = case.sequence(1)
        see = np.ones((1, 50), bool)
        see[0, 16:32] = False
        y, bound = R.attention(K, V, Q[1:2].cpu().double().numpy(), float(np.float32(0.1)), see)
        assert (np.abs(Y[1:2].cpu().double().numpy() - y) <= bound + (np.abs(y) + bound) * 2.0 ** -8 + 1e-5).all()


def test_strided_queries():
    case = R.Case([3, 1], [20, 33], heads=2, hd=128, seed=16)
    cache, batch = case.on_gpu()
    qkv = torch.randn(4, 12, 128).to(bf16).cuda()
    want = ttq.ttq_kv_attention(cache, batch, qkv[:, :8].contiguous(), 0.1)
    assert torch.equal(ttq.ttq_kv_attention(cache, batch, qkv[:, :8], 0.1), want)
    t = qkv[:, :8].transpose(0, 1).contiguous()
    assert torch.equal(ttq.ttq_kv_attention(cache, batch, t.transpose(0, 1), 0.1), want)


def test_same_bits_every_time_and_workspaces_may_be_shared():
    """Two captured graphs and eager calls with one workspace, replayed in turn."""
    a = R.Case([1, 2], [700, 300], heads=2, hd=128, page=64, seed=17)
    b = R.Case([1, 1, 1], [90, 500, 20], heads=2, hd=128, page=64, seed=18)
    state = []
    for case in (a, b):
        cache, batch = case.on_gpu()
        Q = torch.randn(case.rows, 8, 128).to(bf16).cuda()
        state.append((cache, batch, Q, torch.empty_like(Q)))
    ws = ttq.new_kv_workspace(state[0][0], ttq.KVBatch(*[state[0][1].__dict__[k] for k in ("page_table", "kv_len", "cu_new")], 3, 2), 8)
    eager = [ttq.ttq_kv_attention(c, bt, Q, 0.1).clone() for c, bt, Q, _ in state]
    for c, bt, Q, Y in state:
        ttq.ttq_kv_attention(c, bt, Q, 0.1, ws=ws, Y=Y)
    graphs = []
    for c, bt, Q, Y in state:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ttq.ttq_kv_attention(c, bt, Q, 0.1, ws=ws, Y=Y)
        graphs.append(g)
    for _ in range(5):
        for (_, _, _, Y), g, want in zip(state, graphs, eager):
            Y.zero_()
            g.replay()
            g.replay()
            assert torch.equal(Y, want)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)


def test_the_cache_beyond_4_gib():
    page, hd, H = 64, 128, 8
    n = ttq.ttq_kv_page_bytes(page, H, hd, 8, 128)
    P = (5 << 30) // n
    cache = ttq.new_kv_cache(P, page, H, hd, 8, 128, ttq.TTQ_QSCHEME_FP8_E4M3)
    table = torch.tensor([[P - 1, 0, P - 2]], dtype=torch.int32, device="cuda")
    small = ttq.new_kv_cache(3, page, H, hd, 8, 128, ttq.TTQ_QSCHEME_FP8_E4M3)
    kv, i32 = 150, dict(dtype=torch.int32, device="cuda")
    K, V = torch.randn(2, kv, H, hd, device="cuda").to(bf16)
    Q = torch.randn(1, 16, hd, device="cuda").to(bf16)
    out = []
    for c, t in ((cache, table), (small, torch.tensor([[2, 1, 0]], **i32))):
        ttq.ttq_kv_write(c, ttq.KVBatch(t, torch.tensor([kv], **i32), torch.tensor([0, kv], **i32), kv, kv), K, V)
        out.append(ttq.ttq_kv_attention(c, ttq.KVBatch(t, torch.tensor([kv], **i32), torch.tensor([0, 1], **i32), 1, 1), Q, 0.1))
    assert torch.equal(out[0], out[1])


def test_a_decoding_run_as_it_would_be_used():
    """Prompts written in one call, then steps: a tree of drafted tokens is
    written and attended to, its longest accepted path is written again in
    place, and the next step goes on from there; every step's outputs agree
    with dense attention over what the cache stands for."""
    rng = np.random.default_rng(0)
    H, per, hd, page, B = 2, 4, 128, 16, 3
    cache = ttq.new_kv_cache(40, page, H, hd, 4, 64)
    cache.pages.random_(0, 256)
    table = torch.from_numpy(rng.permutation(40)[:36].reshape(B, 12).astype(np.int32)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = [5, 33, 64]

    def batch(new):
        return ttq.KVBatch(table, torch.tensor(kv, **i32), torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32),
                           sum(new), max(new))

    ws = ttq.new_kv_workspace(cache, ttq.KVBatch(table, torch.zeros(B, **i32), torch.zeros(B + 1, **i32), 0, 8), H * per)
    ttq.ttq_kv_write(cache, batch(kv), *torch.randn(2, sum(kv), H, hd, device="cuda").to(bf16), ws=ws)
    for step in range(6):
        new = [8, 5, 1] if step % 2 == 0 else [1, 1, 1]
        kv = [k + n for k, n in zip(kv, new)]
        masks = _trees(new, step)
        K, V = torch.randn(2, sum(new), H, hd, device="cuda").to(bf16)
        Q = torch.randn(sum(new), H * per, hd, device="cuda").to(bf16)
        ttq.ttq_kv_write(cache, batch(new), K, V, ws=ws)
        Y = ttq.ttq_kv_attention(cache, batch(new), Q, 0.1, softcap=20.0, tree=_signed(masks).cuda(), ws=ws)
        k, v = ttq.ttq_kv_read(cache, batch(kv), dtype=f32, ws=ws)
        at, row = 0, 0
        for b in range(B):
            kk, vv = (x[at:at + kv[b]].cpu().double().numpy().transpose(1, 0, 2) for x in (k, v))
            see = R.visible(new[b], kv[b], 0, masks[row:row + new[b]])
            y, bound = R.attention(kk, vv, Q[row:row + new[b]].cpu().double().numpy(), float(np.float32(0.1)), see, 20.0)
            got = Y[row:row + new[b]].cpu().double().numpy()
            assert (np.abs(got - y) <= bound + (np.abs(y) + bound) * 2.0 ** -8 + 1e-5).all()
            at, row = at + kv[b], row + new[b]
        # accept each sequence's deepest path: its rows are written to the positions behind the old ones
        keep, row, kept = [], 0, []
        for b in range(B):
            m = max(masks[row:row + new[b]], key=lambda x: bin(x).count("1"))
            path = [i for i in range(new[b]) if m >> i & 1]
            keep += [row + i for i in path]
            kept.append(len(path))
            row += new[b]
        kv = [k - n + a for k, n, a in zip(kv, new, kept)]
        idx = torch.tensor(keep, device="cuda")
        ttq.ttq_kv_write(cache, batch(kept), K[idx], V[idx], ws=ws)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)


def test_more_new_rows_than_a_mask_holds_are_refused():
    case = R.Case([1], [20], heads=1, hd=64, bits=4, group=64, seed=19)
    cache, batch = case.on_gpu()
    big = ttq.KVBatch(batch.page_table, batch.kv_len, batch.cu_new, 1, 65)
    with pytest.raises(ttq.TTQError) as e:
        ttq.ttq_kv_attention(cache, big, torch.zeros((1, 2, 64), dtype=bf16, device="cuda"), 1.0)
    assert e.value.status == ttq.TTQ_ERR_UNSUPPORTED


WIDE = [(hd, b, g) for hd, b, g in FORMATS if hd <= 128 and hd // g <= 2]
ROOM = 9000     # columns of the page table: those tiles are for batches that may be long


@pytest.mark.parametrize("hd,bits,group", WIDE)
@pytest.mark.parametrize("tree", [False, True])
def test_tiles_of_256_rows_of_every_format(hd, bits, group, tree):
    """Full, ragged and nearly empty tiles of rows; lengths around a step's 64 tokens."""
    new = [64, 61, 0, 3, 64]
    case = R.Case(new, [64, 127, 20, 67, 200], heads=1, hd=hd, bits=bits, group=group, page=32, seed=hd + bits + group,
                  table_extra=ROOM)
    check(case, per=4, masks=_trees(new, 5) if tree else None)


@pytest.mark.parametrize("kw", [dict(cap=7.0), dict(window=1), dict(window=50), dict(window=130), dict(dtype=f32),
                                dict(dtype=f16, y_dtype=f32), dict(stat=True), dict(scheme=R.SYM), dict(rows=5),
                                dict(per=5), dict(per=7), dict(q_scale=3.0), dict(small=True)], ids=str)
def test_tiles_of_256_rows(kw):
    kw = dict(kw)
    new = [48, 64, 50]
    per = kw.pop("per", 4)
    small = kw.pop("small", False)
    case = R.Case(new, [300, 64, 131], heads=2, hd=128, bits=4, group=64, page=16, seed=31, stat=kw.pop("stat", False),
                  scheme=kw.pop("scheme", None), extra_rows=kw.pop("rows", 0), table_extra=ROOM,
                  scale_of=(lambda which, b: 1e-3 * 40.0 ** b) if small else (lambda which, b: 1.0))
    check(case, per=per, masks=_trees(new, 6), **kw)


def test_wide_tiles_of_long_contexts_are_cut_and_joined():
    """Enough steps that a segment's parts are many, their maxima apart; every time the same bits."""
    case = R.Case([64], [7000], heads=1, hd=64, bits=4, group=64, page=64, seed=32, table_extra=ROOM)
    Q = (torch.randn(64, 4, 64, generator=torch.Generator().manual_seed(33)) * 3).to(bf16)
    Y = check(case, per=4, Q=Q)
    for _ in range(3):
        assert torch.equal(check(case, per=4, Q=Q), Y)


def test_wide_tiles_skip_what_is_not_there():
    """NaN scales in sight of some rows, pages that are not the cache's, sequences that are not valid."""
    case = R.Case([64, 64], [150, 100], heads=1, hd=128, bits=4, group=128, page=16, seed=34, table_extra=ROOM)
    masks = [1 << i for i in range(64)] * 2       # every new token sees the old ones and itself
    cache, batch = case.on_gpu()
    Q = torch.randn(128, 4, 128, generator=torch.Generator().manual_seed(35)).to(bf16).cuda()
    tree = _signed(masks).cuda()
    ws = ttq.new_kv_workspace(cache, batch, 4)
    good = ttq.ttq_kv_attention(cache, batch, Q, 0.1, tree=tree, ws=ws)
    # the last new token of sequence 0: a NaN key and value, which it alone sees
    nan = torch.full((1, 1, 128), float("nan"), dtype=bf16, device="cuda")
    one = ttq.KVBatch(batch.page_table[:1], batch.kv_len[:1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, 1)
    ttq.ttq_kv_write(cache, one, nan, nan)
    Y = ttq.ttq_kv_attention(cache, batch, Q, 0.1, tree=tree, ws=ws)
    assert bool(Y[63].isnan().all())
    keep = [r for r in range(128) if r != 63]
    assert torch.equal(Y[keep], good[keep])
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    # a page of sequence 1's old tokens: as if its positions were not there
    batch.page_table[1, 1] = 10 ** 8
    Y = ttq.ttq_kv_attention(cache, batch, Q, 0.1, tree=tree, ws=ws)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws)[1] == ttq.TTQ_FLAG_BAD_INDEX
    assert torch.equal(Y[:63], good[:63])
    K, V = case.sequence(1)
    see = R.visible(64, 100, 0, masks[64:])
    see[:, 16:32] = False
    y, bound = R.attention(K, V, Q[64:].cpu().double().numpy(), float(np.float32(0.1)), see)
    got = Y[64:].cpu().double().numpy()
    assert (np.abs(got - y) <= bound + (np.abs(y) + bound) * 2.0 ** -8 + 1e-5).all()
    # a length beyond the table: its rows stay
    batch.kv_len[1] = 10 ** 6
    Y = torch.full_like(Q, 5.0)
    ttq.ttq_kv_attention(cache, batch, Q, 0.1, tree=tree, ws=ws, Y=Y)
    assert bool((Y[64:] == 5).all())
    # (sequence 0 may be cut at other blocks now, so that its results are the same to their bound, not to the bit)
    K, V = case.sequence(0)
    y, bound = R.attention(K, V, Q[:64].cpu().double().numpy(), float(np.float32(0.1)), R.visible(64, 150, 0, masks[:64]))
    got = Y[:63].cpu().double().numpy()
    assert (np.abs(got - y[:63]) <= bound[:63] + (np.abs(y[:63]) + bound[:63]) * 2.0 ** -8 + 1e-5).all()
