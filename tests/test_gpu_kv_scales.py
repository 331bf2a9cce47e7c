"""Values of very different magnitudes in one context: a token's V counts for a
row as much as its probability says, and not at all where the row does not see
it, however large it is."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from test_gpu_kv_attention import ROOM, _signed, _trees
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def put(case, b, pos, K=None, V=None):
    """Token `pos` of sequence b becomes the codes of K and V [heads][hd] (None: as it is)."""
    f = case.cache
    for which, x in enumerate((K, V)):
        if x is not None:
            for h in range(f.kv_heads):
                q, s, z = R.quantise(f, np.asarray(x[h:h + 1], np.float32))
                R.write(case.host, f, case.table[b, pos // f.page_size], pos % f.page_size, h, which, q[0], s[0], z[0])


def scales(case, b):
    """The largest of each token's V scales, [heads][kv]."""
    s = R.unpack(case.host[case.table[b, :-(-case.kv[b] // case.cache.page_size)]], case.cache)[1][1]
    s = s.transpose(1, 0, 2, 3).reshape(case.cache.kv_heads, -1, s.shape[3])[:, :case.kv[b]].astype(np.uint16)
    return s.view(np.float16).astype(np.float64).max(-1)


def check(case, Q, masks=None, window=0, cap=0.0, y_dtype=f32):
    """Against the definition, within kv_reference.attention's bound without its last term, and for that
    kv 2^-25 times the codes' largest times the largest p_j s_j of the tokens j that the row sees, twice: p s_V is taken
    in units of at most that (s_j lies in [1, 2) powers of two), and rounded to half of binary16's least step, 2^-25."""
    f, hd = case.cache, case.cache.head_dim
    cache, batch = case.on_gpu()
    scale = 1 / math.sqrt(hd)
    ws = ttq.new_kv_workspace(cache, batch, Q.shape[1])
    tree = None if masks is None else _signed(masks).cuda()
    Y = ttq.ttq_kv_attention(cache, batch, Q.cuda(), scale, softcap=cap, window=window, tree=tree, ws=ws, y_dtype=y_dtype)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    got, per = Y.cpu().double().numpy(), Q.shape[1] // f.kv_heads
    code_max = 448.0 if f.bits == 8 else 2.0 ** f.bits - 1
    scale = float(np.float32(scale))
    for b, n in enumerate(case.new):
        r = slice(case.cu[b], case.cu[b] + n)
        K, V = case.sequence(b)
        see = R.visible(n, case.kv[b], window, None if masks is None else masks[r])
        q = Q[r].double().numpy()
        y, bound = R.attention(K, V, q, scale, see, cap, raw=case.sequence(b, of=R.magnitudes), q_rounded=Q.dtype == f32)
        top, s = np.zeros(y.shape[:2]), scales(case, b)
        for i in range(n):
            js = np.nonzero(see[i])[0]
            for h in range(Q.shape[1]):
                t = scale * (K[h // per][js] @ q[i, h])
                t = cap * np.tanh(t / cap) if cap else t
                p = np.exp(t - t.max())
                top[i, h] = (p / p.sum() * s[h // per][js]).max()
        tol = bound + (case.kv[b] * 2.0 ** -25 * 2 * code_max * top)[..., None]
        tol = tol + (np.abs(y) + tol) * R.HALF_STEP[Y.dtype]
        err = np.abs(got[r] - y)
        assert (err <= tol).all(), (b, int((~(err <= tol)).sum()), float(np.nanmax(err / tol)))
        # and the bound says something
        assert np.sqrt(np.mean(tol ** 2)) <= 0.25 * np.sqrt(np.mean(y ** 2)), (np.sqrt(np.mean(tol ** 2)), np.sqrt(np.mean(y ** 2)))
    return Y


SMALL, LARGE = 2.0 ** -6, 2.0 ** 16 / 3     # V's sizes: their scales 2^22 apart
FORMATS = [(64, 4, 64), (64, 2, 32), (128, 4, 128), (128, 4, 32), (128, 2, 64), (128, 8, 64), (256, 4, 64), (256, 8, 256)]


def _case(new, kv, hd, bits, group, seed, heads=1, **kw):
    return R.Case(new, kv, heads=heads, hd=hd, bits=bits, group=group, page=16, seed=seed,
                  scale_of=lambda which, b: SMALL if which else 1.0, **kw)


def _q(case, per, seed=0):
    hd = case.cache.head_dim
    return torch.randn((case.rows, case.cache.kv_heads * per, hd), generator=torch.Generator().manual_seed(seed)).to(bf16)


@pytest.mark.parametrize("hd,bits,group", FORMATS)
@pytest.mark.parametrize("per", [1, 4])
def test_large_values_that_some_rows_do_not_see(hd, bits, group, per):
    """A drafted token with V 2^22 times as large as all others: the rows of the other branches are as exact as without it."""
    new = [7, 3]
    case = _case(new, [75, 40], hd, bits, group, hd + bits)
    masks = [0b1, 0b11, 0b101, 0b1001, 0b10101, 0b100001, 0b1000001] + [0b1, 0b11, 0b101]
    rng = np.random.default_rng(1)
    put(case, 0, 75 - 7 + 1, V=rng.normal(size=(1, hd)) * LARGE)     # rows 1 alone sees it
    put(case, 1, 40 - 3 + 2, V=rng.normal(size=(1, hd)) * LARGE)     # row 2 of the other
    check(case, _q(case, per), masks)


@pytest.mark.parametrize("hd,bits,group", FORMATS)
def test_large_values_behind_the_window(hd, bits, group):
    """In a block of which the window covers a part."""
    case = _case([1, 2], [100, 61], hd, bits, group, hd + bits + 1)
    rng = np.random.default_rng(2)
    for b, kv in enumerate(case.kv):
        n = case.new[b]
        put(case, b, kv - n - 21, V=rng.normal(size=(1, hd)) * LARGE)     # the first row sees 20 positions before its own
    check(case, _q(case, 4), window=21)


def _away(case, per, b, pos, V, seed=0):
    """Q, and a token `pos` of K that scores some 60 (in powers of e) below the others for all rows."""
    hd = case.cache.head_dim
    Q = _q(case, per, seed)
    Q[..., 0] = 30.0
    k = np.zeros((case.cache.kv_heads, hd))
    k[:, 0] = -2.0 * math.sqrt(hd)
    put(case, b, pos, K=k, V=V)
    return Q


@pytest.mark.parametrize("hd,bits,group", FORMATS)
@pytest.mark.parametrize("per", [1, 4])
@pytest.mark.parametrize("pos", [3, 50])
def test_large_values_of_no_probability(hd, bits, group, per, pos):
    """Seen, and with a probability of e^-60 beside the others: before them in their context, and after most of them."""
    case = _case([2], [70], hd, bits, group, hd + bits + 2)
    rng = np.random.default_rng(3)
    check(case, _away(case, per, 0, pos, rng.normal(size=(1, hd)) * LARGE))


@pytest.mark.parametrize("hd,bits,group", [(64, 4, 64), (128, 4, 64), (128, 8, 128), (128, 2, 128)])
def test_large_values_in_tiles_of_256_rows(hd, bits, group):
    new = [60, 64]
    case = _case(new, [200, 164], hd, bits, group, hd + bits + 3, table_extra=ROOM * 2)
    masks = [1 << i for i in range(60)] + [1 << i for i in range(64)]
    rng = np.random.default_rng(4)
    put(case, 0, 140 + 59, V=rng.normal(size=(1, hd)) * LARGE)       # the last new token alone sees itself
    put(case, 1, 100 + 5, V=rng.normal(size=(1, hd)) * LARGE)
    check(case, _away(case, 4, 0, 17, rng.normal(size=(1, hd)) * LARGE), masks)
    check(case, _q(case, 4, 5), masks, window=90)


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 14])
@pytest.mark.parametrize("wide", [False, True])
def test_groups_of_very_different_sizes(ratio, wide):
    """V's channels of one group far above those of the other."""
    new = [64] if wide else [3]
    case = _case(new, [150], 128, 4, 64, 9, table_extra=2 * ROOM if wide else 1)
    rng = np.random.default_rng(5)
    size = np.where(np.arange(128) < 64, SMALL * ratio, SMALL)
    for pos in range(150):
        put(case, 0, pos, V=rng.normal(size=(1, 128)) * size)
    check(case, _q(case, 4), _trees(new, 7))


@pytest.mark.parametrize("per", [1, 4, 8])
def test_values_that_grow_along_the_context(per):
    """Each block's V larger than the one before, by 2^24 in all, over many blocks and thread blocks' parts."""
    case = _case([2], [1500], 64, 4, 64, 10)
    rng = np.random.default_rng(6)
    for pos in range(1500):
        put(case, 0, pos, V=rng.normal(size=(1, 64)) * 2.0 ** (-8 + 24 * pos / 1500))
    check(case, _q(case, per))
    check(case, _q(case, per), cap=20.0)
    Q = _q(case, per) * 8
    check(case, Q)
