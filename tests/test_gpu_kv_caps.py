"""Caps of every size that the cache's attention takes: softcap tanh(t / softcap)
from where it makes all scores equal to where it changes none."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from test_gpu_kv_attention import ROOM, _signed, _trees
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def check(case, per, cap, scale, masks=None, q_scale=1.0, part=0.25):
    """Within kv_reference.attention's bound, but with a capped score's own error relative to the score instead of to
    the cap: 2^-19 of it (tanh of a quarter or more to 2^-21.4, some 4 roundings to 2^-24 and the exponential's and the
    reciprocal's last bits, over tanh(1 / 4) = 0.245; below that a polynomial to 2^-22), where the cap is above 256; at
    most 256 2^-20 below."""
    f, hd = case.cache, case.cache.head_dim
    cache, batch = case.on_gpu()
    g = torch.Generator().manual_seed(3)
    Q = (torch.randn((case.rows, f.kv_heads * per, hd), generator=g) * q_scale).to(bf16)
    ws = ttq.new_kv_workspace(cache, batch, Q.shape[1])
    tree = None if masks is None else _signed(masks).cuda()
    Y = ttq.ttq_kv_attention(cache, batch, Q.cuda(), scale, softcap=cap, tree=tree, ws=ws, y_dtype=f32)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    got = Y.cpu().double().numpy()
    code_max = 448.0 if f.bits == 8 else 2.0 ** f.bits - 1
    cap, scale = float(np.float32(cap)), float(np.float32(scale))
    for b, n in enumerate(case.new):
        r = slice(case.cu[b], case.cu[b] + n)
        K, V = case.sequence(b)
        see = R.visible(n, case.kv[b], 0, None if masks is None else masks[r])
        q = Q[r].double().numpy()
        s = R.unpack(case.host[case.table[b, :-(-case.kv[b] // f.page_size)]], f)[1][1]
        s = s.transpose(1, 0, 2, 3).reshape(f.kv_heads, -1, s.shape[3])[:, :case.kv[b]].astype(np.uint16).view(np.float16)
        # (from 2^30 on the cap moves a score of 2^8 by 2^-45 of it, and its term would drown the others in 64 bits)
        told = 0.0 if cap >= 2.0 ** 30 else cap
        y, bound = R.attention(K, V, q, scale, see, told, raw=case.sequence(b, of=R.magnitudes), smax=float(s.max()),
                               code_max=code_max)
        for i in range(n):
            js = np.nonzero(see[i])[0]
            for h in range(Q.shape[1]):
                t = cap * np.tanh(scale * (K[h // per][js] @ q[i, h]) / cap)
                p = np.exp(t - t.max())
                a = p / p.sum() @ np.abs(V[h // per][js])
                own = min(np.abs(t).max() * 2.0 ** -19, cap) if cap > 256 else cap * 2.0 ** -20
                bound[i, h] += a * 2 * (own - told * 2.0 ** -20)
        tol = bound + (np.abs(y) + bound) * 2.0 ** -24
        err = np.abs(got[r] - y)
        assert (err <= tol).all(), (b, int((~(err <= tol)).sum()), float(np.nanmax(err / tol)))
        assert bound.mean() <= part * np.sqrt(np.mean(y ** 2)), (bound.mean(), np.sqrt(np.mean(y ** 2)))


CAPS = [2.0 ** -149, 1e-40, 2.0 ** -126, 1e-30, 1e-8, 0.01, 1.0, 50.0, 255.0, 257.0, 2000.0, 1e4, 1e6, 1e10, 2.0 ** 64, 1e25,
        2.0 ** 127, 3.4e38]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("hd,bits,group,per", [(64, 4, 64, 1), (128, 2, 64, 4), (256, 8, 64, 2)])
def test_every_cap(cap, hd, bits, group, per):
    case = R.Case([2, 1], [70, 33], heads=1, hd=hd, bits=bits, group=group, page=16, seed=hd + per)
    check(case, per, cap, 1 / math.sqrt(hd))


@pytest.mark.parametrize("cap", CAPS)
def test_every_cap_in_tiles_of_256_rows(cap):
    case = R.Case([64], [150], heads=1, hd=64, bits=4, group=64, page=16, seed=51, table_extra=2 * ROOM)
    check(case, 4, cap, 0.125, masks=_trees([64], 9))


@pytest.mark.parametrize("cap", [0.0, 20.0, 500.0, 1e4])
def test_scores_beyond_what_their_factors_hold(cap):
    """Scores around the cap and well above it; and scales that overflow with the row's own size where the score is zero."""
    case = R.Case([2], [60], heads=1, hd=64, bits=4, group=64, page=16, seed=52)
    if cap:
        # (q times the offset codes adds up to some 4e4, and 6 roundings of that at 2^-22 to 0.06 of a score: the bound
        # is twice that of p |V|, which is some three times |y|)
        check(case, 2, cap, 0.125, q_scale=200.0, part=0.5)
    cache, batch = case.on_gpu()
    cache.pages.zero_()                               # zero codes, scales and zeros: every score is zero
    Q = torch.full((2, 2, 64), 1e4, dtype=bf16, device="cuda")
    for scale in (3e38, -3e38):
        Y = ttq.ttq_kv_attention(cache, batch, Q, scale, softcap=cap)
        assert bool((Y == 0).all())
