"""How much of its precision the cache's attention keeps where the output has
more than bf16 to show it: a statistic D of K, rows of Q in float32."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from test_gpu_kv_attention import ROOM, _signed, _trees
from test_weight_quantization_ttq_b200 import ttq

pytestmark = pytest.mark.gpu
bf16, f32, f16 = torch.bfloat16, torch.float32, torch.float16


def run(case, per, dtype, y_dtype, masks=None, cap=0.0, q_scale=1.0):
    """(Y, its definition in 64 bits, the bound): kv_reference.attention on Q D_k^{-1/2} and the codes' own values, without
    a rounding of Q to binary16 (what is left of it is in the bound's 2^-20 of the row's largest element)."""
    f, hd = case.cache, case.cache.head_dim
    cache, batch = case.on_gpu()
    g = torch.Generator().manual_seed(per)
    Q = (torch.randn((case.rows, f.kv_heads * per, hd), generator=g) * q_scale).to(dtype)
    scale = 1 / math.sqrt(hd)
    ws = ttq.new_kv_workspace(cache, batch, Q.shape[1])
    tree = None if masks is None else _signed(masks).cuda()
    Y = ttq.ttq_kv_attention(cache, batch, Q.cuda(), scale, softcap=cap, tree=tree, ws=ws, y_dtype=y_dtype)
    torch.cuda.synchronize()
    assert ttq.ttq_get_status(ws) == (ttq.TTQ_OK, 0)
    q = Q.double().numpy()
    if case.Dr[0] is not None:
        q = q * np.repeat(case.Dr[0].astype(np.float64), per, 0)
    want, bounds = np.zeros(q.shape), np.zeros(q.shape)
    Dr = (None, case.Dr[1])
    for b, n in enumerate(case.new):
        r = slice(case.cu[b], case.cu[b] + n)
        K, V = case.sequence(b, Dr=Dr)
        s = R.unpack(case.host[case.table[b, :-(-case.kv[b] // f.page_size)]], f)[1][1]
        s = s.transpose(1, 0, 2, 3).reshape(f.kv_heads, -1, s.shape[3])[:, :case.kv[b]].astype(np.uint16).view(np.float16)
        smax = float(s.max()) * (1.0 if Dr[1] is None else float(Dr[1].max()))
        see = R.visible(n, case.kv[b], 0, None if masks is None else masks[r])
        want[r], bounds[r] = R.attention(K, V, q[r], float(np.float32(scale)), see, cap, smax=smax,
                                         code_max=448.0 if f.bits == 8 else 2.0 ** f.bits - 1,
                                         raw=case.sequence(b, Dr=Dr, of=R.magnitudes))
    return Y.cpu().double().numpy(), want, bounds


MODES = [(f16, f16, True), (bf16, f32, True), (f32, f32, False), (f32, f16, True), (f32, f32, True)]


@pytest.mark.parametrize("dtype,y_dtype,stat", MODES, ids=str)
@pytest.mark.parametrize("hd,group,per,n", [(64, 32, 1, 1), (128, 128, 4, 1), (128, 32, 4, 5), (256, 128, 2, 3), (64, 64, 8, 4)])
def test_scores_are_as_exact_as_float32_sums(dtype, y_dtype, stat, hd, group, per, n):
    """E4M3 codes, whose sums hold no offsets, and scores of 20 and more, whose own error shows most."""
    case = R.Case([n, 1], [150, 61], heads=2, hd=hd, bits=8, group=group, page=16, seed=hd + n, stat=stat)
    got, want, bound = run(case, per, dtype, y_dtype, q_scale=16.0)
    tol = bound + (np.abs(want) + bound) * R.HALF_STEP[y_dtype] + 2.0 ** -24
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("hd,bits,group,per,n", [
    (64, 4, 64, 1, 1), (64, 2, 32, 2, 8), (128, 4, 32, 2, 1), (128, 2, 128, 8, 2), (128, 4, 128, 4, 8), (128, 8, 64, 1, 1),
    (256, 4, 256, 2, 1), (256, 2, 64, 4, 8), (64, 4, 64, 4, 64), (128, 4, 64, 4, 64)])
@pytest.mark.parametrize("dtype", [f16, f32], ids=str)
def test_binary16_outputs_lose_less_than_their_own_rounding(hd, bits, group, per, n, dtype):
    """Against 64 bits, in the 2-norm: p s_V is rounded to as many bits as the output is, each token's on its own, so
    that it adds as much as the output's rounding at most, sqrt(2) together; the scores' errors add little to that
    (1.5 leaves them half of the output's rounding)."""
    case = R.Case([n, n], [n + 700, n + 333], heads=2, hd=hd, bits=bits, group=group, page=16, seed=hd + bits + n, stat=True,
                  table_extra=ROOM)     # (wide enough for tiles of 256 rows)
    got, want, _ = run(case, per, dtype, f16, masks=_trees(case.new, 3) if n > 1 else None)
    own = np.linalg.norm(torch.from_numpy(want).to(f16).double().numpy() - want)
    assert np.linalg.norm(got - want) <= 1.5 * own, float(np.linalg.norm(got - want) / own)
