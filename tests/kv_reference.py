"""The quantised key/value cache in numpy: its layout, token by token and
channel by channel as include/ttq_kv.h states it, its values in 64 bits, and
attention over them from the definition."""
from __future__ import annotations

import functools
import math

import numpy as np
import torch

import ttq_oracle
from test_weight_quantization_ttq_b200 import ttq

ASYM, SYM, FP8 = ttq.TTQ_QSCHEME_ASYMMETRIC, ttq.TTQ_QSCHEME_SYMMETRIC, ttq.TTQ_QSCHEME_FP8_E4M3


@functools.lru_cache(None)
def layout(hd: int, bits: int, group: int):
    """(K, V): the first bit of every code within its part, [16][hd]."""
    lane_bytes = hd * bits // 32
    piece = min(16, lane_bytes)
    per_word, per_unit = 32 // bits, 16 // bits

    def place(lane, half, byte):
        return ((byte // piece) * 2 + half) * 32 * piece + lane * piece + byte % piece

    K, V = np.zeros((16, hd), np.int64), np.zeros((16, hd), np.int64)
    for t in range(16):
        for c in range(hd):
            k, r = divmod(c, group)
            e = k * (group // 4) + r % (group // 4)
            word, f = divmod(e, per_word)
            if bits < 8:
                f = f // 2 + f % 2 * (per_word // 2)
            bit = bits * f
            K[t, c] = 8 * place(4 * (t % 8) + r // (group // 4), t // 8, 4 * word + bit // 8) + bit % 8
            e = k * (group // 8) + r % (group // 8)
            unit, f = divmod(e, per_unit)
            bit = bits * f
            V[t, c] = 8 * place(4 * (r // (group // 8)) + t % 8 // 2, t // 8, 4 * unit + 2 * (t % 2) + bit // 8) + bit % 8
    return K, V


def parts(hd, bits, group):
    """Bytes of the codes and of the pairs of a block's K (or V)."""
    return 16 * hd * bits // 8, 16 * (hd // group) * 4


def blocks(pages: np.ndarray, cache) -> np.ndarray:
    """pages uint8 [P][page bytes] as [P][heads][blocks][block bytes]."""
    c, p = parts(cache.head_dim, cache.bits, cache.group)
    return pages.reshape(pages.shape[0], cache.kv_heads, cache.page_size // 16, 2 * (c + p))


def unpack(pages: np.ndarray, cache):
    """For K and V: codes [P][heads][page_size][hd], scales and zeros
    [P][heads][page_size][groups] (binary16 as uint16)."""
    hd, bits, group = cache.head_dim, cache.bits, cache.group
    c, p = parts(hd, bits, group)
    blk = blocks(pages, cache)
    out = []
    for which, at in enumerate(layout(hd, bits, group)):
        part = blk[..., which * (c + p):(which + 1) * (c + p)]
        codes = (part[..., at // 8] >> (at % 8).astype(np.uint8)) & np.uint8((1 << bits) - 1)
        pair = np.ascontiguousarray(part[..., c:]).view(np.uint16).reshape(*part.shape[:-1], 16, hd // group, 2)
        shape = (*blk.shape[:2], cache.page_size)
        out.append((codes.reshape(*shape, hd), pair[..., 0].reshape(*shape, -1), pair[..., 1].reshape(*shape, -1)))
    return out


def write(pages: np.ndarray, cache, page: int, slot: int, head: int, which: int, codes, scales, zeros) -> None:
    """One row's codes [hd], scales and zeros [groups] into pages."""
    hd, bits, group = cache.head_dim, cache.bits, cache.group
    c, p = parts(hd, bits, group)
    t = slot % 16
    part = blocks(pages, cache)[page, head, slot // 16, which * (c + p):(which + 1) * (c + p)]
    at = layout(hd, bits, group)[which][t]
    for i in range(hd):
        byte, sh = divmod(int(at[i]), 8)
        part[byte] = (int(part[byte]) & ~(((1 << bits) - 1) << sh) & 255) | (int(codes[i]) << sh)
    pair = np.stack([scales, zeros], -1).astype(np.uint16).reshape(-1).view(np.uint8)
    width = 4 * (hd // group)
    part[c + t * width:c + (t + 1) * width] = pair


def e4m3(codes: np.ndarray) -> np.ndarray:
    e, m = (codes.astype(np.int64) >> 3) & 15, codes.astype(np.int64) & 7
    v = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9) * np.where(codes & 128, -1.0, 1.0)
    return np.where((codes & 127) == 127, np.nan, v)


def values(cache, codes, scales, zeros, Dr=None) -> np.ndarray:
    """float64 s (q - z) [D^{-1/2}]; Dr [heads][hd] applies to codes [..., heads, positions, hd]."""
    s = np.ascontiguousarray(scales).view(np.float16).astype(np.float64)
    z = np.ascontiguousarray(zeros).view(np.float16).astype(np.float64)
    q = e4m3(codes) if cache.bits == 8 else codes.astype(np.float64)
    q = q.reshape(*q.shape[:-1], -1, cache.group)
    if cache.bits != 8:
        q = q - z[..., None]
    v = (q * s[..., None]).reshape(codes.shape)
    return v if Dr is None else v * Dr.astype(np.float64)[:, None, :]


def quantise(cache, rows: np.ndarray, D=None):
    """The oracle's codes [n][hd], scales and zeros [n][groups] of rows
    [n][hd] of one head (D [hd] float32 or None)."""
    O = ttq_oracle.get()
    x = np.ascontiguousarray(rows, np.float32)
    if cache.bits == 8:
        codes, s, z, _ = O.quantize_fp8(x, D, cache.group)
        q = codes.view(np.uint8).reshape(x.shape)
    else:
        codes, s, z, _ = O.quantize(x, D, cache.bits, cache.group, symmetric=cache.scheme == SYM)
        q = O.unpack(codes, x.shape[1], cache.bits)
    return q, s, z


def magnitudes(cache, codes, scales, zeros, Dr=None) -> np.ndarray:
    """float64 s (64 + max(q, z)) [D^{-1/2}] (s |q| for E4M3): what the sums of offset codes and of offset zeros
    are made of."""
    if cache.bits == 8:
        return np.abs(values(cache, codes, scales, zeros, Dr))
    s = np.ascontiguousarray(scales).view(np.float16).astype(np.float64)
    z = np.ascontiguousarray(zeros).view(np.float16).astype(np.float64)
    q = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, cache.group)
    v = ((64 + np.maximum(q, z[..., None])) * s[..., None]).reshape(codes.shape)
    return v if Dr is None else v * Dr.astype(np.float64)[:, None, :]


class Case:
    """A cache with random contents, and a batch with the given new rows and
    lengths.  Tokens behind a sequence's length are left as random bytes."""

    def __init__(self, new, kv, heads=2, hd=128, bits=4, group=128, scheme=None, page=32, seed=0, stat=False,
                 scale_of=lambda which, g: 1.0, extra_rows=0, spare=2, table_extra=1):
        rng = np.random.default_rng(seed)
        self.rng, self.new, self.kv = rng, list(new), list(kv)
        self.stat = stat
        need = [-(-k // page) for k in kv]
        P = sum(need) + spare
        perm = rng.permutation(P)
        self.table = np.full((len(kv), max(need + [0]) + table_extra), -7, np.int32)   # entries that are never used
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + extra_rows
        self.host = rng.integers(0, 256, (P, ttq.ttq_kv_page_bytes(page, heads, hd, bits, group)), dtype=np.uint8)
        scheme = (FP8 if bits == 8 else ASYM) if scheme is None else scheme
        self.cache = type("Format", (), dict(page_size=page, kv_heads=heads, head_dim=hd, bits=bits, group=group,
                                             scheme=scheme))
        self.D = [np.exp(rng.normal(size=(heads, hd))).astype(np.float32) if stat else None for _ in range(2)]
        # the same tokens' rows, quantised by the oracle, for every position of every sequence
        c, p = parts(hd, bits, group)
        K, V = layout(hd, bits, group)
        ng = hd // group
        for b, n in enumerate(kv):
            for h in range(heads):
                for which in range(2):
                    x = rng.normal(size=(n, hd)) * np.where(rng.random(hd) < 0.03, 6.0, 1.0)
                    x = x * scale_of(which, b)
                    if n == 0:
                        continue
                    q, s, z = quantise(self.cache, x, None if not stat else self.D[which][h])
                    for t in range(n):
                        write(self.host, self.cache, self.table[b, t // page], t % page, h, which, q[t], s[t], z[t])

    def on_gpu(self):
        """(KVCache, KVBatch) on the current device."""
        f = self.cache
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
        D = [dev(d) for d in self.D]
        Dr = [None if d is None else (1 / d.double().sqrt()).float() for d in D]
        self.Dr = [None if d is None else d.cpu().numpy() for d in Dr]
        cache = ttq.KVCache(dev(self.host), f.page_size, f.kv_heads, f.head_dim, f.bits, f.group, f.scheme, D_k=D[0],
                            D_v=D[1], D_k_rsqrt=Dr[0], D_v_rsqrt=Dr[1])
        batch = ttq.KVBatch(dev(self.table), dev(np.asarray(self.kv, np.int32)), dev(self.cu), self.rows,
                            max(self.new + [0]))
        return cache, batch

    def sequence(self, b: int, pages: np.ndarray | None = None, Dr=(None, None), of=values):
        """K and V (or another function `of` their codes) of sequence b, float64 [heads][kv][hd]."""
        pages = self.host if pages is None else pages
        n, page = self.kv[b], self.cache.page_size
        own = self.table[b, :-(-n // page)]
        out = []
        for which, (q, s, z) in enumerate(unpack(pages[own], self.cache)):
            join = lambda a: a.transpose(1, 0, 2, 3).reshape(a.shape[1], -1, a.shape[3])[:, :n]
            out.append(of(self.cache, join(q), join(s), join(z), Dr[which]))
        return out


def visible(n: int, kv: int, window: int = 0, masks=None) -> np.ndarray:
    """bool [n][kv]: which positions each new row sees."""
    old = kv - n
    masks = [(2 << i) - 1 for i in range(n)] if masks is None else [int(m) & (2 ** 64 - 1) for m in masks]
    sees = [[k for k in range(n) if m >> k & 1] for m in masks]
    pos = [old + sum(k != i for k in s) for i, s in enumerate(sees)]
    out = np.zeros((n, kv), bool)
    for i in range(n):
        for j in range(old):
            out[i, j] = window <= 0 or pos[i] - j < window
        for k in sees[i]:
            out[i, old + k] = window <= 0 or pos[i] - pos[k] < window
    return out


def attention(K, V, Q, scale, see, cap=0.0, q_rounded=False, smax=None, code_max=15.0, raw=None):
    """(y, bound) for one sequence: K, V float64 [heads][kv][hd], Q float64
    [n][query heads][hd], see [n][kv]; raw: (K, V) of magnitudes().  The bound
    on the kernel's error, from its own roundings:
      scores: the fp32 sums of q times offset codes, offsets and zeros, hd / 16
        matrix instructions and two more terms at 2^-22 each of the sum of
        magnitudes (truncated sums: a whole unit 2^-23, twice), 8 roundings of
        the score itself at 2^-23, and Q rounded to binary16 (2^-11 each) where
        it is (q_rounded), else 2^-20 of the row's largest for the elements
        that are subnormal beside it;
      probabilities: a relative 2 d for a score error of d, 2^-20 for the
        exponentials and the sums' fp32 roundings;
      p s_V rounded to binary16: 2^-11 relative, or 2^-25 in units of at
        most twice the largest scale where it is subnormal;
      the second product: at most 34 truncated additions of offset codes between
        two times that offsets and zeros are taken off, 2^-23 each."""
    n, hq, hd = Q.shape
    heads, kv = K.shape[:2]
    per = hq // heads
    K_raw, V_raw = raw if raw is not None else (np.abs(K), np.abs(V))
    y, bound = np.zeros((n, hq, hd)), np.zeros((n, hq, hd))
    for h in range(hq):
        k, v = K[h // per], V[h // per]
        for i in range(n):
            js = np.nonzero(see[i])[0]
            if js.size == 0:
                continue
            q = Q[i, h]
            t = scale * (k[js] @ q)
            mag = abs(scale) * (np.abs(k[js]) @ np.abs(q))
            mag_raw = abs(scale) * (K_raw[h // per][js] @ np.abs(q))
            top = abs(scale) * np.abs(k[js]).sum(-1) * np.abs(q).max()
            d = mag_raw * (hd / 16 + 2) * 2.0 ** -22 + np.abs(t) * 8 * 2.0 ** -23
            d = d + (mag * 2.0 ** -11 if q_rounded else 0.0) + top * 2.0 ** -20
            if cap > 0:
                t = cap * np.tanh(t / cap)
                d = d + cap * 2.0 ** -20
            p = np.exp(t - t.max())
            weight = p.sum()       # at most the kernel's: its maximum is never above the largest score
            p /= weight
            y[i, h] = p @ v[js]
            a, a_raw = p @ np.abs(v[js]), p @ V_raw[h // per][js]
            bound[i, h] = a * (2 * d.max() + 2.0 ** -20 + 2.0 ** -11 + js.size * 2.0 ** -24) + a_raw * 34 * 2.0 ** -23
            if smax is not None:
                bound[i, h] += js.size * 2.0 ** -25 * 2 * smax * code_max / weight
    return y, bound


HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
