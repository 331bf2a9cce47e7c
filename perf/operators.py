"""The quantised key/value cache's operators as measured cases: writing rows and reading them back, reading a
cache, and attention over it, in plain torch operations (`own` false) and through the library (`own` true).

The cache is paged.  A page holds, for each key/value head, page_size / 16 blocks of 16 tokens; a block is
[K codes | K (scale, zero) pairs | V codes | V pairs].  Sequence b has n_b rows in a call, standing for its last
n_b positions: row cu_new[b] + i is position kv_len[b] - n_b + i.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    def case(name, op, **kw):
        c = dict(name=name, op=op, batch=1, ctx=0, new=1, ragged=False, hq=32, hkv=8, hd=128, bits=4, group=128,
                 page=64, dtype="bf16", stat=False, cap=0.0, window=0, tree=False)
        c.update(kw)
        return c
    return [
        # one decode step's new tokens of 32 requests, appended and read back as the values the cache now holds
        case("write-step-32", "write", batch=32, ctx=1500, new=1, hkv=8),
        # the prompts of five requests with a 70B-like layer's 8 heads, K and V scaled by their activation statistic
        case("write-prompts", "write", batch=5, ctx=4097, new=4097, ragged=True, group=64, stat=True),
        # a 1000-token chunk of one long prompt in E4M3, 32 heads of a 7B-like layer, starting inside a page
        case("write-chunk-fp8", "write", ctx=5123, new=1000, hkv=32, bits=8, dtype="f16"),
        # a whole long sequence read back, as for the dense attention of its next prompt chunk
        case("read-long", "read", ctx=32785),
        # many short sequences of a small model with 2-bit codes
        case("read-ragged-int2", "read", batch=24, ctx=2111, ragged=True, hkv=4, hd=64, bits=2, group=32, page=16,
             dtype="f16"),
        # one user's next token, 32 heads of a 7B-like layer: launch latency counts
        case("decode-one", "attention", ctx=517, hkv=32),
        # a serving batch with contexts of very different lengths, 64 query heads on 8
        case("decode-batch", "attention", batch=64, ctx=8192, ragged=True, hq=64, group=64),
        # one very long context: the split over the cache
        case("decode-long-fp8", "attention", ctx=131072, hq=64, bits=8),
        # capped scores and a sliding window, wide heads, 2-bit codes
        case("decode-cap-window-int2", "attention", batch=20, ctx=9000, ragged=True, hq=16, hkv=4, hd=256, bits=2,
             group=64, cap=50.0, window=4096, dtype="f16"),
        # a short chain of drafted tokens verified for many requests, one query head per key/value head
        case("chain-5", "attention", batch=48, ctx=1027, new=5, ragged=True, hkv=32, hd=64, group=64, page=32),
        # trees of 24 drafted tokens over ragged contexts
        case("tree-24", "attention", batch=8, ctx=4099, new=24, ragged=True, hq=64, tree=True, stat=True),
        # the largest trees, over a long context, with a cap
        case("tree-64-fp8", "attention", batch=2, ctx=16384, new=64, bits=8, cap=30.0, tree=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention"])
    hd = rng.choice([64, 128, 128, 256])
    bits = rng.choice([2, 4, 4, 8])
    group = rng.choice([g for g in (32, 64, 128, 256) if hd // 4 <= g <= hd])
    hkv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    c = dict(op=op, batch=_log(rng, 1, 64), ctx=0, new=1, ragged=rng.random() < 0.7, hq=32, hkv=hkv, hd=hd, bits=bits,
             group=group, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
             stat=rng.random() < 0.3, cap=0.0, window=0, tree=False)
    per_token = c["batch"] * hkv * hd  # elements of K in one position of every sequence
    if op == "write":
        c["new"] = _log(rng, 1, max(1, min(8192, 20_000_000 // per_token)))
        c["ctx"] = c["new"] + rng.choice([0, rng.randrange(0, 700)])
    elif op == "read":
        c["ctx"] = _log(rng, 1, max(1, min(32768, 30_000_000 // per_token)))
    else:
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        c["new"] = rng.choice([1, 1, 1, 2, 5, 8, 16, 33, 64])
        c["tree"] = c["new"] > 1 and rng.random() < 0.6
        c["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        # bounded by the cache's elements and by the products with every query row
        most = min(131072, 200_000_000 // per_token, 6_000_000_000 // (c["batch"] * c["hq"] * hd * c["new"]))
        c["ctx"] = _log(rng, c["new"], max(c["new"], most))
        c["window"] = rng.choice([0, 0, 0, _log(rng, 16, max(16, c["ctx"]))])
    return c


def _ragged(most, least, batch, ragged):
    """`batch` lengths from the case alone: the first is `most`, the others spread over [least, most]."""
    if not ragged:
        return [most] * batch
    return [most] + [least + (most - least) * ((b * 40503 + 12345) % 65536) // 65536 for b in range(1, batch)]


def _lens(c):
    """(new rows, cache length) of each sequence."""
    if c["op"] == "write":
        n = _ragged(c["new"], 1, c["batch"], c["ragged"])
        return n, [c["ctx"] - c["new"] + k for k in n]
    kv = _ragged(c["ctx"], c["new"] if c["op"] == "attention" else 1, c["batch"], c["ragged"])
    return (kv if c["op"] == "read" else [c["new"]] * c["batch"]), kv


def work(case):
    c = case
    n, kv = _lens(c)
    row = c["hkv"] * 2 * (c["hd"] * c["bits"] // 8 + 4 * (c["hd"] // c["group"]))  # a position's bytes in the cache
    dense = c["hkv"] * 2 * c["hd"] * 2
    if c["op"] == "write":  # the rows in, the cache out, and the rows back
        return {"bytes": sum(n) * (dense + row + dense), "flops": 0}
    if c["op"] == "read":
        return {"bytes": sum(n) * (row + dense), "flops": 0}
    seen = [min(k, c["window"] + m - 1) if c["window"] else k for m, k in zip(n, kv)]
    return {"bytes": sum(seen) * row + 2 * sum(n) * c["hq"] * c["hd"] * 2,
            "flops": 4 * c["hd"] * c["hq"] * sum(m * s for m, s in zip(n, seen))}


# ------------------------------------------------- the cache's format in torch
def _layout(c, device):
    """Where a block's codes are: for K and V, `at` [16][hd] the code's byte within its part, `shift` [hd] its
    first bit there, and `order` [hd * bits / 8][8 / bits] the channels that a token's bytes hold."""
    hd, b, gs = c["hd"], c["bits"], c["group"]
    lane_bytes = hd * b // 32
    piece = min(16, lane_bytes)
    ch, tok = torch.arange(hd, device=device), torch.arange(16, device=device)
    g, j = ch // gs, ch % gs

    def place(lane, half, byte):
        return ((byte // piece) * 2 + half) * 32 * piece + lane * piece + byte % piece

    # K: the channels 2i and 2i + 1 of a 32-bit word's codes are at fields i and i + half of the fields (bytes: in order)
    t, slot, per = j // (gs // 4), g * (gs // 4) + j % (gs // 4), 32 // b
    field = slot if b == 8 else slot // per * per + slot % per // 2 + slot % 2 * (per // 2)
    bit = field * b
    k_at = place((tok % 8)[:, None] * 4 + t, (tok // 8)[:, None], bit // 8)
    k_order = (t * hd + field).argsort().view(-1, 8 // b)
    u, slot = j // (gs // 8), g * (gs // 8) + j % (gs // 8)
    unit, rest = slot // (16 // b), slot % (16 // b) * b
    v_at = place(u * 4 + (tok % 8)[:, None] // 2, (tok // 8)[:, None], unit * 4 + (tok % 2)[:, None] * 2 + rest // 8)
    return {"k": (k_at, bit % 8, k_order),
            "v": (v_at, rest % 8, (u * hd + slot).argsort().view(-1, 8 // b))}


def _part_bytes(c):
    return 16 * c["hd"] * c["bits"] // 8, 16 * (c["hd"] // c["group"]) * 4


def _quantise(c, x, D):
    """(code values, scale, zero) of rows x [..., hd]; D [..., hd] or None."""
    x = x.float()
    if D is not None:
        x = x * D.sqrt()
    x = x.unflatten(-1, (-1, c["group"]))
    if c["bits"] == 8:
        span = x.abs().amax(-1, keepdim=True) / x.new_tensor(448.0)  # a tensor: a true division, not a product
    else:
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
        span = (hi - lo) / x.new_tensor(2.0 ** c["bits"] - 1)
    span = span.clamp(min=2.0 ** -14)
    s = span.half()
    s = torch.where(s.float() < span, (s.view(torch.int16) + 1).view(torch.float16), s)  # rounded up
    inv = 1.0 / s.float()
    if c["bits"] == 8:
        q = (x * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        z = torch.zeros_like(s)
    else:
        top = 2 ** c["bits"] - 1
        # the products next to a rounding border, exact in 64 bits
        z = (-lo.double() * inv.double()).round().clamp(0, top)
        q = ((x.double() * inv.double()).round() + z).clamp(0, top).to(torch.uint8)
        z = z.half()
    return q.flatten(-2), s.squeeze(-1), z.squeeze(-1)


def _code_bytes(c, q, order):
    """A token's codes [..., hd] as the bytes in `order`."""
    per = 8 // c["bits"]
    shift = torch.arange(per, device=q.device, dtype=torch.int32) * c["bits"]
    return (q[..., order].int() << shift).sum(-1).to(torch.uint8)


def _write_plain(c, s):
    k_part, p_part = _part_bytes(c)
    flat = s["pages"].view(-1)
    base, tok = _row_base(c, s)
    for x, D, which, off in ((s["K"], s["D_k"], "k", 0), (s["V"], s["D_v"], "v", k_part + p_part)):
        at, _, order = s["layout"][which]
        q, sc, z = _quantise(c, x, D)
        flat[(base + off)[..., None] + at[:, order[:, 0]][tok][:, None, :]] = _code_bytes(c, q, order)
        pair = torch.stack((sc, z), -1).flatten(-2).view(torch.uint8)
        width = pair.shape[-1]
        flat[(base + off + k_part)[..., None] + (tok * width)[:, None, None]
             + torch.arange(width, device=flat.device)] = pair


def _values(c, q, shift, pair):
    """float32 values [..., hd] from the bytes that hold the codes [..., hd] and the pairs' bytes [..., 4 * groups]."""
    if c["bits"] == 8:
        q = q.view(torch.float8_e4m3fn).float()
    else:
        q = ((q >> shift.to(torch.uint8)) & (2 ** c["bits"] - 1)).float()
    pair = pair.contiguous().view(torch.float16).float().unflatten(-1, (-1, 2))
    q = q.unflatten(-1, (-1, c["group"]))
    if c["bits"] != 8:
        q = q - pair[..., 1, None]
    return (q * pair[..., 0, None]).flatten(-2)


def _gather_plain(c, s):
    """K and V of every page of every sequence: float32 [B][positions][hkv][hd]."""
    k_part, p_part = _part_bytes(c)
    blk = s["pages"].view(-1, c["hkv"], c["page"] // 16, 2 * (k_part + p_part))[s["page_table"].long()]
    out = []
    for which, off, Dr in (("k", 0, s["D_k_rsqrt"]), ("v", k_part + p_part, s["D_v_rsqrt"])):
        at, shift, _ = s["layout"][which]
        pair = blk[..., off + k_part:off + k_part + p_part].unflatten(-1, (16, -1))
        x = _values(c, blk[..., off:off + k_part][..., at], shift, pair)
        x = x.movedim(2, 4).flatten(1, 3)  # [B][pages][blocks][16][hkv][hd]
        out.append(x if Dr is None else x * Dr)
    return out


def _row_base(c, s):
    """[T][hkv]: the first byte of the block that each row of the call is in; [T]: its token there."""
    block = 2 * sum(_part_bytes(c))
    base = (s["slot_page"] * c["hkv"])[:, None] + torch.arange(c["hkv"], device=s["slot_page"].device)
    return (base * (c["page"] // 16) + (s["slot_in"] // 16)[:, None]) * block, s["slot_in"] % 16


def _read_plain(c, s):
    k_part, p_part = _part_bytes(c)
    flat, width = s["pages"].view(-1), 4 * (c["hd"] // c["group"])
    base, tok = _row_base(c, s)
    out = []
    for which, off, Dr in (("k", 0, s["D_k_rsqrt"]), ("v", k_part + p_part, s["D_v_rsqrt"])):
        at, shift, _ = s["layout"][which]
        q = flat[(base + off)[..., None] + at[tok][:, None, :]]
        pair = flat[(base + off + k_part)[..., None] + (tok * width)[:, None, None] + torch.arange(width, device=flat.device)]
        x = _values(c, q, shift, pair)
        out.append((x if Dr is None else x * Dr).to(DTYPES[c["dtype"]]))
    return out


def _attention_plain(c, s):
    K, V = _gather_plain(c, s)
    K, V = K.transpose(1, 2), V.transpose(1, 2)  # [B][hkv][L][hd]
    B, n, per, L = c["batch"], c["new"], c["hq"] // c["hkv"], K.shape[2]
    q = s["Q"].float().view(B, n, c["hkv"], per, c["hd"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    t = (q @ K.transpose(-1, -2)) * s["scale"]
    if c["cap"]:
        t = torch.tanh(t / c["cap"]) * c["cap"]
    # which positions each new token sees
    kv, dev = s["kv_len"].long(), t.device
    pos, first = torch.arange(L, device=dev), (kv - n)[:, None]
    i = torch.arange(n, device=dev)
    mask = s["tree"].view(B, n) if c["tree"] else ((1 << i) * 2 - 1).expand(B, n)
    bit = (mask[:, :, None] >> i) & 1  # [B][n][n]
    depth = bit.sum(-1) - bit.diagonal(dim1=1, dim2=2)
    in_new = (pos - first).clamp(0, n - 1)  # [B][L]
    is_new = (pos >= first) & (pos < kv[:, None])
    at = torch.where(is_new, first + depth.gather(1, in_new), pos)  # a position's distance is counted along the tree
    see = torch.where(is_new[:, None], bit.gather(2, in_new[:, None].expand(B, n, L)) > 0,
                      (pos < first)[:, None].expand(B, n, L))
    if c["window"]:
        see = see & ((first + depth)[:, :, None] - at[:, None] < c["window"])
    t = t.unflatten(2, (n, per)).masked_fill(~see[:, None, :, None], -math.inf)
    p = torch.exp(t - t.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    y = p.flatten(2, 3) @ V
    return y.unflatten(2, (n, per)).permute(0, 2, 1, 3, 4).reshape(B * n, c["hq"], c["hd"]).to(s["Q"].dtype)


# ---------------------------------------------------------------- the state
def _rows(g, shape, dtype, outliers):
    """Rows as a projection gives them: N(0, 1), some channels of K much larger in every token."""
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:
        big = torch.rand(shape[-2:], generator=g, device="cuda") < 0.02
        x = torch.where(big, x * 6.0, x)
    return x.to(dtype)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[c["dtype"]]
    n, kv = _lens(c)
    B, T, ps = c["batch"], sum(n), c["page"]
    need = [-(-k // ps) for k in kv]
    P = sum(need) + 3  # a few pages belong to nobody
    perm = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.zeros((B, max(need)), dtype=torch.int32)
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor(need))
    within = torch.cat([torch.arange(k) for k in need])
    table = table.cuda()
    table[owner.cuda(), within.cuda()] = perm[:sum(need)]
    s = {"case": c, "page_table": table, "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"),
         "cu_new": torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda(), "rows": T,
         "max_new": max(n), "D_k": None, "D_v": None, "D_k_rsqrt": None, "D_v_rsqrt": None, "tree": None,
         "layout": _layout(c, "cuda")}
    # where each row of the call is in the cache
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(n)).cuda()
    pos = torch.cat([torch.arange(k - m, k) for m, k in zip(n, kv)]).cuda()
    s["slot_page"], s["slot_in"] = table.long()[seq, pos // ps], pos % ps
    if c["stat"]:  # (||x||_2 + lambda)^(1/2) of each channel over some earlier tokens
        for w in "kv":
            D = (_rows(g, (64, c["hkv"], c["hd"]), torch.float32, w == "k").norm(dim=0) + 1e-3).sqrt()
            s["D_" + w], s["D_%s_rsqrt" % w] = D, D.rsqrt()
    k_part, p_part = _part_bytes(c)
    shape = (P, c["hkv"] * (ps // 16) * 2 * (k_part + p_part))
    if c["op"] == "write":
        s["pages"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        s["K"] = _rows(g, (T, c["hkv"], c["hd"]), dtype, True)
        s["V"] = _rows(g, (T, c["hkv"], c["hd"]), dtype, False)
        return s
    s["pages"] = torch.empty(shape, dtype=torch.uint8, device="cuda")
    some = max(1, 16_000_000 // (ps * c["hkv"] * c["hd"]))
    for a in range(0, P, some):  # the cache's contents: rows quantised as a write does it
        m = min(some, P - a)
        out = s["pages"][a:a + m].view(m, c["hkv"], ps // 16, 2 * (k_part + p_part))
        for w, off in (("k", 0), ("v", k_part + p_part)):
            x = _rows(g, (m * (ps // 16) * 16, c["hkv"], c["hd"]), dtype, w == "k")
            q, sc, z = _quantise(c, x, s["D_" + w])
            at, _, order = s["layout"][w]
            codes = torch.empty((m, ps // 16, c["hkv"], k_part), dtype=torch.uint8, device="cuda")
            codes[..., at[:, order[:, 0]]] = _code_bytes(c, q, order).view(m, ps // 16, 16, c["hkv"], -1).transpose(2, 3)
            out[..., off:off + k_part] = codes.transpose(1, 2)
            pair = torch.stack((sc, z), -1).flatten(-2).view(m, ps // 16, 16, c["hkv"], -1).transpose(2, 3)
            out[..., off + k_part:off + k_part + p_part] = pair.flatten(-2).contiguous().view(torch.uint8).transpose(1, 2)
    if c["op"] == "attention":
        s["Q"] = _rows(g, (T, c["hq"], c["hd"]), dtype, False)
        s["scale"] = 1.0 / math.sqrt(c["hd"])
        if c["tree"]:  # each drafted token hangs from an earlier one of its sequence, or from the context
            m = c["new"]
            up = (torch.rand((B, m), generator=g, device="cuda") * (torch.arange(m, device="cuda") + 1)).long().cpu() - 1
            bits = torch.zeros((B, m), dtype=torch.int64)
            for i in range(m):
                prev = torch.where(up[:, i] >= 0, bits.gather(1, up[:, i].clamp(min=0)[:, None])[:, 0], 0)
                bits[:, i] = prev | (1 << i if i < 63 else -2 ** 63)
            s["tree"] = bits.view(-1).cuda()
    return s


# ------------------------------------------------------------------ one pass
def _handles(s):
    """The cache's and the batch's handles and the workspace, which a program keeps beside them."""
    from test_weight_quantization_ttq_b200 import ttq

    if "handles" not in s:
        c = s["case"]
        scheme = ttq.TTQ_QSCHEME_FP8_E4M3 if c["bits"] == 8 else ttq.TTQ_QSCHEME_ASYMMETRIC
        cache = ttq.KVCache(s["pages"], c["page"], c["hkv"], c["hd"], c["bits"], c["group"], scheme=scheme, D_k=s["D_k"],
                            D_v=s["D_v"], D_k_rsqrt=s["D_k_rsqrt"], D_v_rsqrt=s["D_v_rsqrt"])
        batch = ttq.KVBatch(s["page_table"], s["kv_len"], s["cu_new"], s["rows"], s["max_new"])
        s["handles"] = cache, batch, ttq.new_kv_workspace(cache, batch, c["hq"])
    return ttq, *s["handles"]


def run(state):
    s, c = state, state["case"]
    if own:
        ttq, cache, batch, ws = _handles(s)
        if c["op"] == "attention":
            return ttq.ttq_kv_attention(cache, batch, s["Q"], s["scale"], softcap=c["cap"], window=c["window"],
                                        tree=s["tree"], ws=ws)
        if c["op"] == "write":
            ttq.ttq_kv_write(cache, batch, s["K"], s["V"], ws=ws)
        return ttq.ttq_kv_read(cache, batch, dtype=DTYPES[c["dtype"]], ws=ws)
    if c["op"] == "attention":
        return _attention_plain(c, s)
    if c["op"] == "write":
        _write_plain(c, s)
    return _read_plain(c, s)


# ------------------------------------------------- from the definition, in 64 bits
def _exact_rows(c, x, D):
    """What a row stands for after the quantiser, x [T][hkv][hd]."""
    h = torch.ones((), device=x.device) if D is None else torch.from_numpy(np.sqrt(D.cpu().numpy())).to(x.device)
    # x sqrt(D) and 1 / step are binary32 values by the quantiser's definition: it breaks ties by them
    y = (x.float() * h).double().reshape(*x.shape[:-1], -1, c["group"])
    if c["bits"] == 8:
        step = (y.abs().max(-1, keepdim=True).values / 448).clamp_min(2.0 ** -14)
    else:
        lo = torch.minimum(y.min(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=y.device))
        hi = torch.maximum(y.max(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=y.device))
        step = ((hi - lo) / (2 ** c["bits"] - 1)).clamp_min(2.0 ** -14)
    ulp = torch.exp2(torch.floor(torch.log2(step)) - 10)
    step = torch.ceil(step / ulp) * ulp  # the binary16 value at or above it
    inv = (1.0 / step).float().double()
    if c["bits"] == 8:
        r = (y * inv).float().double().clamp(-448, 448)
        unit = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))) - 3)
        v = torch.round(r / unit) * unit * step
    else:
        top = 2 ** c["bits"] - 1
        z = torch.round(-lo * inv).clamp(0, top)
        v = ((torch.round(y * inv) + z).clamp(0, top) - z) * step
    return v.reshape(x.shape) / h.double()


def _exact_cache(c, s, b, length):
    """K and V of sequence b, float64 [length][hkv][hd], taken from the blocks piece by piece."""
    hd, bits, gs, hkv, ps = c["hd"], c["bits"], c["group"], c["hkv"], c["page"]
    ng, lane_bytes = hd // gs, hd * bits // 32
    piece = min(16, lane_bytes)
    blocks = -(-length // 16)
    pages = s["page_table"][b, :-(-length // ps)].long()
    raw = s["pages"][pages].reshape(len(pages), hkv, ps // 16, -1).transpose(1, 2).reshape(-1, hkv, 2, 16 * hd * bits // 8 + 64 * ng)
    raw = raw[:blocks]
    vals = []
    for which in (0, 1):
        part = raw[:, :, which]
        codes = part[..., :16 * hd * bits // 8].reshape(blocks, hkv, lane_bytes // piece, 2, 32, piece)
        lanes = codes.permute(0, 1, 3, 4, 2, 5).reshape(blocks, hkv, 2, 32, lane_bytes)  # [half][lane][byte]
        if which == 0:  # lane = (token % 8, quarter of each group)
            lanes = lanes.reshape(blocks, hkv, 16, 4, lane_bytes)
        else:  # lane = (eighth of each group, token pair); bytes = (unit, token parity, 2)
            lanes = lanes.reshape(blocks, hkv, 2, 8, 4, lane_bytes // 4, 2, 2).permute(0, 1, 2, 4, 6, 3, 5, 7)
            lanes = lanes.reshape(blocks, hkv, 16, 8, lane_bytes // 2)
        if bits == 8:
            byte = lanes.long()
            e, m = (byte >> 3) & 15, byte & 7
            q = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9) * (1.0 - 2.0 * (byte >> 7))
        else:
            q = torch.stack([(lanes.long() // 2 ** (bits * i)) % 2 ** bits for i in range(8 // bits)], -1).flatten(-2).double()
        if which == 0 and bits < 8:  # a word's even channels come before its odd ones
            q = q.unflatten(-1, (-1, 2, 16 // bits)).transpose(-1, -2).flatten(-3)
        q = q.reshape(blocks, hkv, 16, q.shape[-2], ng, -1).transpose(3, 4).reshape(blocks, hkv, 16, ng, gs)
        sz = part[..., 16 * hd * bits // 8:].contiguous().view(torch.float16).double().reshape(blocks, hkv, 16, ng, 2)
        v = (q - sz[..., 1:]) * sz[..., :1]
        v = v.reshape(blocks, hkv, 16, hd).transpose(1, 2).reshape(-1, hkv, hd)[:length]
        Dr = s["D_v_rsqrt" if which else "D_k_rsqrt"]
        vals.append(v if Dr is None else v * Dr.double())
    return vals


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    n, kv = _lens(c)
    if c["op"] == "write":
        return [_exact_rows(c, s["K"], s["D_k"]), _exact_rows(c, s["V"], s["D_v"])]
    if c["op"] == "read":
        both = [_exact_cache(c, s, b, k) for b, k in enumerate(kv)]
        return [torch.cat([x[w] for x in both]) for w in (0, 1)]
    out, per = [], c["hq"] // c["hkv"]
    for b in range(c["batch"]):
        K, V = _exact_cache(c, s, b, kv[b])
        past = kv[b] - n[b]
        masks = s["tree"][b * n[b]:(b + 1) * n[b]].tolist() if c["tree"] else [2 ** (i + 1) - 1 for i in range(n[b])]
        sees = [[k for k in range(n[b]) if (m >> k) & 1] for m in masks]
        where = [past + len([k for k in x if k != i]) for i, x in enumerate(sees)]
        for i in range(n[b]):
            ok = torch.zeros(kv[b], dtype=torch.bool)
            ok[max(0, where[i] - c["window"] + 1) if c["window"] else 0:past] = True
            for k in sees[i]:
                ok[past + k] = not c["window"] or where[i] - where[k] < c["window"]
            idx = ok.nonzero()[:, 0].to(K.device)
            q = s["Q"][b * n[b] + i].double().reshape(c["hkv"], per, c["hd"])
            t = torch.einsum("hpd,lhd->hpl", q, K[idx]) * s["scale"]
            if c["cap"]:
                t = c["cap"] * torch.tanh(t / c["cap"])
            out.append(torch.einsum("hpl,lhd->hpd", torch.softmax(t, -1), V[idx]).reshape(c["hq"], c["hd"]))
    return torch.stack(out)
