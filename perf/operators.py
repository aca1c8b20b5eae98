"""Serving operators next to the block-sparse prefill: what is measured of them.

Five operators of one path: queries and keys are normed and rotated
(rope_qk_norm), the prompt's layers with a sliding window attend
(swa_prefill), requests get pages and slots (kv4_extend), keys and values go to
a cache of 4-bit values and come back from it (kv4_append, kv4_load), and new
tokens attend to that cache (kv4_attend).

Every case runs in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's calls on the same inputs.

The 4-bit cache: a key or value of one token and head is 128 dims in 8 groups
of 16; a group holds e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their
negatives) and one e4m3 scale, amax / 6 rounded to nearest.  A page of one KV
head is page_size / 16 sub-blocks of 16 tokens, 2304 bytes each: 1024 bytes of
key codes, 1024 of value codes, 128 of key scales, 128 of value scales.
"""

import math

import torch

own = False

D = 128
GROUP = 16
SUB = 2304  # bytes of a sub-block: 16 tokens of one KV head, keys and values
DEV = "cuda"


# --------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoding step of 64 requests: only latency counts
        dict(name="rope_norm_decode", op="rope", B=64, L=1, Hq=32, Hkv=4, style=0),
        # a prompt's queries and keys out of a packed projection
        dict(name="rope_norm_prompt", op="rope", B=1, L=16384, Hq=32, Hkv=4, style=0),
        # a layer with a wide window over a long prompt
        dict(name="swa_prompt_wide", op="swa", B=1, L=16384, off=0, Hq=32, Hkv=4, window=4096, sinks=4),
        # a layer with a narrow window over a long prompt: bound by memory
        dict(name="swa_prompt_narrow", op="swa", B=1, L=65536, off=0, Hq=32, Hkv=4, window=128, sinks=4),
        # the user's question after the retrieved passages, an odd length
        dict(name="swa_question", op="swa", B=2, L=509, off=8011, Hq=32, Hkv=8, window=1024, sinks=16),
        # new tokens of a decoding step into the cache, and back
        dict(name="cache_decode", op="append", B=64, L=1, Hkv=4, page=64),
        # a prompt's keys and values into the cache, and back for another prompt
        dict(name="cache_prompt", op="append", B=1, L=16384, Hkv=4, page=64),
        # one request of middle length: only latency counts
        dict(name="attend_one", op="attend", B=1, Lq=1, longest=2048, Hq=32, Hkv=4, page=64, window=0, sinks=0),
        # a full batch of requests of unequal lengths
        dict(name="attend_batch", op="attend", B=64, Lq=1, longest=16384, Hq=32, Hkv=4, page=64, window=0, sinks=0),
        # four drafted tokens checked at once against long prompts
        dict(name="attend_long_draft", op="attend", B=4, Lq=4, longest=131072, Hq=32, Hkv=4, page=64, window=0, sinks=0),
        # pages and slots of one decoding step
        dict(name="pages_decode", op="extend", B=64, new=1, longest=16384, page=64),
        # pages and slots of a batch of new prompts
        dict(name="pages_prompts", op="extend", B=64, new=4096, longest=4096, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "swa", "append", "attend", "attend", "extend"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        b = _log(rng, 1, 64)
        return dict(op=op, B=b, L=_log(rng, 1, max(1, 8192 // b)), Hq=hkv * g, Hkv=hkv, style=rng.choice([0, 1]))
    if op == "swa":
        b = rng.choice([1, 1, 2, 3])
        n = _log(rng, 1, 8192 // b)
        return dict(op=op, B=b, L=n, off=rng.choice([0, 0, _log(rng, 1, 16384)]), Hq=hkv * g, Hkv=hkv,
                    window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 64]))
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        b = _log(rng, 1, 128)
        return dict(op=op, B=b, L=_log(rng, 1, max(1, 16384 // b)), Hkv=hkv, page=page)
    if op == "attend":
        b = _log(rng, 1, 128)
        return dict(op=op, B=b, Lq=rng.choice([1, 1, 1, 2, 4, 7]), longest=_log(rng, 8, max(8, 262144 // (b * hkv))),
                    Hq=hkv * g, Hkv=hkv, page=page, window=rng.choice([0, 0, _log(rng, 16, 8192)]),
                    sinks=rng.choice([0, 4, 16]))
    b = _log(rng, 1, 256)
    new = _log(rng, 1, 2048)
    return dict(op=op, B=b, new=new, longest=new + rng.choice([0, _log(rng, 1, 16384)]), page=page)


# --------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _tables(g, lens, longest, page):
    """Block table [B, max pages] over a shuffled pool just large enough for the longest lengths, and its pages."""
    B, width = lens.numel(), -(-longest // page)
    pool = B * width
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    need = (lens + page - 1) // page
    at = torch.arange(width, device=DEV, dtype=torch.int32)
    first = torch.cumsum(need, 0) - need
    idx = (first[:, None] + at[None, :]).clamp(max=pool - 1)
    return torch.where(at[None, :] < need[:, None], order[idx.long()], -1).to(torch.int32).contiguous(), pool


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    if op == "rope":
        qkv = _randn(g, c["B"], c["L"], c["Hq"] + 2 * c["Hkv"], D)
        start = _ints(g, 0, 100000, c["B"])
        pos = (start[:, None] + torch.arange(c["L"], device=DEV, dtype=torch.int32)[None, :]).contiguous()
        return dict(case=c, Q=qkv[:, :, :c["Hq"]], K=qkv[:, :, c["Hq"]:c["Hq"] + c["Hkv"]], pos=pos,
                    wq=(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16),
                    wk=(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16))
    if op == "swa":
        Lk = c["off"] + c["L"]
        return dict(case=c, Q=_randn(g, c["B"], c["L"], c["Hq"], D), K=_randn(g, c["B"], Lk, c["Hkv"], D),
                    V=_randn(g, c["B"], Lk, c["Hkv"], D))
    if op == "append":
        B, L, H, P = c["B"], c["L"], c["Hkv"], c["page"]
        width = -(-L // P) + 1
        pool = B * width
        # one page more than the pool: no request's, it takes the padding of the plain form
        data = torch.zeros(pool + 1, H, P // 16 * SUB, dtype=torch.uint8, device=DEV)
        start = _ints(g, 0, P - 1, B)
        lens = start + (_ints(g, max(1, L // 2), L, B) if B > 1 else L)
        table, _ = _tables(g, torch.full_like(lens, width * P), width * P, P)
        t = start[:, None] + torch.arange(L, device=DEV, dtype=torch.int32)[None, :]
        slots = torch.gather(table, 1, (t // P).long()) * P + t % P
        slots = torch.where(t < lens[:, None], slots, -1).to(torch.int32).contiguous()
        spread = torch.exp(0.5 * torch.randn(H, D, generator=g, device=DEV))  # channels of unequal size
        K = (torch.randn(B, L, H, D, generator=g, device=DEV) * spread).to(torch.bfloat16)
        return dict(case=c, K=K, V=_randn(g, B, L, H, D), slots=slots, data=data, spare=pool * P)
    if op == "attend":
        B, H, P, longest = c["B"], c["Hkv"], c["page"], c["longest"]
        lens = _ints(g, max(1, longest // 2), longest, B)
        lens[0] = longest
        table, pool = _tables(g, lens, longest, P)
        kv = [_quantise(torch.randn(pool * H, P, D, generator=g, device=DEV)) for _ in range(2)]
        data = _page_bytes(*kv[0], *kv[1]).view(pool, H, P // 16 * SUB)
        return dict(case=c, Q=_randn(g, B, c["Lq"], c["Hq"], D), data=data, table=table, lens=lens)
    if op == "extend":
        B, new, P = c["B"], c["new"], c["page"]
        add = _ints(g, max(1, new // 2), new, B)
        old = torch.where(_ints(g, 0, 3, B) > 0, _ints(g, 0, c["longest"] - new, B), 0).to(torch.int32)
        width = -(-c["longest"] // P)
        table, pool = _tables(g, old, c["longest"], P)
        used = ((old + P - 1) // P).sum(dtype=torch.int32).view(1)
        # the free list, in the pool's shuffled order; its first `used` pages are taken
        free = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        return dict(case=c, table=table.view(B, width), old=old, new=(old + add).to(torch.int32), free=free, head=used)
    raise ValueError(op)


# --------------------------------------------------------------------------- the 4-bit format, plainly

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """fp32 values [..., 128] -> codes [..., 128] (0..15) and e4m3 scale bits [..., 8]; to nearest, ties to the even code."""
    x = x.reshape(*x.shape[:-1], D // GROUP, GROUP)
    amax = x.abs().amax(-1)
    s8 = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(torch.float32)[..., None]
    a = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.where((x < 0) & (s > 0), 8, 0).to(torch.uint8)
    return code.reshape(*x.shape[:-2], D), s8.view(torch.uint8)


def _values(code, scale):
    """codes [..., 128] and scale bits [..., 8] -> fp32 values."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device, dtype=torch.float32)
    v = level[code.long()].reshape(*code.shape[:-1], D // GROUP, GROUP)
    return (v * scale.view(torch.float8_e4m3fn).to(torch.float32)[..., None]).reshape(code.shape)


def _page_bytes(kc, ks, vc, vs):
    """Codes [N, P, 128] and scales [N, P, 8] of keys and values -> page bytes [N, P / 16 * 2304].
    Key dim 16 s + 8 e + 2 j + n of token 8 h + r; value dim 16 s + 8 e + r of token 8 h + 2 j + i."""
    N, P = kc.shape[:2]
    n = P // 16
    k = kc.view(N, n, 2, 8, 8, 2, 4, 2).permute(0, 1, 2, 3, 6, 4, 5, 7)
    v = vc.view(N, n, 2, 4, 2, 8, 2, 8).permute(0, 1, 2, 7, 3, 4, 5, 6)
    k = (k[..., 0] | (k[..., 1] << 4)).reshape(N, n, 1024)
    v = (v[..., 0] | (v[..., 1] << 4)).reshape(N, n, 1024)
    vs = vs.view(N, n, 8, 2, 8).permute(0, 1, 2, 4, 3).reshape(N, n, 128)
    return torch.cat([k, v, ks.view(N, n, 128), vs], -1).reshape(N, n * SUB)


def _page_values(data):
    """Page bytes [N, P / 16 * 2304] -> keys and values [N, P, 128] in fp32."""
    N, n = data.shape[0], data.shape[1] // SUB
    data = data.view(N, n, SUB)
    k, v = data[..., :1024], data[..., 1024:2048]
    k = torch.stack([k & 15, k >> 4], -1).view(N, n, 2, 8, 4, 8, 2, 2).permute(0, 1, 2, 3, 5, 6, 4, 7)
    v = torch.stack([v & 15, v >> 4], -1).view(N, n, 2, 8, 4, 2, 8, 2).permute(0, 1, 2, 4, 5, 6, 7, 3)
    vs = data[..., 2176:].reshape(N, n, 8, 8, 2).permute(0, 1, 2, 4, 3).reshape(N, n * 16, 8)
    ks = data[..., 2048:2176].reshape(N, n * 16, 8)
    return _values(k.reshape(N, n * 16, D), ks), _values(v.reshape(N, n * 16, D), vs)


def _token_bytes(slot, H, P):
    """Where the bytes of tokens [T] lie in the flat cache, for each of H heads: key codes [T, H, 64], value codes
    [T, H, 64], key scales [T, H, 8], value scales [T, H, 8], as _page_bytes lays them out."""
    a = lambda n: torch.arange(n, device=slot.device)  # noqa: E731
    slot = slot.long()
    page, t = slot // P, slot % P
    base = ((page[:, None] * H + a(H)[None, :]) * (P // 16) + (t // 16)[:, None])[..., None] * SUB
    t = (t % 16)[:, None, None]
    h, r, j, i = t // 8, t % 8, t % 8 // 2, t % 2
    kc = base + h * 512 + r * 64 + a(64)
    vc = base + 1024 + h * 512 + (a(64) // 8) * 64 + j * 16 + i * 8 + a(64) % 8
    ks = base + 2048 + t * 8 + a(8)
    vs = base + 2176 + (t // 2) * 16 + a(8) * 2 + i
    return kc, vc, ks, vs


# --------------------------------------------------------------------------- the plain forms


def _rope_plain(st):
    style, half = st["case"]["style"], D // 2
    inv = 500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) * 2 / D)
    ang = st["pos"].double()[..., None] * inv
    cos, sin = torch.cos(ang).float()[:, :, None, :], torch.sin(ang).float()[:, :, None, :]

    def one(x, w):
        x = x.float()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (x[..., :half], x[..., half:]) if style == 0 else (x[..., 0::2], x[..., 1::2])
        lo, hi = a * cos - b * sin, a * sin + b * cos
        y = torch.cat([lo, hi], -1) if style == 0 else torch.stack([lo, hi], -1).flatten(-2)
        return y.to(torch.bfloat16)

    return one(st["Q"], st["wq"]), one(st["K"], st["wk"])


def _softmax_rows(s, v_of):
    """Scores s (changed in place) -> (sum of weights times values, ln sum exp); a row with nothing visible gives 0, -inf."""
    m = s.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(safe).exp_()
    l = p.sum(-1, keepdim=True)
    o = v_of(p) / torch.where(l > 0, l, 1.0)
    return o, (torch.log(l) + safe).squeeze(-1)


def _swa_plain(st):
    c = st["case"]
    B, L, off, Hq, H = c["B"], c["L"], c["off"], c["Hq"], c["Hkv"]
    W, S, G = min(c["window"], c["off"] + c["L"]), min(c["sinks"], c["off"] + c["L"]), c["Hq"] // c["Hkv"]
    bq = min(L, max(W, 64))  # queries of a block; a block sees the W - 1 keys before it and its own
    n = -(-L // bq)
    first = off - (W - 1)  # key position of the first block's first column

    def band(x):
        x = x[:, max(0, first):].float()
        pad = torch.zeros(B, max(0, -first), H, D, device=DEV)
        tail = torch.zeros(B, n * bq - L, H, D, device=DEV)
        return torch.cat([pad, x, tail], 1).unfold(1, bq + W - 1, bq)  # [B, n, H, D, keys]

    q = torch.cat([st["Q"].float(), torch.zeros(B, n * bq - L, Hq, D, device=DEV)], 1)
    q = q.view(B, n, bq, H, G, D).permute(0, 1, 3, 4, 2, 5).reshape(B, n, H, G * bq, D) / math.sqrt(D)
    kb, vb = band(st["K"]), band(st["V"])
    s = torch.empty(B, n, H, G * bq, S + bq + W - 1, device=DEV)
    torch.matmul(q, kb, out=s[..., S:]) if S == 0 else s[..., S:].copy_(torch.matmul(q, kb))
    qp = torch.arange(bq, device=DEV)[:, None] + W - 1  # a query's own column in its block's band
    kc = torch.arange(bq + W - 1, device=DEV)[None, :]
    blocks = (torch.arange(n, device=DEV) * bq + first)[:, None, None]
    hide = (kc > qp) | (kc <= qp - W) | (blocks + kc < S) | (blocks + kc < 0)  # [n, bq, keys]
    s.view(B, n, H, G, bq, -1)[..., S:].masked_fill_(hide[None, :, None, None], -math.inf)
    if S:
        ks, vs = (st[k][:, :S].float().permute(0, 2, 1, 3)[:, None] for k in ("K", "V"))  # [B, 1, H, S, D]
        s[..., :S] = torch.matmul(q, ks.transpose(-1, -2))
        late = torch.arange(S, device=DEV)[None, None, :] > blocks + qp
        s.view(B, n, H, G, bq, -1)[..., :S].masked_fill_(late[None, :, None, None], -math.inf)

    def values(p):
        o = torch.matmul(p[..., S:], vb.transpose(-1, -2))
        return o + torch.matmul(p[..., :S], vs) if S else o

    o, lse = _softmax_rows(s, values)
    o = o.view(B, n, H, G, bq, D).permute(0, 1, 4, 2, 3, 5).reshape(B, n * bq, Hq, D)[:, :L]
    lse = lse.view(B, n, H, G, bq).permute(0, 2, 3, 1, 4).reshape(B, Hq, n * bq)[..., :L]
    return o.to(torch.bfloat16), lse.contiguous()


def _append_plain(st):
    c = st["case"]
    B, L, H, P = c["B"], c["L"], c["Hkv"], c["page"]
    slots, flat = st["slots"].view(-1), st["data"].view(-1)
    kc, ks = _quantise(st["K"].float().view(B * L, H, D))
    vc, vs = _quantise(st["V"].float().view(B * L, H, D))
    where = _token_bytes(torch.where(slots >= 0, slots, st["spare"]), H, P)
    k = kc.view(B * L, H, 8, 2, 4, 2).permute(0, 1, 4, 2, 3, 5)
    v = vc.view(B * L, H, 8, 2, 8).permute(0, 1, 4, 2, 3)
    parts = ((k[..., 0] | (k[..., 1] << 4)).reshape(B * L, H, 64), (v[..., 0] | (v[..., 1] << 4)).reshape(B * L, H, 64),
             ks, vs)
    flat[torch.cat(where, -1)] = torch.cat(parts, -1)
    # and back
    got = flat[torch.cat(where, -1)]
    k, v = got[..., :64], got[..., 64:128]
    k = torch.stack([k & 15, k >> 4], -1).view(B * L, H, 4, 8, 2, 2).permute(0, 1, 3, 4, 2, 5).reshape(B * L, H, D)
    v = torch.stack([v & 15, v >> 4], -1).view(B * L, H, 8, 8, 2).permute(0, 1, 3, 4, 2).reshape(B * L, H, D)
    there = (slots >= 0)[:, None, None]
    return tuple(torch.where(there, _values(x, s.contiguous()), 0.0).to(torch.bfloat16).view(B, L, H, D)
                 for x, s in ((k, got[..., 128:136]), (v, got[..., 136:])))


def _attend_plain(st):
    c = st["case"]
    B, Lq, Hq, H, P, W, S = (c[k] for k in ("B", "Lq", "Hq", "Hkv", "page", "window", "sinks"))
    pages, width = st["data"].shape[0], st["table"].shape[1]
    k, v = _page_values(st["data"].view(pages * H, -1))
    at = st["table"].clamp(min=0).long()
    k, v = (x.view(pages, H, P, D)[at].permute(0, 2, 1, 3, 4).reshape(B, H, width * P, D) for x in (k, v))
    q = st["Q"].float().view(B, Lq, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D) / math.sqrt(D)
    s = torch.matmul(q, k.transpose(-1, -2)).view(B, H, Hq // H, Lq, -1)
    qp = (st["lens"][:, None] - Lq + torch.arange(Lq, device=DEV, dtype=torch.int32)[None, :])[:, :, None]
    kp = torch.arange(width * P, device=DEV, dtype=torch.int32)[None, None, :]
    see = kp <= qp
    if W:
        see &= (kp > qp - W) | (kp < S)
    s.masked_fill_(~see[:, None, None], -math.inf)
    o, lse = _softmax_rows(s.view(B, H, -1, width * P), lambda p: torch.matmul(p, v))
    o = o.view(B, H, Hq // H, Lq, D).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D)
    return o.to(torch.bfloat16), lse.view(B, Hq, Lq)


def _extend_plain(st):
    c = st["case"]
    P, table, old, new, free = c["page"], st["table"], st["old"], st["new"], st["free"]
    had, has = (old + P - 1) // P, (new + P - 1) // P
    need = has - had
    first = st["head"] + torch.cumsum(need, 0, dtype=torch.int32) - need
    at = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)[None, :]
    idx = (first[:, None] + at - had[:, None]).clamp(0, free.numel() - 1).long()
    table.copy_(torch.where((at >= had[:, None]) & (at < has[:, None]), free[idx], table))
    pos = old[:, None] + torch.arange(c["new"], device=DEV, dtype=torch.int32)[None, :]
    live = pos < new[:, None]
    page = torch.gather(table, 1, (pos // P).clamp(max=table.shape[1] - 1).long())
    slots = torch.where(live, page * P + pos % P, -1).to(torch.int32)
    pos = torch.where(live, pos, -1).to(torch.int32)
    return table, slots, pos, (st["head"] + need.sum(dtype=torch.int32)).to(torch.int32)


# --------------------------------------------------------------------------- one pass


def _run_own(st):
    import block_sparse_long_rbs_b200 as rbs

    c, op = st["case"], st["case"]["op"]
    if op == "rope":
        return rbs.rope_qk_norm(st["Q"], st["K"], st["wq"], st["wk"], st["pos"], 500000.0, rope_style=c["style"])
    if op == "swa":
        return rbs.swa_prefill(st["Q"], st["K"], st["V"], c["window"], c["sinks"], q_offset=c["off"], return_lse=True)
    if op == "append":
        cache = rbs.KV4Cache(st["data"], c["page"])
        rbs.kv4_append(cache, st["K"], st["V"], st["slots"])
        return rbs.kv4_load(cache, st["slots"])
    if op == "attend":
        cache = rbs.KV4Cache(st["data"], c["page"])
        return rbs.kv4_attend(st["Q"], cache, st["table"], st["lens"], window=c["window"], sinks=c["sinks"],
                              return_lse=True)
    slots, pos, head = rbs.kv4_extend(st["table"], st["old"], st["new"], st["free"], st["head"], c["new"], c["page"])
    return st["table"], slots, pos, head


def run(state):
    if own:
        return _run_own(state)
    plain = dict(rope=_rope_plain, swa=_swa_plain, append=_append_plain, attend=_attend_plain, extend=_extend_plain)
    return plain[state["case"]["op"]](state)


# --------------------------------------------------------------------------- work


def _seen(q, W, S):
    """Keys that the query at position q >= 0 sees."""
    if not W or W > q:
        return q + 1
    return W + min(S, q + 1 - W)


def work(case):
    c, op = case, case["op"]
    if op == "rope":
        n = c["B"] * c["L"] * (c["Hq"] + c["Hkv"]) * D
        return {"bytes": 4 * n + 4 * c["B"] * c["L"] + 4 * D, "flops": 8 * n}
    if op == "swa":
        pairs = sum(_seen(c["off"] + t, c["window"], c["sinks"]) for t in range(c["L"]))
        Lk = c["off"] + c["L"]
        lo = max(0, c["off"] - c["window"] + 1)
        keys = Lk - lo + min(lo, c["sinks"])
        return {"bytes": c["B"] * (c["L"] * c["Hq"] * (4 * D + 4) + keys * c["Hkv"] * 4 * D),
                "flops": 4 * D * c["B"] * c["Hq"] * pairs}
    if op == "append":
        n = c["B"] * c["L"] * c["Hkv"]
        return {"bytes": n * (2 * 2 * 2 * D + 2 * 144) + 8 * c["B"] * c["L"], "flops": 2 * n * 3 * D}
    if op == "attend":
        # lengths are drawn from the longest's upper half; the first is the longest
        B, Lq, W, S = c["B"], c["Lq"], c["window"], c["sinks"]
        mean = (c["longest"] + (B - 1) * 0.75 * c["longest"]) / B
        held = min(mean, W + Lq - 1 + S) if W else mean
        return {"bytes": B * (held * c["Hkv"] * 144 + Lq * c["Hq"] * (4 * D + 4)),
                "flops": 4 * D * B * Lq * c["Hq"] * held}
    B, new = c["B"], c["new"]
    pages = B * (0.75 * new / c["page"] + 1)
    return {"bytes": B * new * 8 + pages * 8 + B * 8, "flops": B * new * 4}


# --------------------------------------------------------------------------- the definitions, in 64 bits


def _rope_exact(st):
    f = torch.tensor([500000.0 ** (-2 * m / D) for m in range(D // 2)], dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), st["pos"].double()[..., None] * f)[:, :, None]
    out = []
    for x, w in ((st["Q"], st["wq"]), (st["K"], st["wk"])):
        x = x.double()
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
        if st["case"]["style"] == 0:
            z = torch.complex(x[..., :64], x[..., 64:]) * turn
            out.append(torch.cat([z.real, z.imag], -1))
        else:
            z = torch.view_as_complex(x.reshape(*x.shape[:-1], 64, 2)) * turn
            out.append(torch.view_as_real(z).reshape(x.shape))
    return tuple(out)


def _attention_exact(q, k, v, qp, kp, W, S):
    """q [R, n, D], k, v [m, D] in fp64, positions qp [n], kp [m] -> outputs [R, n, D] and ln sum exp [R, n]."""
    see = kp[None, :] <= qp[:, None]
    if W:
        see = see & ((qp[:, None] - kp[None, :] < W) | (kp[None, :] < S))
    s = torch.einsum("rnd,md->rnm", q, k) * D ** -0.5
    s = torch.where(see[None], s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    w = torch.where(see[None], torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None]), 0.0)
    return torch.einsum("rnm,md->rnd", w, v), lse


def _swa_exact(st):
    c = st["case"]
    B, L, off, Hq, H, W, S = (c[k] for k in ("B", "L", "off", "Hq", "Hkv", "window", "sinks"))
    G, step = Hq // H, 1024
    out = torch.empty(B, L, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, L, dtype=torch.float64, device=DEV)
    for t in range(0, L, step):
        e = min(L, t + step)
        lo = max(0, off + t - W + 1)
        kp = torch.cat([torch.arange(min(S, lo), device=DEV), torch.arange(lo, off + e, device=DEV)])
        qp = torch.arange(off + t, off + e, device=DEV)
        for b in range(B):
            for h in range(H):
                q = st["Q"][b, t:e, h * G:(h + 1) * G].double().transpose(0, 1)
                o, z = _attention_exact(q, st["K"][b, kp, h].double(), st["V"][b, kp, h].double(), qp, kp, W, S)
                out[b, t:e, h * G:(h + 1) * G] = o.transpose(0, 1)
                lse[b, h * G:(h + 1) * G, t:e] = z
    return out, lse


def _round_trip_exact(x):
    """What the 4-bit format holds of x, by looking for the nearest level in 64 bits (the even code of two equally near)."""
    x = x.double().unflatten(-1, (D // GROUP, GROUP))
    e4m3 = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    scale = e4m3[_nearest((x.abs().amax(-1) / 6).reshape(-1), e4m3)].view(x.shape[:-1])
    level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    ratio = (x.abs() / torch.where(scale > 0, scale, 1.0)[..., None]).reshape(-1)
    mag = level[_nearest(ratio, level)].view(x.shape) * scale[..., None]
    return torch.where(x < 0, -mag, mag).flatten(-2)


def _nearest(a, grid):
    up = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    d0, d1 = a - grid[up - 1], grid[up] - a
    return torch.where((d0 < d1) | ((d0 == d1) & (up % 2 == 1)), up - 1, up)


def _append_exact(st):
    there = (st["slots"] >= 0)[:, :, None, None]
    return tuple(torch.where(there, _round_trip_exact(st[k]), 0.0) for k in ("K", "V"))


def _attend_exact(st):
    c = st["case"]
    B, Lq, Hq, H, P = (c[k] for k in ("B", "Lq", "Hq", "Hkv", "page"))
    G = Hq // H
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=DEV)
    out = torch.empty(B, Lq, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, Lq, dtype=torch.float64, device=DEV)
    flat = st["data"].view(-1)
    for b in range(B):
        n = int(st["lens"][b])
        kp = torch.arange(n, device=DEV)
        slot = st["table"][b].long()[kp // P] * P + kp % P
        kc, vc, ks, vs = _token_bytes(slot, H, P)
        k, v = flat[kc], flat[vc]
        k = level[torch.stack([k & 15, k >> 4], -1).long()].view(n, H, 4, 8, 2, 2).permute(0, 1, 3, 4, 2, 5).reshape(n, H, D)
        v = level[torch.stack([v & 15, v >> 4], -1).long()].view(n, H, 8, 8, 2).permute(0, 1, 3, 4, 2).reshape(n, H, D)
        k, v = (x * flat[s].view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, -1) for x, s in ((k, ks), (v, vs)))
        qp = n - Lq + torch.arange(Lq, device=DEV)
        for h in range(H):
            q = st["Q"][b, :, h * G:(h + 1) * G].double().transpose(0, 1)
            o, z = _attention_exact(q, k[:, h], v[:, h], qp, kp, c["window"], c["sinks"])
            out[b, :, h * G:(h + 1) * G] = o.transpose(0, 1)
            lse[b, h * G:(h + 1) * G] = z
    return out, lse


def exact(case, seed):
    if case["op"] == "extend":  # whole numbers
        return None
    st = prepare(case, seed)
    return dict(rope=_rope_exact, swa=_swa_exact, append=_append_exact, attend=_attend_exact)[case["op"]](st)
