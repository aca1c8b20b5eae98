"""GPU parity of the 4-bit cache with the fp64 oracle: pages and slots,
writing and reading tokens (to the byte), and attention over it."""

import numpy as np
import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from helpers import host_bits
from oracle import serving_oracle as S
from serving_helpers import FP16, check_attention, f64, ints, randn

pytestmark = pytest.mark.gpu


# ---- writing and reading tokens


def _special(rng, B, L, H):
    """Values of every size: unequal channels, zero groups, borders of the codes, sizes at and past the scales' ends."""
    x = rng.standard_normal((B, L, H, 128)) * np.exp(rng.standard_normal(128))
    x[0, 0, 0, :16] = 0
    x[0, 0, 0, 16:32] = [6, -6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]
    x[0, 0, 0, 32:48] = 1e4
    x[0, 0, 0, 48:64] = rng.standard_normal(16) * 1e-3
    x[0, 0, 0, 64:80] = rng.standard_normal(16) * 1e-6
    x[0, 0, 0, 80:96] = -0.0
    # scales on the border between two e4m3 values: amax = 6 * (s + half a step)
    for i in range(16):
        x[-1, -1, -1, 8 * i:8 * i + 8] = 6 * (1 + (2 * i + 1) / 16) * 2.0 ** (i - 8)
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("B,L,H,page,gk,gv", [(1, 1, 1, 16, 1.0, 1.0), (2, 37, 3, 48, 0.25, 4.0),
                                              (5, 9, 4, 256, 2.0 ** -20, 2.0 ** 20), (1, 130, 2, 64, 1.0, 2.0)])
def test_append_writes_the_documented_bytes_and_load_reads_them(cuda_ok, B, L, H, page, gk, gv):
    rng = np.random.default_rng(L + page)
    K, V = _special(rng, B, L, H), _special(rng, B, L, H)
    pages = -(-B * L // page) + 2
    slots = rng.permutation(pages * page)[:B * L].reshape(B, L)
    if L > 8:
        slots[-1, -3:-1] = [-1, -77]  # padding
    cache = rbs.KV4Cache.empty(pages, page, H, k_scale=gk, v_scale=gv)
    cache.data.fill_(0xA5)
    rbs.kv4_append(cache, K, V, ints(slots))
    (kc, ks), (vc, vs) = S.quantise(f64(K), gk), S.quantise(f64(V), gv)
    want = np.full(tuple(cache.data.shape), 0xA5, dtype=np.uint8)
    for b in range(B):
        for t in range(L):
            for h in range(H):
                if slots[b, t] >= 0:
                    S.write_token(want, slots[b, t], page, h, kc[b, t, h], ks[b, t, h], vc[b, t, h], vs[b, t, h])
    assert np.array_equal(cache.data.cpu().numpy(), want)
    k, v = rbs.kv4_load(cache, ints(slots))
    there = (slots >= 0)[:, :, None, None]
    assert np.array_equal(f64(k), np.where(there, S.values(kc, ks, gk), 0))
    assert np.array_equal(f64(v), np.where(there, S.values(vc, vs, gv), 0))
    assert rbs.rbs_get_device_error() == 0


def test_nan_and_infinity_take_their_group(cuda_ok):
    rng = np.random.default_rng(3)
    K, V = randn(rng, 1, 4, 1, 128), randn(rng, 1, 4, 1, 128)
    K[0, 1, 0, 20], V[0, 2, 0, 127] = float("inf"), float("nan")
    cache = rbs.KV4Cache.empty(1, 16, 1)
    slots = ints([[3, 2, 9, 8]])
    rbs.kv4_append(cache, K, V, slots)
    for x, y in zip((K, V), rbs.kv4_load(cache, slots)):
        assert np.array_equal(f64(y), S.round_trip(f64(x)), equal_nan=True)


def test_views_and_strides(cuda_ok):
    """Keys and values as views of a packed projection; outputs in another head order."""
    rng = np.random.default_rng(4)
    qkv = randn(rng, 2, 21, 10, 128)
    K, V = qkv[:, :, 6:8], qkv[:, :, 8:]
    cache = rbs.KV4Cache.empty(4, 16, 2)
    slots = ints(rng.permutation(64)[:42].reshape(2, 21))
    rbs.kv4_append(cache, K, V, slots)
    hold = torch.full((2, 2, 30, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = rbs.kv4_load(cache, slots, k_out=hold.transpose(1, 2)[:, 3:24])
    assert np.array_equal(f64(k), S.round_trip(f64(K))) and np.array_equal(f64(v), S.round_trip(f64(V)))
    assert (hold[:, :, :3] == 7).all() and (hold[:, :, 24:] == 7).all()


def test_slots_past_the_cache_are_reported_and_skipped(cuda_ok):
    rng = np.random.default_rng(5)
    K = randn(rng, 1, 3, 2, 128)
    cache = rbs.KV4Cache.empty(2, 16, 2)
    cache.data.zero_()
    rbs.rbs_get_device_error()
    bad = ints([[32, 5, (1 << 31) - 1]])
    rbs.kv4_append(cache, K, K, bad)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_SLOT
    k, _ = rbs.kv4_load(cache, bad)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_SLOT
    assert not f64(k)[0, [0, 2]].any() and np.array_equal(f64(k)[0, 1], S.round_trip(f64(K)[0, 1]))


# ---- pages and slots


def _extend_case(rng, B, page, width, max_new):
    old = rng.integers(0, width * page - max_new + 1, B) * (rng.random(B) > 0.3)
    new = old + rng.integers(0, max_new + 1, B)
    need = -(-new // page) - -(-old // page)
    had = -(-old // page)
    pages = rng.permutation(int(had.sum() + need.sum()) + 3)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :had[b]] = pages[at:at + had[b]]
        at += had[b]
    free = np.concatenate([rng.permutation(7) + 10000, pages[at:]])  # seven pages of the list are taken
    return table, old, new, free, 7


@pytest.mark.parametrize("B,page,width,max_new", [(1, 16, 1, 1), (1, 64, 700, 40000), (64, 64, 20, 1), (300, 16, 9, 33),
                                                  (1000, 48, 5, 100), (3, 256, 10, 513), (2049, 16, 3, 2)])
def test_extend(cuda_ok, B, page, width, max_new):
    rng = np.random.default_rng(B + max_new)
    table, old, new, free, head = _extend_case(rng, B, page, width, max_new)
    t = ints(table)
    args = (ints(old), ints(new), ints(free), ints([head]), max_new, page)
    want = S.extend(table, old, new, free, head, max_new, page)
    rbs.rbs_get_device_error()
    for _ in range(2):  # the same call again changes nothing
        slots, pos, out = rbs.kv4_extend(t, *args)
        for got, w in zip((t, slots, pos), want):
            assert np.array_equal(got.cpu().numpy(), w)
        assert out.item() == want[3]
    assert rbs.rbs_get_device_error() == 0


def test_extend_row_views(cuda_ok):
    rng = np.random.default_rng(1)
    table, old, new, free, head = _extend_case(rng, 5, 16, 6, 20)
    hold = torch.full((5, 11), -9, dtype=torch.int32, device="cuda")
    hold[:, :6] = ints(table)
    rbs.kv4_extend(hold[:, :6], ints(old), ints(new), ints(free), ints([head]), 20, 16)
    want = S.extend(table, old, new, free, head, 20, 16)
    assert np.array_equal(hold[:, :6].cpu().numpy(), want[0]) and (hold[:, 6:] == -9).all()


def test_extend_errors(cuda_ok):
    """A list that runs out, and lengths out of range: reported, and nothing beyond the buffers is touched."""
    rbs.rbs_get_device_error()
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    i0 = ints([0, 0, 0])
    slots, pos, head = rbs.kv4_extend(table, i0, ints([16, 40, 17]), ints([5, 6, 7]), ints([0]), 40, 16)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_PAGES
    assert table.cpu().tolist() == [[5, -1, -1, -1], [6, 7, -1, -1], [-1, -1, -1, -1]] and head.item() == 3
    s = slots.cpu().numpy()
    assert (s[0, :16] == 80 + np.arange(16)).all() and (s[1, :32] >= 0).all() and (s[1, 32:] == -1).all()
    assert (s[2] == -1).all() and pos.cpu().numpy()[2, :17].tolist() == list(range(17))
    rbs.kv4_extend(table, i0, i0, ints([5]), ints([2]), 1, 16)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_PAGES  # the count itself is past the list
    for old, new, want in (([-3, 0, 0], [1, 0, 0], [1, 0, 0]), ([9, 0, 0], [4, 0, 0], [0, 0, 0]),
                           ([0, 0, 0], [0, 0, 9], [0, 0, 8]), ([62, 0, 0], [70, 1, 0], [2, 1, 0])):
        slots, _, _ = rbs.kv4_extend(table.zero_(), ints(old), ints(new), ints(np.arange(9)), ints([0]), 8, 16)
        assert rbs.rbs_get_device_error() == rbs.DEVERR_LENGTH
        assert (slots >= 0).sum(1).tolist() == want


def test_extend_entries_that_are_no_pages(cuda_ok):
    """An entry whose slots would pass 2^31 - 1 gives none, in the table as held and in the free list."""
    top = (2 ** 31 - 1 - 16) // 16
    table = ints([[top + 1, -1], [2 ** 31 - 1, -1], [top, -1], [5, -1]])
    slots, pos, _ = rbs.kv4_extend(table, ints([3, 3, 3, 16]), ints([4, 4, 4, 17]), ints([2 ** 31 - 1]), ints([0]), 1, 16)
    assert slots.cpu().tolist() == [[-1], [-1], [16 * top + 3], [-1]] and pos.cpu().tolist() == [[3], [3], [3], [16]]


# ---- attention


class Held:
    """Requests of the given lengths in a cache whose other bytes are 0xff (NaN scales), and what it holds in fp64."""

    def __init__(self, rng, lens, H, page, width=None, gk=1.0, gv=1.0, k_scale=1.0):
        self.lens, B = np.asarray(lens), len(lens)
        need = -(-self.lens // page)
        self.width = max(1, int(need.max())) if width is None else width
        total = int(need.sum())
        order = rng.permutation(total + 2)
        self.table = np.full((B, self.width), 1 << 30)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.cache = rbs.KV4Cache.empty(total + 2, page, H, k_scale=gk, v_scale=gv)
        self.cache.data.fill_(0xFF)
        n = max(1, int(self.lens.max()))
        K, V = randn(rng, B, n, H, 128, scale=k_scale), randn(rng, B, n, H, 128)
        t = np.arange(n)
        slots = np.where(t < self.lens[:, None],
                         self.table[np.arange(B)[:, None], np.minimum(t // page, self.width - 1)] * page + t % page, -1)
        self.slots = slots
        rbs.kv4_append(self.cache, K, V, ints(slots))
        self.k, self.v = S.round_trip(f64(K), gk), S.round_trip(f64(V), gv)

    def expect(self, Q, starts=None, window=0, sinks=0, scale=None):
        Q = f64(Q)
        B, Lq, Hq, D = Q.shape
        G = Hq // self.k.shape[2]
        scale = D ** -0.5 if scale is None else scale
        out, a = np.zeros_like(Q), np.zeros_like(Q)
        lse, z = np.zeros((B, Hq, Lq)), np.zeros((B, Hq, Lq))
        for b in range(B):
            n = int(self.lens[b])
            qp = (n - Lq if starts is None else starts[b]) + np.arange(Lq)
            see = S.visible(qp, np.arange(n), window, sinks) & ((qp >= 0) & (qp < n))[:, None]
            for h in range(Hq):
                o, e, aa, zz = S.attend(Q[b, :, h], self.k[b, :n, h // G], self.v[b, :n, h // G], see, scale)
                out[b, :, h], lse[b, h], a[b, :, h], z[b, h] = o, e, aa, zz
        return out, lse, a, z


def _check(o, lse, held, Q, what="", **kw):
    """A weight p (relative to the running maximum; the row sum is at least 1) is held as fp16 of 2^6 p: below fp16's
    normal range it is off by up to half of 2^-24 instead of p * 2^-11, so by 2^-31 of the largest weight for each key."""
    floor = 2.0 ** -31 * np.abs(held.v[np.isfinite(held.v)]).max(initial=0) * held.lens.max()
    check_attention(o, lse, held.expect(Q, **kw), FP16, what, floor)


def _attend(held, Q, starts=None, **kw):
    o, lse = rbs.kv4_attend(Q, held.cache, ints(held.table), ints(held.lens),
                            starts=None if starts is None else ints(starts), return_lse=True, **kw)
    return o, lse


@pytest.mark.parametrize("G", [1, 2, 5, 8, 16, 40])
@pytest.mark.parametrize("Lq", [1, 3])
def test_attend_heads_and_tokens(cuda_ok, G, Lq):
    rng = np.random.default_rng(G * 10 + Lq)
    held = Held(rng, [1, 15, 16, 17, 0, 128, 129, 500, 2], 2, 16)
    Q = randn(rng, 9, Lq, 2 * G, 128)
    o, lse = _attend(held, Q)
    _check(o, lse, held, Q)
    assert not f64(o)[4].any() and rbs.rbs_get_device_error() == 0


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (100, 0), (100, 40), (333, 1000), (5000, 4)])
def test_attend_windows_and_pages(cuda_ok, page, window, sinks):
    rng = np.random.default_rng(page + window + sinks)
    held = Held(rng, [700, 1, 333, 64, 350], 1, page)
    Q = randn(rng, 5, 2, 4, 128)
    o, lse = _attend(held, Q, window=window, sinks=sinks)
    _check(o, lse, held, Q, window=window, sinks=sinks)


@pytest.mark.parametrize("lens,H,G,Lq", [([20000], 1, 8, 1), ([9001, 3], 2, 4, 2), ([5000] * 3, 4, 1, 1),
                                         ([30, 4000, 700, 1, 0, 2500], 8, 2, 1), ([6000, 100], 1, 8, 9),
                                         ([2000], 1, 3, 50)])
def test_attend_split_over_many_blocks(cuda_ok, lens, H, G, Lq):
    rng = np.random.default_rng(len(lens) + G + Lq)
    held = Held(rng, lens, H, 64)
    Q = randn(rng, len(lens), Lq, H * G, 128)
    o, lse = _attend(held, Q)
    _check(o, lse, held, Q)
    again, lse2 = _attend(held, Q)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_attend_starts_and_padded_rows(cuda_ok):
    """Queries left-aligned in a padded batch: rows past a request's length and before its first token are empty."""
    rng = np.random.default_rng(20)
    held = Held(rng, [40, 7, 0, 300], 2, 32)
    Q = randn(rng, 4, 5, 4, 128)
    for starts in ([35, 5, 0, 100], [-2, 0, 3, 298], [40, 50, -9, (1 << 31) - 1], [-(1 << 31), 6, 0, 299]):
        for kw in ({}, dict(window=3, sinks=2)):
            o, lse = _attend(held, Q, starts=starts, **kw)
            _check(o, lse, held, Q, str(starts), starts=starts, **kw)


@pytest.mark.parametrize("qs,ks", [(30.0, 1.0), (1e-20, 1.0), (1e20, 1e-3), (1.0, 100.0)])
def test_attend_score_sizes(cuda_ok, qs, ks):
    """Peaked and flat rows, and queries far outside fp16's range."""
    rng = np.random.default_rng(21)
    held = Held(rng, [777, 50], 1, 48, k_scale=ks)
    Q = randn(rng, 2, 1, 8, 128, scale=qs)
    scale = 1e-18 if qs > 1e10 else 0.3
    o, lse = _attend(held, Q, softmax_scale=scale)
    _check(o, lse, held, Q, scale=scale)


def test_attend_rising_scores_and_scales(cuda_ok):
    """Keys whose scores rise along the cache (every block moves the maximum); k_scale, v_scale other than 1."""
    rng = np.random.default_rng(22)
    held = Held(rng, [900], 1, 64, gk=0.125, gv=8.0)
    q = f64(randn(rng, 1, 1, 1, 128))[0, 0, 0]
    K = np.linspace(-3, 3, 900)[None, :, None, None] * q + 0.1 * rng.standard_normal((1, 900, 1, 128))
    K, V = (torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda() for x in (K, rng.standard_normal((1, 900, 1, 128))))
    rbs.kv4_append(held.cache, K, V, ints(held.slots))
    held.k, held.v = S.round_trip(f64(K), 0.125), S.round_trip(f64(V), 8.0)
    Q = torch.from_numpy(np.stack([q, -q, 0 * q]).astype(np.float32)).to(torch.bfloat16).cuda().view(1, 1, 3, 128)
    o, lse = _attend(held, Q)
    _check(o, lse, held, Q)


def test_nan_in_masked_places_stays_there(cuda_ok):
    """NaN keys and values reach the queries that see them and no others: not earlier drafted tokens, not rows whose
    window has passed them."""
    rng = np.random.default_rng(23)
    held = Held(rng, [60, 60], 1, 16)
    K, V = randn(rng, 2, 60, 1, 128), randn(rng, 2, 60, 1, 128)
    K[0, 58, 0, 3] = float("nan")
    V[1, 57, 0, 30] = float("nan")
    V[1, 20, 0, 90] = float("inf")
    rbs.kv4_append(held.cache, K, V, ints(held.slots))
    held.k, held.v = S.round_trip(f64(K)), S.round_trip(f64(V))
    Q = randn(rng, 2, 8, 2, 128)
    for kw in ({}, dict(window=36), dict(window=36, sinks=21)):
        o, _ = _attend(held, Q, **kw)
        for b in range(2):
            for t in range(8):
                p = 52 + t
                see = S.visible([p], np.arange(60), kw.get("window", 0), kw.get("sinks", 0))[0]
                hit = np.isnan(held.v[b, see, 0]).any(0) | np.isnan(held.k[b, see, 0]).any()
                assert np.array_equal(np.isnan(f64(o)[b, t]), np.broadcast_to(hit, (2, 128))), (b, t, kw)


def test_bad_pages_and_lengths(cuda_ok):
    rng = np.random.default_rng(24)
    held = Held(rng, [200, 90], 2, 32)
    Q = randn(rng, 2, 1, 4, 128)
    want = held.expect(Q)
    rbs.rbs_get_device_error()
    held.table[0, 2] = held.cache.data.shape[0]  # tokens 64 .. 95 of request 0 are nowhere
    o, lse = _attend(held, Q)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_BLOCK_INDEX
    keep = np.r_[0:64, 96:200]
    short = Held.__new__(Held)
    short.lens, short.k, short.v = np.array([168]), held.k[:1, keep], held.v[:1, keep]
    r = short.expect(Q[:1])
    check_attention(o[:1], lse[:1], r, FP16)
    check_attention(o[1:], lse[1:], tuple(x[1:] for x in want), FP16)
    held.table[0, 2] = -5
    _attend(held, Q)
    assert rbs.rbs_get_device_error() == rbs.DEVERR_BLOCK_INDEX
    held.table[0, 2] = 0
    for n in (-1, 7 * 32 + 1):
        held.lens[1] = n
        _attend(held, Q)
        assert rbs.rbs_get_device_error() & rbs.DEVERR_LENGTH


def test_attend_layouts_streams_graph(cuda_ok):
    """Queries as a view of a packed projection, outputs in another order, a given workspace, another stream, and a
    graph replayed on changed lengths."""
    rng = np.random.default_rng(25)
    held = Held(rng, [300, 45], 2, 16, width=40)
    qkv = randn(rng, 2, 1, 20, 128)
    Q = qkv[:, :, 2:18]
    want, lse = _attend(held, Q)
    _check(want, lse, held, Q)
    hold = torch.zeros(2, 16, 3, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((rbs.rbs_kv4_attend_workspace_bytes(1, 16, 2),), 255, dtype=torch.uint8, device="cuda")
    table, lens = ints(held.table), ints(held.lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rbs.kv4_attend(Q, held.cache, table, lens, out=hold.transpose(1, 2)[:, 1:2], workspace=ws)
    s.synchronize()
    assert torch.equal(hold.transpose(1, 2)[:, 1:2], want) and not hold[:, :, [0, 2]].any()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, z = rbs.kv4_attend(Q, held.cache, table, lens, return_lse=True)
    for n in ([300, 45], [17, 0], [299, 32]):
        lens.copy_(ints(n))
        g.replay()
        a, b = rbs.kv4_attend(Q, held.cache, table, lens, return_lse=True)
        assert torch.equal(o, a) and torch.equal(z, b)


@pytest.mark.parametrize("B", [1500, 4096])
def test_attend_many_requests(cuda_ok, B):
    """Up to the most requests of a call, of a few tokens each, some of none."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, B)
    held = Held(rng, lens, 1, 16)
    Q = randn(rng, B, 1, 2, 128)
    o, lse = _attend(held, Q)
    pick = np.r_[0:20, rng.integers(0, B, 100), B - 20:B]
    part = Held.__new__(Held)
    part.lens, part.k, part.v = held.lens[pick], held.k[pick], held.v[pick]
    _check(o[pick], lse[pick], part, Q[pick])
    assert (f64(lse)[lens == 0] == -np.inf).all() and not f64(o)[lens == 0].any()


def test_cache_past_32_bits(cuda_ok):
    """Pages whose bytes lie beyond 2^31 and 2^32 of a cache of 4.7 GB."""
    rng = np.random.default_rng(60)
    page, H, pages = 256, 8, 16000
    data = torch.empty(pages, H, rbs.rbs_kv4_page_bytes(page), dtype=torch.uint8, device="cuda")
    assert data.numel() > 1 << 32
    cache = rbs.KV4Cache(data, page)
    table = np.array([[pages - 1, 7, 15000], [7300, 14600, 0]])
    lens = np.array([600, 300])
    K, V = randn(rng, 2, 600, H, 128), randn(rng, 2, 600, H, 128)
    t = np.arange(600)
    slots = np.where(t < lens[:, None], table[np.arange(2)[:, None], t // page] * page + t % page, -1)
    rbs.kv4_append(cache, K, V, ints(slots))
    k, v = rbs.kv4_load(cache, ints(slots))
    held = Held.__new__(Held)
    held.lens, held.k, held.v = lens, S.round_trip(f64(K)), S.round_trip(f64(V))
    for b in range(2):
        assert np.array_equal(f64(k)[b, :lens[b]], held.k[b, :lens[b]])
        assert np.array_equal(f64(v)[b, :lens[b]], held.v[b, :lens[b]])
    Q = randn(rng, 2, 1, 16, 128)
    o, lse = rbs.kv4_attend(Q, cache, ints(table), ints(lens), return_lse=True)
    _check(o, lse, held, Q)


def test_attend_a_prompt(cuda_ok):
    """Many query tokens per request: tiles of rows that end inside a token's heads, and several of them per request."""
    rng = np.random.default_rng(61)
    held = Held(rng, [150, 64], 2, 32)
    Q = randn(rng, 2, 64, 6, 128)
    for kw in ({}, dict(window=20, sinks=2)):
        o, lse = _attend(held, Q, **kw)
        _check(o, lse, held, Q, **kw)


def test_windows_and_sinks_past_32_bits(cuda_ok):
    """A window or a count of sinks that no int32 holds is one that reaches every key."""
    rng = np.random.default_rng(62)
    held = Held(rng, [200, 90], 2, 32)
    Q = randn(rng, 2, 3, 4, 128)
    full, _ = _attend(held, Q)
    for big in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 128, 2 ** 64 + 5):
        a, _ = _attend(held, Q, window=big)
        b, _ = _attend(held, Q, window=3, sinks=big)
        assert torch.equal(a, full)
        _check(b, None, held, Q)
    for bad in (-1, -2 ** 31 - 1, -2 ** 32 + 7, -2 ** 64):
        for kw in (dict(window=bad), dict(window=4, sinks=bad)):
            with pytest.raises(rbs.RbsError, match=">= 0"):
                _attend(held, Q, **kw)


def test_integers_past_32_bits_are_refused(cuda_ok):
    rng = np.random.default_rng(63)
    K, cache = randn(rng, 1, 4, 2, 128), rbs.KV4Cache.empty(2, 16, 2)
    table, n = ints([[0]]), ints([1])
    for bad in (2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="page_size"):
            rbs.kv4_extend(table, n, n, n, n, 1, bad)
        with pytest.raises(ValueError, match="max_new"):
            rbs.kv4_extend(table, n, n, n, n, bad, 16)
        with pytest.raises(ValueError, match="page_size"):
            rbs.kv4_load(rbs.KV4Cache(cache.data, bad), n[None])
        with pytest.raises(ValueError, match="rope_style"):
            rbs.rope_qk_norm(K, K, None, None, ints(np.arange(4)), 1e4, rope_style=bad)


@pytest.mark.parametrize("qs,gk,scale", [(1e-30, 2.0 ** -64, None), (1.0, 2.0 ** -64, 1e-44), (1e-37, 2.0 ** 64, 2e19)])
def test_attend_factors_of_the_scores_beyond_fp32(cuda_ok, qs, gk, scale):
    """softmax_scale, k_scale and the size of a query row, whose product leaves fp32's range while the scores do not: rows
    of equal weights, and ordinary ones."""
    rng = np.random.default_rng(64)
    held = Held(rng, [40, 7, 200], 1, 32, gk=gk, k_scale=gk)
    Q = randn(rng, 3, 2, 4, 128, scale=qs)
    for kw in ({}, dict(window=9, sinks=3)):
        o, lse = _attend(held, Q, softmax_scale=scale, **kw)
        _check(o, lse, held, Q, scale=scale, **kw)


@pytest.mark.parametrize("lens", [[60], [3000, 50]])
def test_attend_scores_far_below_zero(cuda_ok, lens):
    """Every score of a row below -1e34: the largest one takes the whole weight all the same."""
    rng = np.random.default_rng(65)
    held = Held(rng, lens, 1, 32)
    B, n = held.slots.shape
    K = torch.full((B, n, 1, 128), -2.0, dtype=torch.bfloat16, device="cuda")
    K[:, 17] = -1.0
    K[:, 18:] = -6.0
    rbs.kv4_append(held.cache, K, randn(rng, B, n, 1, 128), ints(held.slots))
    k, v = rbs.kv4_load(held.cache, ints(held.slots))
    o, lse = _attend(held, torch.full((B, 1, 2, 128), 1e33, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(o, v[:, 17:18].expand(B, 1, 2, 128))
    # (the cache holds -1 as code 6 times the scale e4m3(1 / 6) = 11 / 64: -1.03125)
    want = f64(k)[:, 17].sum() / B * float(torch.tensor(1e33, dtype=torch.bfloat16)) / 128 ** 0.5
    assert (np.abs(f64(lse) / want - 1) < 2.0 ** -20).all()  # a handful of fp32 roundings


@pytest.mark.parametrize("size", [1e4, 1e5, 1e7])
@pytest.mark.parametrize("Lq", [1, 2])
def test_attend_scores_far_apart(cuda_ok, size, Lq):
    """Queries and keys whose scores are far past 2^28: each row is the value of its highest key."""
    rng = np.random.default_rng(68)
    held = Held(rng, [500, 3000, 40], 2, 32, gk=2.0 ** 12, k_scale=size)
    Q = randn(rng, 3, Lq, 6, 128, scale=size)
    o, lse = _attend(held, Q)
    _check(o, lse, held, Q)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("lens,G,Lq", [([700, 90, 16, 5], 2, 4), ([5000, 3], 8, 4), ([2000, 40], 6, 20)])
def test_attend_padded_rows_that_hold_anything(cuda_ok, lens, G, Lq):
    """Rows of a padded batch past a request's tokens or before its first: empty, whatever their queries hold, and the
    rows beside them are what they are alone."""
    rng = np.random.default_rng(66)
    held = Held(rng, lens, 2, 32)
    Q = randn(rng, len(lens), Lq, 2 * G, 128)
    for back in (1, Lq - 1, -2):  # live rows at the front, or two dead ones there
        starts = held.lens - back if back > 0 else np.full(len(lens), -2)
        p = starts[:, None] + np.arange(Lq)
        dead = (p < 0) | (p >= held.lens[:, None])
        odd = Q.clone()
        odd[torch.from_numpy(dead).cuda()] = float("nan")
        for kw in ({}, dict(window=40, sinks=21)):
            o, lse = _attend(held, odd, starts=starts, **kw)
            _check(o, lse, held, Q, starts=starts, **kw)


def test_attend_padded_rows_cost_what_full_rows_do(cuda_ok):
    """Three of four drafted tokens live, over long caches: the sub-blocks that every live row sees whole take one pass.
    (Measured ratio of the times 1.0; four passes over each sub-block made it 2 and more.)"""
    rng = np.random.default_rng(67)
    n, page, B = 65536, 64, 4
    data = torch.zeros(B * n // page, 4, rbs.rbs_kv4_page_bytes(page), dtype=torch.uint8, device="cuda")
    cache, table = rbs.KV4Cache(data, page), ints(np.arange(B * n // page).reshape(B, -1))
    Q, lens = randn(rng, B, 4, 32, 128), ints([n] * B)
    took = []
    for live in (4, 3):
        starts, times = ints([n - live] * B), []
        for i in range(13):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                rbs.kv4_attend(Q, cache, table, lens, starts=starts)
            b.record()
            b.synchronize()
            if i >= 3:
                times.append(a.elapsed_time(b))
        took.append(sorted(times)[5])
    assert took[1] < 1.5 * took[0], took


def test_extend_as_many_new_tokens_as_int32_holds(cuda_ok):
    """max_new = 2^31 - 1: every slot and position of the row is written, and nothing beside them."""
    n = 2 ** 31 - 1
    hold = [torch.full((n + 4096,), 77, dtype=torch.int32, device="cuda") for _ in range(2)]
    slots, pos = (x[2048:2048 + n].view(1, n) for x in hold)
    table = ints([[-1, -1, -1]])
    assert rbs.rbs_get_device_error() == 0
    rbs.kv4_extend(table, ints([0]), ints([40]), ints([7, 3, 5, 9]), ints([1]), n, 16, slots=slots, pos=pos)
    assert rbs.rbs_get_device_error() == 0 and table.tolist() == [[3, 5, 9]]
    assert pos[0, :40].tolist() == list(range(40)) and slots[0, :40].tolist() == [(3, 5, 9)[t // 16] * 16 + t % 16 for t in range(40)]
    for x in hold:
        assert (x[:2048] == 77).all() and (x[2048 + n:] == 77).all()
        assert x[2088:2048 + n].amax() == -1 and x[2088:2048 + n].amin() == -1
