"""The serving operators one after another, as a model with per-head norms and
windowed layers uses them: pages, norm and rotation, cache, attention -- for
the prompts, for decoding steps, in a captured graph, and for a passage taken
back out of the cache and moved to another position."""

import numpy as np
import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from helpers import host_bits
from oracle import rbs_oracle as O
from oracle import serving_oracle as S
from serving_helpers import BF16, FP16, assert_within, check_attention, f64, ints, randn

pytestmark = pytest.mark.gpu

THETA, HQ, H, PAGE, WINDOW, SINKS = 10000.0, 8, 2, 16, 24, 4


class Layer:
    def __init__(self, rng, B, width):
        self.wq, self.wk = randn(rng, 128), randn(rng, 128)
        pages = B * width + 1
        self.cache = rbs.KV4Cache.empty(pages, PAGE, H)
        self.cache.data.fill_(0xFF)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.free = ints(rng.permutation(pages))
        self.head = ints([0])

    def step(self, qkv, old, new, **kw):
        """One call's work for qkv [B, n, HQ + 2 H, 128] of tokens old .. new - 1 (the rest of n is padding)."""
        q, k, v = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + H], qkv[:, :, HQ + H:]
        slots, pos, head = rbs.kv4_extend(self.table, old, new, self.free, self.head, qkv.shape[1], PAGE)
        self.head.copy_(head)
        q, k = rbs.rope_qk_norm(q, k, self.wq, self.wk, pos, THETA)
        rbs.kv4_append(self.cache, k, v, slots)
        o, lse = rbs.kv4_attend(q, self.cache, self.table, new, starts=old, return_lse=True, **kw)
        return q, k, v, slots, pos, o, lse


class Held:
    """What the requests hold, in fp64: rotated keys and values as the cache stores them."""

    def __init__(self, B, n):
        self.k, self.v = np.zeros((B, n, H, 128)), np.zeros((B, n, H, 128))

    def add(self, k, v, pos):
        for b, t in zip(*np.nonzero(pos >= 0)):
            self.k[b, pos[b, t]], self.v[b, pos[b, t]] = S.round_trip(k[b, t]), S.round_trip(v[b, t])

    def expect(self, q, pos, window, sinks):
        B, n = q.shape[:2]
        out, a = np.zeros(q.shape), np.zeros(q.shape)
        lse, z = np.full((B, HQ, n), -np.inf), np.zeros((B, HQ, n))
        for b in range(B):
            see = S.visible(pos[b], np.arange(self.k.shape[1]), window, sinks) & (pos[b] >= 0)[:, None]
            for h in range(HQ):
                out[b, :, h], lse[b, h], a[b, :, h], z[b, h] = S.attend(
                    q[b, :, h], self.k[b, :, h // (HQ // H)], self.v[b, :, h // (HQ // H)], see, 128 ** -0.5)
        return out, lse, a, z


@pytest.mark.parametrize("window,sinks", [(0, 0), (WINDOW, SINKS)])
def test_prompts_and_decoding(cuda_ok, window, sinks):
    rng = np.random.default_rng(window)
    lens = np.array([37, 5, 64])
    layer, held = Layer(rng, 3, 6), Held(3, 96)
    old, new = np.zeros(3, int), lens
    for step in range(5):
        n = int((new - old).max()) if step else 64
        qkv = randn(rng, 3, n, HQ + 2 * H, 128)
        q, k, v, slots, pos, o, lse = layer.step(qkv, ints(old), ints(new), window=window, sinks=sinks)
        p = pos.cpu().numpy()
        assert np.array_equal(p, np.where(np.arange(n) < (new - old)[:, None], old[:, None] + np.arange(n), -1))
        for x, y, w in ((qkv[:, :, :HQ], q, layer.wq), (qkv[:, :, HQ:HQ + H], k, layer.wk)):
            ref, size = S.qk_norm_rope(host_bits(x), host_bits(w), p, THETA, 1e-6)
            assert_within(f64(y), ref, BF16 * np.abs(ref) + 2.0 ** -19 * size, "rotated")
        held.add(f64(k), f64(v), p)
        check_attention(o, lse, held.expect(f64(q), p, window, sinks), FP16, f"step {step}", 2.0 ** -31 * 96 * 6)
        if step == 0 and window:  # the prompts' own attention: the same window over keys that were not rounded to 4 bits
            full, flse = rbs.swa_prefill(q, k, v, window, sinks, return_lse=True)
            check_attention(full, flse, S.window_attention(f64(q), f64(k), f64(v), window, sinks), BF16, "prompt")
        old = new
        new = old + np.array([[1, 1, 0], [2, 3, 1], [1, 0, 1], [4, 4, 4]][step % 4])
    taken = layer.table.cpu().numpy()
    used = taken[taken >= 0]
    assert used.size == np.unique(used).size == layer.head.item() == (-(-old // PAGE)).sum()
    assert rbs.rbs_get_device_error() == 0


def test_captured_decoding_step(cuda_ok):
    """A decoding step captured once, with the request lengths advanced inside the graph, gives what eager steps give."""
    outs = []
    for captured in (False, True):
        rng = np.random.default_rng(5)
        layer = Layer(rng, 2, 8)
        prompt = randn(rng, 2, 40, HQ + 2 * H, 128)
        old, new = ints([0, 0]), ints([40, 13])
        layer.step(prompt, old, new)
        steps = randn(rng, 20, 2, 1, HQ + 2 * H, 128)
        x = torch.empty_like(steps[0])
        got = []

        def one():
            old.copy_(new)
            new.add_(1)
            return layer.step(x, old, new, window=WINDOW, sinks=SINKS)[5:]

        if captured:
            torch.cuda.synchronize()
            keep = [t.clone() for t in (layer.table, layer.head, old, new, layer.cache.data)]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                o, lse = one()
            for t, s in zip((layer.table, layer.head, old, new, layer.cache.data), keep):
                assert torch.equal(t, s)  # capturing runs nothing
        for s in range(20):
            x.copy_(steps[s])
            if captured:
                g.replay()
            else:
                o, lse = one()
            got.append((o.clone(), lse.clone()))
        outs.append((got, layer.table.clone(), layer.head.item(), new.clone()))
    for (a, la), (b, lb) in zip(outs[0][0], outs[1][0]):
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(outs[0][1], outs[1][1]) and outs[0][2] == outs[1][2] and torch.equal(outs[0][3], outs[1][3])
    assert rbs.rbs_get_device_error() == 0


def test_two_requests_streams_at_once(cuda_ok):
    """Two groups of requests decoded on two streams over one cache, each with a workspace of its own."""
    rng = np.random.default_rng(6)
    layer = Layer(rng, 2, 40)
    layer.step(randn(rng, 2, 600, HQ + 2 * H, 128), ints([0, 0]), ints([600, 411]))
    Q, lens = randn(rng, 2, 1, HQ, 128), ints([600, 411])
    want = rbs.kv4_attend(Q, layer.cache, layer.table, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate(streams * 5):
        with torch.cuda.stream(s):
            b = i % 2
            got.append((b, rbs.kv4_attend(Q[b:b + 1], layer.cache, layer.table[b:b + 1], lens[b:b + 1])))
    torch.cuda.synchronize()
    for b, o in got:
        assert (f64(o) - f64(want[b:b + 1]) <= 2 * BF16 * np.abs(f64(want[b:b + 1])) + 2.0 ** -9).all()


def test_cached_passage_moved_and_attended(cuda_ok):
    """A passage's keys come back from the cache, move to another position and are attended to as a passage of a new
    prompt (Block-attention's cached passages)."""
    rng = np.random.default_rng(7)
    layer = Layer(rng, 1, 8)
    L, shift, L2 = 100, 60, 192
    _, k, v, slots, pos, _, _ = layer.step(randn(rng, 1, L, HQ + 2 * H, 128), ints([0]), ints([L]))
    ck, cv = rbs.kv4_load(layer.cache, slots)
    assert np.array_equal(f64(ck), S.round_trip(f64(k))) and np.array_equal(f64(cv), S.round_trip(f64(v)))
    at = ints(np.arange(L))
    moved = rbs.rope_reencode(ck, at, at + shift, THETA)
    ref = O.rope_rotate(f64(ck), np.full(L, shift), THETA)
    size = np.concatenate([np.abs(f64(ck)[..., :64]) + np.abs(f64(ck)[..., 64:])] * 2, -1)
    assert_within(f64(moved), ref, BF16 * np.abs(ref) + 2.0 ** -19 * size, "moved")
    K, V = randn(rng, 1, L2, H, 128), randn(rng, 1, L2, H, 128)
    K[:, shift:shift + L], V[:, shift:shift + L] = moved, cv
    Q = randn(rng, 1, L2, HQ, 128)
    seg, final = [0, shift], shift + L
    lists = rbs.rbs_lists_block_attention(seg, final, 64, 1, HQ, 0, L2 // 64)
    out = rbs.bsa_prefill_segments(Q, K, V, lists, seg, final, 64, 64)
    q, kk, vv = f64(Q), f64(K), f64(V)
    lo = O.block_attention_key_start(seg, final, np.arange(L2))
    see = (np.arange(L2)[None] <= np.arange(L2)[:, None]) & (np.arange(L2)[None] >= np.asarray(lo)[:, None])
    for h in range(HQ):
        o, _, _, _ = S.attend(q[0, :, h], kk[0, :, h // 4], vv[0, :, h // 4], see, 128 ** -0.5)
        assert np.abs(f64(out)[0, :, h] - o).max() <= 2e-2  # the library's bound for this call
