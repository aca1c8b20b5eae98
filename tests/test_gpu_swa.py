"""GPU parity of swa_prefill with the fp64 oracle."""

import numpy as np
import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from block_sparse_long_rbs_b200 import _abi, _stream, _t
from oracle import serving_oracle as S
from serving_helpers import BF16, check_attention, f64, randn

pytestmark = pytest.mark.gpu


def _check(Q, K, V, window, sinks, off=0, scale=None, rows=None, **kw):
    o, lse = rbs.swa_prefill(Q, K, V, window, sinks, q_offset=off, softmax_scale=scale, return_lse=True, **kw)
    W = window if window else off + Q.shape[1]
    ref = S.window_attention(f64(Q), f64(K), f64(V), W, sinks, off, scale, rows)
    got = (o, lse) if rows is None else (o[:, rows], lse[:, :, rows])
    check_attention(*got, ref, BF16)
    assert rbs.rbs_get_device_error() == 0
    return o, lse


def _qkv(rng, B, Lq, Hq, Hkv, Lk=None, scale=1.0):
    Lk = Lq if Lk is None else Lk
    return randn(rng, B, Lq, Hq, 128, scale=scale), randn(rng, B, Lk, Hkv, 128), randn(rng, B, Lk, Hkv, 128)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 48, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (64, 16), (100, 17), (300, 150)])
def test_heads_windows_sinks(cuda_ok, G, window, sinks):
    rng = np.random.default_rng(G + window + sinks)
    n = 333 if G < 48 else 70
    H = 2 if G < 48 else 1
    _check(*_qkv(rng, 1, n, H * G, H), window, sinks)


@pytest.mark.parametrize("Lq", [1, 2, 15, 16, 17, 64, 129])
@pytest.mark.parametrize("off", [0, 1, 63, 1000])
def test_lengths_and_offsets(cuda_ok, Lq, off):
    rng = np.random.default_rng(Lq + off)
    Q, K, V = _qkv(rng, 2, Lq, 4, 1, off + Lq)
    for window, sinks in ((0, 0), (1, 1), (50, 4), (200, 70), (5000, 4)):
        _check(Q, K, V, window, sinks, off)


@pytest.mark.parametrize("window", [1, 16, 64, 128, 1000, 4096])
def test_long(cuda_ok, window):
    rng = np.random.default_rng(window)
    Q, K, V = _qkv(rng, 1, 6000, 8, 1)
    rows = np.unique(np.r_[0:3, 15:18, 127:130, rng.integers(0, 6000, 60), 5997:6000])
    for sinks in (0, 4, 100):
        _check(Q, K, V, window, sinks, rows=rows)


def test_every_block_works_on_many_items(cuda_ok):
    """More items than CTAs: ring, buffer and barrier phases carried from item to item, tile counts odd and even."""
    rng = np.random.default_rng(77)
    Q, K, V = _qkv(rng, 3, 1500, 16, 4)
    rows = np.unique(rng.integers(0, 1500, 80))
    for window, sinks in ((1, 0), (70, 0), (130, 4), (130, 20), (0, 0)):
        a, la = _check(Q, K, V, window, sinks, rows=rows)
        b, lb = rbs.swa_prefill(Q, K, V, window, sinks, return_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("Lk,off", [(50, 0), (200, 100), (100, 200), (5, 300), (400, 0)])
def test_keys_that_end_before_or_after_the_queries(cuda_ok, Lk, off):
    """Keys past Lk do not exist; a query whose window lies past them sees the sinks or nothing (O 0, lse -inf)."""
    rng = np.random.default_rng(Lk + off)
    Q, K, V = _qkv(rng, 1, 150, 2, 1, Lk)
    for window, sinks in ((40, 0), (40, 3), (40, 30), (0, 0), (1, 0)):
        _check(Q, K, V, window, sinks, off)


@pytest.mark.parametrize("scale,spread", [(2.0, 3.0), (1e-6, 1.0), (0.09, 20.0)])
def test_score_sizes(cuda_ok, scale, spread):
    rng = np.random.default_rng(31)
    Q, K, V = _qkv(rng, 1, 500, 4, 2, scale=spread)
    _check(Q, K, V, 150, 4, scale=scale)


def test_rising_scores(cuda_ok):
    """Keys whose scores rise along the sequence: every tile moves the maximum and scales the outputs."""
    rng = np.random.default_rng(32)
    Q, K, V = _qkv(rng, 1, 700, 2, 1)
    d = f64(Q)[0, 0, 0]
    K = torch.from_numpy((np.linspace(-4, 4, 700)[None, :, None, None] * d + 0.1 * f64(K)).astype(np.float32))
    Q = torch.from_numpy((d + 0.1 * f64(Q)).astype(np.float32))
    _check(Q.to(torch.bfloat16).cuda(), K.to(torch.bfloat16).cuda(), V, 300, 8, scale=0.5)


def test_views_outputs_stream_graph(cuda_ok):
    rng = np.random.default_rng(33)
    qkv = randn(rng, 2, 200, 12, 128)
    Q, K, V = qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:]
    want, lse = _check(Q, K, V, 60, 4)
    hold = torch.full((2, 8, 210, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rbs.swa_prefill(Q, K, V, 60, 4, out=hold.transpose(1, 2)[:, 5:205])
    s.synchronize()
    assert torch.equal(hold.transpose(1, 2)[:, 5:205], want) and (hold[:, :, :5] == 7).all() and (hold[:, :, 205:] == 7).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, z = rbs.swa_prefill(Q, K, V, 60, 4, return_lse=True)
    qkv.neg_()
    qkv[:, 50:60] *= 2
    g.replay()
    a, b = rbs.swa_prefill(Q, K, V, 60, 4, return_lse=True)
    assert torch.equal(o, a) and torch.equal(z, b)


@pytest.mark.parametrize("G", [1, 4])
def test_nan_and_infinity_in_masked_places(cuda_ok, G):
    """NaN and infinite keys and values reach exactly the queries that see them; the others keep their results."""
    rng = np.random.default_rng(34)
    Q, K, V = _qkv(rng, 1, 400, 2 * G, 2)
    want, wlse = rbs.swa_prefill(Q, K, V, 90, 5, return_lse=True)
    K[0, 100, 0, 7] = float("nan")
    V[0, 200, 0, 9] = float("inf")
    V[0, 2, 1, 11] = float("nan")
    V[0, 300, 1] = float("nan")
    o, lse = rbs.swa_prefill(Q, K, V, 90, 5, return_lse=True)
    see = S.visible(np.arange(400), np.arange(400), 90, 5)
    off = 2 * BF16 * np.abs(f64(want)) + 2.0 ** -6  # the two ways round P differently
    for h in range(2 * G):
        k, v = f64(K)[0, :, h // G], f64(V)[0, :, h // G]
        bad_k = (see & np.isnan(k).any(-1)[None]).any(1)
        got = f64(o)[0, :, h]
        assert np.isnan(got[bad_k]).all() and np.isnan(f64(lse)[0, h, bad_k]).all()
        odd = (see[:, :, None] & ~np.isfinite(v)[None]).any(1) | bad_k[:, None]  # [token, dim]
        assert np.array_equal(~np.isfinite(got), odd)
        assert (np.abs(got - f64(want)[0, :, h])[~odd] <= off[0, :, h][~odd]).all()
        assert np.array_equal(f64(lse)[0, h, ~bad_k], f64(wlse)[0, h, ~bad_k])


def test_values_that_spoil_every_row_of_a_long_prompt(cuda_ok):
    """Rows made again one by one, all 12,000 keys of each, stay far inside the waits' limit."""
    rng = np.random.default_rng(44)
    Q, K, V = _qkv(rng, 1, 12000, 8, 1)
    want, wlse = rbs.swa_prefill(Q, K, V, 0, return_lse=True)
    V[0, 0, 0, 3] = float("nan")
    V[0, 1, 0, 4] = float("-inf")
    rbs.rbs_get_device_error()
    o, lse = rbs.swa_prefill(Q, K, V, 0, return_lse=True)
    assert rbs.rbs_get_device_error() == 0
    assert torch.isnan(o[..., 3]).all() and torch.isneginf(o[:, 1:, :, 4]).all() and torch.isfinite(o[:, 0, :, 4]).all()
    o[..., 3:5] = want[..., 3:5]
    # P's rounding here and there (2^-9 of values whose weighted mean size is below 1), the output's twice
    assert (f64(o) - f64(want) <= 2 * BF16 * np.abs(f64(want)) + 2.0 ** -6).all()
    assert (f64(want) - f64(o) <= 2 * BF16 * np.abs(f64(want)) + 2.0 ** -6).all()
    assert torch.equal(lse, wlse)


def test_batches_far_apart(cuda_ok):
    """Batch entries more than 2^31 bytes apart (views of one buffer)."""
    rng = np.random.default_rng(35)
    big = torch.empty(2, (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    x = randn(rng, 2, 100, 12, 128)
    qkv = big[:, :x[0].numel()].view(2, 100, 12, 128)
    qkv.copy_(x)
    out = big[:, 1 << 20:(1 << 20) + 100 * 8 * 128].view(2, 100, 8, 128)
    _check(qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:], 30, 3, out=out)
    w = randn(rng, 128)
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    got = rbs.rope_qk_norm(qkv[:, :, :8], qkv[:, :, 8:10], w, None, pos, 1e4, q_out=out)
    want = rbs.rope_qk_norm(x[:, :, :8], x[:, :, 8:10], w, None, pos, 1e4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("stall", [0, 1, 5])
def test_wait_that_runs_out_returns_timeout_and_the_next_call_is_correct(cuda_ok, stall):
    """The producer of key tiles stops early (a testing hook): the waits for the missing tiles run out, the kernel records
    it and returns with nothing in flight, and the next call is correct."""
    rng = np.random.default_rng(36)
    Q, K, V = _qkv(rng, 1, 3000, 8, 2)
    out = torch.zeros_like(Q)
    L_ = _abi.lib()
    assert rbs.rbs_get_device_error() == 0
    args = (_t(Q, "Q"), _t(K, "K"), _t(V, "V"), 500)
    assert L_.rbs_testing_swa_prefill_stalled(*args, 1_000_000, stall, _t(out, "O"), _stream()) == 0, L_.rbs_last_error()
    torch.cuda.synchronize()
    assert rbs.rbs_get_device_error() & rbs.DEVERR_TIMEOUT
    _check(Q, K, V, 500, 4, rows=np.unique(rng.integers(0, 3000, 40)))
    for wait, n in ((10, 5), (3_000_000_000, 5), (1_000_000, -1)):
        assert L_.rbs_testing_swa_prefill_stalled(*args, wait, n, _t(out, "O"), _stream()) == 1


def test_windows_and_sinks_past_32_bits(cuda_ok):
    """A window or a count of sinks that no int32 holds is one that reaches every key."""
    rng = np.random.default_rng(47)
    Q, K, V = _qkv(rng, 1, 200, 4, 2)
    full = rbs.swa_prefill(Q, K, V, 0)
    for big in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 128, 2 ** 64 + 5):
        assert torch.equal(rbs.swa_prefill(Q, K, V, big), full)
        assert torch.equal(rbs.swa_prefill(Q, K, V, 3, big), full)
    for bad in (-1, -2 ** 31 - 1, -2 ** 32 + 7, -2 ** 64):
        with pytest.raises(rbs.RbsError, match=">= 0"):
            rbs.swa_prefill(Q, K, V, bad)
        with pytest.raises(rbs.RbsError, match=">= 0"):
            rbs.swa_prefill(Q, K, V, 4, bad)
    with pytest.raises(ValueError, match="q_offset"):
        rbs.swa_prefill(Q, K, V, 4, q_offset=2 ** 64 + 5)
    with pytest.raises(rbs.RbsError, match="2\\^31"):
        rbs.swa_prefill(Q, K, V, 4, q_offset=2 ** 32 + 5)


def _with_odd_values(o, see, v):
    """Outputs [n, D] of finite values, and what they become where visible keys (see [n, keys]) hold the v's that are not."""
    nan, up, down = (see.astype(np.float32) @ m.astype(np.float32) > 0 for m in (np.isnan(v), np.isposinf(v), np.isneginf(v)))
    o = np.where(up, np.inf, np.where(down, -np.inf, o))
    return np.where(nan | (up & down), np.nan, o)


@pytest.mark.parametrize("G,Lq,off", [(1, 300, 0), (2, 333, 70), (8, 300, 0), (48, 70, 200), (128, 40, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (1, 1), (40, 0), (64, 16), (100, 17), (150, 70)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_alone(cuda_ok, G, Lq, off, window, sinks):
    """Anywhere, many of them, and in keys that no query sees: the other outputs do not change by a bit."""
    rng = np.random.default_rng(G + window)
    n = off + Lq
    Lk = n + 50  # keys past the last query
    Q, K, V = _qkv(rng, 1, Lq, 2 * G, 2, Lk)
    want, wlse = rbs.swa_prefill(Q, K, V, window, sinks, q_offset=off, return_lse=True)
    see = S.visible(off + np.arange(Lq), np.arange(Lk), window, sinks)
    values = np.array([np.nan, np.inf, -np.inf])
    few = [(k, int(rng.integers(2)), int(rng.integers(128))) for k in (0, max(0, sinks - 1), sinks, sinks + 5, n // 2, n - 1, n, Lk - 1)]
    many = [(int(k), h, int(d)) for k in rng.integers(0, Lk, 60) for h in range(2) for d in rng.integers(0, 128, 2)]
    whole = [(k, 0, 9) for k in range(Lk)]
    past = [(k, h, d) for k in range(n, Lk) for h in range(2) for d in range(128)]
    for places in (few, many, whole, past):
        W = V.clone()
        k, h, d = (torch.tensor(x, device="cuda") for x in zip(*places))
        W[0, k, h, d] = torch.from_numpy(rng.choice(values, len(places))).to(torch.bfloat16).cuda()
        o, lse = rbs.swa_prefill(Q, K, W, window, sinks, q_offset=off, return_lse=True)
        assert torch.equal(lse, wlse)
        for h in range(2 * G):
            assert np.array_equal(f64(o)[0, :, h], _with_odd_values(f64(want)[0, :, h], see, f64(W)[0, :, h // G]), equal_nan=True)
    assert rbs.rbs_get_device_error() == 0


def _time(f):
    took = []
    for i in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        took.append(a.elapsed_time(b))
    return sorted(took[3:])[2]


def test_a_value_that_every_row_of_a_very_long_prompt_sees_costs_nothing(cuda_ok):
    """A NaN and an infinity among the first keys of 131,072 tokens, and a dim of infinities alone: rows that see them are
    not finite there, every other output is what it was, in about the same time."""
    rng = np.random.default_rng(48)
    Q, K, V = _qkv(rng, 1, 131072, 4, 1)
    want, wlse = rbs.swa_prefill(Q, K, V, 0, return_lse=True)
    clean = _time(lambda: rbs.swa_prefill(Q, K, V, 0))
    V[0, 0, 0, 3] = float("nan")
    V[0, 5, 0, 7] = float("inf")
    V[..., 9] = float("-inf")
    o, lse = rbs.swa_prefill(Q, K, V, 0, return_lse=True)
    odd = _time(lambda: rbs.swa_prefill(Q, K, V, 0))
    assert rbs.rbs_get_device_error() == 0
    assert torch.isnan(o[..., 3]).all() and torch.isposinf(o[:, 5:, :, 7]).all() and torch.isneginf(o[..., 9]).all()
    o[..., [3, 9]] = want[..., [3, 9]]
    o[:, 5:, :, 7] = want[:, 5:, :, 7]
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    assert odd < 1.5 * clean, (odd, clean)
