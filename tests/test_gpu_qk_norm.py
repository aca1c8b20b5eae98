"""GPU parity of rope_qk_norm with the fp64 oracle."""

import numpy as np
import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from helpers import host_bits
from oracle import serving_oracle as S
from serving_helpers import BF16, assert_within, f64, ints, randn

pytestmark = pytest.mark.gpu

# fp32 between the roundings: the mean of squares, its root and the two
# products are within 2^-20 of the pair's size, the angle within 2^-22
SLACK = 2.0 ** -19


def _check(Q, K, wq, wk, pos, theta, eps, style, out):
    p = np.broadcast_to(pos, (Q.shape[0], Q.shape[1]))
    for x, w, y, what in ((Q, wq, out[0], "q"), (K, wk, out[1], "k")):
        ref, size = S.qk_norm_rope(host_bits(x), None if w is None else host_bits(w), p, theta, eps, style)
        assert_within(f64(y), ref, BF16 * np.abs(ref) + SLACK * size, what)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("B,L,Hq,Hkv", [(1, 1, 1, 1), (3, 1, 32, 4), (2, 77, 5, 5), (1, 300, 7, 1), (70, 2, 9, 3)])
def test_matches_oracle(cuda_ok, B, L, Hq, Hkv, style):
    rng = np.random.default_rng(B * 100 + L + style)
    qkv = randn(rng, B, L, Hq + 2 * Hkv, 128, scale=3.0)
    Q, K = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]  # views of a packed projection
    wq, wk = randn(rng, 128), randn(rng, 128)
    pos = rng.integers(0, 1 << 20, (B, L))
    out = rbs.rope_qk_norm(Q, K, wq, wk, ints(pos), 500000.0, rope_style=style)
    _check(Q, K, wq, wk, pos, 500000.0, 1e-6, style, out)


@pytest.mark.parametrize("style", [0, 1])
def test_positions_weights_eps(cuda_ok, style):
    """Positions to both ends of int32, shared by the batch; no weights; a large eps; zero rows."""
    rng = np.random.default_rng(7)
    pos = np.array([0, 1, 131071, (1 << 31) - 1, -(1 << 31), -5, 12345678])
    Q, K = randn(rng, 2, pos.size, 4, 128, scale=1e-3), randn(rng, 2, pos.size, 2, 128, scale=100.0)
    Q[0, 2, 1] = 0
    for wq, wk, eps in ((None, randn(rng, 128), 1e-5), (randn(rng, 128), None, 0.5)):
        out = rbs.rope_qk_norm(Q, K, wq, wk, ints(pos), 10000.0, eps=eps, rope_style=style)
        _check(Q, K, wq, wk, pos[None], 10000.0, eps, style, out)
        assert not f64(out[0])[0, 2, 1].any()


def test_in_place_and_given_outputs(cuda_ok):
    rng = np.random.default_rng(9)
    qkv = randn(rng, 2, 33, 12, 128)
    wq, wk, pos = randn(rng, 128), randn(rng, 128), ints(np.arange(33) + 5)
    want = rbs.rope_qk_norm(qkv[:, :, :8], qkv[:, :, 8:10], wq, wk, pos, 1e5)
    # outputs with a batch stride and a head order of their own
    hold = torch.full((2, 8, 40, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = hold.permute(0, 2, 1, 3)[:, :33]
    got = rbs.rope_qk_norm(qkv[:, :, :8], qkv[:, :, 8:10], wq, wk, pos, 1e5, q_out=q_out)
    assert got[0] is q_out and torch.equal(q_out, want[0]) and torch.equal(got[1], want[1])
    assert (hold[:, :, 33:] == 7).all()
    rest = qkv[:, :, 10:].clone()
    q, k = qkv[:, :, :8], qkv[:, :, 8:10]
    rbs.rope_qk_norm(q, k, wq, wk, pos, 1e5, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 10:], rest)


def test_agrees_with_rope_reencode(cuda_ok):
    """Keys normed and rotated to p, then moved by rope_reencode, are the keys normed and rotated to where they went:
    one more rounding of each value and of its pair's other member."""
    rng = np.random.default_rng(10)
    K, w = randn(rng, 1, 64, 2, 128), randn(rng, 128)
    a, b = ints(np.arange(64)), ints(np.arange(64) + 4321)
    at_a = rbs.rope_qk_norm(K, K, w, w, a, 5e5)[1]
    at_b = rbs.rope_qk_norm(K, K, w, w, b, 5e5)[1]
    moved = rbs.rope_reencode(at_a, a, b, 5e5)
    ref, size = S.qk_norm_rope(host_bits(K), host_bits(w), np.arange(64)[None] + 4321, 5e5, 1e-6)
    tol = BF16 * np.abs(ref) + (BF16 + SLACK) * size
    assert_within(f64(moved), ref, tol * (1 + BF16), "moved")
    assert_within(f64(at_b), ref, BF16 * np.abs(ref) + SLACK * size, "direct")


def test_nan_and_infinity_stay_in_their_row(cuda_ok):
    rng = np.random.default_rng(11)
    Q, K = randn(rng, 1, 8, 4, 128), randn(rng, 1, 8, 4, 128)
    pos = ints(np.arange(8))
    want = rbs.rope_qk_norm(Q, K, None, None, pos, 1e4)[0]
    Q[0, 3, 1, 17], Q[0, 5, 2, 100] = float("nan"), float("inf")
    got = rbs.rope_qk_norm(Q, K, None, None, pos, 1e4)[0]
    hit = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    hit[3, 1] = hit[5, 2] = True
    assert torch.equal(got[0][~hit], want[0][~hit])
    assert got[0, 3, 1].isnan().all() and got[0, 5, 2, [36, 100]].isnan().all()


def test_stream_and_graph(cuda_ok):
    rng = np.random.default_rng(12)
    Q, K, w = randn(rng, 2, 40, 8, 128), randn(rng, 2, 40, 2, 128), randn(rng, 128)
    pos = ints(np.arange(80).reshape(2, 40))
    want = rbs.rope_qk_norm(Q, K, w, w, pos, 1e4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = rbs.rope_qk_norm(Q, K, w, w, pos, 1e4)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = rbs.rope_qk_norm(Q, K, w, w, pos, 1e4)
    for shift in (0, 1000):
        pos += shift
        Q.neg_()
        g.replay()
        want = rbs.rope_qk_norm(Q, K, w, w, pos, 1e4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
