"""The serving calls' native marshalling against the Python code behind it: the
same outputs, layouts and errors, on a stream of its own and with given outputs."""

import numpy as np
import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from serving_helpers import ints, randn

pytestmark = pytest.mark.gpu


class _Nothing:
    """A marshalling module that leaves every call to the Python code."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture
def both(monkeypatch):
    """Runs a call through the native marshalling, then through the Python code alone."""
    def run(f):
        real, used = rbs.fast(), []

        class Spy:
            def __getattr__(self, name):
                def g(*a):
                    r = getattr(real, name)(*a)
                    used.append(r is not None)
                    return r
                return g
        monkeypatch.setattr(rbs, "fast", lambda: Spy())
        a = f()
        assert used and all(used)  # the native way was taken
        monkeypatch.setattr(rbs, "fast", lambda: _Nothing())
        b = f()
        monkeypatch.setattr(rbs, "fast", lambda: real)
        return a, b
    return run


def _same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y) and x.dtype == y.dtype and x.stride() == y.stride() and not x.requires_grad


def test_same_results_and_layouts(cuda_ok, both):
    rng = np.random.default_rng(1)
    qkv = randn(rng, 2, 40, 12, 128)
    Q, K, V = qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:]
    w = torch.nn.Parameter(randn(rng, 128), requires_grad=False)
    for pos in (ints(np.arange(40)), ints(np.arange(80).reshape(2, 40))):
        for ww in (w, None):
            _same(*both(lambda: rbs.rope_qk_norm(Q, K, ww, w, pos, 1e4, rope_style=1)))
    swapped = randn(rng, 2, 8, 40, 128).transpose(1, 2)  # heads outside tokens
    _same(*both(lambda: rbs.rope_qk_norm(swapped, K, w, w, pos, 10000, 0)))
    for kw in ({}, dict(return_lse=True), dict(softmax_scale=0.3, sinks=2, q_offset=3)):
        _same(*both(lambda: rbs.swa_prefill(Q, K, V, 9, **kw)))
    page, table = 16, ints(np.arange(8).reshape(2, 4))
    cache = rbs.KV4Cache.empty(9, page, 2)
    lens, slots = ints([40, 33]), ints(np.arange(80).reshape(2, 40) % 128)

    def write():
        cache.data.zero_()
        rbs.kv4_append(cache, K, V, slots)
        return cache.data.clone()
    _same(*both(write))
    _same(*both(lambda: rbs.kv4_load(cache, slots)))
    for kw in ({}, dict(return_lse=True, window=7, sinks=1), dict(starts=ints([0, 1]), softmax_scale=1.0)):
        _same(*both(lambda: rbs.kv4_attend(Q, cache, table, lens, **kw)))
    _same(*both(lambda: rbs.kv4_attend(Q[:1], cache, table[:1, :3], lens[:1])))
    _same(*both(lambda: rbs.kv4_extend(table.clone(), ints([20, 0]), lens, ints(np.arange(20)), ints([3]), 40, page)))


def test_given_outputs_are_returned(cuda_ok, both):
    rng = np.random.default_rng(2)
    Q, K = randn(rng, 1, 5, 4, 128), randn(rng, 1, 5, 2, 128)
    pos, q, k = ints(np.arange(5)), torch.empty_like(Q), torch.empty_like(K)
    for got in both(lambda: rbs.rope_qk_norm(Q, K, None, None, pos, 1e4, q_out=q, k_out=k)):
        assert got[0] is q and got[1] is k
    for got in both(lambda: rbs.swa_prefill(Q, K, K, 3, out=q)):
        assert got is q
    cache = rbs.KV4Cache.empty(2, 16, 2)
    ws = torch.empty(rbs.rbs_kv4_attend_workspace_bytes(5, 4, 2), dtype=torch.uint8, device="cuda")
    for got in both(lambda: rbs.kv4_attend(Q, cache, ints([[0]]), ints([0]), out=q, workspace=ws)):
        assert got is q and not q.any()
    for got in both(lambda: rbs.kv4_load(cache, ints([[0] * 5]), k_out=k)):
        assert got[0] is k


def test_same_errors(cuda_ok):
    """Both ways refuse alike: arguments the library refuses, and those the binding does."""
    rng = np.random.default_rng(3)
    Q, K = randn(rng, 1, 4, 4, 128), randn(rng, 1, 4, 2, 128)
    pos, cache = ints(np.arange(4)), rbs.KV4Cache.empty(2, 16, 2)
    t, n = ints([[0]]), ints([1])
    real = rbs.fast
    for f, e in ((lambda: rbs.rope_qk_norm(Q, K, None, None, pos, -1.0), rbs.RbsError),
                 (lambda: rbs.rope_qk_norm(Q, K, None, None, pos.long(), 1e4), TypeError),
                 (lambda: rbs.rope_qk_norm(Q, K, None, None, pos[:3], 1e4), ValueError),
                 (lambda: rbs.rope_qk_norm(Q, K, Q[0, 0, 0, :64], None, pos, 1e4), ValueError),
                 (lambda: rbs.rope_qk_norm(Q.float(), K, None, None, pos, 1e4), TypeError),
                 (lambda: rbs.swa_prefill(Q, K, K[:, :3], 4), rbs.RbsError),
                 (lambda: rbs.swa_prefill(Q, K, K, -1), rbs.RbsError),
                 (lambda: rbs.swa_prefill(Q, K, K.cpu(), 4), TypeError),
                 (lambda: rbs.kv4_append(cache, Q, Q, pos[None]), rbs.RbsError),
                 (lambda: rbs.kv4_append(rbs.KV4Cache(cache.data, 32), K, K, pos[None]), ValueError),
                 (lambda: rbs.kv4_append(rbs.KV4Cache(cache.data, 16, 3.0), K, K, pos[None]), rbs.RbsError),
                 (lambda: rbs.kv4_append(cache, K, K, pos), ValueError),
                 (lambda: rbs.kv4_load(cache, pos), TypeError),
                 (lambda: rbs.kv4_attend(Q, cache, t, n, window=-2), rbs.RbsError),
                 (lambda: rbs.kv4_attend(Q, cache, t.long(), n), TypeError),
                 (lambda: rbs.kv4_attend(Q, cache, t, ints([1, 1])), ValueError),
                 (lambda: rbs.kv4_attend(Q, cache, t, n, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), rbs.RbsError),
                 (lambda: rbs.kv4_extend(t, n, n, pos, n, 0, 16), rbs.RbsError),
                 (lambda: rbs.kv4_extend(t, n, n, pos, n, 1, 17), rbs.RbsError),
                 (lambda: rbs.kv4_extend(t, n, n, pos, n, 1, 16, free_head_out=n), rbs.RbsError),
                 (lambda: rbs.kv4_extend(t[0], n, n, pos, n, 1, 16), TypeError)):
        for way in (real, lambda: _Nothing()):
            rbs.fast = way
            try:
                with pytest.raises(e):
                    f()
            finally:
                rbs.fast = real


def test_threads(cuda_ok):
    """Calls from several threads at once, each on its own stream."""
    import threading

    rng = np.random.default_rng(4)
    cache, table = rbs.KV4Cache.empty(8, 16, 2), ints(np.arange(8).reshape(2, 4))
    K = randn(rng, 2, 64, 2, 128)
    rbs.kv4_append(cache, K, K, ints(np.arange(128).reshape(2, 64)))
    Q = [randn(rng, 2, 3, 8, 128) for _ in range(4)]
    lens, pos = ints([64, 50]), ints([7, 8, 9])

    def chain(q):
        x, _ = rbs.rope_qk_norm(q, K[:, :3], None, None, pos, 1e4)
        return rbs.kv4_attend(x, cache, table, lens, return_lse=True)
    want = [chain(q) for q in Q]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    o, z = chain(Q[i])
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(o, want[i][0]) and torch.equal(z, want[i][1])):
                        wrong.append(i)
        except Exception as e:  # a thread's own would be lost
            wrong.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong
