"""Refusals of the serving operators before any launch (no GPU): through the
C ABI with made-up addresses, and in the Python binding with host tensors."""

import ctypes

import pytest
import torch

import block_sparse_long_rbs_b200 as rbs
from block_sparse_long_rbs_b200 import _abi

INVALID, UNSUPPORTED, CAPACITY, CUDA = 1, 2, 3, 4  # CUDA: past every check, no GPU here


@pytest.fixture(scope="module")
def L():
    from block_sparse_long_rbs_b200 import build
    build.build()
    return _abi.lib()


def _fake(B=2, L=8, H=4, D=128, ptr=0x10000, ss=None):
    ss = H * D if ss is None else ss
    return _abi.Bf16Tensor(ptr, B, L, H, D, L * ss, ss, D)


def _cache(**kw):
    f = dict(data=0x40000, num_pages=10, kv_heads=2, page_size=64, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return _abi.KV4CacheC(*f.values())


def test_rope_qk_norm(L):
    def call(q=None, qo=None, k=None, ko=None, wq=0x1000, wk=0x2000, eps=1e-6, pos=0x3000, pb=0, theta=1e4, style=0):
        q, k = q or _fake(H=8), k or _fake(ptr=0x20000)
        return L.rope_qk_norm(q, qo or q, k, ko or k, wq, wk, eps, pos, pb, theta, style, None)
    assert call() == CUDA
    assert call(wq=None, wk=None, pb=8, style=1, eps=0.0) == CUDA
    assert call(q=_fake(H=8, D=64)) == UNSUPPORTED
    assert call(q=_fake(H=8, ptr=None)) == INVALID
    assert call(qo=_fake(H=4)) == INVALID
    assert call(ko=_fake(L=7)) == INVALID
    assert call(k=_fake(L=7)) == INVALID  # other tokens than the queries'
    assert call(qo=_fake(H=8, ss=8 * 128 + 8)) == INVALID  # in place with other strides
    assert call(wq=0x1008) == INVALID
    assert call(pos=None) == INVALID
    assert call(pb=7) == INVALID
    for bad in (float("nan"), float("inf"), -1.0):
        assert call(eps=bad) == INVALID
        assert call(theta=bad) == INVALID
    assert call(theta=0.0) == INVALID
    assert call(style=2) == INVALID
    assert call(q=_fake(H=8, ss=8 * 128 + 4)) == INVALID


def test_page_bytes(L):
    assert [rbs.rbs_kv4_page_bytes(p) for p in (16, 48, 256)] == [2304, 3 * 2304, 16 * 2304]
    for bad in (0, -16, 8, 24, 272):
        with pytest.raises(rbs.RbsError, match="page_size"):
            rbs.rbs_kv4_page_bytes(bad)


def test_cache_and_slots(L):
    for f in (lambda c, k, v, s: L.kv4_append(c, k, v, s, None), lambda c, k, v, s: L.kv4_load(c, s, k, v, None)):
        k = _fake(H=2)
        assert f(_cache(), k, k, 0x1000) == CUDA
        assert f(_cache(data=None), k, k, 0x1000) == INVALID
        assert f(_cache(data=0x40008), k, k, 0x1000) == INVALID
        assert f(_cache(num_pages=0), k, k, 0x1000) == INVALID
        assert f(_cache(kv_heads=4), k, k, 0x1000) == INVALID
        assert f(_cache(page_size=24), k, k, 0x1000) == UNSUPPORTED
        assert f(_cache(page_size=512), k, k, 0x1000) == UNSUPPORTED
        assert f(_cache(num_pages=(1 << 31) // 64), k, k, 0x1000) == UNSUPPORTED
        assert f(_cache(num_pages=(1 << 31) // 64 - 1), k, k, 0x1000) == CUDA
        for bad in (0.0, -1.0, 3.0, float("nan"), float("inf"), 2.0 ** 65, 2.0 ** -65):
            assert f(_cache(k_scale=bad), k, k, 0x1000) == INVALID
            assert f(_cache(v_scale=bad), k, k, 0x1000) == INVALID
        assert f(_cache(k_scale=2.0 ** -64, v_scale=2.0 ** 64), k, k, 0x1000) == CUDA
        assert f(_cache(), k, _fake(H=2, L=9), 0x1000) == INVALID
        assert f(_cache(), k, k, None) == INVALID


def test_extend(L):
    base = dict(table=0x1000, stride=4, B=3, width=4, old=0x2000, new=0x3000, free=0x4000, n=9, head=0x5000, page=16,
                max_new=5, slots=0x6000, pos=0x7000, out=0x8000)

    def call(**kw):
        return L.kv4_extend(*{**base, **kw}.values(), None)
    assert call() == CUDA
    for p in ("table", "old", "new", "free", "head", "slots", "pos", "out"):
        assert call(**{p: None}) == INVALID
    for p in ("B", "width", "n", "max_new"):
        assert call(**{p: 0}) == INVALID
    assert call(stride=3) == INVALID
    assert call(out=0x5000) == INVALID  # the count is read by every block while one writes it
    assert call(page=20) == UNSUPPORTED
    assert call(page=256, width=1 << 23, stride=1 << 23) == UNSUPPORTED
    assert call(n=1 << 31) == UNSUPPORTED


def test_attend(L):
    need = rbs.rbs_kv4_attend_workspace_bytes(2, 8, 2)
    assert need > 0 and rbs.rbs_kv4_attend_workspace_bytes(1, 7, 2) == 0

    def call(q=None, o=None, c=None, table=0x1000, stride=4, width=4, lens=0x2000, starts=None, window=0, sinks=0,
             scale=0.0, ws=0x50000, n=need, lse=None):
        q = q or _fake(L=2, H=8)
        return L.kv4_attend(q, c or _cache(), table, stride, width, lens, starts, window, sinks, scale, ws, n,
                            o or _fake(L=2, H=8, ptr=0x20000), lse, None)
    assert call() == CUDA
    assert call(starts=0x3000, window=5, sinks=3, scale=0.5, lse=0x9000) == CUDA
    assert call(o=_fake(L=3, H=8)) == INVALID
    assert call(c=_cache(kv_heads=3)) == INVALID
    assert call(c=_cache(page_size=40)) == UNSUPPORTED
    assert call(table=None) == INVALID and call(lens=None) == INVALID
    assert call(width=0) == INVALID and call(stride=3) == INVALID
    assert call(window=-1) == INVALID and call(sinks=-1) == INVALID
    assert call(scale=float("nan")) == INVALID
    assert call(ws=None) == INVALID and call(ws=0x50008) == INVALID
    assert call(n=need - 1) == CAPACITY
    big = dict(B=4097, L=2, H=8)
    assert call(q=_fake(**big), o=_fake(**big)) == UNSUPPORTED
    assert call(width=1 << 25, stride=1 << 25) == UNSUPPORTED
    assert call(q=_fake(L=2, H=8, D=64)) == UNSUPPORTED


def test_swa(L):
    def call(q=None, k=None, v=None, o=None, window=4, sinks=1, off=0, scale=0.0, lse=None):
        k = k or _fake(H=2, ptr=0x20000)
        return L.swa_prefill(q or _fake(), k, v or k, window, sinks, off, scale, o or _fake(ptr=0x30000), lse, None)
    assert call() == CUDA
    assert call(window=0, sinks=0, off=77, scale=0.5, lse=0x9000) == CUDA
    assert call(window=(1 << 31) - 1, sinks=(1 << 31) - 1) == CUDA
    assert call(k=_fake(B=1, H=2)) == INVALID
    assert call(v=_fake(L=7, H=2)) == INVALID
    assert call(o=_fake(L=7)) == INVALID
    assert call(k=_fake(H=3)) == INVALID
    assert call(window=-1) == INVALID and call(sinks=-1) == INVALID and call(off=-1) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(off=(1 << 31) - 8) == UNSUPPORTED
    assert call(q=_fake(H=129), o=_fake(H=129), k=_fake(H=1)) == UNSUPPORTED
    swapped = _abi.Bf16Tensor(0x20000, 2, 8, 2, 128, 2048, 128, 1024)  # heads outside tokens
    assert call(k=swapped) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    cache = rbs.KV4Cache(torch.zeros(3, 4, 2304, dtype=torch.uint8), 16)
    with pytest.raises(TypeError, match="CUDA"):
        rbs.rope_qk_norm(q, q, None, None, i, 1e4)
    with pytest.raises(TypeError, match="CUDA"):
        rbs.swa_prefill(q, q, q, 4)
    with pytest.raises(TypeError, match="CUDA"):
        rbs.kv4_append(cache, q, q, i)
    with pytest.raises(TypeError, match="CUDA"):
        rbs.kv4_load(cache, i)
    with pytest.raises(TypeError, match="CUDA"):
        rbs.kv4_attend(q, cache, i, i[0])
    with pytest.raises(TypeError, match="CUDA"):
        rbs.kv4_extend(i, i[0, :1], i[0, :1], i[0], i[0, :1], 1, 16)


def test_binding_refuses_shapes_and_types():
    dev = torch.device("cpu")
    i = torch.zeros(2, 3, dtype=torch.int32)
    assert rbs._ints(i, "x", dev, 2, 3) == i.data_ptr()
    with pytest.raises(ValueError, match="x: expected shape"):
        rbs._ints(i, "x", dev, 6)
    with pytest.raises(TypeError, match="x: expected a contiguous int32"):
        rbs._ints(i.long(), "x", dev, 2, 3)
    with pytest.raises(TypeError, match="x: expected a contiguous int32"):
        rbs._ints(i.t(), "x", dev, 3, 2)
    with pytest.raises(TypeError, match="torch.Tensor"):
        rbs._ints([0], "x", dev, 1)
    with pytest.raises(ValueError, match="one device"):
        rbs._ints(i, "x", torch.device("cuda", 0), 2, 3)
    wide = torch.zeros(2, 8, dtype=torch.int32)
    assert rbs._table(wide[:, :3], "t", dev, 2) == (wide.data_ptr(), 8, 3)
    with pytest.raises(TypeError, match="contiguous rows"):
        rbs._table(wide.t(), "t", dev, 8)
    with pytest.raises(ValueError, match="rows"):
        rbs._table(wide, "t", dev, 3)


def test_native_marshalling_leaves_odd_arguments_alone(L):
    """What is not plainly a call's argument (host tensors, other types, wrong counts) comes back as None, undone."""
    f = _abi.fast()
    q = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    i, data = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(3, 4, 2304, dtype=torch.uint8)
    assert f.rope_qk_norm(q, q, None, None, i, 1e4, 1e-6, 0, None, None) is None
    assert f.rope_qk_norm(q, "k", None, None, i, 1e4, 1e-6, 0, None, None) is None
    assert f.rope_qk_norm(q, q) is None
    assert f.swa_prefill(q, q, q, 4, 0, 0, None, None, False) is None
    assert f.swa_prefill(q, q, q, 4, 0, 0, None, None, "yes") is None
    assert f.kv4_extend(i, i[0, :1], i[0, :1], i[0], i[0, :1], 1, 16, None, None, None) is None
    assert f.kv4_append(data, 16, 1.0, 1.0, q, q, i) is None
    assert f.kv4_append([], 16, 1.0, 1.0, q, q, i) is None
    assert f.kv4_load(data, 16, 1.0, 1.0, i, None, None) is None
    assert f.kv4_attend(data, 16, 1.0, 1.0, q, i, i[0, :1], None, 0, 0, None, None, True, None) is None
    assert f.kv4_attend() is None
    with pytest.raises(TypeError, match="seven"):
        f.bind(1, 2)
    with pytest.raises(ValueError, match="null"):
        f.bind(*[0] * 7)


def test_binding_integers():
    """Integers that their C type does not hold are refused, and windows and sinks past 32 bits reach every key."""
    assert rbs._i32(-2 ** 31, "x") == -2 ** 31 and rbs._i32(2 ** 31 - 1, "x") == 2 ** 31 - 1
    assert rbs._i64(-2 ** 63, "x") == -2 ** 63 and rbs._i64(2 ** 63 - 1, "x") == 2 ** 63 - 1
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 5, 2 ** 64):
        with pytest.raises(ValueError, match="x: .* 32 bits"):
            rbs._i32(bad, "x")
    for bad in (2 ** 63, -2 ** 63 - 1, 2 ** 64 + 5):
        with pytest.raises(ValueError, match="x: .* 64 bits"):
            rbs._i64(bad, "x")
    for f in (rbs._i32, rbs._i64, rbs._reach):
        with pytest.raises(TypeError, match="x: expected an integer"):
            f(4.0, "x")
    assert [rbs._reach(n, "x") for n in (0, 7, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 128, 2 ** 64)] == [0, 7] + [2 ** 31 - 1] * 4
    assert all(rbs._reach(n, "x") < 0 for n in (-1, -2 ** 31 - 1, -2 ** 32 + 7, -2 ** 64))  # the library refuses them
    for bad in (2 ** 32 + 64, -2 ** 32 + 64):
        with pytest.raises(ValueError, match="page_size"):
            rbs.rbs_kv4_page_bytes(bad)
        with pytest.raises(ValueError, match="page_size"):
            rbs.KV4Cache.empty(1, bad, 1, device="cpu")
    for sizes in ((2 ** 64 + 1, 8, 2), (1, 2 ** 64 + 8, 2), (1, 8, 2 ** 64 + 2)):
        with pytest.raises(ValueError, match="64 bits"):
            rbs.rbs_kv4_attend_workspace_bytes(*sizes)
