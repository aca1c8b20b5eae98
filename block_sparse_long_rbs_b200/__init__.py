"""Block-sparse prefill attention with radius-bounded block selection (RBS)
and the Block-attention mask, on NVIDIA B200 (sm_100a).

A thin binding over the C ABI of librbs (include/rbs.h): argument
marshalling only.  Torch tensors supply device memory and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels.
Functions carry the same names as the C entry points.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import operator

import torch

from ._abi import (  # noqa: F401
    DEVERR_BLOCK_INDEX,
    DEVERR_LENGTH,
    DEVERR_NONCAUSAL,
    DEVERR_PAGES,
    DEVERR_ROW_PTR,
    DEVERR_SLOT,
    DEVERR_TIMEOUT,
    MAX_KV_BLOCKS,
    BlockListsC,
    Bf16Tensor,
    KV4CacheC,
    RbsError,
    SelectParamsC,
    check,
    fast,
    lib,
)

__all__ = [
    "SelectParams", "BlockLists", "rbs_block_stats", "rbs_block_beta", "rbs_pool_queries", "rbs_select",
    "rbs_select_capacity", "rbs_select_workspace_bytes", "rbs_lists_causal_full", "rbs_lists_block_attention",
    "bsa_prefill", "bsa_prefill_rescue_weighted", "bsa_prefill_segments", "rope_reencode", "rbs_get_device_error",
    "rope_qk_norm", "swa_prefill", "KV4Cache", "rbs_kv4_page_bytes", "kv4_extend", "kv4_append", "kv4_load", "kv4_attend",
    "rbs_kv4_attend_workspace_bytes", "RbsError",
]


@dataclasses.dataclass
class SelectParams:
    """Selection parameters (field meanings and defaults as in include/rbs.h)."""

    block_q: int = 128
    block_k: int = 128
    rho_centroid: float = 0.05
    rho_rescue: float = 0.05
    beta_mode: int = 0
    beta_const: float = 1.0
    beta_p_lo: float = 0.0
    beta_p_hi: float = 1.0
    force_diag: int = 1
    force_sink: int = 0
    causal: int = 1
    q_block_offset: int = 0
    threshold_mode: int = 0  # 0 = top-k fraction, 1 = within delta of the row maximum
    delta_centroid: float = 0.0
    delta_rescue: float = 0.0
    list_mode: int = 0  # 0 = one list per q head, 1 = one per KV head (union of its q heads)
    query_pool: int = 0  # 0 = mean query of the block, 1 = best query token of the block

    def c(self) -> SelectParamsC:
        return SelectParamsC(*[getattr(self, f.name) for f in dataclasses.fields(self)])


@dataclasses.dataclass
class BlockLists:
    """CSR key-block lists on the device: one row per (batch, q head, query block)."""

    row_ptr: torch.Tensor  # int32 [num_rows + 1]
    col_idx: torch.Tensor  # int32 [capacity]
    flags: torch.Tensor | None  # uint8 [capacity]
    num_rows: int

    def c(self) -> BlockListsC:
        # the kernels write row_ptr[0 .. num_rows] and col_idx / flags up to
        # the capacity: every buffer must be a contiguous CUDA tensor that long
        if self.row_ptr.numel() < self.num_rows + 1:
            raise ValueError(f"lists.row_ptr: {self.row_ptr.numel()} entries for {self.num_rows} rows")
        if self.flags is not None and self.flags.numel() < self.col_idx.numel():
            raise ValueError(f"lists.flags: {self.flags.numel()} entries, capacity {self.col_idx.numel()}")
        _dev(self.row_ptr, "lists.row_ptr", torch.int32)
        _dev(self.col_idx, "lists.col_idx", torch.int32)
        if self.flags is not None:
            _dev(self.flags, "lists.flags", torch.uint8)
        return BlockListsC(self.row_ptr.data_ptr(), self.col_idx.data_ptr(),
                           self.flags.data_ptr() if self.flags is not None else None,
                           self.col_idx.numel(), self.num_rows)

    def nnz(self) -> int:
        return int(self.row_ptr[-1].item())

    @staticmethod
    def empty(num_rows: int, capacity: int, device, flags: bool = True) -> "BlockLists":
        return BlockLists(torch.empty(num_rows + 1, dtype=torch.int32, device=device),
                          torch.empty(max(1, capacity), dtype=torch.int32, device=device),
                          torch.empty(max(1, capacity), dtype=torch.uint8, device=device) if flags else None,
                          num_rows)


def _dev(x, name: str, dtype: torch.dtype) -> int:
    """Check a contiguous CUDA tensor of the given dtype and return its
    device pointer."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not x.is_cuda or x.dtype != dtype or not x.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} CUDA tensor")
    return x.data_ptr()


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _one_device(ref_name: str, ref, **others) -> torch.device:
    """The device every tensor of one call must live on (ref's).  The library
    launches on the current device and its current stream, so a tensor on
    another GPU would hand a kernel a pointer it cannot use: refuse it here.
    None entries (optional arguments) are skipped."""
    dev = ref.device
    for name, x in others.items():
        if x is not None and x.device != dev:
            raise ValueError(f"{name} is on {x.device} but {ref_name} is on {dev}: "
                             "every tensor of a call must be on one device")
    return dev


def _lists_tensors(lists) -> dict:
    return {"lists.row_ptr": lists.row_ptr, "lists.col_idx": lists.col_idx, "lists.flags": lists.flags}


def _t(x: torch.Tensor, name: str) -> Bf16Tensor:
    """Describe a [B, L, H, 128] bf16 CUDA tensor (head_dim contiguous) for the C ABI."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if x.dtype != torch.bfloat16 or x.dim() != 4 or x.stride(3) != 1:
        raise TypeError(f"{name}: expected bf16 [B, L, H, 128] with a contiguous last dimension")
    B, L, H, D = x.shape
    return Bf16Tensor(x.data_ptr(), B, L, H, D, x.stride(0), x.stride(1), x.stride(2))


def _f32(x: torch.Tensor, name: str) -> int:
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous float32 CUDA tensor")
    return x.data_ptr()


def rbs_block_stats(K: torch.Tensor, block_k: int):
    """Centroids [B, Hkv, nKB, 128] and radii [B, Hkv, nKB] (fp32) of every key block."""
    B, L, H, D = K.shape
    nkb = -(-L // block_k)  # a last, partial block holds the remaining keys
    C = torch.empty(B, H, nkb, D, dtype=torch.float32, device=K.device)
    R = torch.empty(B, H, nkb, dtype=torch.float32, device=K.device)
    tK = _t(K, "K")
    with torch.cuda.device(K.device):
        check(lib().rbs_block_stats(ctypes.byref(tK), block_k, C.data_ptr(), R.data_ptr(), _stream()),
              "rbs_block_stats")
    return C, R


def rbs_block_beta(radii: torch.Tensor, params: SelectParams):
    """beta [B, Hkv, nKB] and the (R_lo, R_hi) range [B, Hkv, 2] from the radii."""
    B, H, n = radii.shape
    beta = torch.empty_like(radii)
    rng = torch.empty(B, H, 2, dtype=torch.float32, device=radii.device)
    p = params.c()
    r_ptr = _f32(radii, "radii")
    with torch.cuda.device(radii.device):
        check(lib().rbs_block_beta(r_ptr, B, H, n, ctypes.byref(p), beta.data_ptr(), rng.data_ptr(), _stream()),
              "rbs_block_beta")
    return beta, rng


def rbs_pool_queries(Q: torch.Tensor, block_q: int):
    """qbar [B, Hq, nQB, 128] and qnorm [B, Hq, nQB] (fp32)."""
    B, L, H, D = Q.shape
    nqb = -(-L // block_q)
    qbar = torch.empty(B, H, nqb, D, dtype=torch.float32, device=Q.device)
    qnorm = torch.empty(B, H, nqb, dtype=torch.float32, device=Q.device)
    tQ = _t(Q, "Q")
    with torch.cuda.device(Q.device):
        check(lib().rbs_pool_queries(ctypes.byref(tQ), block_q, qbar.data_ptr(), qnorm.data_ptr(), _stream()),
              "rbs_pool_queries")
    return qbar, qnorm


def rbs_select_capacity(batch: int, heads_q: int, num_q_blocks: int, num_kv_blocks: int, params: SelectParams) -> int:
    p = params.c()
    return int(lib().rbs_select_capacity(batch, heads_q, num_q_blocks, num_kv_blocks, ctypes.byref(p)))


def rbs_select_workspace_bytes(batch: int, heads_q: int, num_q_blocks: int, kv_heads: int, num_kv_blocks: int,
                               params: SelectParams) -> int:
    p = params.c()
    return int(lib().rbs_select_workspace_bytes(batch, heads_q, num_q_blocks, kv_heads, num_kv_blocks,
                                                ctypes.byref(p)))


def rbs_select(Q: torch.Tensor, centroids: torch.Tensor, radii: torch.Tensor, params: SelectParams,
               workspace: torch.Tensor | None = None, out: BlockLists | None = None, beta_out: torch.Tensor | None = None,
               flags: bool = True) -> BlockLists:
    """Two-branch selection -> CSR key-block lists, rows = (batch, q head, query block), or
    (batch, KV head, query block) when params.list_mode == 1."""
    B, L, Hq, D = Q.shape
    if centroids.dim() != 4:
        raise ValueError(f"centroids: expected [B, Hkv, nKB, {D}], got {tuple(centroids.shape)}")
    Hkv, nkb = centroids.shape[1], centroids.shape[2]
    # every shape first, then where the tensors live
    for x, name, shape in ((centroids, "centroids", (B, Hkv, nkb, D)), (radii, "radii", (B, Hkv, nkb)),
                           (beta_out, "beta_out", (B, Hkv, nkb))):
        if x is not None and tuple(x.shape) != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(x.shape)}")
    c_ptr = _dev(centroids, "centroids", torch.float32)
    r_ptr = _dev(radii, "radii", torch.float32)
    b_ptr = _dev(beta_out, "beta_out", torch.float32) if beta_out is not None else None
    nqb = -(-L // params.block_q)
    rows = B * (Hkv if params.list_mode == 1 else Hq) * nqb
    if out is None:
        out = BlockLists.empty(rows, rbs_select_capacity(B, Hq, nqb, nkb, params), Q.device, flags)
    if workspace is None:
        workspace = torch.empty(rbs_select_workspace_bytes(B, Hq, nqb, Hkv, nkb, params), dtype=torch.uint8,
                                device=Q.device)
    ws_ptr = _dev(workspace, "workspace", torch.uint8)
    p = params.c()
    lc = out.c()
    tQ = _t(Q, "Q")
    dev = _one_device("Q", Q, centroids=centroids, radii=radii, beta_out=beta_out, workspace=workspace,
                      **_lists_tensors(out))
    with torch.cuda.device(dev):
        check(lib().rbs_select(ctypes.byref(tQ), c_ptr, r_ptr, Hkv, nkb, ctypes.byref(p), ws_ptr,
                               workspace.numel(), ctypes.byref(lc), b_ptr, _stream()), "rbs_select")
    return out


def rbs_lists_causal_full(batch: int, heads_q: int, num_q_blocks: int, q_block_offset: int = 0, device="cuda",
                          flags: bool = False) -> BlockLists:
    """Every causally visible block for every row (the dense reference point)."""
    nnz = int(lib().rbs_lists_causal_full_nnz(batch, heads_q, num_q_blocks, q_block_offset))
    out = BlockLists.empty(batch * heads_q * num_q_blocks, nnz, device, flags)
    lc = out.c()
    with torch.cuda.device(out.row_ptr.device):
        check(lib().rbs_lists_causal_full(batch, heads_q, num_q_blocks, q_block_offset, ctypes.byref(lc), _stream()),
              "rbs_lists_causal_full")
    return out


def rbs_lists_block_attention(seg_start, final_start: int, block: int, batch: int, heads_q: int, q_first_block: int,
                              q_num_blocks: int, device="cuda", flags: bool = False) -> BlockLists:
    """Block-attention mask lists (passages self-attend, the final block sees all)."""
    seg = (ctypes.c_int32 * len(seg_start))(*[int(s) for s in seg_start])
    nnz = int(lib().rbs_lists_block_attention_nnz(seg, len(seg_start), final_start, block, batch, heads_q,
                                                  q_first_block, q_num_blocks))
    if nnz < 0:
        raise RbsError(1, "rbs_lists_block_attention_nnz", lib().rbs_last_error().decode())
    out = BlockLists.empty(batch * heads_q * q_num_blocks, nnz, device, flags)
    lc = out.c()
    with torch.cuda.device(out.row_ptr.device):
        check(lib().rbs_lists_block_attention(seg, len(seg_start), final_start, block, batch, heads_q, q_first_block,
                                              q_num_blocks, ctypes.byref(lc), _stream()), "rbs_lists_block_attention")
    return out


def bsa_prefill(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lists: BlockLists, block_q: int = 128,
                block_k: int = 128, q_offset: int = 0, softmax_scale: float | None = None, causal: bool = True,
                out: torch.Tensor | None = None, return_lse: bool = False):
    """Exact softmax attention of every query block over its listed key blocks."""
    if out is None:
        out = torch.empty_like(Q)
    lse = None
    if return_lse:
        lse = torch.empty(Q.shape[0], Q.shape[2], Q.shape[1], dtype=torch.float32, device=Q.device)
    scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(Q.shape[-1])
    lc = lists.c()
    tQ, tK, tV, tO = _t(Q, "Q"), _t(K, "K"), _t(V, "V"), _t(out, "O")
    dev = _one_device("Q", Q, K=K, V=V, out=out, lse=lse, **_lists_tensors(lists))
    with torch.cuda.device(dev):
        check(lib().bsa_prefill(ctypes.byref(tQ), ctypes.byref(tK), ctypes.byref(tV), ctypes.byref(lc), block_q,
                                block_k, q_offset, scale, 1 if causal else 0, ctypes.byref(tO),
                                lse.data_ptr() if lse is not None else None, _stream()), "bsa_prefill")
    return (out, lse) if return_lse else out


def bsa_prefill_rescue_weighted(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lists: BlockLists,
                                rescue_weight: float, block_q: int = 128, block_k: int = 128, q_offset: int = 0,
                                softmax_scale: float | None = None, causal: bool = True,
                                out: torch.Tensor | None = None, return_lse: bool = False):
    """bsa_prefill with the rescue-only blocks' softmax mass scaled by rescue_weight
    (the lists' flags say which entries those are)."""
    if out is None:
        out = torch.empty_like(Q)
    lse = None
    if return_lse:
        lse = torch.empty(Q.shape[0], Q.shape[2], Q.shape[1], dtype=torch.float32, device=Q.device)
    scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(Q.shape[-1])
    lc = lists.c()
    tQ, tK, tV, tO = _t(Q, "Q"), _t(K, "K"), _t(V, "V"), _t(out, "O")
    dev = _one_device("Q", Q, K=K, V=V, out=out, lse=lse, **_lists_tensors(lists))
    with torch.cuda.device(dev):
        check(lib().bsa_prefill_rescue_weighted(
            ctypes.byref(tQ), ctypes.byref(tK), ctypes.byref(tV), ctypes.byref(lc), block_q, block_k, q_offset, scale,
            1 if causal else 0, float(rescue_weight), ctypes.byref(tO), lse.data_ptr() if lse is not None else None,
            _stream()), "bsa_prefill_rescue_weighted")
    return (out, lse) if return_lse else out


def bsa_prefill_segments(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lists: BlockLists, seg_start,
                         final_start: int, block_q: int = 128, block_k: int = 128, q_offset: int = 0,
                         softmax_scale: float | None = None, out: torch.Tensor | None = None,
                         return_lse: bool = False):
    """bsa_prefill with the Block-attention mask applied token by token: a query
    token of a passage sees only its own passage's earlier keys, a token of the
    final block every earlier key (passage starts may be any token offsets)."""
    if out is None:
        out = torch.empty_like(Q)
    lse = None
    if return_lse:
        lse = torch.empty(Q.shape[0], Q.shape[2], Q.shape[1], dtype=torch.float32, device=Q.device)
    scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(Q.shape[-1])
    seg = (ctypes.c_int32 * len(seg_start))(*[int(s) for s in seg_start])
    lc = lists.c()
    tQ, tK, tV, tO = _t(Q, "Q"), _t(K, "K"), _t(V, "V"), _t(out, "O")
    dev = _one_device("Q", Q, K=K, V=V, out=out, lse=lse, **_lists_tensors(lists))
    with torch.cuda.device(dev):
        check(lib().bsa_prefill_segments(ctypes.byref(tQ), ctypes.byref(tK), ctypes.byref(tV), ctypes.byref(lc),
                                         block_q, block_k, q_offset, seg, len(seg_start), int(final_start), scale,
                                         ctypes.byref(tO), lse.data_ptr() if lse is not None else None, _stream()),
              "bsa_prefill_segments")
    return (out, lse) if return_lse else out


def rope_reencode(x: torch.Tensor, old_pos: torch.Tensor, new_pos: torch.Tensor, theta: float, rope_style: int = 0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Move RoPE-encoded vectors from old_pos to new_pos (out may be x for in place)."""
    if out is None:
        out = torch.empty_like(x)
    for name, p in (("old_pos", old_pos), ("new_pos", new_pos)):
        if not p.is_cuda or p.dtype != torch.int32 or p.numel() != x.shape[1]:
            raise TypeError(f"{name}: expected int32 CUDA tensor of length {x.shape[1]}")
    tx, to = _t(x, "x"), _t(out, "out")
    dev = _one_device("x", x, out=out, old_pos=old_pos, new_pos=new_pos)
    with torch.cuda.device(dev):
        check(lib().rope_reencode(ctypes.byref(tx), ctypes.byref(to), old_pos.data_ptr(), new_pos.data_ptr(), theta,
                                  rope_style, _stream()), "rope_reencode")
    return out


# ---- serving: norm and rotation, the 4-bit cache ----------------------------
# These run once per layer and decoding step, where the call itself counts.
# Each first hands its arguments to the native marshalling (csrc/fastcall.cpp),
# which makes the call when they are plainly what it takes, on the current
# device; otherwise the code here checks them one by one, says what is wrong,
# and makes the call on another device.


def _made(result, where: str):
    """What the native marshalling returned: the outputs, or a status that is an error."""
    if type(result) is int:
        check(result, where)
    return result


def _int(x, name: str, bits: int) -> int:
    """An integer that a signed C integer of that many bits holds (ctypes would cut off the rest)."""
    try:
        n = operator.index(x)
    except TypeError:
        raise TypeError(f"{name}: expected an integer") from None
    if not -(1 << bits - 1) <= n < 1 << bits - 1:
        raise ValueError(f"{name}: {n} does not fit {bits} bits")
    return n


def _i32(x, name: str) -> int:
    return _int(x, name, 32)


def _i64(x, name: str) -> int:
    return _int(x, name, 64)


def _reach(x, name: str) -> int:
    """A window or a count of sinks: positions end below 2^31, so what lies past that reaches every key as 2^31 - 1 does
    (and anything negative is left to the library to refuse)."""
    try:
        return max(-1, min(operator.index(x), 2 ** 31 - 1))
    except TypeError:
        raise TypeError(f"{name}: expected an integer") from None


def _b(x, name: str) -> Bf16Tensor:
    """_t with the passing case first."""
    try:
        if x.dtype is torch.bfloat16 and x.is_cuda:
            B, L, H, D = x.shape
            sb, ss, sh, sd = x.stride()
            if sd == 1:
                return Bf16Tensor(x.data_ptr(), B, L, H, D, sb, ss, sh)
    except (AttributeError, ValueError):
        pass
    return _t(x, name)


def _call(dev: torch.device, fn, where: str, *args) -> None:
    """fn(*args, stream) on dev's current stream."""
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        check(st, where)


def _ints(x, name: str, dev: torch.device, *shape: int) -> int:
    """Device pointer of a contiguous int32 tensor of the given shape on dev."""
    if isinstance(x, torch.Tensor) and x.dtype is torch.int32 and x.shape == shape and x.device == dev and x.is_contiguous():
        return x.data_ptr()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype != torch.int32 or not x.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous int32 CUDA tensor")
    if tuple(x.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(x.shape)}")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, expected {dev}: every tensor of a call must be on one device")
    return x.data_ptr()


def _table(x, name: str, dev: torch.device, rows: int) -> tuple[int, int, int]:
    """Pointer, row stride and width of an int32 [rows, width] table with contiguous rows on dev."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype is not torch.int32 or x.dim() != 2:
        raise TypeError(f"{name}: expected an int32 CUDA tensor [batch, max_pages] with contiguous rows")
    (n, width), (stride, inner) = x.shape, x.stride()
    if inner != 1 and width > 1:
        raise TypeError(f"{name}: expected an int32 CUDA tensor [batch, max_pages] with contiguous rows")
    if n != rows:
        raise ValueError(f"{name}: expected {rows} rows, got {n}")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, expected {dev}: every tensor of a call must be on one device")
    _i32(n, f"rows of {name}"), _i32(width, f"width of {name}")
    return x.data_ptr(), stride if rows > 1 else max(stride, width), width


def rope_qk_norm(Q: torch.Tensor, K: torch.Tensor, q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                 pos: torch.Tensor, theta: float, eps: float = 1e-6, rope_style: int = 0,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Per-head norm of queries and keys and their rotation to pos ([L] or [B, L] int32), one pass.
    Returns (q_out, k_out); an output may be its input, for in place."""
    made = fast().rope_qk_norm(Q, K, q_weight, k_weight, pos, theta, eps, rope_style, q_out, k_out)
    if made is not None:
        return _made(made, "rope_qk_norm")
    rope_style = _i32(rope_style, "rope_style")
    if q_out is None:
        q_out = torch.empty_like(Q)
    if k_out is None:
        k_out = torch.empty_like(K)
    tq, tk, to, tp = _b(Q, "Q"), _b(K, "K"), _b(q_out, "q_out"), _b(k_out, "k_out")
    dev = Q.device
    if K.device != dev or q_out.device != dev or k_out.device != dev:
        _one_device("Q", Q, K=K, q_out=q_out, k_out=k_out)
    B, L = Q.shape[:2]
    shared = isinstance(pos, torch.Tensor) and pos.dim() == 1
    p_ptr = _ints(pos, "pos", dev, L) if shared else _ints(pos, "pos", dev, B, L)
    w = []
    for x, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if x is not None:
            if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 1 or not x.is_contiguous():
                raise TypeError(f"{name}: expected a contiguous bfloat16 CUDA tensor [128]")
            if x.shape[0] != Q.shape[3]:
                raise ValueError(f"{name}: expected {Q.shape[3]} weights, got {x.shape[0]}")
            if x.device != dev:
                _one_device("Q", Q, **{name: x})
        w.append(None if x is None else x.data_ptr())
    _call(dev, lib().rope_qk_norm, "rope_qk_norm", tq, to, tk, tp, w[0], w[1], eps, p_ptr, 0 if shared else L, theta,
          rope_style)
    return q_out, k_out


def swa_prefill(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, window: int, sinks: int = 0, q_offset: int = 0,
                softmax_scale: float | None = None, out: torch.Tensor | None = None, return_lse: bool = False):
    """Causal attention of Q [B, Lq, Hq, 128] over K, V [B, Lk, Hkv, 128] where the query at position p = t + q_offset
    sees the last `window` keys up to its own and the first `sinks` (window 0: every key up to its own)."""
    made = fast().swa_prefill(Q, K, V, window, sinks, q_offset, softmax_scale, out, return_lse)
    if made is not None:
        return _made(made, "swa_prefill")
    window, sinks, q_offset = _reach(window, "window"), _reach(sinks, "sinks"), _i64(q_offset, "q_offset")
    tq, tk, tv = _b(Q, "Q"), _b(K, "K"), _b(V, "V")
    dev = Q.device
    if out is None:
        out = torch.empty_like(Q)
    B, Lq, Hq, D = Q.shape
    lse = Q.new_empty((B, Hq, Lq), dtype=torch.float32) if return_lse else None
    to = _b(out, "out")
    if K.device != dev or V.device != dev or out.device != dev:
        _one_device("Q", Q, K=K, V=V, out=out)
    _call(dev, lib().swa_prefill, "swa_prefill", tq, tk, tv, window, sinks, q_offset,
          1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale, to, None if lse is None else lse.data_ptr())
    return (out, lse) if return_lse else out


def rbs_kv4_page_bytes(page_size: int) -> int:
    """Bytes of one page of one KV head of the 4-bit cache."""
    n = int(lib().rbs_kv4_page_bytes(_i32(page_size, "page_size")))
    if n < 0:
        raise RbsError(2, "rbs_kv4_page_bytes", lib().rbs_last_error().decode())
    return n


@dataclasses.dataclass
class KV4Cache:
    """A paged key/value cache in 4 bits (format and layout in include/rbs.h)."""

    data: torch.Tensor  # uint8 [num_pages, Hkv, rbs_kv4_page_bytes(page_size)]
    page_size: int
    k_scale: float = 1.0  # powers of two that the stored scales are relative to
    v_scale: float = 1.0

    @staticmethod
    def empty(num_pages: int, page_size: int, kv_heads: int, device="cuda", k_scale: float = 1.0,
              v_scale: float = 1.0) -> "KV4Cache":
        return KV4Cache(torch.empty(num_pages, kv_heads, rbs_kv4_page_bytes(page_size), dtype=torch.uint8,
                                    device=device), page_size, k_scale, v_scale)

    def c(self) -> KV4CacheC:
        x = self.data
        if not isinstance(x, torch.Tensor):
            raise TypeError("cache.data: expected a torch.Tensor")
        if not x.is_cuda or x.dtype is not torch.uint8 or not x.is_contiguous() or x.dim() != 3:
            raise TypeError("cache.data: expected a contiguous uint8 CUDA tensor [num_pages, Hkv, page bytes]")
        pages, heads, size = x.shape
        page_size = _i32(self.page_size, "cache.page_size")
        # a page is page_size / 16 sub-blocks of 2304 bytes; the library checks the page size itself
        if size != page_size // 16 * 2304:
            raise ValueError(f"cache.data: pages of {size} bytes, expected {page_size // 16 * 2304}")
        return KV4CacheC(x.data_ptr(), pages, heads, page_size, self.k_scale, self.v_scale)


def kv4_extend(block_table: torch.Tensor, old_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
               free_head: torch.Tensor, max_new: int, page_size: int, slots: torch.Tensor | None = None,
               pos: torch.Tensor | None = None, free_head_out: torch.Tensor | None = None):
    """Pages from the free list for requests that grow from old_lens to new_lens ([B] int32): updates block_table
    [B, max_pages] in place and returns (slots, pos, free_head_out), the slots and positions [B, max_new] of the new
    tokens (-1 past a request's last one) and the count of free pages taken so far."""
    made = fast().kv4_extend(block_table, old_lens, new_lens, free_pages, free_head, max_new, page_size, slots, pos,
                             free_head_out)
    if made is not None:
        return _made(made, "kv4_extend")
    max_new, page_size = _i32(max_new, "max_new"), _i32(page_size, "page_size")
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise TypeError("block_table: expected a CUDA tensor")
    dev, B = block_table.device, block_table.shape[0]
    t_ptr, stride, width = _table(block_table, "block_table", dev, B)
    if max_new < 0:
        raise ValueError("max_new must be positive")
    if slots is None:
        slots = block_table.new_empty((B, max_new))
    if pos is None:
        pos = block_table.new_empty((B, max_new))
    if free_head_out is None:
        free_head_out = block_table.new_empty((1,))
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise TypeError("free_pages: expected a contiguous int32 CUDA tensor [num_free]")
    n = free_pages.shape[0]
    _call(dev, lib().kv4_extend, "kv4_extend", t_ptr, stride, B, width, _ints(old_lens, "old_lens", dev, B),
          _ints(new_lens, "new_lens", dev, B), _ints(free_pages, "free_pages", dev, n), n,
          _ints(free_head, "free_head", dev, 1), page_size, max_new, _ints(slots, "slots", dev, B, max_new),
          _ints(pos, "pos", dev, B, max_new), _ints(free_head_out, "free_head_out", dev, 1))
    return slots, pos, free_head_out


def kv4_append(cache: KV4Cache, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantise K and V [B, L, Hkv, 128] into the cache's slots [B, L] (int32; negative: padding, skipped)."""
    made = fast().kv4_append(cache.data, cache.page_size, cache.k_scale, cache.v_scale, K, V, slots)
    if made is not None:
        _made(made, "kv4_append")
        return
    tk, tv, c = _b(K, "K"), _b(V, "V"), cache.c()
    dev = K.device
    if V.device != dev or cache.data.device != dev:
        _one_device("K", K, V=V, cache=cache.data)
    _call(dev, lib().kv4_append, "kv4_append", c, tk, tv, _ints(slots, "slots", dev, K.shape[0], K.shape[1]))


def kv4_load(cache: KV4Cache, slots: torch.Tensor, k_out: torch.Tensor | None = None,
             v_out: torch.Tensor | None = None):
    """The cached keys and values of slots [B, L] as bf16 [B, L, Hkv, 128] (zeros for negative slots)."""
    made = fast().kv4_load(cache.data, cache.page_size, cache.k_scale, cache.v_scale, slots, k_out, v_out)
    if made is not None:
        return _made(made, "kv4_load")
    c = cache.c()
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        raise TypeError("slots: expected a contiguous int32 CUDA tensor [B, L]")
    dev, shape = cache.data.device, (slots.shape[0], slots.shape[1], cache.data.shape[1], 128)
    if k_out is None:
        k_out = slots.new_empty(shape, dtype=torch.bfloat16)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    tk, tv = _b(k_out, "k_out"), _b(v_out, "v_out")
    if k_out.device != dev or v_out.device != dev:
        _one_device("cache", cache.data, k_out=k_out, v_out=v_out)
    _call(dev, lib().kv4_load, "kv4_load", c, _ints(slots, "slots", dev, k_out.shape[0], k_out.shape[1]), tk, tv)
    return k_out, v_out


@functools.lru_cache(maxsize=256)  # a function of the sizes alone
def rbs_kv4_attend_workspace_bytes(seqlen_q: int, heads_q: int, kv_heads: int) -> int:
    return int(lib().rbs_kv4_attend_workspace_bytes(_i64(seqlen_q, "seqlen_q"), _i64(heads_q, "heads_q"),
                                                    _i64(kv_heads, "kv_heads")))


def kv4_attend(Q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, lens: torch.Tensor,
               starts: torch.Tensor | None = None, window: int = 0, sinks: int = 0,
               softmax_scale: float | None = None, out: torch.Tensor | None = None, return_lse: bool = False,
               workspace: torch.Tensor | None = None):
    """Attention of new tokens Q [B, Lq, Hq, 128] over the cached keys and values of their requests: query t of
    request b is at position starts[b] + t (lens[b] - Lq + t without starts) and sees the keys up to its own, with
    window > 0 only the last `window` of them and the first `sinks`."""
    made = fast().kv4_attend(cache.data, cache.page_size, cache.k_scale, cache.v_scale, Q, block_table, lens, starts, window,
                             sinks, softmax_scale, out, return_lse, workspace)
    if made is not None:
        return _made(made, "kv4_attend")
    window, sinks = _reach(window, "window"), _reach(sinks, "sinks")
    tq, c = _b(Q, "Q"), cache.c()
    dev = Q.device
    B, Lq, Hq, D = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    lse = Q.new_empty((B, Hq, Lq), dtype=torch.float32) if return_lse else None
    if workspace is None:
        workspace = Q.new_empty((rbs_kv4_attend_workspace_bytes(Lq, Hq, cache.data.shape[1]),), dtype=torch.uint8)
    to, w_ptr = _b(out, "out"), _dev(workspace, "workspace", torch.uint8)
    if cache.data.device != dev or out.device != dev or workspace.device != dev:
        _one_device("Q", Q, cache=cache.data, out=out, workspace=workspace)
    t_ptr, stride, width = _table(block_table, "block_table", dev, B)
    _call(dev, lib().kv4_attend, "kv4_attend", tq, c, t_ptr, stride, width, _ints(lens, "lens", dev, B),
          None if starts is None else _ints(starts, "starts", dev, B), window, sinks,
          1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale, w_ptr, workspace.numel(), to,
          None if lse is None else lse.data_ptr())
    return (out, lse) if return_lse else out


def rbs_get_device_error() -> int:
    """Read and clear the library's device error word (synchronises the current stream)."""
    code = ctypes.c_int32(0)
    st = lib().rbs_get_device_error(ctypes.byref(code), _stream())
    if st not in (0, 5):
        check(st, "rbs_get_device_error")
    return int(code.value)
