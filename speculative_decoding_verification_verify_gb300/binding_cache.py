"""The operators over a paged cache whose rows may have 8 bits, and a prompt's chunks: the same marshalling as `binding`,
whose helpers these entry points use."""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import binding as b


class Rows(NamedTuple):
    k: torch.Tensor
    v: torch.Tensor


@functools.lru_cache(maxsize=256)
def spec_verify_kv_e4m3_row_bytes(kv_heads: int, head_dim: int) -> int:
    """Bytes of a slot's row of e4m3 values and their heads' powers of two (0: unsupported sizes)."""
    return int(b.load_library().spec_verify_kv_e4m3_row_bytes(kv_heads, head_dim))


def _caches(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_heads: Optional[int], D: int, dtype, device: int):
    """A pair of caches of dtype's rows [num_slots, Hkv, D], or of 8-bit rows [num_slots, row bytes] (uint8):
    (code of the rows' type, slots, key heads, strides from slot to slot)."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}")
    if k_cache.shape != v_cache.shape or k_cache.dtype is not v_cache.dtype:
        raise ValueError("k_cache and v_cache must have one shape and type")
    if k_cache.dtype is not torch.uint8:
        if k_cache.dtype is not dtype:
            raise TypeError(f"k_cache must be {dtype}, or uint8 rows, got {k_cache.dtype}")
        if k_cache.dim() != 3 or k_cache.shape[2] != D or kv_heads not in (None, k_cache.shape[1]):
            raise ValueError(f"k_cache and v_cache must be [num_slots, Hkv, {D}]")
        S, Hkv, _ = k_cache.shape
        return (b._HALF[dtype], S, Hkv, b._slot_stride("k_cache", k_cache, Hkv, D), b._slot_stride("v_cache", v_cache, Hkv, D))
    if kv_heads is None:
        raise ValueError("kv_heads is needed for a cache of 8-bit rows")
    need = spec_verify_kv_e4m3_row_bytes(kv_heads, D)
    if k_cache.dim() != 2 or not need or k_cache.shape[1] != need:
        raise ValueError(f"a cache of 8-bit rows must be [num_slots, {need}] for {kv_heads} heads of {D}")
    strides = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.stride(1) != 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        strides.append(t.stride(0) if t.shape[0] > 1 else max(t.stride(0), need))
    return b.E4M3, k_cache.shape[0], kv_heads, *strides


def _weight(name: str, t: Optional[torch.Tensor], D: int, dtype, device: int):
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (D,) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor [{D}] on cuda:{device}")
    return t.data_ptr()


def spec_verify_kv_append_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, slot_table: torch.Tensor, committed: torch.Tensor,
                             cos_sin: Optional[torch.Tensor], *, q_norm=None, k_norm=None, eps: float = 1e-6,
                             parents=None, num_nodes=None, interleaved: bool = False, q_out=None,
                             dev_status=None, stream=None) -> torch.Tensor:
    """spec_verify_kv_append with an RMS norm of each head of q and k before the rotation (q_norm, k_norm [D] of
    q's type; None: no norm), into a cache of 16-bit rows [num_slots, Hkv, D] or of 8-bit ones, uint8 [num_slots,
    spec_verify_kv_e4m3_row_bytes(Hkv, D)]: e4m3 with a power of two for each head."""
    lib = b._lib or b.load_library()
    code, dt, dev = b._half_dtype(q), q.dtype, b._device_of("q", q)
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, D) or v.shape != (B, N, Hkv, D):
        raise ValueError(f"k and v must be {[B, N, 'Hkv', D]}")
    b._same(dt, dev, k=k, v=v)
    rows, S, Hkv, ks, vs = _caches(k_cache, v_cache, Hkv, D, dt, dev)
    cs, rot_positions, rot = b._angles(cos_sin, dev)
    max_pos = slot_table.shape[-1]
    q_out = b._result("q_out", q_out, (B, N, Hq, D), dt, dev, stream)
    rc = b._on(dev, lib.spec_verify_kv_append_ex)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), code, b._row_stride("q", q, B, N, Hq, D),
        b._row_stride("k", k, B, N, Hkv, D), b._row_stride("v", v, B, N, Hkv, D), q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), rows, S, ks, vs,
        b._index("slot_table", slot_table, (B, max_pos), dev), max_pos, b._index("committed", committed, (B,), dev),
        None if parents is None else b._index("parents", parents, (B, N), dev),
        None if num_nodes is None else b._index("num_nodes", num_nodes, (B,), dev), cs, rot_positions, rot,
        bool(interleaved), _weight("q_norm", q_norm, D, dt, dev), _weight("k_norm", k_norm, D, dt, dev), eps, B, N,
        Hq, Hkv, D, b._status(dev_status, dev), b._raw_stream(stream, dev))
    if rc != b.OK:
        raise b.SpecVerifyError("spec_verify_kv_append_ex", rc)
    return q_out


def spec_verify_kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, slot_table: torch.Tensor, first: torch.Tensor,
                        N: int, *, num_rows=None, kv_heads: Optional[int] = None, head_dim: Optional[int] = None,
                        dtype: Optional[torch.dtype] = None, k_out=None, v_out=None, dev_status=None,
                        stream=None) -> Rows:
    """The cache's rows at positions first[b] .. first[b] + num_rows[b] (None: N) - 1 as contiguous k, v
    [B, N, Hkv, D], zeros behind.  A cache of 8-bit rows needs kv_heads, head_dim and the outputs' dtype."""
    lib = b._lib or b.load_library()
    dev = b._device_of("k_cache", k_cache)
    if k_cache.dtype is not torch.uint8:
        if k_cache.dim() != 3 or k_cache.dtype not in b._HALF:
            raise TypeError("k_cache must be bfloat16 or float16 [num_slots, Hkv, D], or uint8 rows")
        dtype, head_dim = dtype or k_cache.dtype, head_dim or k_cache.shape[2]
    if dtype not in b._HALF or head_dim is None:
        raise ValueError("a cache of 8-bit rows needs head_dim and dtype (bfloat16 or float16)")
    rows, S, Hkv, ks, vs = _caches(k_cache, v_cache, kv_heads, head_dim, dtype, dev)
    B, max_pos = slot_table.shape
    k_out = b._result("k_out", k_out, (B, N, Hkv, head_dim), dtype, dev, stream)
    v_out = b._result("v_out", v_out, (B, N, Hkv, head_dim), dtype, dev, stream)
    rc = b._on(dev, lib.spec_verify_kv_read)(
        k_cache.data_ptr(), v_cache.data_ptr(), rows, S, ks, vs, b._index("slot_table", slot_table, (B, max_pos), dev),
        max_pos, b._index("first", first, (B,), dev),
        None if num_rows is None else b._index("num_rows", num_rows, (B,), dev), B, N, Hkv, head_dim,
        k_out.data_ptr(), v_out.data_ptr(), b._HALF[dtype], b._status(dev_status, dev), b._raw_stream(stream, dev))
    if rc != b.OK:
        raise b.SpecVerifyError("spec_verify_kv_read", rc)
    return Rows(k_out, v_out)


@functools.lru_cache(maxsize=256)
def spec_verify_attention_e4m3_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int, max_pos: int) -> int:
    return int(b.load_library().spec_verify_attention_e4m3_workspace_bytes(B, N, Hq, Hkv, D, max_pos))


def spec_verify_attention_e4m3(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               slot_table: torch.Tensor, committed: torch.Tensor, *, kv_heads: int, parents=None,
                               num_nodes=None, scale: Optional[float] = None, out=None, lse=None,
                               want_lse: bool = False, workspace=None, dev_status=None,
                               stream=None) -> b.Attention:
    """spec_verify_attention over a cache of 8-bit rows: uint8 [num_slots, row bytes], as
    spec_verify_kv_append_ex wrote them from rows of q's type."""
    lib = b._lib or b.load_library()
    code, dt, dev = b._half_dtype(q), q.dtype, b._device_of("q", q)
    B, N, Hq, D = q.shape
    if k_cache.dtype is not torch.uint8:
        raise TypeError(f"k_cache must be uint8 rows, got {k_cache.dtype}")
    _, S, Hkv, ks, vs = _caches(k_cache, v_cache, kv_heads, D, dt, dev)
    max_pos = slot_table.shape[-1]
    out = b._result("out", out, (B, N, Hq, D), dt, dev, stream)
    if lse is not None or want_lse:
        lse = b._result("lse", lse, (B, N, Hq), b._FP32, dev, stream)
    raw = b._raw_stream(stream, dev)
    if workspace is None:
        nbytes = spec_verify_attention_e4m3_workspace_bytes(B, N, Hq, Hkv, D, max_pos)
        workspace = b._workspaces.get(nbytes, dev, stream, raw)
    rc = b._on(dev, lib.spec_verify_attention_e4m3)(
        q.data_ptr(), code, b._row_stride("q", q, B, N, Hq, D), k_cache.data_ptr(), v_cache.data_ptr(), S, ks, vs,
        b._index("slot_table", slot_table, (B, max_pos), dev), max_pos, b._index("committed", committed, (B,), dev),
        None if parents is None else b._index("parents", parents, (B, N), dev),
        None if num_nodes is None else b._index("num_nodes", num_nodes, (B,), dev), B, N, Hq, Hkv, D,
        D ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), b._status(dev_status, dev), raw)
    if rc != b.OK:
        raise b.SpecVerifyError("spec_verify_attention_e4m3", rc)
    return b.Attention(out, lse)


@functools.lru_cache(maxsize=256)
def spec_verify_attention_chunk_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int, max_pos: int) -> int:
    return int(b.load_library().spec_verify_attention_chunk_workspace_bytes(B, N, Hq, Hkv, D, max_pos))


def spec_verify_attention_chunk(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                slot_table: torch.Tensor, committed: torch.Tensor, *,
                                kv_heads: Optional[int] = None, num_nodes=None, scale: Optional[float] = None,
                                out=None, lse=None, want_lse: bool = False, workspace=None, dev_status=None,
                                stream=None) -> b.Attention:
    """Causal attention of a chunk of a prompt: q [B, N, Hq, D] rotated, node n at position committed + n, over
    one layer's paged cache that holds the chunk's own rows too.  k_cache and v_cache are 16-bit rows [num_slots,
    Hkv, D] or, with kv_heads, 8-bit ones (uint8 [num_slots, row bytes]); the rest as for spec_verify_attention."""
    lib = b._lib or b.load_library()
    code, dt, dev = b._half_dtype(q), q.dtype, b._device_of("q", q)
    B, N, Hq, D = q.shape
    rows, S, Hkv, ks, vs = _caches(k_cache, v_cache, kv_heads, D, dt, dev)
    max_pos = slot_table.shape[-1]
    out = b._result("out", out, (B, N, Hq, D), dt, dev, stream)
    if lse is not None or want_lse:
        lse = b._result("lse", lse, (B, N, Hq), b._FP32, dev, stream)
    raw = b._raw_stream(stream, dev)
    if workspace is None:
        nbytes = spec_verify_attention_chunk_workspace_bytes(B, N, Hq, Hkv, D, max_pos)
        workspace = b._chunk_workspaces.get(nbytes, dev, stream, raw)
    rc = b._on(dev, lib.spec_verify_attention_chunk)(
        q.data_ptr(), code, b._row_stride("q", q, B, N, Hq, D), k_cache.data_ptr(), v_cache.data_ptr(), rows, S, ks, vs,
        b._index("slot_table", slot_table, (B, max_pos), dev), max_pos, b._index("committed", committed, (B,), dev),
        None if num_nodes is None else b._index("num_nodes", num_nodes, (B,), dev), B, N, Hq, Hkv, D,
        D ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), b._status(dev_status, dev), raw)
    if rc != b.OK:
        raise b.SpecVerifyError("spec_verify_attention_chunk", rc)
    return b.Attention(out, lse)
