"""GB300-native paged KV cache: decode attention, KV write and block copy.

A thin binding over ``libpagedkv.so`` (C ABI: ``include/pagedkv.h``).  Each
function checks and marshals its tensors (device, dtype, contiguity) and
passes raw pointers and the CUDA stream to the library; every step of the
computation runs in the library's CUDA kernels.  PyTorch supplies device
memory and streams only.  There is no CPU fallback: if the library is not
built, the first call raises.

Cache layout: ``k_cache`` and ``v_cache`` are ``[num_blocks, kv_heads,
block_size, head_dim]`` tensors of one dtype (float32, float16 or bfloat16).
"""

import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import (PKV_DEV_FREE_LIST, PKV_DEV_NOMEM, PKV_DEV_PAIR_RANGE,  # noqa: F401
                   PKV_DEV_SEQ_LEN, PKV_DEV_SLOT_RANGE, PKV_DEV_TABLE_RANGE, PKV_DEV_TIMEOUT,
                   PKV_DEV_TOKENS, PKV_ERR_NOMEM, PKV_SWAP_IN,
                   PKV_SWAP_OUT)

_DTYPE_CODE = {torch.float32: _lib.PKV_F32, torch.float16: _lib.PKV_F16, torch.bfloat16: _lib.PKV_BF16,
               torch.float8_e4m3fn: _lib.PKV_FP8_E4M3}

__all__ = [
    "PagedKVCache", "BlockManager", "paged_kv_write", "paged_attention_decode",
    "paged_attention_prefill",
    "paged_attention_workspace_bytes", "paged_attention_partition_size",
    "paged_block_copy", "paged_block_swap", "paged_get_device_error",
    "paged_selftest_wait_timeout", "paged_selftest_read_stream", "paged_attention_decode_shared",
    "paged_build_tables", "RotaryAxes", "paged_rope_kv_write", "paged_attention_cross",
    "paged_attention_cross_workspace_bytes",
    "library_path",
]


def library_path():
    return _lib.LIB_PATH


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The current stream's handle on a device (the raw accessor where torch has
# it: a Stream object costs ten times as much to make).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(device, stream):
    """The context to enter before a call whose tensors are on ``device``, so
    that it launches there and its allocations belong to ``stream``; None
    where the current device and stream are the ones."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return None
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _need(t, name, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, device))


def _int32(x, name):
    """``x`` as an int that the library's 32-bit argument holds."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError("%s must fit 32 bits, got %d" % (name, x))
    return x


class PagedKVCache:
    """The physical pool: two ``[N, Hk, b, D]`` tensors (keys, values).

    FP8 pools (``torch.float8_e4m3fn``) also take ``k_scale`` / ``v_scale``
    (float32 CUDA tensors ``[Hk]``: a key of head h is its code's value times
    ``k_scale[h]``) and ``io_dtype`` (float16 or bfloat16: the type of q, out
    and the new keys/values).  For other pools ``io_dtype`` is the pool's.
    """

    def __init__(self, k_cache, v_cache, k_scale=None, v_scale=None, io_dtype=None):
        _need(k_cache, "k_cache")
        _need(v_cache, "v_cache", k_cache.dtype, k_cache.device)
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
            raise ValueError("k_cache and v_cache must both be [N, Hk, b, D]")
        if k_cache.dtype not in _DTYPE_CODE:
            raise ValueError("cache dtype must be float32, float16, bfloat16 or float8_e4m3fn")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim = k_cache.shape
        self.dtype, self.device = k_cache.dtype, k_cache.device
        self.k_scale = self.v_scale = None
        if self.dtype == torch.float8_e4m3fn:
            if io_dtype not in (torch.float16, torch.bfloat16):
                raise ValueError("an FP8 pool needs io_dtype float16 or bfloat16")
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need(t, name, torch.float32, self.device)
                if t.shape != (self.num_kv_heads,):
                    raise ValueError("%s must be [kv_heads]" % name)
            self.k_scale, self.v_scale = k_scale, v_scale
            self.io_dtype = io_dtype
        else:
            self.io_dtype = self.dtype
        self._c = _lib.pkv_cache(k_cache.data_ptr(), v_cache.data_ptr(), self.num_blocks,
                                 self.block_size, self.num_kv_heads, self.head_dim,
                                 _DTYPE_CODE[self.dtype],
                                 self.k_scale.data_ptr() if self.k_scale is not None else None,
                                 self.v_scale.data_ptr() if self.v_scale is not None else None,
                                 _DTYPE_CODE[self.io_dtype])

    @classmethod
    def empty(cls, num_blocks, block_size, num_kv_heads, head_dim, dtype, device="cuda"):
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device))

    @property
    def ref(self):
        return ctypes.byref(self._c)


def paged_kv_write(cache, k, v, slot_mapping, stream=None):
    """Store ``k``/``v`` ``[T, Hk, D]`` at ``slot_mapping`` (int64 ``[T]``)."""
    _need(k, "k", cache.io_dtype, cache.device)
    _need(v, "v", cache.io_dtype, cache.device)
    _need(slot_mapping, "slot_mapping", torch.int64, cache.device)
    n = slot_mapping.numel()
    if k.shape != (n, cache.num_kv_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError("k and v must be [num_tokens, kv_heads, head_dim]")
    _lib.check(_lib.lib().paged_kv_write(cache.ref, _ptr(k), _ptr(v), _ptr(slot_mapping), n,
                                         _stream(stream)), "paged_kv_write")


class RotaryAxes:
    """A rotary embedding with one or several position axes.

    ``rotary_dim``: leading elements of a head that rotate (even);
    ``inv_freq``: radians per position of each of the ``rotary_dim / 2``
    pairs; ``pair_axis``: the axis whose position turns each pair (None: axis
    0); ``interleaved``: pairs are neighbours (2i, 2i + 1) instead of halves
    (i, i + rotary_dim / 2); ``num_axes``: rows of the positions, for plans
    whose last axes turn no pair (None: up to the last axis that does).
    """

    def __init__(self, rotary_dim, inv_freq, pair_axis=None, interleaved=False, num_axes=None):
        freq = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
        if freq.shape != (rotary_dim // 2,):
            raise ValueError("inv_freq must hold rotary_dim / 2 frequencies")
        axes = None
        if pair_axis is None and num_axes is not None:
            pair_axis = np.zeros(freq.shape, dtype=np.int32)
        if pair_axis is not None:
            axes = np.ascontiguousarray(np.asarray(pair_axis, dtype=np.int32))
            if axes.shape != freq.shape or axes.min(initial=0) < 0:
                raise ValueError("pair_axis must name an axis for each pair")
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        used = 1 if axes is None else int(axes.max(initial=0)) + 1
        self.num_axes = used if num_axes is None else int(num_axes)
        if self.num_axes < used:
            raise ValueError("pair_axis names axis %d of %d" % (used - 1, self.num_axes))
        self._c = _lib.pkv_rotary()
        _lib.check(_lib.lib().paged_rotary_init(
            ctypes.byref(self._c), self.rotary_dim, self.num_axes, freq.ctypes.data,
            None if axes is None else axes.ctypes.data, int(self.interleaved)), "RotaryAxes")

    @classmethod
    def sections(cls, sections, base=10000.0, interleaved=False):
        """Contiguous runs of pairs, one per axis (``[16, 24, 24]``: the first
        16 of 64 pairs turn with axis 0, ...; an axis may have none), at
        frequencies ``base ** (-2 i / rotary_dim)``."""
        pairs = int(sum(sections))
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        return cls(2 * pairs, [float(base) ** (-i / pairs) for i in range(pairs)], axis, interleaved,
                   num_axes=len(sections))

    @property
    def ref(self):
        return ctypes.byref(self._c)


def _need_rows(t, name, heads, dim, dtype, device):
    """The token stride of ``t``: [T, heads, dim] whose heads are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype or t.device != device:
        raise ValueError("%s must be %s on %s, got %s on %s" % (name, dtype, device, t.dtype, t.device))
    if t.dim() != 3 or t.shape[1:] != (heads, dim):
        raise ValueError("%s must be [num_tokens, %d, %d]" % (name, heads, dim))
    row, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError("%s must have contiguous heads" % name)
    return row


def paged_rope_kv_write(cache, rotary, q, k, v, positions, slot_mapping, q_out=None, stream=None):
    """Rotate ``q`` ``[T, H, D]`` and ``k`` ``[T, Hk, D]`` by the tokens'
    positions and store ``k`` and ``v`` at ``slot_mapping`` (int64 ``[T]``).

    ``positions``: int32 ``[num_axes, T]`` (or ``[T]`` with one axis).  q, k
    and v may be slices of one projection (heads contiguous, tokens strided
    by a multiple of 16 bytes).  ``q_out`` may be ``q``; it is allocated when
    not given.  Returns ``q_out``.
    """
    dev, io, dim = cache.device, cache.io_dtype, cache.head_dim
    if q.dim() != 3:
        raise ValueError("q must be [num_tokens, num_heads, head_dim]")
    n, heads = q.shape[0], q.shape[1]
    qs = _need_rows(q, "q", heads, dim, io, dev)
    ks = _need_rows(k, "k", cache.num_kv_heads, dim, io, dev)
    vs = _need_rows(v, "v", cache.num_kv_heads, dim, io, dev)
    _need(positions, "positions", torch.int32, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if k.shape[0] != n or v.shape[0] != n or slot_mapping.shape != (n,):
        raise ValueError("q, k, v and slot_mapping must hold one entry per token")
    if positions.shape != (rotary.num_axes, n) and not (rotary.num_axes == 1 and
                                                        positions.shape == (n,)):
        raise ValueError("positions must be [num_axes, num_tokens]")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_rope_kv_write(cache, rotary, q, k, v, positions, slot_mapping, q_out)
    if q_out is None:
        q_out = torch.empty((n, heads, dim), dtype=io, device=dev)
        os = heads * dim
    else:
        os = _need_rows(q_out, "q_out", heads, dim, io, dev)
        if q_out.shape[0] != n:
            raise ValueError("q_out must have q's shape")
    rc = _lib.lib().paged_rope_kv_write(
        cache.ref, rotary.ref, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
        positions.data_ptr(), slot_mapping.data_ptr(), n, heads, q_out.data_ptr(), os,
        _raw_stream(dev.index))
    if rc:
        _lib.check(rc, "paged_rope_kv_write")
    return q_out


def paged_attention_partition_size(cache, num_seqs, num_heads, max_seq_len, partition_size=0):
    r = _lib.lib().paged_attention_partition_size(cache.ref, num_seqs, num_heads, max_seq_len,
                                                  partition_size)
    if r < 0:
        _lib.check(r, "paged_attention_partition_size")
    return r


def paged_attention_workspace_bytes(cache, num_seqs, num_heads, max_seq_len, partition_size=0):
    return int(_lib.lib().paged_attention_workspace_bytes(cache.ref, num_seqs, num_heads,
                                                          max_seq_len, partition_size))


def paged_attention_decode(cache, q, block_tables, seq_lens, scale, out=None, max_seq_len=0,
                           workspace=None, partition_size=0, stream=None):
    """Decode attention of ``q`` ``[S, H, D]`` through the block tables.

    ``block_tables``: int32 ``[S, max_blocks]``; ``seq_lens``: int32 ``[S]``;
    ``max_seq_len``: host bound on ``seq_lens`` (0 = table width x block
    size).  Allocates ``out`` and the split-K workspace when not given.
    Returns ``out``.
    """
    _need(q, "q", cache.io_dtype, cache.device)
    _need(block_tables, "block_tables", torch.int32, cache.device)
    _need(seq_lens, "seq_lens", torch.int32, cache.device)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [num_seqs, num_heads, head_dim]")
    num_seqs, num_heads = q.shape[0], q.shape[1]
    if block_tables.dim() != 2 or block_tables.shape[0] != num_seqs or seq_lens.shape != (num_seqs,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", cache.io_dtype, cache.device)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    bound = max_seq_len if max_seq_len else block_tables.shape[1] * cache.block_size
    need = paged_attention_workspace_bytes(cache, num_seqs, num_heads, bound, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    ws_ptr = _ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _lib.check(_lib.lib().paged_attention_decode(
        cache.ref, _ptr(q), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        num_heads, max_seq_len, float(scale), _ptr(out), ws_ptr, ws_len, partition_size,
        _stream(stream)), "paged_attention_decode")
    return out


def paged_attention_decode_shared(cache, q, block_tables, seq_lens, scale, group_starts,
                                  group_prefix, max_group_size, out=None, max_seq_len=0,
                                  workspace=None, partition_size=0, tail_parts=0, stream=None):
    """Decode attention like :func:`paged_attention_decode` for a batch whose
    groups of consecutive sequences share a table prefix.

    ``group_starts``: int32 ``[num_groups + 1]`` (group g is sequences
    ``group_starts[g] .. group_starts[g+1] - 1``); ``group_prefix``: int32
    ``[num_groups]`` positions shared by every member; ``max_group_size``:
    host bound on group sizes; ``tail_parts``: partitions per sequence that
    the partition pass covers after its group's shared ones (0: all of
    them).  Returns ``out``.
    """
    _need(q, "q", cache.io_dtype, cache.device)
    _need(block_tables, "block_tables", torch.int32, cache.device)
    _need(seq_lens, "seq_lens", torch.int32, cache.device)
    _need(group_starts, "group_starts", torch.int32, cache.device)
    _need(group_prefix, "group_prefix", torch.int32, cache.device)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [num_seqs, num_heads, head_dim]")
    num_seqs, num_heads = q.shape[0], q.shape[1]
    if block_tables.dim() != 2 or block_tables.shape[0] != num_seqs or seq_lens.shape != (num_seqs,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    num_groups = group_prefix.numel()
    if group_starts.numel() != num_groups + 1:
        raise ValueError("group_starts must hold num_groups + 1 entries")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", cache.io_dtype, cache.device)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    bound = max_seq_len if max_seq_len else block_tables.shape[1] * cache.block_size
    need = paged_attention_workspace_bytes(cache, num_seqs, num_heads, bound, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    ws_ptr = _ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _lib.check(_lib.lib().paged_attention_decode_shared(
        cache.ref, _ptr(q), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        num_heads, max_seq_len, float(scale), _ptr(out), _ptr(group_starts), _ptr(group_prefix),
        num_groups, int(max_group_size), int(tail_parts), ws_ptr, ws_len, partition_size,
        _stream(stream)),
        "paged_attention_decode_shared")
    return out


def paged_attention_prefill(cache, q, query_starts, block_tables, seq_lens, scale, max_queries,
                            out=None, stream=None):
    """Causal attention of each sequence's chunk of new queries.

    ``q``: ``[total_queries, H, D]``; ``query_starts``: int32 ``[S + 1]``;
    ``block_tables``: int32 ``[S, max_blocks]``; ``seq_lens``: int32 ``[S]``
    (positions including the chunk); ``max_queries``: host bound on any
    chunk's length.  Returns ``out``.
    """
    _need(q, "q", cache.io_dtype, cache.device)
    _need(query_starts, "query_starts", torch.int32, cache.device)
    _need(block_tables, "block_tables", torch.int32, cache.device)
    _need(seq_lens, "seq_lens", torch.int32, cache.device)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [total_queries, num_heads, head_dim]")
    num_seqs = seq_lens.shape[0]
    if query_starts.shape != (num_seqs + 1,) or block_tables.dim() != 2 or \
            block_tables.shape[0] != num_seqs:
        raise ValueError("query_starts must be [S + 1] and block_tables [S, max_blocks]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", cache.io_dtype, cache.device)
    _lib.check(_lib.lib().paged_attention_prefill(
        cache.ref, _ptr(q), q.shape[0], _ptr(query_starts), num_seqs, int(max_queries),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), q.shape[1], float(scale),
        _ptr(out), _stream(stream)), "paged_attention_prefill")
    return out


def paged_attention_cross_workspace_bytes(cache, total_queries, num_seqs, num_heads, max_queries,
                                          max_enc_len):
    """Bytes of workspace that :func:`paged_attention_cross` needs.

    ``max_enc_len`` is the bound itself: table width x block size where the
    call is given 0.
    """
    there = _elsewhere(cache.device, None)  # the plan goes by the device's size
    if there is not None:
        with there:
            return paged_attention_cross_workspace_bytes(cache, total_queries, num_seqs, num_heads,
                                                         max_queries, max_enc_len)
    return int(_lib.lib().paged_attention_cross_workspace_bytes(
        cache.ref, total_queries, _int32(num_seqs, "num_seqs"), _int32(num_heads, "num_heads"),
        _int32(max_queries, "max_queries"), _int32(max_enc_len, "max_enc_len")))


def paged_attention_cross(cache, q, query_starts, block_tables, enc_lens, scale, max_queries,
                          max_enc_len=0, out=None, workspace=None, stream=None):
    """Attention of each sequence's queries to all of its encoder's cached
    states (no causal mask).

    ``q``: ``[total_queries, H, D]``, sequence s's queries at
    ``query_starts[s] .. query_starts[s + 1] - 1``; ``query_starts``: int32
    ``[S + 1]``; ``block_tables``: int32 ``[S, max_blocks]`` of the encoder's
    states; ``enc_lens``: int32 ``[S]``, how many there are (0: zero rows);
    ``max_queries``: host bound on a sequence's queries; ``max_enc_len``:
    host bound on ``enc_lens`` (0 = table width x block size).  Rows of
    ``out`` behind the last sequence's are left as they were.  Returns
    ``out``.
    """
    dev = cache.device
    _need(q, "q", cache.io_dtype, dev)
    _need(query_starts, "query_starts", torch.int32, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(enc_lens, "enc_lens", torch.int32, dev)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [total_queries, num_heads, head_dim]")
    num_seqs = enc_lens.numel()
    if enc_lens.shape != (num_seqs,) or query_starts.shape != (num_seqs + 1,) or \
            block_tables.dim() != 2 or block_tables.shape[0] != num_seqs:
        raise ValueError("enc_lens must be [S], query_starts [S + 1] and block_tables [S, max_blocks]")
    max_queries = _int32(max_queries, "max_queries")
    max_enc_len = _int32(max_enc_len, "max_enc_len")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_attention_cross(cache, q, query_starts, block_tables, enc_lens, scale,
                                         max_queries, max_enc_len, out, workspace)
    lib, total, heads, width = _lib.lib(), q.shape[0], q.shape[1], block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", cache.io_dtype, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        need = lib.paged_attention_cross_workspace_bytes(
            cache.ref, total, num_seqs, heads, max_queries, max_enc_len or width * cache.block_size)
        ws, ws_len = None, need
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            ws = workspace.data_ptr()
    else:
        _need(workspace, "workspace", None, dev)
        ws, ws_len = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = lib.paged_attention_cross(
        cache.ref, q.data_ptr(), total, query_starts.data_ptr(), num_seqs, max_queries,
        block_tables.data_ptr(), width, enc_lens.data_ptr(), max_enc_len, heads, scale,
        out.data_ptr(), ws, ws_len, _raw_stream(dev.index))
    if rc:
        _lib.check(rc, "paged_attention_cross")
    return out


def paged_block_copy(cache, pairs, stream=None):
    """Copy blocks ``pairs[i, 0] -> pairs[i, 1]`` (int64 ``[n, 2]``)."""
    _need(pairs, "pairs", torch.int64, cache.device)
    if pairs.numel() and (pairs.dim() != 2 or pairs.shape[1] != 2):
        raise ValueError("pairs must be [num_pairs, 2]")
    n = pairs.shape[0] if pairs.numel() else 0
    _lib.check(_lib.lib().paged_block_copy(cache.ref, _ptr(pairs), n, _stream(stream)),
               "paged_block_copy")


def paged_block_swap(cache, host_k, host_v, pairs, direction, stream=None):
    """Move blocks between the device pool and a pinned host pool.

    ``host_k``/``host_v``: pinned CPU tensors ``[M, Hk, b, D]`` of the cache
    dtype; ``pairs``: int64 ``[n, 2]`` on the device as (src, dst);
    ``direction``: ``PKV_SWAP_OUT`` (device -> host) or ``PKV_SWAP_IN``.
    """
    for t, name in ((host_k, "host_k"), (host_v, "host_v")):
        if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned():
            raise ValueError("%s must be a pinned CPU tensor" % name)
        if not t.is_contiguous() or t.dtype != cache.dtype:
            raise ValueError("%s must be contiguous with the cache dtype" % name)
        if t.dim() != 4 or tuple(t.shape[1:]) != (cache.num_kv_heads, cache.block_size, cache.head_dim):
            raise ValueError("%s must be [M, kv_heads, block_size, head_dim]" % name)
    if host_k.shape != host_v.shape:
        raise ValueError("host_k and host_v must have one shape")
    _need(pairs, "pairs", torch.int64, cache.device)
    if pairs.numel() and (pairs.dim() != 2 or pairs.shape[1] != 2):
        raise ValueError("pairs must be [num_pairs, 2]")
    n = pairs.shape[0] if pairs.numel() else 0
    _lib.check(_lib.lib().paged_block_swap(cache.ref, _ptr(host_k), _ptr(host_v), host_k.shape[0],
                                           _ptr(pairs), n, int(direction), _stream(stream)),
               "paged_block_swap")


def _output(t, name, size, dtype, device):
    """``t`` checked against what the call writes, or a new tensor."""
    if t is None:
        return torch.empty(size, dtype=dtype, device=device)
    _need(t, name, dtype, device)
    if t.shape != (size,):
        raise ValueError("%s must be [%d], got %s" % (name, size, list(t.shape)))
    return t


def paged_build_tables(free_list, free_state, old_lens, new_lens, block_tables, block_size,
                       max_tokens, seq_lens=None, free_state_out=None, query_starts=None,
                       slot_mapping=None, positions=None, stream=None):
    """Block tables, slot map, query starts and positions of one step, on the
    device: rows go from ``old_lens`` to ``new_lens`` positions, taking blocks
    from a ring of free ones or giving them back.

    ``free_list``: int32 ``[num_blocks]`` ring, updated in place;
    ``free_state``: int64 ``[2]`` (head, count); ``old_lens``/``new_lens``:
    int32 ``[S]``; ``block_tables``: int32 ``[S, max_blocks]``, updated in
    place; ``max_tokens``: length of the slot map (tokens past the step's are
    padding, slot -1).  Outputs are allocated when not given;
    ``seq_lens`` may be ``old_lens`` and ``free_state_out`` may be
    ``free_state``.  Returns ``(seq_lens, free_state_out, query_starts,
    slot_mapping, positions)``.  A step that cannot be taken whole changes
    nothing and sets a device error bit (``PKV_DEV_NOMEM`` when blocks run
    out).
    """
    _need(free_list, "free_list", torch.int32)
    dev = free_list.device
    _need(free_state, "free_state", torch.int64, dev)
    _need(old_lens, "old_lens", torch.int32, dev)
    _need(new_lens, "new_lens", torch.int32, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    n = old_lens.numel()
    if free_list.dim() != 1 or free_state.shape != (2,):
        raise ValueError("free_list must be [num_blocks] and free_state [2]")
    width = block_tables.shape
    if len(width) != 2 or width[0] != n or old_lens.dim() != 1 or new_lens.shape != (n,):
        raise ValueError("old_lens and new_lens must be [S] and block_tables [S, max_blocks]")
    block_size, max_tokens = _int32(block_size, "block_size"), int(max_tokens)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_build_tables(free_list, free_state, old_lens, new_lens, block_tables,
                                      block_size, max_tokens, seq_lens, free_state_out, query_starts,
                                      slot_mapping, positions)
    seq_lens = torch.empty_like(old_lens) if seq_lens is None else \
        _output(seq_lens, "seq_lens", n, torch.int32, dev)
    free_state_out = torch.empty_like(free_state) if free_state_out is None else \
        _output(free_state_out, "free_state_out", 2, torch.int64, dev)
    query_starts = _output(query_starts, "query_starts", n + 1, torch.int32, dev)
    slot_mapping = _output(slot_mapping, "slot_mapping", max_tokens, torch.int64, dev)
    positions = _output(positions, "positions", max_tokens, torch.int32, dev)
    rc = _lib.lib().paged_build_tables(
        free_list.numel(), block_size, free_list.data_ptr(), free_state.data_ptr(),
        old_lens.data_ptr(), new_lens.data_ptr(), n, block_tables.data_ptr(),
        width[1], seq_lens.data_ptr(), free_state_out.data_ptr(), query_starts.data_ptr(),
        slot_mapping.data_ptr(), positions.data_ptr(), max_tokens, _raw_stream(dev.index))
    if rc:
        _lib.check(rc, "paged_build_tables")
    return seq_lens, free_state_out, query_starts, slot_mapping, positions


def paged_get_device_error(stream=None):
    """Synchronise the stream; return and clear the device error bits."""
    bits = ctypes.c_uint32(0)
    _lib.check(_lib.lib().paged_get_device_error(_stream(stream), ctypes.byref(bits)),
               "paged_get_device_error")
    return int(bits.value)


def paged_selftest_wait_timeout(limit_ns=10_000_000, stream=None):
    """Run the bounded-wait self-test: a wait that nothing completes gives up
    after ``limit_ns`` and sets PKV_DEV_TIMEOUT (read it with
    :func:`paged_get_device_error`)."""
    _lib.check(_lib.lib().paged_selftest_wait_timeout(int(limit_ns), _stream(stream)),
               "paged_selftest_wait_timeout")


def paged_selftest_read_stream(buf, sink, stream=None):
    """Read every byte of the device tensor ``buf`` once (read-only
    streaming bandwidth); ``sink`` is a device int32 tensor of one element
    that the kernel XOR-updates."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    _need(sink, "sink", torch.int32, buf.device)
    _lib.check(_lib.lib().paged_selftest_read_stream(_ptr(buf), buf.numel() * buf.element_size(),
                                                     _ptr(sink), _stream(stream)),
               "paged_selftest_read_stream")


def _i64(a):
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64))


class BlockManager:
    """Host block manager (native): tables, slots and copy-on-write pairs."""

    def __init__(self, num_blocks, block_size, free_order=None):
        self._lib = _lib.lib()
        order = None
        if free_order is not None:
            order = _i64(free_order)
            if order.shape != (num_blocks,):
                raise ValueError("free_order must list every block once")
        self._h = self._lib.pkv_bm_create(num_blocks, block_size,
                                          None if order is None else order.ctypes.data)
        if not self._h:
            raise ValueError("bad block manager arguments")
        self.num_blocks, self.block_size = num_blocks, block_size

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.pkv_bm_destroy(h)
            self._h = None

    def admit(self, seq, num_tokens):
        rc = self._lib.pkv_bm_admit(self._h, seq, num_tokens)
        if rc == PKV_ERR_NOMEM:
            raise MemoryError("not enough free blocks (or host memory) to admit %d positions"
                              % num_tokens)
        _lib.check(rc, "admit")

    def fork(self, parent, child):
        _lib.check(self._lib.pkv_bm_fork(self._h, parent, child), "fork")

    def append(self, seqs):
        """Append one position to each sequence; returns (slots, pairs)."""
        s = _i64(seqs)
        n = s.shape[0]
        slots = np.empty(n, dtype=np.int64)
        pairs = np.empty((max(n, 1), 2), dtype=np.int64)
        npairs = ctypes.c_int64(0)
        rc = self._lib.pkv_bm_append(self._h, s.ctypes.data, n, slots.ctypes.data,
                                     pairs.ctypes.data, ctypes.byref(npairs))
        if rc == PKV_ERR_NOMEM:
            raise MemoryError("not enough free blocks (or host memory) for this step")
        _lib.check(rc, "append")
        return slots, pairs[: npairs.value].copy()

    def release(self, seq):
        _lib.check(self._lib.pkv_bm_release(self._h, seq), "release")

    def tables(self, seqs, max_blocks):
        s = _i64(seqs)
        tab = np.empty((s.shape[0], max_blocks), dtype=np.int32)
        lens = np.empty(s.shape[0], dtype=np.int32)
        _lib.check(self._lib.pkv_bm_tables(self._h, s.ctypes.data, s.shape[0], max_blocks,
                                           tab.ctypes.data, lens.ctypes.data), "tables")
        return tab, lens

    def slots(self, seq, start, count):
        """Slots of positions ``start .. start+count-1`` of a sequence."""
        out = np.empty(count, dtype=np.int64)
        _lib.check(self._lib.pkv_bm_slots(self._h, seq, start, count, out.ctypes.data), "slots")
        return out

    def num_free(self):
        return int(self._lib.pkv_bm_num_free(self._h))

    def seq_len(self, seq):
        return int(self._lib.pkv_bm_seq_len(self._h, seq))

    def num_seq_blocks(self, seq):
        return int(self._lib.pkv_bm_num_seq_blocks(self._h, seq))

    def refcount(self, block):
        return int(self._lib.pkv_bm_refcount(self._h, block))

    def check(self):
        return self._lib.pkv_bm_check(self._h) == 0
